// Attention of one new token per request where all requests begin with the same keys.
//
// The shared keys meet B g query rows a key head (g heads share it), 4 g B D operations per 4 D
// bytes: with 287 rows the tensor cores are as busy as the memory.  So they go through
// the forward's tensor-core kernels (LAYOUT_SHARED of ffpa_single.cu, ffpa_dual.cu,
// ffpa_split.cu, ffpa_cluster.cu): a query tile holds the heads of whole requests, the keys come
// from their pages by boxes, and because a decode batch has few tiles the keys are cut into parts,
// an item each, that leave fp32 sums.  The requests' own keys go through the decode kernels
// (DECODE_OWN of ffpa_decode.cuh), which leave normalised fp32 rows.  A last launch
// weighs both by their maxima and sums, in a fixed order, and rounds once.
//
// B64 Hq32 Hkv8 D512 behind 16384 shared keys: 133 us, 520 TFLOPS (its floor: 79 us of the memory's rate, 36 of the tensor
// cores'); the shared keys alone take 92 us on 128 SMs, 16 rounds of 4.75 us behind a first one of 12, own keys 50 us, most
// of them beside and behind those.  B128 Hq32 Hkv8 D128 behind 32768: 120 us (61, 36); shared 60 to 68 us, bound by the
// softmax of the dual-tile kernel, own keys 63.
#include "ffpa_decode.cuh"

namespace ffpa {
namespace {

struct SharedPlan {
  SharedKernel kernel;
  int ctas, per, tile_rows, n_qt, items, splits;
  double us;                                       // the estimate, for a number of keys
  int64_t parts() const { return (int64_t)items * splits * per; }
};

// sms: of the device, or the most that any has (for the workspace).  keys: at most so many are shared (0:
// any number, for the workspace).
SharedPlan shared_plan(int B, int Hq, int Hkv, int D, int sms, long long keys) {
  SharedPlan p;
  const int group = Hq / Hkv;
  const int requests = BM / group;                 // of a query tile
  const int tiles = (B + requests - 1) / requests;
  p.tile_rows = requests * group;
  p.kernel = shared_kernel(D, tiles > 1);
  p.ctas = shared_ctas(p.kernel, D);
  p.per = p.kernel == SharedKernel::DUAL ? 2 : 1;
  p.n_qt = (tiles + p.per - 1) / p.per;
  p.items = Hkv * p.n_qt;
  // Parts of the keys: as many as fill the SMs, in one wave or two, where the time that this
  // takes off the longest chain of tiles is more than the parts' sums cost (written and read).
  const int slots = sms / p.ctas;
  int most = 2 * slots / p.items;
  if (most < 1) most = 1;
  p.splits = most;
  p.us = 0;
  if (keys > 0) {
    const double tiles_all = (double)((keys + BN - 1) / BN);
    const double tile_us = 4.0 * BM * BN * D * p.per / p.ctas / 8.4e6, part_us = p.items * p.per * (double)BM * D * 8.0 / 6e6;
    // Beside other launches a tile of a CTA takes longer: 6 TFLOPS (4.2 with Q streamed), at D = 64 the 1 us of its
    // softmax.  (Cut by that estimate, B16 S4096 Hkv4 D128 took 24 us in place of 16: more parts are dear to join.)
    const double slow_us = 4.0 * BM * BN * D * p.per / p.ctas / (D > 512 ? 4.2e6 : 6e6), real_us = slow_us > 1.0 ? slow_us : 1.0;
    double best = 0;
    for (int s = 1; s <= most && s <= tiles_all; ++s) {
      const int waves = (p.items * s + slots - 1) / slots;
      const double longest = (double)(long long)((tiles_all + s - 1) / s);
      const double us = waves * (longest * tile_us + 3.0) + s * part_us;
      if (s == 1 || us < best) {
        best = us;
        p.splits = s;
        p.us = waves * (longest * real_us + 3.0) + s * (part_us + 0.1);   // (the merge of a row takes its parts in turn)
      }
    }
  }
  return p;
}

// Workspace: what own keys need, their rows and log-sum-exps, the parts and their maxima and sums.
struct SharedSpace {
  size_t o32, lse, part, ml, total;
};
SharedSpace shared_space(int B, int Hq, int Hkv, int D, int64_t parts) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  SharedSpace s;
  s.o32 = up(decode_bytes(Hq, Hkv, D));
  s.lse = s.o32 + up((size_t)B * Hq * D * 4);
  s.part = s.lse + up((size_t)B * Hq * 4);
  s.ml = s.part + up((size_t)parts * BM * D * 4);
  s.total = s.ml + up((size_t)parts * BM * 8);
  return s;
}

struct MergeParams {
  const float* part;
  const float2* part_ml;
  const float* own;        // [B][Hq][D]
  const float* own_lse;    // [B][Hq]
  const int32_t* shared_len;
  char* o;
  float* lse;
  int* err;
  int64_t o_sb, o_sh;      // bytes
  int B, Hq, D, group, tile_rows, tiles, splits;   // query tiles of a part (with the empty one of a last pair)
};

// One decode over all keys of each request takes two launches in place of four, and its reads of the shared keys
// come from L2 but for the first: 10.6 TB/s with up to 8 heads a key head; more take one CTA an SM, 5.6 TB/s, and above
// 16 heads every pass of 16 reads the keys again.  One request in one pass reads no more than the split.  It is taken where the
// estimates say so.  Measured, one pass and split (us): B2 S5003 Hkv4 D1024 32 and 48, B2 S18858 Hkv1 D512 17 and 30, B3 S3305
// Hkv8 D128 13.7 and 16.6, B4 S30111 Hkv4 D64 20 and 27.5, B16 S1010 Hkv4 D128 12.4 and 13.8, B8 S1024 Hkv8 D512 23 and 19.5,
// B4 S8192 Hkv8 D256 36 and 25, B16 S3353 Hkv2 D512 29 and 21; of one key head with 128 heads, B1 S31552 D512 98 and 35,
// B16 S54432 D192 1007 and 114.  Of 34916 sizes (1 to 4 key heads, groups of 1 to 128, B 1 to 32, 512 to 65536 shared keys) the
// estimates take a way that is more than 10 % slower for 3 %, more than 25 % for 0.8 %, 1.7 times as slow at most.
bool one_pass(int B, int Hkv, int group, int D, double keys, const SharedPlan& split) {
  const int heads = 8 * decode_nt(group), passes = (group + heads - 1) / heads;
  if (B == 1 && passes == 1) return true;          // (at most 4 % slower than the split in 4016 sizes)
  return 9.0 + B * Hkv * passes * keys * D * 4.0 / (heads == 8 ? 10.6e6 : 5.6e6) <= 10.0 + split.us;
}

constexpr int MERGE_WARPS = 4;
constexpr int MERGE_FLIGHT = 8;   // parts on their way
constexpr float LOG2E = 1.4426950408889634f;

// A warp joins 128 columns of a row: the row's parts in order, then its own keys.
template <bool F16>
__global__ void __launch_bounds__(MERGE_WARPS * 32) merge_kernel(const __grid_constant__ MergeParams P) {
  const int lane = threadIdx.x % 32;
  const int cols = (P.D + 127) / 128;
  const long long task = (long long)blockIdx.x * MERGE_WARPS + threadIdx.x / 32;
  dependency_wait();
  if (blockIdx.x == 0 && threadIdx.x == 0 && *P.shared_len < 0) report_invalid(P.err);
  const long long row = task / cols;               // b Hq + hq
  if (row >= (long long)P.B * P.Hq) return;
  const int col = (int)(task - row * cols) * 128 + lane * 4;
  const int b = (int)(row / P.Hq), hq = (int)(row - (long long)b * P.Hq);
  const int hk = hq / P.group, r = b * P.group + hq - hk * P.group;   // row of the key head
  const int tile = r / P.tile_rows;
  // Part s of the row: ((hk splits + s) tiles + tile) 128 + its row of the tile.
  const int64_t first = ((int64_t)hk * P.splits * P.tiles + tile) * BM + (r - tile * P.tile_rows), step = (int64_t)P.tiles * BM;
  const bool mine = col < P.D;
  const int at = min(col, P.D - 4);
  const float* from = P.part + first * P.D + at;
  const float own2 = P.own_lse[row] * LOG2E;
  const float4 own = *reinterpret_cast<const float4*>(P.own + row * P.D + at);
  // Parts four at a time, in order, with the maximum so far; a part without keys for this row has no
  // sums (and its memory may hold anything).
  float top = own2, l = own2 == -INFINITY ? 0.0f : 1.0f;
  float4 a = own2 == -INFINITY ? make_float4(0, 0, 0, 0) : own;
  for (int s0 = 0; s0 < P.splits; s0 += MERGE_FLIGHT) {
    float2 ml[MERGE_FLIGHT];
    float4 x[MERGE_FLIGHT];
    float now = top;
#pragma unroll
    for (int i = 0; i < MERGE_FLIGHT; ++i) {
      const int s = min(s0 + i, P.splits - 1);
      ml[i] = P.part_ml[first + s * step];
      x[i] = *reinterpret_cast<const float4*>(from + s * step * P.D);
      if (s0 + i >= P.splits) ml[i].y = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < MERGE_FLIGHT; ++i)
      if (ml[i].y != 0.0f) now = fmaxf(now, ml[i].x);
    const float base = now == -INFINITY ? 0.0f : now, f0 = ex2_approx(top - base);
    top = now;
    l *= f0;
    a.x *= f0;
    a.y *= f0;
    a.z *= f0;
    a.w *= f0;
#pragma unroll
    for (int i = 0; i < MERGE_FLIGHT; ++i) {
      if (ml[i].y == 0.0f) continue;
      const float f = ex2_approx(ml[i].x - base);
      l += f * ml[i].y;
      a.x += f * x[i].x;
      a.y += f * x[i].y;
      a.z += f * x[i].z;
      a.w += f * x[i].w;
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (mine)
    *reinterpret_cast<uint2*>(P.o + b * P.o_sb + hq * P.o_sh + col * 2) =
        make_uint2(pack2<F16>(a.x * inv, a.y * inv), pack2<F16>(a.z * inv, a.w * inv));
  if (P.lse && col == 0) P.lse[row] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
}

}  // namespace
}  // namespace ffpa

extern "C" {

size_t ffpa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int D) {
  using namespace ffpa;
  if (B < 0 || decode_bytes(Hq, Hkv, D) == 0 || D % 64 != 0 || Hq / Hkv > BM) return 0;
  return shared_space(B, Hq, Hkv, D, B == 0 ? 0 : shared_plan(B, Hq, Hkv, D, DEC_SMS_MAX, 0).parts()).total;
}

ffpa_status ffpa_decode_shared(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                               ffpa_dtype dt, int B, int Hq, int Hkv, int D, int num_pages, int page_size,
                               int max_pages, int n_shared, const int64_t q_str[3], const int64_t k_str[4],
                               const int64_t v_str[4], const int64_t o_str[3], const int32_t* shared_pages,
                               const int32_t* shared_len, const int32_t* block_table, int64_t table_str,
                               const int32_t* seq_lens, const float* scale, int enable_gqa, void* workspace,
                               size_t workspace_bytes, ffpa_stream_t stream, const ffpa_options* options) {
  using namespace ffpa;
  const DecodeShape shape{B, Hq, Hkv, D, num_pages, page_size, max_pages, k_str, v_str};
  float sc = 0.0f;
  ffpa_status st = check_decode(DECODE_OWN, dt, shape, scale, enable_gqa, &sc);
  if (st != FFPA_OK) return st;
  const int way = options ? options->kernel : FFPA_VARIANT_AUTO;
  if (n_shared < 0 || (way != FFPA_VARIANT_AUTO && way != FFPA_VARIANT_SINGLE && way != FFPA_VARIANT_SPLIT)) return FFPA_ERR_INVALID;
  if (D % 64 != 0 || page_size % 8 != 0 || Hq / Hkv > BM) return FFPA_ERR_UNSUPPORTED;
  if (B == 0) return FFPA_OK;
  st = check_decode_rows(DECODE_OWN, shape, q, k_cache, v_cache, o, lse, q_str, o_str, block_table, table_str, seq_lens, workspace);
  if (st != FFPA_OK) return st;
  if (!shared_len || !on_boundary(shared_len, 4) || (n_shared > 0 && (!shared_pages || !on_boundary(shared_pages, 4))))
    return FFPA_ERR_INVALID;
  if (workspace_bytes < ffpa_decode_shared_workspace_bytes(B, Hq, Hkv, D)) return FFPA_ERR_INVALID;
  if ((long long)B * Hq > 0x7fffffffLL / 8) return FFPA_ERR_INVALID;
  const bool held = shape.held();
  int dev = 0;
  st = call_device({q, o, lse, seq_lens, workspace, shared_len, held ? k_cache : nullptr, held ? v_cache : nullptr,
                    held ? (const void*)block_table : nullptr, n_shared > 0 ? (const void*)shared_pages : nullptr},
                   &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  int* err = nullptr;
  int sms = 0;
  if ((st = call_status(dev, options, &err, &sms)) != FFPA_OK) return st;
  if (sms > DEC_SMS_MAX) sms = DEC_SMS_MAX;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int pages = held ? (n_shared < max_pages ? n_shared : max_pages) : 0;
  char* ws = static_cast<char*>(workspace);
  MergeParams M{};
  SharedPlan pl = shared_plan(B, Hq, Hkv, D, sms, pages > 0 ? (long long)pages * page_size : 1);
  if (pages == 0) pl.splits = 0;
  const SharedSpace sp = shared_space(B, Hq, Hkv, D, pl.parts());

  DecodeParams P{};
  P.err = err;
  P.q = static_cast<const char*>(q);
  P.k = static_cast<const char*>(k_cache);
  P.v = static_cast<const char*>(v_cache);
  P.table = block_table;
  P.lens = seq_lens;
  P.q_sb = q_str[0] * 2;
  P.q_sh = q_str[1] * 2;
  P.table_str = table_str;
  P.shared_len = shared_len;
  P.shared_table = shared_pages;
  P.shared_pages = pages;
  if (way == FFPA_VARIANT_SINGLE ||
      (way == FFPA_VARIANT_AUTO && one_pass(B, Hkv, Hq / Hkv, D, (double)pages * page_size, pl))) {
    P.o = static_cast<char*>(o);
    P.lse = lse;
    P.o_sb = o_str[0] * 2;
    P.o_sh = o_str[1] * 2;
    return run_decode_16(P, shape, dt, sc, sms, dev, ws, options, s);
  }

  // ---- the shared keys
  if (pages > 0) {
    Params P{};                                      // (of the forward kernels)
    const size_t smem = plan_shared(pl.kernel, D, &P);
    const int group = Hq / Hkv;
    // Queries as (64, heads of a group, requests, chunks, key heads); a box is a chunk of a tile.
    {
      const uint64_t qh = Hq > 1 ? (uint64_t)q_str[1] * 2 : (uint64_t)D * 2, qb = B > 1 ? (uint64_t)q_str[0] * 2 : (uint64_t)D * 2;
      const uint64_t dims[5] = {DK, (uint64_t)group, (uint64_t)B, (uint64_t)(D / DK), (uint64_t)Hkv};
      const uint64_t str[4] = {qh, qb, DK * 2, qh * group};
      const uint32_t box[5] = {DK, (uint32_t)group, (uint32_t)(pl.tile_rows / group), 1, 1};
      if ((st = encode_rows(&P.tm_q, dt, 5, q, dims, str, box)) != FFPA_OK) return st;
    }
    SharedKeys& S = P.sh;
    S.box_rows = BM;
    while (page_size % S.box_rows != 0) S.box_rows /= 2;
    S.v_rows = S.box_rows < P.vk ? S.box_rows : P.vk;   // a stage of V holds whole boxes
    for (int i = 0; i < 2; ++i) {
      // K a chunk a box, V the chunks of a stage.
      const int64_t* of = i ? v_str : k_str;
      const uint64_t one = (uint64_t)D * 2, head = Hkv > 1 ? (uint64_t)of[2] * 2 : one;
      const uint64_t dims[5] = {DK, (uint64_t)page_size, (uint64_t)(D / DK), (uint64_t)Hkv, (uint64_t)num_pages};
      const uint64_t str[4] = {(uint64_t)of[1] * 2, DK * 2, head, num_pages > 1 ? (uint64_t)of[0] * 2 : one};
      const uint32_t box[5] = {DK, (uint32_t)(i ? S.v_rows : S.box_rows), (uint32_t)(i ? P.vchunks : 1), 1, 1};
      if ((st = encode_rows(i ? &P.tm_v : &P.tm_k, dt, 5, i ? v_cache : k_cache, dims, str, box)) != FFPA_OK) return st;
    }
    S.pages = shared_pages;
    S.len = shared_len;
    S.lens = seq_lens;
    S.part = reinterpret_cast<float*>(ws + sp.part);
    S.part_ml = reinterpret_cast<float2*>(ws + sp.ml);
    S.n_pages = pages;
    S.num_pages = num_pages;
    S.page_size = page_size;
    S.tile_rows = pl.tile_rows;
    S.splits = pl.splits;
    // fp16 weights: up to 2^8 above the kept maximum, and the smallest that counts 2^-31 of it.
    S.lift = dt == FFPA_FP16 ? 7.0f : 0.0f;
    P.B = B;
    P.Hq = Hq;
    P.group = group;
    P.D = D;
    P.n_qt = pl.n_qt;
    P.scale_log2 = sc * LOG2E;
    P.fp16 = dt == FFPA_FP16;
    P.mask_kind = FFPA_MASK_NONE;
    P.inject = options && options->test_drop_first_copy ? 1 : 0;
    P.timeout_ns = options && options->wait_timeout_ns ? options->wait_timeout_ns : 2000000000ull;
    P.err = err;
    P.device = dev;
    const int items = pl.items * pl.splits;
    st = pl.kernel == SharedKernel::DUAL    ? launch_dual_shared(P, items, smem, s)
         : pl.kernel == SharedKernel::SPLIT ? launch_split_shared(P, items, smem, s)
         : pl.kernel == SharedKernel::CLUSTER ? launch_cluster_shared(P, items, smem, s)
                                              : launch_single_shared(P, items * P.n_slices, smem, s);
    if (st != FFPA_OK) return st;
  }

  // ---- the requests' own keys
  P.o32 = reinterpret_cast<float*>(ws + sp.o32);
  P.lse = reinterpret_cast<float*>(ws + sp.lse);
  st = run_decode<DECODE_OWN>(P, shape, dt, sc, sms, dev, ws, options, s);
  if (st != FFPA_OK) return st;

  // ---- both
  M.part = reinterpret_cast<const float*>(ws + sp.part);
  M.part_ml = reinterpret_cast<const float2*>(ws + sp.ml);
  M.own = P.o32;
  M.own_lse = P.lse;
  M.shared_len = shared_len;
  M.o = static_cast<char*>(o);
  M.lse = lse;
  M.err = err;
  M.o_sb = o_str[0] * 2;
  M.o_sh = o_str[1] * 2;
  M.B = B;
  M.Hq = Hq;
  M.D = D;
  M.group = Hq / Hkv;
  M.tile_rows = pl.tile_rows;
  M.tiles = pl.n_qt * pl.per;
  M.splits = pl.splits;
  const long long tasks = (long long)B * Hq * ((D + 127) / 128);
  const int grid = (int)((tasks + MERGE_WARPS - 1) / MERGE_WARPS);
  return launch_dependent(dt == FFPA_FP16 ? merge_kernel<true> : merge_kernel<false>, grid, MERGE_WARPS * 32, 0, s, M);
}

}  // extern "C"
