// RMS norm of query and key heads with the rotation by position, forward, and
// the same with keys and values going to their slots of a paged cache.
//
// Each row is read once and written once: the memory's bandwidth is the bound.
//  - A work item is some heads of one token, so that the token's cosines and
//    sines (two polynomials a pair) are shared by its heads; with the weights
//    they make four factors a pair, and a row costs two products and the
//    row's scale for each value.
//  - Rows come through shared memory by asynchronous copies, DEPTH - 1 of them
//    ahead: each thread copies the very bytes that it will work on, so the
//    ring needs no barrier and the rows on their way no registers.  Some 100 KB an
//    SM are in flight, which the memory's latency takes (with loads into
//    registers, one row at a time read and wrote 3.1 TB/s, four at a time 3.9).
#include "ffpa_rope.cuh"

namespace ffpa {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_DEPTH = 4;

// Where the rows of a work item are: queries, keys or (append) values.
struct RopeItem {
  const char* src;
  int64_t src_h;
  int which, wt, heads, h0, b, n;
};
__device__ __forceinline__ RopeItem rope_item(const RopeParams& P, unsigned item) {
  RopeItem r;
  const bool in = item < P.items[0] + P.items[1] + P.items_v;
  r.which = item < P.items[0] ? 0 : item < P.items[0] + P.items[1] ? 1 : 2;
  r.wt = r.which == 0 ? 0 : 1;
  const unsigned local = !in ? 0 : r.which == 0 ? item : r.which == 1 ? item - P.items[0] : item - P.items[0] - P.items[1];
  const unsigned token = local / P.chunks[r.wt];
  r.h0 = (local - token * P.chunks[r.wt]) * P.heads_per[r.wt];
  r.heads = in ? min(P.t[r.wt].H - r.h0, P.heads_per[r.wt]) : 0;
  r.b = P.B == 1 ? 0 : token / P.N;
  r.n = token - r.b * P.N;
  if (r.which == 2) {
    r.src_h = P.vs[0];
    r.src = P.v + r.n * P.vs[1] + r.h0 * r.src_h;
  } else {
    const RopeTensor& t = P.t[r.wt];
    r.src_h = t.xs[1];
    r.src = t.x + r.b * t.xs[0] + r.n * t.xs[2] + r.h0 * r.src_h;
  }
  return r;
}

template <int VEC, int ITER>
__host__ __device__ constexpr int rope_row_bytes() {   // of one row, for all threads of a block
  return ROPE_THREADS * ITER * 2 * VEC * 2;
}

// Resident blocks an SM.  The 4-wide vectors fit three (T16384 D120: 54 us, with
// two 64); more rows on their way than those of two blocks of 8-wide vectors
// only slow the memory down (T8192 D512: 110 us, with three blocks 112).
template <int VEC, int ITER>
__host__ __device__ constexpr int rope_blocks() {
  return VEC == 4 && ITER == 1 ? 3 : 2;
}

template <bool F16, int VEC, int LPR, int ITER, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS, rope_blocks<VEC, ITER>()) rope_kernel(const __grid_constant__ RopeParams P) {
  constexpr int ROW = rope_row_bytes<VEC, ITER>(), PIECE = ROPE_THREADS * VEC * 2;
  extern __shared__ __align__(16) char ring[];     // [ROPE_DEPTH][ITER][2][thread] vectors
  __shared__ long long freq_s[512];
  // The weights in fp32, behind the ring: queries', then keys'.
  float* weight_s = reinterpret_cast<float*>(ring + ROPE_DEPTH * ROW);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (P.t[i].w)
      for (int d = threadIdx.x; d < P.D; d += ROPE_THREADS) weight_s[i * P.D + d] = one_weight<F16>(P.t[i].w, P.w32, d);
  load_freqs<VEC, INTER>(P, freq_s);
  const int np = P.rot / (2 * VEC);                // rotated chunks
  const int lane = threadIdx.x % LPR;
  const unsigned all = P.items[0] + P.items[1] + P.items_v;
  const unsigned stride = gridDim.x * (ROPE_THREADS / LPR);
  RopeChunk<VEC> ch[ITER];
#pragma unroll
  for (int k = 0; k < ITER; ++k) ch[k] = rope_chunk<VEC>(lane + k * LPR, P.D, P.rot);
  const float inv_d = 1.0f / P.D;
  // Whole warps stay in the loop: the lanes of a row talk through shuffles.
  const int sub = threadIdx.x % 32 / LPR;
  unsigned first = blockIdx.x * (ROPE_THREADS / LPR) + threadIdx.x / 32 * (32 / LPR);
  // Rows that the items first .. of a warp take (queries' and keys' items differ).
  auto steps = [&](unsigned f) {
    const int q = f < P.items[0] ? P.heads_per[0] : 0;
    return f + (32 / LPR - 1) >= P.items[0] && P.heads_per[1] > q ? P.heads_per[1] : q;
  };
  char* own = ring + threadIdx.x * (VEC * 2);
  const uint32_t own_at = smem_u32(own);

  // The copying runs ahead of the work by DEPTH - 1 steps, into later items too.
  unsigned ahead = first;
  int ahead_h = 0, ahead_heads = 0, ahead_slot = 0, ahead_steps = 0;
  const char* ahead_src = nullptr;
  int64_t ahead_stride = 0;
  auto issue = [&] {
    if (ahead < all) {
      if (ahead_h == 0) {
        const RopeItem it = rope_item(P, ahead + sub);
        ahead_steps = steps(ahead);
        ahead_heads = it.heads;
        ahead_src = it.src;
        ahead_stride = it.src_h;
      }
      if (ahead_h < ahead_heads) {
#pragma unroll
        for (int k = 0; k < ITER; ++k)
          if (ch[k].live) {
            const uint32_t to = own_at + ahead_slot * ROW + 2 * k * PIECE;
            copy_async<VEC * 2>(to, ahead_src + ch[k].a * 2);
            copy_async<VEC * 2>(to + PIECE, ahead_src + ch[k].b * 2);
          }
        ahead_src += ahead_stride;
      }
      if (++ahead_h == ahead_steps) {
        ahead_h = 0;
        ahead += stride;
      }
      if (++ahead_slot == ROPE_DEPTH) ahead_slot = 0;
    }
    copy_commit();
  };
#pragma unroll 1
  for (int i = 0; i < ROPE_DEPTH - 1; ++i) issue();

  int ring_slot = 0;
  for (; first < all; first += stride) {
    const RopeItem it = rope_item(P, first + sub);
    const int64_t pos = P.rot && it.which < 2 ? position_of(P, it.b, it.n) : 0;
    int64_t slot = P.slots && it.which > 0 && it.heads > 0 ? P.slots[it.n] : -1;
    const RopeTensor& t = P.t[it.wt];
    const bool norm = it.which < 2 && t.w;
    int heads = it.heads;
    char* dst;
    int64_t dst_h;
    if (it.which > 0 && P.slots) {
      // The slot of a cached row; a negative one is padding and is not stored.
      if (slot >= P.n_slots) {
        report_invalid(P.err);
        slot = -1;
      }
      if (slot < 0) heads = 0;
      const int64_t page = slot / P.slot_page;
      slot -= page * P.slot_page;
      dst_h = it.which == 2 ? P.vcs[2] : P.kcs[2];
      dst = it.which == 2 ? P.vc + page * P.vcs[0] + slot * P.vcs[1] : P.kc + page * P.kcs[0] + slot * P.kcs[1];
    } else {
      dst_h = t.ys[1];
      dst = t.y + it.b * t.ys[0] + it.n * t.ys[2];
    }
    dst += it.h0 * dst_h;
    // The factors of a value: itself times f0, its partner times f1 (not of
    // columns that are not rotated).
    float2 f0[ITER][VEC], f1[ITER][VEC];
    if (it.which < 2 && heads > 0) {
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        if (!ch[k].live) continue;
#pragma unroll
        for (int i = 0; i < VEC; ++i) f0[k][i] = make_float2(1.0f, 1.0f);
        if (norm) {
          const float* w = weight_s + it.wt * P.D;
#pragma unroll
          for (int i = 0; i < VEC; i += 2) {
            const float4 v = *reinterpret_cast<const float4*>(w + (i < VEC / 2 ? ch[k].a + 2 * i : ch[k].b + 2 * i - VEC));
            f0[k][i] = make_float2(v.x, v.y);
            f0[k][i + 1] = make_float2(v.z, v.w);
          }
        }
        if (ch[k].pair) {
          float c[VEC], s[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) turn(pos, freq_s[i * np + lane + k * LPR], P.rope_scale, c[i], s[i]);
#pragma unroll
          for (int i = 0; i < VEC; ++i) f1[k][i] = partner<VEC, INTER>(f0[k], i);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int p0 = pair_of<VEC, INTER>(i, 0), p1 = pair_of<VEC, INTER>(i, 1);
            f0[k][i].x *= c[p0];
            f0[k][i].y *= c[p1];
            f1[k][i].x *= second_of<VEC, INTER>(i, 0) ? s[p0] : -s[p0];
            f1[k][i].y *= second_of<VEC, INTER>(i, 1) ? s[p1] : -s[p1];
          }
        }
      }
    }
    const int per = steps(first);
#pragma unroll 1
    for (int h = 0; h < per; ++h) {
      copy_wait<ROPE_DEPTH - 2>();
      const char* row = own + ring_slot * ROW;
      if (++ring_slot == ROPE_DEPTH) ring_slot = 0;
      const bool on = h < heads;
      Raw<VEC> ra[ITER], rb[ITER];
      float2 sq = make_float2(0.0f, 0.0f);
      if (on) {
#pragma unroll
        for (int k = 0; k < ITER; ++k)
          if (ch[k].live) {
            ra[k] = own_load<VEC>(row + 2 * k * PIECE);
            rb[k] = own_load<VEC>(row + (2 * k + 1) * PIECE);
            if (norm) {
              float2 x[VEC];
              widen<F16, VEC>(ra[k], x);
              widen<F16, VEC>(rb[k], x + VEC / 2);
#pragma unroll
              for (int i = 0; i < VEC; ++i) sq = fma2(x[i], x[i], sq);
            }
          }
      }
      issue();
      const float sum = row_sum<LPR>(sq.x + sq.y);
      if (!on) continue;
      const float r = norm ? rsqrtf(sum * inv_d + P.eps) : 1.0f;
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int k = 0; k < ITER; ++k)
        if (ch[k].live) {
          if (it.which < 2) {
            float2 x[VEC], y[VEC];
            widen<F16, VEC>(ra[k], x);
            widen<F16, VEC>(rb[k], x + VEC / 2);
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = mul2(x[i], f0[k][i]);
            if (ch[k].pair) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) y[i] = fma2(partner<VEC, INTER>(x, i), f1[k][i], y[i]);
            }
#pragma unroll
            for (int i = 0; i < VEC; ++i) y[i] = mul2(y[i], r2);
            ra[k] = narrow<F16, VEC>(y);
            rb[k] = narrow<F16, VEC>(y + VEC / 2);
          }
          *reinterpret_cast<Raw<VEC>*>(dst + ch[k].a * 2) = ra[k];
          *reinterpret_cast<Raw<VEC>*>(dst + ch[k].b * 2) = rb[k];
        }
      dst += dst_h;
    }
  }
  copy_wait<0>();
}

template <bool F16, int VEC, int LPR, int ITER>
ffpa_status launch_rope_as(const RopeParams& P, bool inter, int sms, int dev, cudaStream_t stream) {
  const int64_t all = P.items[0] + P.items[1] + P.items_v;
  const int64_t per = ROPE_THREADS / LPR;
  int64_t grid = (all + per - 1) / per;
  // As many blocks as are resident, so that the frequencies are formed once
  // and no last wave is left over.
  const int64_t resident = (int64_t)sms * rope_blocks<VEC, ITER>();
  if (grid > resident) grid = resident;
  const int smem = ROPE_DEPTH * rope_row_bytes<VEC, ITER>() + 2 * P.D * 4;
  auto fn = inter ? &rope_kernel<F16, VEC, LPR, ITER, true> : &rope_kernel<F16, VEC, LPR, ITER, false>;
  const ffpa_status st = set_smem_attr_once(reinterpret_cast<const void*>(fn), dev, smem);
  if (st != FFPA_OK) return st;
  fn<<<(int)grid, ROPE_THREADS, smem, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? FFPA_OK : FFPA_ERR_CUDA;
}

template <bool F16>
ffpa_status launch_rope(RopeParams& P, bool inter, int sms, int dev, cudaStream_t stream) {
  const int64_t tokens = (int64_t)P.B * P.N;
  for (int i = 0; i < 2; ++i) {
    const int per = rope_heads(P.D, P.rot, tokens, P.t[i].H, sms);
    P.chunks[i] = (P.t[i].H + per - 1) / per;
    P.heads_per[i] = (P.t[i].H + P.chunks[i] - 1) / P.chunks[i];
    P.items[i] = P.t[i].x ? (unsigned)(tokens * P.chunks[i]) : 0;
  }
  P.items_v = P.slots ? P.items[1] : 0;
  if (rope_vec(P.D, P.rot) == 8) {
    const int n = P.D / 16;
    if (n <= 4) return launch_rope_as<F16, 8, 4, 1>(P, inter, sms, dev, stream);
    if (n <= 8) return launch_rope_as<F16, 8, 8, 1>(P, inter, sms, dev, stream);
    if (n <= 16) return launch_rope_as<F16, 8, 16, 1>(P, inter, sms, dev, stream);
    if (n <= 32) return launch_rope_as<F16, 8, 32, 1>(P, inter, sms, dev, stream);
    return launch_rope_as<F16, 8, 32, 2>(P, inter, sms, dev, stream);
  }
  const int n = P.D / 8;
  if (n <= 16) return launch_rope_as<F16, 4, 16, 1>(P, inter, sms, dev, stream);
  if (n <= 32) return launch_rope_as<F16, 4, 32, 1>(P, inter, sms, dev, stream);
  if (n <= 64) return launch_rope_as<F16, 4, 32, 2>(P, inter, sms, dev, stream);
  return launch_rope_as<F16, 4, 32, 4>(P, inter, sms, dev, stream);
}

}  // namespace

ffpa_status rope_params(const ffpa_rope* r, ffpa_dtype dt, int B, int Hq, int Hkv, int N, int D, RopeParams* P) {
  if (dt != FFPA_BF16 && dt != FFPA_FP16) return FFPA_ERR_DTYPE;
  if (B < 0 || N < 0 || Hq < 1 || Hkv < 1 || !r) return FFPA_ERR_INVALID;
  if (D < 64 || D > 1024 || D % 8 != 0) return FFPA_ERR_UNSUPPORTED;
  if (r->rot_dim < 0 || r->rot_dim > D || r->rot_dim % 8 != 0) return FFPA_ERR_INVALID;
  if (r->rot_dim > 0 && (!r->inv_freq || (!r->positions && B > 0 && N > 0))) return FFPA_ERR_INVALID;
  if (r->rot_dim > 0 && r->position_bits != 32 && r->position_bits != 64) return FFPA_ERR_INVALID;
  if (r->rot_dim > 0 && (!on_boundary(r->inv_freq, 8) || !on_boundary(r->positions, r->position_bits / 8)))
    return FFPA_ERR_INVALID;
  if (!std::isfinite(r->eps) || r->eps < 0.0f || !std::isfinite(r->rope_scale)) return FFPA_ERR_INVALID;
  const size_t wa = r->weight_f32 ? 4 : 2;
  if (!on_boundary(r->q_weight, wa) || !on_boundary(r->k_weight, wa)) return FFPA_ERR_INVALID;
  if ((int64_t)B * N > 0x7fffffffLL / ((int64_t)Hq + 2 * (int64_t)Hkv)) return FFPA_ERR_INVALID;   // rows in 31 bits
  P->pos = static_cast<const char*>(r->positions);
  const int64_t pb = r->position_bits / 8;
  P->pos_s[0] = r->position_str[0] * pb;
  P->pos_s[1] = r->position_str[1] * pb;
  P->pos64 = r->position_bits == 64;
  P->inv_freq = r->inv_freq;
  P->rot = r->rot_dim;
  P->w32 = r->weight_f32 != 0;
  P->B = B;
  P->N = N;
  P->D = D;
  P->eps = r->eps;
  P->rope_scale = r->rope_scale;
  P->t[0].w = r->q_weight;
  P->t[1].w = r->k_weight;
  P->t[0].H = Hq;
  P->t[1].H = Hkv;
  return FFPA_OK;
}

}  // namespace ffpa

extern "C" {

ffpa_status ffpa_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, ffpa_dtype dt, int B, int Hq,
                              int Hkv, int N, int D, const int64_t q_str[4], const int64_t k_str[4],
                              const int64_t qo_str[4], const int64_t ko_str[4], const ffpa_rope* rope,
                              ffpa_stream_t stream) {
  using namespace ffpa;
  RopeParams P{};
  ffpa_status st = rope_params(rope, dt, B, Hq, Hkv, N, D, &P);
  if (st != FFPA_OK) return st;
  if (B == 0 || N == 0) return FFPA_OK;
  if (!q || !k || !q_out || !k_out || !q_str || !k_str || !qo_str || !ko_str) return FFPA_ERR_INVALID;
  if (!rows_ok(q_str, {B, Hq, N, D}) || !rows_ok(qo_str, {B, Hq, N, D}) || !rows_ok(k_str, {B, Hkv, N, D}) ||
      !rows_ok(ko_str, {B, Hkv, N, D}))
    return FFPA_ERR_INVALID;
  if (!on_boundary(q, 16) || !on_boundary(k, 16) || !on_boundary(q_out, 16) || !on_boundary(k_out, 16))
    return FFPA_ERR_INVALID;
  int dev = 0;
  const bool turns = rope->rot_dim > 0;
  st = call_device({q, k, q_out, k_out, turns ? rope->positions : nullptr, turns ? rope->inv_freq : nullptr,
                    rope->q_weight, rope->k_weight},
                   &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  int sms = 0;
  if ((st = call_status(dev, nullptr, &P.err, &sms)) != FFPA_OK) return st;
  const void* x[2] = {q, k};
  void* y[2] = {q_out, k_out};
  const int64_t* xs[2] = {q_str, k_str};
  const int64_t* ys[2] = {qo_str, ko_str};
  for (int i = 0; i < 2; ++i) {
    P.t[i].x = static_cast<const char*>(x[i]);
    P.t[i].y = static_cast<char*>(y[i]);
    for (int j = 0; j < 3; ++j) {
      P.t[i].xs[j] = xs[i][j] * 2;
      P.t[i].ys[j] = ys[i][j] * 2;
    }
  }
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FFPA_FP16 ? launch_rope<true>(P, rope->interleaved != 0, sms, dev, s)
                         : launch_rope<false>(P, rope->interleaved != 0, sms, dev, s);
}

ffpa_status ffpa_kv_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                           ffpa_dtype dt, int T, int Hq, int Hkv, int D, int num_pages, int page_size,
                           const int64_t q_str[3], const int64_t k_str[3], const int64_t v_str[3],
                           const int64_t qo_str[3], const int64_t kc_str[4], const int64_t vc_str[4],
                           const int64_t* slots, const ffpa_rope* rope, ffpa_stream_t stream,
                           const ffpa_options* options) {
  using namespace ffpa;
  RopeParams P{};
  ffpa_status st = rope_params(rope, dt, 1, Hq, Hkv, T, D, &P);
  if (st != FFPA_OK) return st;
  if (num_pages < 1 || page_size < 1) return FFPA_ERR_INVALID;
  if (T == 0) return FFPA_OK;
  if (!k || !v || !k_cache || !v_cache || !slots || !k_str || !v_str || !kc_str || !vc_str) return FFPA_ERR_INVALID;
  if (q && (!q_out || !q_str || !qo_str)) return FFPA_ERR_INVALID;
  if (!rows_ok(k_str, {T, Hkv, D}) || !rows_ok(v_str, {T, Hkv, D}) ||
      !rows_ok(kc_str, {num_pages, page_size, Hkv, D}) || !rows_ok(vc_str, {num_pages, page_size, Hkv, D}))
    return FFPA_ERR_INVALID;
  if (q && (!rows_ok(q_str, {T, Hq, D}) || !rows_ok(qo_str, {T, Hq, D}))) return FFPA_ERR_INVALID;
  if (!on_boundary(q, 16) || !on_boundary(k, 16) || !on_boundary(v, 16) || !on_boundary(q_out, 16) ||
      !on_boundary(k_cache, 16) || !on_boundary(v_cache, 16) || !on_boundary(slots, 8))
    return FFPA_ERR_INVALID;
  int dev = 0;
  const bool turns = rope->rot_dim > 0;
  st = call_device({k, v, q, q ? q_out : nullptr, k_cache, v_cache, slots, turns ? rope->positions : nullptr,
                    turns ? rope->inv_freq : nullptr, rope->q_weight, rope->k_weight},
                   &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  int sms = 0;
  if ((st = call_status(dev, options, &P.err, &sms)) != FFPA_OK) return st;
  // (t, h, d) strides as (b, h, n)
  if (q) {
    P.t[0].x = static_cast<const char*>(q);
    P.t[0].y = static_cast<char*>(q_out);
    P.t[0].xs[1] = q_str[1] * 2;
    P.t[0].xs[2] = q_str[0] * 2;
    P.t[0].ys[1] = qo_str[1] * 2;
    P.t[0].ys[2] = qo_str[0] * 2;
  }
  P.t[1].x = static_cast<const char*>(k);
  P.t[1].xs[1] = k_str[1] * 2;
  P.t[1].xs[2] = k_str[0] * 2;
  P.v = static_cast<const char*>(v);
  P.vs[0] = v_str[1] * 2;
  P.vs[1] = v_str[0] * 2;
  P.kc = static_cast<char*>(k_cache);
  P.vc = static_cast<char*>(v_cache);
  for (int j = 0; j < 3; ++j) {
    P.kcs[j] = kc_str[j] * 2;
    P.vcs[j] = vc_str[j] * 2;
  }
  P.slots = slots;
  P.n_slots = (int64_t)num_pages * page_size;
  P.slot_page = page_size;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FFPA_FP16 ? launch_rope<true>(P, rope->interleaved != 0, sms, dev, s)
                         : launch_rope<false>(P, rope->interleaved != 0, sms, dev, s);
}

}  // extern "C"
