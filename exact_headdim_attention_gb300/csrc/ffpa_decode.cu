// Attention of one new token per request over a paged key/value cache.
//
//   o[b,h] = sum_n softmax_n(scale * q[b,h] . K[n]) V[n],   n < seq_lens[b],
//
// where key n of request b lies in page block_table[b][n / page_size].  Every
// key and value is read once and takes part in 4 g D operations per 4 D bytes
// (g query heads share it), so the cache's bandwidth is the bound, and the work
// is laid out for it:
//
//  - The keys of all (request, key head) pairs form one line of T-key tiles,
//    cut into equal runs, one run per CTA (two CTAs per SM, or one): a long
//    request is shared by many CTAs and short ones share a CTA, whatever the
//    mix, and the host needs no lengths.  A pair that ends inside its CTA is
//    written at once; a pair cut between CTAs leaves fp32 partial sums with
//    their maximum and sum, which the second launch joins in the order of the CTAs.
//  - Two rings of shared-memory tiles, one of K and one of V, are kept full by warps
//    of their own.  They hold what fits of whole tiles: 192 KB an SM up to D = 256,
//    and with two CTAs an SM 128 KB at D = 512 and 1024 (one K and one V tile of 32 KB
//    a CTA; a third misses by 0.5 and 2.5 KB), 144 to 168 KB between.
//    Where pages hold a multiple of 8 keys a tile arrives as tensor boxes of
//    up to T rows of one page, with the 128-byte swizzle that the matrix
//    loads want.  Of other page sizes the larger ones have tiles that end with
//    their page, one box each, and the smaller ones take 16-byte asynchronous
//    copies into the same layout.  (One bulk copy per row was slower: an SM
//    starts one every 45 to 64 cycles, 1.65 TB/s with the 256-byte rows of D = 128.)
//  - Keys (then columns of V) are the 16 rows of mma.m16n8k16 and the heads its
//    8 columns: K and V are the operands read once, and up to 8 heads cost one
//    instruction per 256 elements.  For the scores each of eight warps takes 16
//    keys and a part of D; for the output it takes 32 keys and a share of the
//    columns.  Between them lies the only barrier of a tile: each
//    warp reads the scores of its keys from shared memory, adds the parts and
//    forms its own P operand in registers (the warps that share keys repeat
//    the 8 exponentials a lane, which costs less than a second barrier).
//  - A tile is a chain of dependent steps that leaves most issue slots empty,
//    so two CTAs share an SM where the registers allow it, each with half of
//    the rings.
//  - Maximum and sum are kept in fp32 by each group of warps that has keys of
//    its own and joined at the pair's end in the order of the groups.  P goes
//    into the second product as two values of the input type (off by 2^-16 of
//    P, fp16 2^-21), so that numerator and sum see the same weights.  (With P
//    rounded once the error of O was 20 to 35 % larger.  The second value costs
//    0 to 4 % with up to 8 heads, B32 Hkv8 D512 201.3 -> 201.8 us, and 3 to 8 % with
//    more: B2 Hq16 Hkv1 D256 104 -> 107, B32 Hq32 Hkv2 D512 98 -> 104.)
//
// Every wait on a copy has a time limit, after which the call's status word
// receives FFPA_ERR_DEVICE_TIMEOUT and the CTA runs out without waiting.
#include "ffpa_paged.cuh"

namespace ffpa {
namespace {

constexpr int DEC_WARPS = 8;          // that multiply
constexpr int DEC_THREADS = (DEC_WARPS + 2) * 32;   // and one each that brings K and V
constexpr int DEC_RING_MAX = 8;       // tiles of K (and of V) in the ring
// Powers of two above the maximum at which fp16 forms its exponentials: the largest is
// 2^15, and 2^-39 of it is the smallest that counts.
constexpr float P_LIFT = 15.0f;
// SMs of any sm_103 part; the workspace is sized for them without asking a device.
constexpr int DEC_SMS_MAX = 160;

struct DecodeParams {
  CUtensorMap map_k, map_v;
  const char *q, *k, *v;
  char* o;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  float* part;      // [2 grid][8 NT][D] unnormalised partial outputs
  float2* part_ml;  // [2 grid][8 NT] (maximum in log2 units, sum)
  int4* cuts;       // [grid][2] the pairs that CTA c shares with earlier and with later CTAs:
                    // (first CTA + 65536 x CTAs or 0, heads, request, first head)
  int* err;
  int64_t q_sb, q_sh, o_sb, o_sh;       // bytes
  int64_t k_sp, k_ss, k_sh, v_sp, v_ss, v_sh;
  int64_t table_str;
  unsigned long long timeout_ns;
  int B, Hq, Hkv, group, D, head_tiles;
  int num_pages, page_size, max_pages;
  int chunks;       // 64-column chunks of a row
  int boxed;        // tiles arrive as tensor boxes
  int page_tiles;   // tiles of a page where a tile ends with its page, else 0
  int box_rows;     // rows of a box (all T where not boxed), a power of two >= 8
  int box_chunks;   // chunks of a box: all, or 1 when D ends inside a chunk
  int ring_k, ring_v, drop;
  float scale_log2;
};

// Sizes of one call.  A tile has T = 16 keys for D > 512 and twice as many each
// time D halves (at most 32 KB).
struct DecodePlan {
  int nt, ctas, tile, chunks, ring_k, ring_v, head_tiles;
  size_t smem;
};

// Heads of one pass: 8 NT.  A larger group is split over pairs that read the
// same keys again (B64 Hq32 Hkv1 D512 of 4096 keys: 192 us in two passes of 16 heads; one
// pass of 32 heads, whose accumulators leave the registers, took 1.56 times as long).
__host__ __device__ constexpr int decode_nt(int group) { return group <= 8 ? 1 : 2; }
// CTAs of an SM: two leave 96 registers a thread, too few for 16 heads (B32 Hq32
// Hkv2 D512 of 4096 keys: 104 us with 8 computing warps an SM; 16 took 1.14 times as long).
__host__ __device__ constexpr int decode_ctas(int nt) { return nt == 1 ? 2 : 1; }
// Parts of D in the first product, and groups of warps with keys of their own in the second.
__host__ __device__ constexpr int decode_parts(int tile) { return tile >= 128 ? 1 : 128 / tile; }
__host__ __device__ constexpr int decode_groups(int tile) { return tile >= 32 ? tile / 32 : 1; }
// Scores of two tiles (of one where a warp reads no other's).
__host__ __device__ constexpr bool decode_own_keys(int tile) { return tile / 16 > DEC_WARPS; }
__host__ __device__ constexpr size_t decode_score_bytes(int nt, int tile) {
  return ((size_t)(decode_own_keys(tile) ? 1 : 2) * decode_parts(tile) * 8 * nt * (tile + 8) * 4 + 1023) / 1024 * 1024;
}

DecodePlan decode_plan(int D, int group) {
  DecodePlan p;
  p.nt = decode_nt(group);
  p.ctas = decode_ctas(p.nt);
  p.head_tiles = (group + 8 * p.nt - 1) / (8 * p.nt);
  p.tile = D > 512 ? 16 : D > 256 ? 32 : D > 128 ? 64 : D > 64 ? 128 : 256;
  p.chunks = (D + 63) / 64;
  const size_t fixed = decode_score_bytes(p.nt, p.tile);
  const size_t stage = (size_t)p.tile * p.chunks * 128;
  // 8 KB a CTA stay for static shared memory, the alignment of the boxes, the system,
  // and a block of the joining kernel that is set up early (with 4 KB left 1 us more).
  int n = static_cast<int>((SMEM_LIMIT / p.ctas - 8192 - fixed) / stage);
  if (n > 2 * DEC_RING_MAX) n = 2 * DEC_RING_MAX;
  p.ring_v = n / 2;
  p.ring_k = n - n / 2;
  p.smem = 1024 + fixed + (size_t)(p.ring_k + p.ring_v) * stage;
  return p;
}

// A place on the line of tiles: tile t of `tiles` of pair u of request b.
struct Place {
  int b, u, t, tiles, len;
};

__device__ __forceinline__ int clamped_len(const DecodeParams& P, int n) {
  const long long cap = (long long)P.max_pages * P.page_size;
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}

// Tiles of a request, and a tile's first key.  (Tiles that end with their page are a
// kernel of their own: with the other path's code beside it a call took 0.2 to 1 us more.)
template <bool PAGED>
__device__ __forceinline__ int tiles_of(const DecodeParams& P, int len, int T) {
  if (!PAGED) return (len + T - 1) / T;
  const int pages = len / P.page_size;
  return pages * P.page_tiles + (len - pages * P.page_size + T - 1) / T;
}
template <bool PAGED>
__device__ __forceinline__ int first_key(const DecodeParams& P, int t, int T) {
  if (!PAGED) return t * T;
  const int pages = t / P.page_tiles;
  return pages * P.page_size + (t - pages * P.page_tiles) * T;
}

template <bool PAGED>
__device__ __forceinline__ void advance(const DecodeParams& P, int pairs, Place& p, int T) {
  if (++p.t < p.tiles) return;
  p.t = 0;
  if (++p.u < pairs) return;
  p.u = 0;
  do {
    if (p.b + 1 >= P.B) {      // behind the last request: never used (one empty tile)
      p.len = 0;
      p.tiles = 1;
      return;
    }
    ++p.b;
    p.len = clamped_len(P, P.lens[p.b]);
  } while (p.len == 0);
  p.tiles = tiles_of<PAGED>(P, p.len, T);
}

// A run [lo, lo + n) of the line's `total` tiles, which are dealt to `runs` CTAs.
struct Run {
  long long lo, total, runs;
  int n;
  __device__ __forceinline__ int cta_of(long long tile) const { return (int)(((tile + 1) * runs - 1) / total); }
};

// Notes for the joining kernel that the pair of the run's tile i, the first one
// here, goes over several CTAs.
__device__ __forceinline__ void note_cut(const DecodeParams& P, const Place& p, const Run& run, int i, int heads) {
  const int side = p.t == 0;
  if (side ? i + p.tiles <= run.n : i != 0) return;
  const long long begin = run.lo + i - p.t;
  const int first = run.cta_of(begin), n = run.cta_of(begin + p.tiles - 1) - first + 1;
  const int hk = p.u / P.head_tiles, ht = p.u % P.head_tiles;
  P.cuts[2 * blockIdx.x + side] = make_int4(first + (n << 16), min(heads, P.group - ht * heads), p.b, hk * P.group + ht * heads);
}

// A whole warp's bounded wait; false for all its lanes when the limit expired for one.
__device__ __forceinline__ bool all_waited(uint32_t bar, uint32_t parity, const DecodeParams& P, volatile int* abort_flag) {
  return __all_sync(~0u, mbar_try_wait(bar, parity) || wait_bounded(bar, parity, abort_flag, P.timeout_ns, P.err));
}

// The queries of the next pair on their way to L2, when its first values are asked
// for: read by the pair itself they came 1 us late (B110 D512 of 1 to 87 keys 28.6 us
// in place of 27.4).
__device__ __forceinline__ void fetch_queries(const DecodeParams& P, const Place& p, int heads) {
  const int hk = p.u / P.head_tiles, ht = p.u % P.head_tiles;
  const int rows = min(heads, P.group - ht * heads), lines = (P.D * 2 + 127) / 128;
  const char* q = P.q + p.b * P.q_sb + (int64_t)(hk * P.group + ht * heads) * P.q_sh;
  for (int x = threadIdx.x % 32; x < rows * lines; x += 32) fetch_l2(q + x / lines * P.q_sh + x % lines * 128);
}

// K (or V) tiles of the run as tensor boxes, a box a lane, its page looked up
// one tile ahead.  A page that does not exist, and rows that belong to no key,
// have a coordinate behind the last page: the copy writes zeros there.
template <bool PAGED>
__device__ __forceinline__ void produce_boxes(const DecodeParams& P, int T, int heads, bool is_v, Place at, const Run& run,
                                              uint32_t ring, int slots, uint64_t* full, uint64_t* empty, volatile int* abort_flag) {
  const int lane = threadIdx.x % 32, pairs = P.Hkv * P.head_tiles, n_tiles = run.n;
  const CUtensorMap* map = is_v ? &P.map_v : &P.map_k;
  const int per_row = P.chunks / P.box_chunks;          // boxes side by side (at most 32 boxes a tile)
  const int row = lane / per_row * P.box_rows, chunk = lane % per_row;
  const bool mine = row < T;
  const uint32_t box_bytes = P.box_rows * P.box_chunks * 128, stage = T * P.chunks * 128;
  const uint32_t to = row * P.chunks * 128 + chunk * box_bytes;
  int page = -1, in_page = 0;
  bool keyed = false;
  auto look_up = [&](const Place& p) {
    const int key = first_key<PAGED>(P, p.t, T) + row;
    keyed = mine && key < p.len;
    page = -1;
    if (keyed) {
      const int j = key / P.page_size;
      in_page = key - j * P.page_size;
      page = P.table[p.b * P.table_str + j];
    }
  };
  look_up(at);
  int slot = 0, i = 0;
  uint32_t lap = 0;
  for (; i < n_tiles; ++i) {
    const int head = at.u / P.head_tiles;
    const bool good = page >= 0 && page < P.num_pages;
    if (keyed && !good) report_invalid(P.err);
    const int y = good ? in_page : 0, z = good ? page : P.num_pages;
    if (is_v && lane == 0 && (at.t == 0 || i == 0)) note_cut(P, at, run, i, heads);
    advance<PAGED>(P, pairs, at, T);
    if (i + 1 < n_tiles) {
      look_up(at);
      if (is_v && at.t == 0) fetch_queries(P, at, heads);
    }
    if (!all_waited(smem_u32(empty + slot), lap ^ 1u, P, abort_flag) || P.drop) break;
    const uint32_t bar = smem_u32(full + slot);
    if (lane == 0) mbar_arrive_expect_tx(bar, stage);
    __syncwarp();
    if (mine) {
      const uint32_t dst = ring + slot * stage + to;
      if (P.box_chunks == 1)
        tma_load_4d(dst, map, bar, chunk * 64, y, head, z);
      else
        tma_load_5d(dst, map, bar, 0, y, 0, head, z);
    }
    if (++slot == slots) {
      slot = 0;
      lap ^= 1u;
    }
  }
  // Copies still in flight land before the CTA ends (the computing warps wait for them,
  // unless they gave up).
  for (int j = i < slots ? i : slots; j > 0; --j) {
    if (slot == 0) {
      slot = slots;
      lap ^= 1u;
    }
    --slot;
    wait_drain(smem_u32(full + slot), lap, P.timeout_ns, P.err);
  }
}

// The same tile for any page size: the warp looks its rows up lane by lane,
// one tile ahead, and copies them in pieces of 16 bytes, a power of two of
// lanes to a row.  A row without a key, or of a page that does not exist,
// becomes zeros.
__device__ __forceinline__ void produce_pieces(const DecodeParams& P, int T, int heads, bool is_v, Place at,
                                               const Run& run, uint32_t ring, int slots, uint64_t* full, uint64_t* empty,
                                               volatile int* abort_flag) {
  const int lane = threadIdx.x % 32, pairs = P.Hkv * P.head_tiles, n_tiles = run.n;
  const int cpr = P.D / 8;                         // pieces of a row
  int wide = 8;                                    // lanes of a row
  while (wide < cpr && wide < 32) wide *= 2;
  const int c0 = lane % wide, r0 = lane / wide, step = 32 / wide;
  const char* base = is_v ? P.v : P.k;
  const int64_t sp = is_v ? P.v_sp : P.k_sp, ss = is_v ? P.v_ss : P.k_ss, sh = is_v ? P.v_sh : P.k_sh;
  const uint32_t stage = T * P.chunks * 128;
  int page[8];
  auto look_up = [&](const Place& p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (32 * j >= T) break;
      const int r = lane + 32 * j, key = p.t * T + r;
      page[j] = r < T && key < p.len ? P.table[p.b * P.table_str + key / P.page_size] : -1;
    }
  };
  look_up(at);
  int slot = 0;
  uint32_t lap = 0;
  for (int i = 0; i < n_tiles; ++i) {
    // Offsets of this tile's rows (-1: zeros), then the pages of the next.
    const char* head = base + (at.u / P.head_tiles) * sh;
    int64_t from[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      from[j] = -1;
      if (32 * j >= T) break;
      const int r = lane + 32 * j, key = at.t * T + r;
      if (r < T && key < at.len) {
        if (page[j] >= 0 && page[j] < P.num_pages)
          from[j] = page[j] * sp + key % P.page_size * ss;
        else
          report_invalid(P.err);
      }
    }
    if (is_v && lane == 0 && (at.t == 0 || i == 0)) note_cut(P, at, run, i, heads);
    advance<false>(P, pairs, at, T);
    if (i + 1 < n_tiles) {
      look_up(at);
      if (is_v && at.t == 0) fetch_queries(P, at, heads);
    }
    if (!all_waited(smem_u32(empty + slot), lap ^ 1u, P, abort_flag) || P.drop) break;
    const uint32_t tile = ring + slot * stage;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (32 * j >= T) break;
      const int end = min(32, T - 32 * j);
      // Four rows a lane at a time: their offsets first, then the copies.
      for (int r = 0; r < end; r += 4 * step) {
        int64_t row_at[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) row_at[y] = __shfl_sync(~0u, from[j], (r + y * step + r0) & 31);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int in = r + y * step + r0;
          if (in >= end) continue;
          const int row = 32 * j + in;
          const char* src = row_at[y] >= 0 ? head + row_at[y] : base;
          const uint32_t bytes = row_at[y] >= 0 ? 16 : 0;
          for (int c = c0; c < cpr; c += wide)
            copy16_async(tile + (c >> 3) * (T * 128) + row * 128 + ((c ^ row) & 7) * 16, bytes ? src + c * 16 : base, bytes);
        }
      }
    }
    copy_arrive(smem_u32(full + slot));
    if (++slot == slots) {
      slot = 0;
      lap ^= 1u;
    }
  }
  copy_wait_all();
}

// Word i of lane q of each four lanes becomes word q of lane i.
__device__ __forceinline__ void trade_words(uint32_t (&r)[4]) {
  const int q = threadIdx.x % 4;
  auto trade = [&](uint32_t& x, uint32_t& y, int mask) {   // y of the lower lane for x of the upper
    const bool up = q & mask;
    const uint32_t got = __shfl_xor_sync(~0u, up ? x : y, mask);
    if (up)
      x = got;
    else
      y = got;
  };
  trade(r[0], r[1], 1);
  trade(r[2], r[3], 1);
  trade(r[0], r[2], 2);
  trade(r[1], r[3], 2);
}

// Two column tiles of 8 heads, as the second product leaves them (a lane holds
// heads c, c + 1 of columns r and r + 8 of a tile, c = lane % 4 * 2, r = lane / 4),
// times f0 and f1, become 64 bytes of each head: 8 x 8 transpositions, then one of
// pieces among four lanes, and 16 bytes a lane.  (Written as they lie, two bytes at a
// time, the output took 3 us of a pair of D = 1024.)
template <bool F16>
__device__ __forceinline__ void write_columns(char* out, int64_t o_sh, int heads, int d0, int D, const float (&a)[4],
                                              const float (&b)[4], float f0, float f1) {
  const int q = threadIdx.x % 4, head = threadIdx.x % 32 / 4, d = d0 + q * 8;
  uint32_t r[4] = {transpose8(pack2<F16>(a[0] * f0, a[1] * f1)), transpose8(pack2<F16>(a[2] * f0, a[3] * f1)),
                   transpose8(pack2<F16>(b[0] * f0, b[1] * f1)), transpose8(pack2<F16>(b[2] * f0, b[3] * f1))};
  trade_words(r);
  if (head < heads && d < D) *reinterpret_cast<uint4*>(out + head * o_sh + d * 2) = make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool F16, int NT, int T, bool PAGED>
__global__ void __launch_bounds__(DEC_THREADS, decode_ctas(NT)) decode_kernel(const __grid_constant__ DecodeParams P) {
  constexpr int HEADS = 8 * NT, THREADS = DEC_THREADS;
  constexpr int PARTS = decode_parts(T), GROUPS = decode_groups(T), MT = T / 16;
  constexpr int KSTEPS = T < 32 ? 1 : 2;      // of 16 keys, of a warp in the second product
  constexpr int DT = T < 32 ? 8 : 4;          // column tiles of a warp there
  constexpr int WDS = DEC_WARPS / GROUPS;     // warps that share keys there
  constexpr int SPITCH = T + 8, SBUF = PARTS * HEADS * SPITCH;
  constexpr bool OWN = decode_own_keys(T);    // a warp's scores are those of its own keys
  extern __shared__ char smem_raw[];
  __shared__ uint64_t full_k[DEC_RING_MAX], full_v[DEC_RING_MAX], empty_k[DEC_RING_MAX], empty_v[DEC_RING_MAX];
  __shared__ float2 ml_s[GROUPS][HEADS];
  __shared__ long long scan_s[DEC_THREADS / 32 + 1];
  __shared__ int start_s[2];
  __shared__ Place next_s[2];
  __shared__ int abort_flag;
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pairs = P.Hkv * P.head_tiles;
  const uint32_t stage = T * P.chunks * 128;

  // ---- this CTA's run of tiles
  long long total, lo, hi;
  Place cur;
  {
    const int per = (P.B + THREADS - 1) / THREADS;
    const int b0 = tid * per, b1 = min(P.B, b0 + per);
    int n0 = b0 < b1 ? P.lens[b0] : 0;             // on its way while the barriers are made
    if (P.boxed && tid == 32) {
      prefetch_tmap(&P.map_k);
      prefetch_tmap(&P.map_v);
    }
    if (tid < DEC_RING_MAX) {
      const int arrivals = P.boxed ? 1 : 32;
      mbar_init(smem_u32(full_k + tid), arrivals);
      mbar_init(smem_u32(full_v + tid), arrivals);
      mbar_init(smem_u32(empty_k + tid), DEC_WARPS);
      mbar_init(smem_u32(empty_v + tid), DEC_WARPS);
      fence_mbar_init();
    }
    if (tid == 64) {
      abort_flag = 0;
      P.cuts[2 * blockIdx.x] = P.cuts[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    }
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = b == b0 ? n0 : P.lens[b];
      const int len = clamped_len(P, n);
      if (n != len && blockIdx.x == 0) report_invalid(P.err);
      mine += tiles_of<PAGED>(P, len, T);
    }
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long x = __shfl_up_sync(~0u, incl, d);
      if (lane >= d) incl += x;
    }
    if (lane == 31) scan_s[warp] = incl;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before += scan_s[w];
      total += scan_s[w];
    }
    total *= pairs;
    long long at = (before + incl - mine) * pairs;   // first tile of request b0
    const long long runs = total < gridDim.x ? total : gridDim.x;
    const long long c = blockIdx.x;
    // c total / runs by way of total = q runs + rest
    const uint32_t cut = (uint32_t)max(runs, 1LL);
    const long long q = total >> 32 ? total / cut : (uint32_t)total / cut;
    const uint32_t rest = (uint32_t)(total - q * cut);
    lo = c < runs ? c * q + (uint32_t)c * rest / cut : 0;
    hi = c < runs ? (c + 1) * q + (uint32_t)(c + 1) * rest / cut : 0;
    if (c < runs && lo >= at && lo < at + mine * pairs) {
      int b = b0;
      for (; b < b1; ++b) {
        const long long tiles = tiles_of<PAGED>(P, clamped_len(P, b == b0 ? n0 : P.lens[b]), T);
        if (lo < at + tiles * pairs) break;
        at += tiles * pairs;
      }
      b = min(b, P.B - 1);
      start_s[0] = b;
      start_s[1] = max(1, clamped_len(P, b == b0 ? n0 : P.lens[b]));
      scan_s[DEC_THREADS / 32] = lo - at;
    }
    // Requests without keys have no tile: their rows are written here.
    for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
      if (clamped_len(P, P.lens[b]) != 0) continue;
      for (int i = tid; i < P.Hq * (P.D / 8); i += THREADS) {
        const int h = i / (P.D / 8), d = i % (P.D / 8);
        *reinterpret_cast<uint4*>(P.o + b * P.o_sb + h * P.o_sh + d * 16) = make_uint4(0, 0, 0, 0);
      }
      if (P.lse)
        for (int h = tid; h < P.Hq; h += THREADS) P.lse[(int64_t)b * P.Hq + h] = -INFINITY;
    }
    if (c >= runs) return;   // (an exit counts for the dependent launch too)
    // Columns behind D meet zeros of Q and must be finite (boxes bring zeros).
    if (!P.boxed && P.D % 16 != 0) {
      char* ring = smem + decode_score_bytes(NT, T);
      const int c16 = P.D / 8;
      for (int i = tid; i < (P.ring_k + P.ring_v) * T; i += THREADS)
        *reinterpret_cast<uint4*>(ring + (size_t)(i / T) * stage + (c16 >> 3) * (T * 128) + (i % T) * 128 +
                                  ((c16 ^ i) & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    __syncthreads();
    cur.b = start_s[0];
    cur.len = start_s[1];
    cur.tiles = tiles_of<PAGED>(P, cur.len, T);
    const long long r = scan_s[DEC_THREADS / 32];
    cur.u = (int)(r >> 32 ? r / cur.tiles : (uint32_t)r / (uint32_t)cur.tiles);
    cur.t = (int)(r - (long long)cur.u * cur.tiles);
  }
  dependents_launch();
  const int n_tiles = (int)(hi - lo);
  float* scores = reinterpret_cast<float*>(smem);                  // [2, or 1 when OWN][PARTS][HEADS][SPITCH]
  const uint32_t ring_k = smem_u32(smem + decode_score_bytes(NT, T));
  const uint32_t ring_v = ring_k + P.ring_k * stage;

  if (warp >= DEC_WARPS) {
    const bool is_v = warp > DEC_WARPS;
    uint64_t *full = is_v ? full_v : full_k, *empty = is_v ? empty_v : empty_k;
    const uint32_t ring = is_v ? ring_v : ring_k;
    const int slots = is_v ? P.ring_v : P.ring_k;
    const Run run{lo, total, total < gridDim.x ? total : gridDim.x, n_tiles};
    if (PAGED || P.boxed)
      produce_boxes<PAGED>(P, T, HEADS, is_v, cur, run, ring, slots, full, empty, &abort_flag);
    else
      produce_pieces(P, T, HEADS, is_v, cur, run, ring, slots, full, empty, &abort_flag);
    return;
  }

  // ---- the computing warps
  const int ksteps = (P.D + 15) / 16;
  // Shares of D are whole chunks, so that a chunk's swizzle is a constant of the code.
  const int part = warp / MT;                        // in the first product (0 when a warp has two key tiles)
  const int kper = (P.chunks + PARTS - 1) / PARTS * 4;
  const int k0 = part * kper, kn = max(0, min(kper, ksteps - k0));
  const int wkey = warp / WDS, wd = warp % WDS;    // group of keys, share of columns
  const int dper = (P.chunks + WDS - 1) / WDS * 4;
  const int d0 = wd * dper, dn = max(0, min(dper, ksteps - d0));
  const int c2 = (lane % 4) * 2, hq = lane / 4;
  const uint32_t chunk_bytes = P.box_rows * 128;
  // Row r of a tile: boxes of box_rows rows, in each chunk after chunk.
  auto row_at = [&](int r) { return r / P.box_rows * (P.chunks * chunk_bytes) + r % P.box_rows * 128; };
  const int key0 = OWN ? warp * 32 : warp % MT * 16;   // first key of the first product
  const int kr = key0 + (lane & 15), vr = wkey * 32 + (lane >> 4) * 8 + (lane & 7);
  const uint32_t k_at = ring_k + row_at(kr) + (k0 >> 2) * chunk_bytes + (((lane >> 4) ^ (lane & 7)) << 4);
  const uint32_t k_at2 = OWN ? k_at - row_at(kr) + row_at(kr + 16) : 0;
  const uint32_t v_x = (d0 >> 2) * chunk_bytes + ((((lane >> 3) & 1) ^ (lane & 7)) << 4);
  const uint32_t v_at = ring_v + row_at(vr) + v_x, v_at2 = ring_v + row_at(vr + 16) + v_x;
  uint32_t qf[8][NT][2];
  float acc[DT][NT][4];
  float top[NT], sum[NT];                          // of head 8 n + lane / 4
  int slot_k = 0, slot_v = 0;
  uint32_t lap_k = 0, lap_v = 0;
  bool alive = true;
  int buf = 0;
  constexpr int N = DEC_WARPS * 32;

  for (int i0 = 0, turn = 0; i0 < n_tiles; turn ^= 1) {
    // ---- one pair's tiles of this run: [i0, i1)
    const int i1 = min(n_tiles, i0 + cur.tiles - cur.t);
    // One warp finds the pair after it; the others read that at the pair's end,
    // behind one barrier at least, so that all warps agree on every pair.
    if (warp == 0) {
      Place next = cur;
      next.t = next.tiles - 1;
      advance<PAGED>(P, pairs, next, T);
      if (lane == 0) next_s[turn] = next;
    }
    const int hk = cur.u / P.head_tiles, ht = cur.u % P.head_tiles;
    const int hq0 = hk * P.group + ht * HEADS;
    const int rows = min(HEADS, P.group - ht * HEADS);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = n * 8 + hq;
      const char* src = P.q + cur.b * P.q_sb + (int64_t)(hq0 + head) * P.q_sh;
#pragma unroll
      for (int s = 0; s < 8; s += 2) {             // 16 bytes a lane
        const int d = (k0 + s) * 16 + lane % 4 * 8;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (head < rows && s < kn && d < P.D) x = *reinterpret_cast<const uint4*>(src + d * 2);
        qf[s][n][0] = x.x;
        qf[s][n][1] = x.y;
        qf[s + 1][n][0] = x.z;
        qf[s + 1][n][1] = x.w;
      }
#pragma unroll
      for (int s = 0; s < DT; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[s][n][j] = 0.0f;
      top[n] = -INFINITY;
      sum[n] = 0.0f;
    }
    int key = first_key<PAGED>(P, cur.t, T);              // of the tile
    int in_page = PAGED ? P.page_size - key % P.page_size : 0;   // keys of its page from the tile on
    for (int i = i0; i < i1; ++i) {
      const int left = (PAGED ? min(in_page, cur.len - key) : cur.len - key) - wkey * 32;   // keys from this warp's first one on
      if (!PAGED) {
        key += T;
      } else {
        const int step = min(in_page, T);
        key += step;
        in_page -= step;
        if (in_page == 0) in_page = P.page_size;
      }
      float* sc = scores + (OWN ? 0 : buf) * SBUF;
      buf ^= 1;
      if (OWN) __syncwarp();

      // ---- scores of 16 keys over this warp's part of D
      if (alive) alive = all_waited(smem_u32(full_k + slot_k), lap_k, P, &abort_flag);
      if (i == i0) {                               // Q is here too: dealt out to the four lanes of a head
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int s = 0; s < 8; s += 2) {
            uint32_t r[4] = {qf[s][n][0], qf[s][n][1], qf[s + 1][n][0], qf[s + 1][n][1]};
            trade_words(r);
            qf[s][n][0] = r[0];
            qf[s][n][1] = r[1];
            qf[s + 1][n][0] = r[2];
            qf[s + 1][n][1] = r[3];
          }
      }
#pragma unroll
      for (int y = 0; y < (OWN ? 2 : 1); ++y) {
        const uint32_t a0 = (y ? k_at2 : k_at) + slot_k * stage;
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[n][j] = 0.0f;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          if (x >= kn) break;
          uint32_t a[4];
          ldm_x4((a0 + (x >> 2) * chunk_bytes) ^ ((x & 3) << 5), a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<F16>(s[n], a, qf[x][n]);
        }
        float* dst = sc + (part * HEADS + c2) * SPITCH + key0 + y * 16 + hq;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          dst[n * 8 * SPITCH] = s[n][0];
          dst[(n * 8 + 1) * SPITCH] = s[n][1];
          dst[n * 8 * SPITCH + 8] = s[n][2];
          dst[(n * 8 + 1) * SPITCH + 8] = s[n][3];
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(empty_k + slot_k));
      if (++slot_k == P.ring_k) {
        slot_k = 0;
        lap_k ^= 1u;
      }
      // The scores are complete (the next tile writes the other buffer).
      if (!OWN) named_bar_sync(1, N);

      // ---- P of this warp's keys, as the operand of the second product
      uint32_t pf[KSTEPS][NT][2], pr[KSTEPS][NT][2];   // and the rest of it
      float fac[NT];
      bool moved = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 x[2 * KSTEPS];
        float most = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2 * KSTEPS; ++j) {
          const float* src = sc + (n * 8 + hq) * SPITCH + wkey * 32 + j * 8 + c2;
          x[j] = *reinterpret_cast<const float2*>(src);
#pragma unroll
          for (int p = 1; p < PARTS; ++p) {
            const float2 w = *reinterpret_cast<const float2*>(src + p * HEADS * SPITCH);
            x[j].x += w.x;
            x[j].y += w.y;
          }
          x[j].x *= P.scale_log2;
          x[j].y *= P.scale_log2;
        }
        if (left < 16 * KSTEPS) {
#pragma unroll
          for (int j = 0; j < 2 * KSTEPS; ++j) {
            if (j * 8 + c2 >= left) x[j].x = -INFINITY;
            if (j * 8 + c2 + 1 >= left) x[j].y = -INFINITY;
          }
        }
#pragma unroll
        for (int j = 0; j < 2 * KSTEPS; ++j) most = fmax3(most, x[j].x, x[j].y);
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
        if (F16) most -= P_LIFT;
        const float now = fmaxf(top[n], most);
        const float base = now == -INFINITY ? 0.0f : now;
        fac[n] = ex2_approx(top[n] - base);
        moved |= now != top[n];
        top[n] = now;
        float add = 0.0f;
#pragma unroll
        for (int j = 0; j < 2 * KSTEPS; ++j) {
          x[j].x = ex2_approx(x[j].x - base);
          x[j].y = ex2_approx(x[j].y - base);
          add += x[j].x + x[j].y;
          split2<F16>(x[j].x, x[j].y, pf[j >> 1][n][j & 1], pr[j >> 1][n][j & 1]);
        }
        sum[n] = sum[n] * fac[n] + add;
      }
      if (__any_sync(~0u, moved)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float f0 = __shfl_sync(~0u, fac[n], c2 * 4), f1 = __shfl_sync(~0u, fac[n], c2 * 4 + 4);
#pragma unroll
          for (int s = 0; s < DT; ++s) {
            acc[s][n][0] *= f0;
            acc[s][n][1] *= f1;
            acc[s][n][2] *= f0;
            acc[s][n][3] *= f1;
          }
        }
      }

      // ---- this warp's columns += V^T P
      if (alive) alive = all_waited(smem_u32(full_v + slot_v), lap_v, P, &abort_flag);
      const bool tail = left < 16 * KSTEPS;        // rows behind the last key hold anything: zeros, not 0 * NaN
#pragma unroll
      for (int s = 0; s < DT; ++s) {
        if (s >= dn) break;
#pragma unroll
        for (int g = 0; g < KSTEPS; ++g) {
          uint32_t a[4];
          ldm_x4_trans(((g ? v_at2 : v_at) + slot_v * stage + (s >> 2) * chunk_bytes) ^ ((s & 3) << 5), a);
          if (tail) {
            const int k = g * 16 + c2;
            const uint32_t m0 = (k < left ? 0xffffu : 0u) | (k + 1 < left ? 0xffff0000u : 0u);
            const uint32_t m1 = (k + 8 < left ? 0xffffu : 0u) | (k + 9 < left ? 0xffff0000u : 0u);
            a[0] &= m0;
            a[1] &= m0;
            a[2] &= m1;
            a[3] &= m1;
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<F16>(acc[s][n], a, pf[g][n]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<F16>(acc[s][n], a, pr[g][n]);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(empty_v + slot_v));
      if (++slot_v == P.ring_v) {
        slot_v = 0;
        lap_v ^= 1u;
      }
    }

    // ---- the pair's sums: written (a whole pair), or left for the second launch (a cut one)
    const bool done = i1 - i0 == cur.tiles - cur.t;
    const bool whole = done && cur.t == 0;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (cur.t == 0 ? 1 : 0);
    float* part_o = P.part + slot * HEADS * P.D;
    float2* part_ml = P.part_ml + slot * HEADS;
    char* out = P.o + cur.b * P.o_sb + (int64_t)hq0 * P.o_sh;
    float* lse = P.lse + (int64_t)cur.b * P.Hq + hq0;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      sum[n] += __shfl_xor_sync(~0u, sum[n], 1);
      sum[n] += __shfl_xor_sync(~0u, sum[n], 2);
    }
    if (GROUPS == 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (whole) {
          const float inv = sum[n] == 0.0f ? 0.0f : 1.0f / sum[n];
          const float f0 = __shfl_sync(~0u, inv, c2 * 4), f1 = __shfl_sync(~0u, inv, c2 * 4 + 4);
#pragma unroll
          for (int s = 0; s < DT; s += 2)
            if (s < dn)
              write_columns<F16>(out + n * 8 * P.o_sh, P.o_sh, rows - n * 8, (d0 + s) * 16, P.D, acc[s][n], acc[s + 1][n], f0, f1);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int head = n * 8 + c2 + (j & 1), d = d0 * 16 + (j >> 1) * 8;
            const int some = (P.D - d + 8) / 16;       // column tiles with these 8 columns
            if (head >= rows) continue;
            float* to = part_o + head * P.D + d + hq;
#pragma unroll
            for (int s = 0; s < DT; ++s)
              if (s < some) to[s * 16] = acc[s][n][j];
          }
        }
        const int head = n * 8 + hq;
        if (wd == 0 && lane % 4 == 0 && head < rows) {
          if (!whole)
            part_ml[head] = make_float2(top[n], sum[n]);
          else if (P.lse)
            lse[head] = sum[n] == 0.0f ? -INFINITY : (top[n] + log2f(sum[n])) * 0.69314718055994531f;
        }
      }
    } else {
      // Every group leaves its sums where the scores were, as many heads at a
      // time as fit, and all threads join them two columns at a time.
      constexpr int RP = WDS * DT * 16 + 4, ROUND = decode_score_bytes(NT, T) / (GROUPS * RP * 4);
      static_assert(ROUND >= 1, "a head's sums fit");
      const int half_d = P.D / 2;
#pragma unroll 1
      for (int r0 = 0; r0 < rows; r0 += ROUND) {
        const int rn = min(ROUND, rows - r0);
        named_bar_sync(1, N);                      // the scores (the last heads' sums) are read
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (r0 == 0 && wd == 0 && lane % 4 == 0) ml_s[wkey][n * 8 + hq] = make_float2(top[n], sum[n]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = n * 8 + c2 + (j & 1) - r0;
            if (row < 0 || row >= rn) continue;
            float* to = scores + (wkey * ROUND + row) * RP + d0 * 16 + hq + (j >> 1) * 8;
#pragma unroll
            for (int s = 0; s < DT; ++s)
              if (s < dn) to[s * 16] = acc[s][n][j];
          }
        }
        named_bar_sync(1, N);
        for (int x = tid; x < rn * half_d; x += N) {
          const int r = x / half_d, d = (x - r * half_d) * 2, row = r0 + r;
          float m = -INFINITY, l = 0.0f;
#pragma unroll
          for (int g = 0; g < GROUPS; ++g) m = fmaxf(m, ml_s[g][row].x);
          const float base = m == -INFINITY ? 0.0f : m;
          float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int g = 0; g < GROUPS; ++g) {
            const float2 ml = ml_s[g][row];
            const float f = ex2_approx(ml.x - base);
            const float2 v = *reinterpret_cast<const float2*>(scores + (g * ROUND + r) * RP + d);
            l += f * ml.y;
            o.x += f * v.x;
            o.y += f * v.y;
          }
          if (whole) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            *reinterpret_cast<uint32_t*>(out + row * P.o_sh + d * 2) = pack2<F16>(o.x * inv, o.y * inv);
            if (d == 0 && P.lse) lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
          } else {
            *reinterpret_cast<float2*>(part_o + (int64_t)row * P.D + d) = o;
            if (d == 0) part_ml[row] = make_float2(m, l);
          }
        }
      }
      named_bar_sync(1, N);                        // before the next pair's scores
    }
    i0 = i1;
    cur = next_s[turn];
  }
}

// Joins the partial sums of the pairs cut between CTAs.  A pair over n CTAs is
// joined by n blocks, one for each of its CTAs, 128 columns of a head at a time:
// by a warp each where n is small (most often 2), by the warps of a block, a
// share of the CTAs each, where it is large.  The order of the sums is fixed.
// The kernel is one chain of latencies (the cut, the sums, the store), so it has
// no division and no sum over lanes: 2 us of one request of 777 keys, against 4 us
// for a block of 512 threads a head, and 2 to 3 us of batches of 110 requests,
// against 4 to 7 us.  With a warp for up to 16 CTAs, 5 requests of up to 208 keys,
// 64 heads of 1024, take 4 us less than for up to 4; for up to 32 CTAs the request
// of 777 keys takes 2.4 us more.
constexpr int JOIN_WARPS = 8, JOIN_FEW = 16;

struct Joined {
  float top, l;
  float4 a;
  __device__ __forceinline__ void rescale(float t) {
    const float f = ex2_approx(top - (t == -INFINITY ? 0.0f : t));
    top = t;
    l *= f;
    a.x *= f;
    a.y *= f;
    a.z *= f;
    a.w *= f;
  }
  __device__ __forceinline__ void add(float2 ml, const float4& x) {   // (behind rescale)
    const float f = ex2_approx(ml.x - (top == -INFINITY ? 0.0f : top));
    l += f * ml.y;
    a.x += f * x.x;
    a.y += f * x.y;
    a.z += f * x.z;
    a.w += f * x.w;
  }
};

// Sums i, i + stride, .. of the pair, at most N below n, heads rows apart.
// The first CTA's sums are its second partial pair, the others' their first.
template <int N>
__device__ __forceinline__ void join_add(Joined& s, const float2* mls, const float* from, int heads, int D, int i, int stride, int n) {
  mls += (2 * i + (i == 0)) * heads;
  from += (2 * i + (i == 0)) * heads * D;
  const int step = 2 * stride * heads, first = i == 0 ? heads : 0;
  float2 ml[N];
  float4 x[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    ml[k] = make_float2(-INFINITY, 0.0f);
    x[k] = make_float4(0, 0, 0, 0);
    if (i + k * stride < n) {
      const int at = k == 0 ? 0 : k * step - first;
      ml[k] = mls[at];
      x[k] = *reinterpret_cast<const float4*>(from + at * D);
    }
  }
  float t = s.top;
#pragma unroll
  for (int k = 0; k < N; ++k) t = fmaxf(t, ml[k].x);
  s.rescale(t);
#pragma unroll
  for (int k = 0; k < N; ++k) s.add(ml[k], x[k]);
}

template <bool F16>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4) join_kernel(const __grid_constant__ DecodeParams P, int heads, int log_rows) {
  __shared__ float4 acc_s[JOIN_WARPS][32];
  __shared__ float2 ml_s[JOIN_WARPS];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tasks = (P.D + 127) / 128 << log_rows;
  dependency_wait();
  const int4 m = P.cuts[blockIdx.x];
  const int n = m.x >> 16, first = m.x & 0xffff;   // CTAs of the pair
  if (n == 0) return;
  const bool few = n <= JOIN_FEW;
  const int mine = blockIdx.x / 2 - first;
  for (int task = few ? mine * JOIN_WARPS + warp : mine; task < tasks; task += few ? n * JOIN_WARPS : n) {
    const int row = task & ((1 << log_rows) - 1), col = (task >> log_rows) * 128 + lane * 4;
    if (row >= m.y) continue;
    const float2* mls = P.part_ml + 2 * first * heads + row;
    const float* from = P.part + (int64_t)(2 * first * heads + row) * P.D + min(col, P.D - 4);
    Joined s{-INFINITY, 0.0f, make_float4(0, 0, 0, 0)};
    if (n == 2) {
      join_add<2>(s, mls, from, heads, P.D, 0, 1, n);
    } else if (few) {
      for (int i = 0; i < n; i += 4) join_add<4>(s, mls, from, heads, P.D, i, 1, n);
    } else {
      for (int i = warp; i < n; i += 4 * JOIN_WARPS) join_add<4>(s, mls, from, heads, P.D, i, JOIN_WARPS, n);
      acc_s[warp][lane] = s.a;
      if (lane == 0) ml_s[warp] = make_float2(s.top, s.l);
      __syncthreads();
      if (warp == 0) {
        float t = s.top;
        for (int w = 1; w < JOIN_WARPS; ++w) t = fmaxf(t, ml_s[w].x);
        s.rescale(t);
        for (int w = 1; w < JOIN_WARPS; ++w) s.add(ml_s[w], acc_s[w][lane]);
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    const int64_t hq = m.w + row;
    const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;
    if (col < P.D)
      *reinterpret_cast<uint2*>(P.o + m.z * P.o_sb + hq * P.o_sh + col * 2) =
          make_uint2(pack2<F16>(s.a.x * inv, s.a.y * inv), pack2<F16>(s.a.z * inv, s.a.w * inv));
    if (P.lse && col == 0)
      P.lse[(int64_t)m.z * P.Hq + hq] = s.l == 0.0f ? -INFINITY : (s.top + log2f(s.l)) * 0.69314718055994531f;
  }
}

// Workspace: partial outputs, their maxima and sums, the cut pairs.
struct DecodeSpace {
  size_t part, ml, cuts, total;
};
DecodeSpace decode_space(int grid, int heads, int D) {
  DecodeSpace s;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  s.part = 0;
  s.ml = up((size_t)2 * grid * heads * D * 4);
  s.cuts = s.ml + up((size_t)2 * grid * heads * 8);
  s.total = s.cuts + up((size_t)2 * grid * sizeof(int4));
  return s;
}

template <bool F16, int NT, int T>
ffpa_status launch_decode_as(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  const auto fn = P.page_tiles ? &decode_kernel<F16, NT, T, true> : &decode_kernel<F16, NT, T, false>;
  const ffpa_status st = set_smem_attr_once(reinterpret_cast<const void*>(fn), dev, (int)pl.smem);
  if (st != FFPA_OK) return st;
  fn<<<grid, DEC_THREADS, pl.smem, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return FFPA_ERR_CUDA;
  const int heads = 8 * NT;
  int log_rows = 0;
  while ((1 << log_rows) < (P.group < heads ? P.group : heads)) ++log_rows;
  // A dependent launch: its blocks are set up while the first kernel runs out.
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * grid);
  cfg.blockDim = dim3(JOIN_WARPS * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, join_kernel<F16>, P, heads, log_rows) != cudaSuccess) {
    cudaGetLastError();
    return FFPA_ERR_CUDA;
  }
  return FFPA_OK;
}

template <bool F16, int T>
ffpa_status launch_decode_tile(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  return pl.nt == 1 ? launch_decode_as<F16, 1, T>(P, pl, grid, dev, stream)
                    : launch_decode_as<F16, 2, T>(P, pl, grid, dev, stream);
}

template <bool F16>
ffpa_status launch_decode(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  switch (pl.tile) {
    case 16: return launch_decode_tile<F16, 16>(P, pl, grid, dev, stream);
    case 32: return launch_decode_tile<F16, 32>(P, pl, grid, dev, stream);
    case 64: return launch_decode_tile<F16, 64>(P, pl, grid, dev, stream);
    case 128: return launch_decode_tile<F16, 128>(P, pl, grid, dev, stream);
    default: return launch_decode_tile<F16, 256>(P, pl, grid, dev, stream);
  }
}

}  // namespace
}  // namespace ffpa

extern "C" {

size_t ffpa_decode_paged_workspace_bytes(int Hq, int Hkv, int D) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 64 || D > 1024 || D % 8 != 0) return 0;
  const int nt = ffpa::decode_nt(Hq / Hkv);
  return ffpa::decode_space(ffpa::DEC_SMS_MAX * ffpa::decode_ctas(nt), 8 * nt, D).total;
}

ffpa_status ffpa_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                              ffpa_dtype dt, int B, int Hq, int Hkv, int D, int num_pages, int page_size,
                              int max_pages, const int64_t q_str[3], const int64_t k_str[4],
                              const int64_t v_str[4], const int64_t o_str[3], const int32_t* block_table,
                              int64_t table_str, const int32_t* seq_lens, const float* scale, int enable_gqa,
                              void* workspace, size_t workspace_bytes, ffpa_stream_t stream,
                              const ffpa_options* options) {
  using namespace ffpa;
  if (dt != FFPA_BF16 && dt != FFPA_FP16) return FFPA_ERR_DTYPE;
  if (B < 0 || Hq < 1 || Hkv < 1 || num_pages < 0 || page_size < 1 || max_pages < 0) return FFPA_ERR_INVALID;
  if (D < 64 || D > 1024 || D % 8 != 0) return FFPA_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0 || (Hq != Hkv && !enable_gqa)) return FFPA_ERR_INVALID;
  if ((long long)max_pages * page_size > 0x7fff0000LL) return FFPA_ERR_INVALID;   // key numbers are int32
  const float sc = scale ? *scale : 1.0f / std::sqrt(static_cast<float>(D));
  if (!std::isfinite(sc)) return FFPA_ERR_INVALID;
  if (B == 0) return FFPA_OK;
  if (!q || !o || !seq_lens || !workspace || !q_str || !k_str || !v_str || !o_str) return FFPA_ERR_INVALID;
  const bool held = num_pages > 0 && max_pages > 0;
  if (held && (!k_cache || !v_cache || !block_table)) return FFPA_ERR_INVALID;
  if (!rows_ok(q_str, {B, Hq, D}) || !rows_ok(o_str, {B, Hq, D})) return FFPA_ERR_INVALID;
  if (held && (!rows_ok(k_str, {num_pages, page_size, Hkv, D}) || !rows_ok(v_str, {num_pages, page_size, Hkv, D})))
    return FFPA_ERR_INVALID;
  if (held && B > 1 && table_str < max_pages) return FFPA_ERR_INVALID;
  if (!on_boundary(q, 16) || !on_boundary(o, 16) || !on_boundary(lse, 4) || !on_boundary(seq_lens, 4) ||
      !on_boundary(workspace, 256))
    return FFPA_ERR_INVALID;
  if (held && (!on_boundary(k_cache, 16) || !on_boundary(v_cache, 16) || !on_boundary(block_table, 4)))
    return FFPA_ERR_INVALID;
  const DecodePlan pl = decode_plan(D, Hq / Hkv);
  if (workspace_bytes < ffpa_decode_paged_workspace_bytes(Hq, Hkv, D)) return FFPA_ERR_INVALID;
  if ((long long)B * Hkv * pl.head_tiles > 0x7fffffffLL) return FFPA_ERR_INVALID;
  int dev = 0;
  ffpa_status st = call_device({q, o, lse, seq_lens, workspace, held ? k_cache : nullptr, held ? v_cache : nullptr,
                                held ? (const void*)block_table : nullptr},
                               &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  int* err = nullptr;
  int sms = 0;
  if ((st = call_status(dev, options, &err, &sms)) != FFPA_OK) return st;
  const int grid = (sms < DEC_SMS_MAX ? sms : DEC_SMS_MAX) * pl.ctas;

  DecodeParams P{};
  P.q = static_cast<const char*>(q);
  P.k = static_cast<const char*>(k_cache);
  P.v = static_cast<const char*>(v_cache);
  P.o = static_cast<char*>(o);
  P.lse = lse;
  P.table = block_table;
  P.lens = seq_lens;
  const DecodeSpace sp = decode_space(grid, 8 * pl.nt, D);
  char* ws = static_cast<char*>(workspace);
  P.part = reinterpret_cast<float*>(ws + sp.part);
  P.part_ml = reinterpret_cast<float2*>(ws + sp.ml);
  P.cuts = reinterpret_cast<int4*>(ws + sp.cuts);
  P.err = err;
  P.q_sb = q_str[0] * 2;
  P.q_sh = q_str[1] * 2;
  P.o_sb = o_str[0] * 2;
  P.o_sh = o_str[1] * 2;
  if (held) {
    P.k_sp = k_str[0] * 2;
    P.k_ss = k_str[1] * 2;
    P.k_sh = k_str[2] * 2;
    P.v_sp = v_str[0] * 2;
    P.v_ss = v_str[1] * 2;
    P.v_sh = v_str[2] * 2;
  }
  P.table_str = table_str;
  P.B = B;
  P.Hq = Hq;
  P.Hkv = Hkv;
  P.group = Hq / Hkv;
  P.D = D;
  P.head_tiles = pl.head_tiles;
  P.num_pages = num_pages;
  P.page_size = page_size;
  P.max_pages = held ? max_pages : 0;   // without pages every request is empty
  P.chunks = pl.chunks;
  // Boxes of as many rows as divide a page, down to the 8 of the swizzle.  Where a
  // page's size is no multiple of 8 but fills enough of a tile, a tile is one box that
  // ends with its page (B32 Hkv8 D512 of 4096 keys, pages of 100: 321 us, in pieces
  // 454); smaller pages of that kind come in pieces.  "Enough" is where both cost the
  // same: a half (that case with pages of 12, of 32 keys a tile: 580 us, in pieces 455), and a
  // third of the tiles of 128 and 256 keys (B64 Hkv2 D64 of 3000 keys, pages of 100: 34 us, in
  // pieces 45; D128 of 2000 keys, pages of 36: 51, 45).
  const bool by_page = page_size % 8 != 0 && page_size > (pl.tile - 1) / (pl.tile >= 128 ? 3 : 2);
  P.boxed = held && (page_size % 8 == 0 || by_page);
  P.page_tiles = by_page ? (page_size + pl.tile - 1) / pl.tile : 0;
  P.box_rows = pl.tile;
  P.box_chunks = D % 64 == 0 ? pl.chunks : 1;
  if (P.boxed) {
    while (!by_page && page_size % P.box_rows != 0) P.box_rows /= 2;
    for (int i = 0; i < 2; ++i) {
      // (bytes; a dimension of one entry may have any stride, a tensor map takes multiples of 16)
      const int64_t* of = i ? v_str : k_str;
      const uint64_t row = (uint64_t)of[1] * 2, one = (uint64_t)D * 2;
      const uint64_t head = Hkv > 1 ? (uint64_t)of[2] * 2 : one, page = num_pages > 1 ? (uint64_t)of[0] * 2 : one;
      CUtensorMap* map = i ? &P.map_v : &P.map_k;
      const void* base = i ? v_cache : k_cache;
      if (P.box_chunks > 1) {
        const uint64_t dims[5] = {64, (uint64_t)page_size, (uint64_t)pl.chunks, (uint64_t)Hkv, (uint64_t)num_pages};
        const uint64_t str[4] = {row, 128, head, page};
        const uint32_t box[5] = {64, (uint32_t)P.box_rows, (uint32_t)pl.chunks, 1, 1};
        st = encode_rows(map, dt, 5, base, dims, str, box);
      } else {
        const uint64_t dims[4] = {(uint64_t)D, (uint64_t)page_size, (uint64_t)Hkv, (uint64_t)num_pages};
        const uint64_t str[3] = {row, head, page};
        const uint32_t box[4] = {64, (uint32_t)P.box_rows, 1, 1};
        st = encode_rows(map, dt, 4, base, dims, str, box);
      }
      if (st != FFPA_OK) return st;
    }
  }
  P.ring_k = pl.ring_k;
  P.ring_v = pl.ring_v;
  P.timeout_ns = options && options->wait_timeout_ns ? options->wait_timeout_ns : 2000000000ull;
  P.drop = options && options->test_drop_first_copy ? 1 : 0;
  P.scale_log2 = sc * 1.4426950408889634f;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FFPA_FP16 ? launch_decode<true>(P, pl, grid, dev, s) : launch_decode<false>(P, pl, grid, dev, s);
}

}  // extern "C"
