#pragma once
// Attention of one new token per request over a paged key/value cache: the
// kernels and the checks of its entry points (ffpa_decode.cu: a cache of 16-bit
// values; ffpa_decode_fp8.cu: of e4m3 codes with a scale for each row;
// ffpa_shared.cu: the requests' own keys behind pages that all of them share).
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
// With e4m3 codes a tile has as many bytes and twice the keys.  The codes become fp16 between the matrix
// load and the product: its 32 bits a lane are four columns of a key (the first product's queries
// are permuted to match), transposed two neighbouring columns of two keys (and so are the outputs).  The
// keys' scales multiply the scores; the values' scales the weights, which have a unit of their own
// so that a row's scale may be anything.  B32 Hkv8 D512 of up to 8192 keys: 197 us, 6.3 TB/s; B64 Hkv8 D128 of
// 4000 keys: 97 us, 5.6 TB/s; B128 Hkv16 D128 of up to 2048 keys: 120 us, 4.4 TB/s (a tile's chain).
//
// Every wait on a copy has a time limit, after which the call's status word
// receives FFPA_ERR_DEVICE_TIMEOUT and the CTA runs out without waiting.
#include "ffpa_paged.cuh"

namespace ffpa {

// What a kernel reads and writes.
enum DecodeKind {
  DECODE_16 = 0,    // a 16-bit cache
  DECODE_E4M3 = 1,  // e4m3 codes and fp32 scales
  DECODE_OWN = 2    // a 16-bit cache behind the shared pages; normalised fp32 outputs for the merge
};
__host__ __device__ constexpr int cache_bytes(int kind) { return kind == DECODE_E4M3 ? 1 : 2; }

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
  const float *ks, *vs;                 // e4m3: scales [page][head][slot], element strides
  int64_t ks_sp, ks_sh, vs_sp, vs_sh;
  int scale4;                           // four slots' scales are 16 bytes on a boundary
  const int32_t* shared_len;            // own keys (and 16 bits, else 0): keys that all requests share, in whole pages
  const int32_t* shared_table;          // their pages
  int shared_pages;                     // at most so many of them
  float* o32;                           // own keys: [B][Hq][D] outputs
  unsigned long long timeout_ns;
  int B, Hq, Hkv, group, D, head_tiles;
  int num_pages, page_size, max_pages;
  int chunks;       // 128-byte chunks of a row
  int boxed;        // tiles arrive as tensor boxes
  int page_tiles;   // tiles of a page where a tile ends with its page, else 0
  int box_rows;     // rows of a box (all T where not boxed), a power of two >= 8
  int box_chunks;   // chunks of a box: all, or 1 when D ends inside a chunk
  int ring_k, ring_v, drop;
  float scale_log2;
};

struct DecodeShape {
  int B, Hq, Hkv, D, num_pages, page_size, max_pages;
  const int64_t *k_str, *v_str;
  bool held() const { return num_pages > 0 && max_pages > 0; }
};

// Decode over a 16-bit cache with P's pointers set (ffpa_decode.cu); shared_len, shared_table and shared_pages name
// pages that stand before every request's own, or are 0.
ffpa_status run_decode_16(DecodeParams& P, const DecodeShape& s, ffpa_dtype dt, float sc, int sms, int dev, char* ws,
                          const ffpa_options* options, cudaStream_t stream);

namespace {

constexpr int DEC_WARPS = 8;          // that multiply
constexpr int DEC_THREADS = (DEC_WARPS + 2) * 32;   // and one each that brings K and V
constexpr int DEC_RING_MAX = 8;       // tiles of K (and of V) in the ring
// Powers of two above the maximum at which fp16 forms its exponentials: the largest is
// 2^15, and 2^-39 of it is the smallest that counts.
constexpr float P_LIFT = 15.0f;
// SMs of any sm_103 part; the workspace is sized for them without asking a device.
constexpr int DEC_SMS_MAX = 160;

// Sizes of one call.  A tile has T = 16 keys for rows of more than 1 KB and twice as many each
// time they halve (at most 32 KB).
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
// Column tiles of a warp in the second product (e4m3: twice the columns, as its tiles hold twice the keys).
__host__ __device__ constexpr int decode_columns(int kind, int tile) { return kind == DECODE_E4M3 || tile < 32 ? 8 : 4; }
// A head's sums of all groups of warps, as they are joined at a pair's end.
__host__ __device__ constexpr size_t decode_join_bytes(int kind, int tile) {
  return (size_t)decode_groups(tile) * (DEC_WARPS / decode_groups(tile) * decode_columns(kind, tile) * 16 + 4) * 4;
}
// (e4m3: room for the sums of eight heads where the ring leaves it, else four.)
__host__ __device__ constexpr size_t decode_score_bytes(int kind, int nt, int tile) {
  const size_t scores = (size_t)(decode_own_keys(tile) ? 1 : 2) * decode_parts(tile) * 8 * nt * (tile + 8) * 4;
  const size_t join = kind == DECODE_E4M3 && tile >= 64 ? decode_join_bytes(kind, tile) * (tile >= 128 ? 8 : 4) : 0;
  return ((scores > join ? scores : join) + 1023) / 1024 * 1024;
}
// e4m3: the queries of a pair as operands of the first product, 16 bytes a lane for 32 columns, and their units.
__host__ __device__ constexpr size_t decode_query_bytes(int nt, int D) { return ((size_t)(D + 31) / 32 * nt * 512 + 64 * nt + 1023) / 1024 * 1024; }

DecodePlan decode_plan(int D, int group, int kind) {
  DecodePlan p;
  p.nt = decode_nt(group);
  p.ctas = decode_ctas(p.nt);
  p.head_tiles = (group + 8 * p.nt - 1) / (8 * p.nt);
  const int row = D * cache_bytes(kind);
  p.tile = row > 1024 ? 16 : row > 512 ? 32 : row > 256 ? 64 : row > 128 ? 128 : 256;
  p.chunks = (row + 127) / 128;
  const size_t fixed = decode_score_bytes(kind, p.nt, p.tile) + (kind == DECODE_E4M3 ? decode_query_bytes(p.nt, D) : 0);
  const size_t stage = (size_t)p.tile * (p.chunks * 128 + (kind == DECODE_E4M3 ? 4 : 0));
  // 8 KB a CTA stay for static shared memory, the alignment of the boxes, the system,
  // and a block of the joining kernel that is set up early (with 4 KB left 1 us more).
  int n = static_cast<int>((SMEM_LIMIT / p.ctas - 8192 - fixed) / stage);
  if (n > 2 * DEC_RING_MAX) n = 2 * DEC_RING_MAX;
  p.ring_v = n / 2;
  p.ring_k = kind == DECODE_E4M3 ? n / 2 : n - n / 2;   // (e4m3: filled in turn)
  p.smem = 1024 + fixed + (size_t)(p.ring_k + p.ring_v) * stage;
  return p;
}

// A place on the line of tiles: tile t of `tiles` of pair u of request b.
struct Place {
  int b, u, t, tiles, len;
};

// Keys of a request behind the `skip` pages that are shared; all of one that ends among those.
__device__ __forceinline__ int clamped_len(const DecodeParams& P, int n, int skip) {
  const long long cap = (long long)P.max_pages * P.page_size;
  n = n < 0 ? 0 : n > cap ? (int)cap : n;
  return n < skip * P.page_size ? n : n - skip * P.page_size;
}
// Page j of those keys (16 bits: of all keys of a request, the first of them in the shared pages).
template <int KIND>
__device__ __forceinline__ int page_of(const DecodeParams& P, int b, int j, int shared) {
  const int32_t* t = P.table + b * P.table_str;
  if (KIND == DECODE_16 && j < shared) t = P.shared_table;
  if (KIND == DECODE_OWN) t = shared > 0 && P.lens[b] < shared * P.page_size ? P.shared_table : t + shared;
  return t[j];
}
// A length out of range.
__device__ __forceinline__ bool bad_len(const DecodeParams& P, int n) { return n < 0 || n > (long long)P.max_pages * P.page_size; }

// The pages that all requests share, of which only whole ones count.
template <int KIND>
__device__ __forceinline__ int pages_shared(const DecodeParams& P) {
  if (KIND == DECODE_E4M3 || !P.shared_len) return 0;
  const int n = *P.shared_len;
  return n < 0 ? 0 : min(n / P.page_size, min(P.shared_pages, P.max_pages));
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
__device__ __forceinline__ void advance(const DecodeParams& P, int pairs, Place& p, int T, int skip) {
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
    p.len = clamped_len(P, P.lens[p.b], skip);
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

// The scales of `per` keys (or values) of a page, of which `there` exist: zeros for the others.
__device__ __forceinline__ void copy_scales(const DecodeParams& P, bool is_v, uint32_t dst, int there, int per, int page, int head, int in_page) {
  const float* src = is_v ? P.vs : P.ks;
  if (there > 0) src += page * (is_v ? P.vs_sp : P.ks_sp) + head * (is_v ? P.vs_sh : P.ks_sh) + in_page;
  if (per == 4)
    copy16_async(dst, src, there <= 0 ? 0 : min(there, 4) * 4);
  else
    copy4_async(dst, src, there > 0 ? 4 : 0);
}

// K (or V) tiles of the run as tensor boxes, a box a lane, its page looked up
// one tile ahead.  A page that does not exist, and rows that belong to no key,
// have a coordinate behind the last page: the copy writes zeros there.
template <int KIND, bool PAGED>
__device__ __forceinline__ void produce_boxes(const DecodeParams& P, int T, int heads, bool is_v, int skip, int shared, Place at,
                                              const Run& run, uint32_t ring, int slots, uint64_t* full, uint64_t* empty,
                                              volatile int* abort_flag) {
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
      page = page_of<KIND>(P, p.b, j, shared);
    }
  };
  // L2 fetches 256 bytes at a time: where a head's row is shorter, the next head's comes with it and has to stay
  // until it is asked for (loads that leave first, B32 Hq64 Hkv2 D64 of 8192 keys 63 -> 79 us, B8 Hkv8 D64 of 16666 64 -> 70).
  const bool alone = P.Hkv == 1 || P.D * cache_bytes(KIND) >= 256;
  const uint64_t once = once_policy();
  look_up(at);
  int slot = 0, i = 0;
  uint32_t lap = 0;
  for (; i < n_tiles; ++i) {
    const int head = at.u / P.head_tiles;
    const bool good = page >= 0 && page < P.num_pages;
    if (keyed && !good) report_invalid(P.err);
    const int y = good ? in_page : 0, z = good ? page : P.num_pages;
    if (is_v && lane == 0 && (at.t == 0 || i == 0)) note_cut(P, at, run, i, heads);
    advance<PAGED>(P, pairs, at, T, skip);
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
      if (P.box_chunks == 1 && alone)
        tma_load_4d(dst, map, bar, chunk * 64, y, head, z, once);
      else if (P.box_chunks == 1)
        tma_load_4d(dst, map, bar, chunk * 64, y, head, z);
      else
        tma_load_5d(dst, map, bar, 0, y, 0, head, z, once);
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

// e4m3: the same by two warps, each with half of the rows of every K and V tile (and their scales, which an
// arrival of every lane reports): the pages are looked up once for both, and a tile of small pages, whose boxes an
// SM starts one in 85 cycles a warp, is on its way in half the time (B128 Hkv16 D128, pages of 16, with a warp for K
// and one for V: 121 us).
template <bool PAGED>
__device__ __forceinline__ void produce_halves(const DecodeParams& P, int T, int heads, int half, Place at, const Run& run,
                                               uint32_t ring_k, uint32_t ring_v, uint32_t scale_k, uint32_t scale_v,
                                               uint64_t* full_k, uint64_t* full_v, uint64_t* empty_k, uint64_t* empty_v,
                                               volatile int* abort_flag) {
  const int lane = threadIdx.x % 32, pairs = P.Hkv * P.head_tiles, n_tiles = run.n, slots = P.ring_k;
  const int per_row = P.chunks / P.box_chunks;
  const int boxes = T / P.box_rows;                 // one: the first warp's
  const int mine_n = boxes > 1 ? boxes / 2 : half == 0 ? 1 : 0, row0 = boxes > 1 ? half * (T / 2) : 0;
  const int row = row0 + lane / per_row * P.box_rows, chunk = lane % per_row;
  const bool mine = lane < mine_n * per_row;
  const uint32_t box_bytes = P.box_rows * P.box_chunks * 128, stage = T * P.chunks * 128;
  const uint32_t to = row * P.chunks * 128 + chunk * box_bytes, bytes = mine_n * per_row * box_bytes;
  // Rows whose scales this warp brings, and the row of the page that this lane knows (as many as boxes, or one).
  const int s0 = half * (T / 2), per = !PAGED && P.scale4 ? 4 : 1;
  const int known = boxes > 1 ? row : 0;
  int page = -1, in_page = 0;
  bool keyed = false;
  auto look_up = [&](const Place& p) {
    const int key = first_key<PAGED>(P, p.t, T) + known;
    keyed = (boxes > 1 ? mine : true) && key < p.len;
    page = -1;
    in_page = 0;
    if (keyed) {
      const int j = key / P.page_size;
      in_page = key - j * P.page_size;
      page = P.table[p.b * P.table_str + j];
    }
  };
  const uint64_t once = once_policy();
  look_up(at);
  int slot = 0, i = 0;
  uint32_t lap = 0;
  bool alive = true, v_missing = false;
  for (; i < n_tiles; ++i) {
    const int head = at.u / P.head_tiles;
    const bool good = page >= 0 && page < P.num_pages;
    if (keyed && !good) report_invalid(P.err);
    const int y = good ? in_page : 0, z = good ? page : P.num_pages;
    if (half && lane == 0 && (at.t == 0 || i == 0)) note_cut(P, at, run, i, heads);
    const int key0 = first_key<PAGED>(P, at.t, T);
    int keys = at.len - key0;
    if (PAGED) keys = min(keys, P.page_size - key0 % P.page_size);
    advance<PAGED>(P, pairs, at, T, 0);
    if (i + 1 < n_tiles) {
      look_up(at);
      if (half && at.t == 0) fetch_queries(P, at, heads);
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      uint64_t* empty = v ? empty_v : empty_k;
      alive = all_waited(smem_u32(empty + slot), lap ^ 1u, P, abort_flag) && !P.drop;
      if (!alive) {
        v_missing = v;
        break;
      }
      const uint32_t bar = smem_u32((v ? full_v : full_k) + slot);
      if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
      __syncwarp();
      if (mine) {
        const uint32_t dst = (v ? ring_v : ring_k) + slot * stage + to;
        const CUtensorMap* map = v ? &P.map_v : &P.map_k;
        if (P.box_chunks == 1)
          tma_load_4d(dst, map, bar, chunk * 128, y, head, z, once);
        else
          tma_load_5d(dst, map, bar, 0, y, 0, head, z, once);
      }
      for (int r0 = s0; r0 < s0 + T / 2; r0 += 32 * per) {
        const int r = r0 + lane * per, in = min(r, s0 + T / 2 - 1);
        const int owner = boxes > 1 ? (in - row0) / P.box_rows * per_row : 0, in_box = boxes > 1 ? r % P.box_rows : r;
        const int rz = __shfl_sync(~0u, z, owner), ry = __shfl_sync(~0u, y, owner) + in_box;
        if (r < s0 + T / 2)
          copy_scales(P, v, (v ? scale_v : scale_k) + (slot * T + r) * 4, rz < P.num_pages ? keys - r : 0, per, rz, head, ry);
      }
      copy_arrive(bar);
    }
    if (!alive) break;
    if (++slot == slots) {
      slot = 0;
      lap ^= 1u;
    }
  }
  // Copies still in flight land before the CTA ends: the tiles before this one, and its K where only V is missing.
  if (v_missing) wait_drain(smem_u32(full_k + slot), lap, P.timeout_ns, P.err);
  for (int j = i < slots ? i : slots; j > 0; --j) {
    if (slot == 0) {
      slot = slots;
      lap ^= 1u;
    }
    --slot;
    wait_drain(smem_u32(full_k + slot), lap, P.timeout_ns, P.err);
    wait_drain(smem_u32(full_v + slot), lap, P.timeout_ns, P.err);
  }
}

// The same tile for any page size: the warp looks its rows up lane by lane,
// one tile ahead, and copies them in pieces of 16 bytes, a power of two of
// lanes to a row.  A row without a key, or of a page that does not exist,
// becomes zeros.
template <int KIND>
__device__ __forceinline__ void produce_pieces(const DecodeParams& P, int T, int heads, bool is_v, int skip, int shared, Place at,
                                               const Run& run, uint32_t ring, uint32_t scale_ring, int slots, uint64_t* full,
                                               uint64_t* empty, volatile int* abort_flag) {
  const int lane = threadIdx.x % 32, pairs = P.Hkv * P.head_tiles, n_tiles = run.n;
  const int cpr = P.D * cache_bytes(KIND) / 16;    // pieces of a row
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
      page[j] = r < T && key < p.len ? page_of<KIND>(P, p.b, key / P.page_size, shared) : -1;
    }
  };
  look_up(at);
  int slot = 0;
  uint32_t lap = 0;
  for (int i = 0; i < n_tiles; ++i) {
    // Offsets of this tile's rows (-1: zeros), then the pages of the next.
    const int hk = at.u / P.head_tiles;
    const char* head = base + hk * sh;
    int64_t from[8];
    int scale_page[8], scale_at[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      from[j] = -1;
      if (32 * j >= T) break;
      const int r = lane + 32 * j, key = at.t * T + r;
      if (r < T && key < at.len) {
        if (page[j] >= 0 && page[j] < P.num_pages) {
          from[j] = page[j] * sp + key % P.page_size * ss;
          if (KIND == DECODE_E4M3) {
            scale_page[j] = page[j];
            scale_at[j] = key % P.page_size;
          }
        } else {
          report_invalid(P.err);
        }
      }
    }
    if (is_v && lane == 0 && (at.t == 0 || i == 0)) note_cut(P, at, run, i, heads);
    advance<false>(P, pairs, at, T, skip);
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
      if (KIND == DECODE_E4M3 && lane < end)
        copy_scales(P, is_v, scale_ring + (slot * T + 32 * j + lane) * 4, from[j] >= 0, 1, scale_page[j], hk, scale_at[j]);
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

// One head's queries as fp16 operands of the first product with e4m3 keys, by a warp: of
// 32 columns, lane 4 head + c of a matrix load gets columns 4 c .. 4 c + 3 of either half; the
// first two of each are column pair c of one step of 16, the others of the next.  bf16 queries
// come in units of a power of two that lifts the largest of the row to 2^14 .. 2^15: exact from 2^-31 of it on
// and off by 2^-39 of it below.
template <bool F16>
__device__ __forceinline__ void bring_queries(const char* q, bool there, int D, char* query_s, int step, int head, float* unit) {
  const int lane = threadIdx.x % 32;
  uint4 x[4];
  float most = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = (i * 32 + lane) * 8;
    x[i] = there && d < D ? *reinterpret_cast<const uint4*>(q + d * 2) : make_uint4(0, 0, 0, 0);
  }
  if (!F16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = unpack2<false>(w[j]);
        most = fmax3(most, fabsf(y.x), fabsf(y.y));
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  }
  const int e = min(max((int)(__float_as_uint(most) >> 23), 16), 254);
  const float up = __uint_as_float((268 - e) << 23);
  if (lane == 0) *unit = F16 ? 1.0f : __uint_as_float((e - 14) << 23);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = (i * 32 + lane) * 8;               // columns d .. d + 7: c = 0, 1 or 2, 3 of a half
    if (d >= (D + 31) / 32 * 32) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h = w[j];
      if (!F16) {
        const float2 y = unpack2<false>(h);
        h = pack_f16(y.x * up, y.y * up);
      }
      const int c = d % 16 / 4 + j / 2;
      *reinterpret_cast<uint32_t*>(query_s + d / 32 * step + (head * 4 + c) * 16 + (j % 2 * 2 + d % 32 / 16) * 4) = h;
    }
  }
}

// Two column tiles as they come of e4m3 values (a lane holds columns 2 r and 2 r + 1
// of a tile, r = lane / 4, in place of r and r + 8): 32 bytes of each head and tile.
template <bool F16>
__device__ __forceinline__ void write_columns8(char* out, int64_t o_sh, int heads, int d0, const float (&a)[4], float f0, float f1) {
  const int q = threadIdx.x % 4, head = threadIdx.x % 32 / 4;
  const uint32_t even = transpose8(pack2<F16>(a[0] * f0, a[1] * f1)), odd = transpose8(pack2<F16>(a[2] * f0, a[3] * f1));
  if (head < heads)
    *reinterpret_cast<uint2*>(out + head * o_sh + (d0 + 4 * q) * 2) =
        make_uint2(__byte_perm(even, odd, 0x5410), __byte_perm(even, odd, 0x7632));
}

// Own keys need nothing of the launch before (the shared keys'), beside which they run, but what
// follows waits for this kernel alone: its last block, and with it the kernel, ends behind that one.
// (With every block waiting, the SMs that the shared keys leave free took one round of blocks.)
__device__ __forceinline__ void end_behind_launch_before() {
  if (blockIdx.x == gridDim.x - 1) dependency_wait();
}

template <int KIND, bool F16, int NT, int T, bool PAGED>
__global__ void __launch_bounds__(DEC_THREADS, decode_ctas(NT)) decode_kernel(const __grid_constant__ DecodeParams P) {
  constexpr bool E4M3 = KIND == DECODE_E4M3;
  constexpr bool P16 = F16 || E4M3;                  // P (and what it meets) is fp16
  constexpr bool TWO = !E4M3 || F16;                 // P as two values (e4m3 with bf16 outputs: as one, see below)
  constexpr int CHUNK = 8 / cache_bytes(KIND);       // 16-column steps of a 128-byte chunk
  constexpr int HEADS = 8 * NT, THREADS = DEC_THREADS;
  constexpr int PARTS = decode_parts(T), GROUPS = decode_groups(T), MT = T / 16;
  constexpr int KSTEPS = T < 32 ? 1 : 2;      // of 16 keys, of a warp in the second product
  constexpr int DT = decode_columns(KIND, T); // column tiles of a warp there
  constexpr int WDS = DEC_WARPS / GROUPS;     // warps that share keys there
  constexpr int SPITCH = T + 8, SBUF = PARTS * HEADS * SPITCH;
  constexpr int N = DEC_WARPS * 32;           // threads that compute
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
  const int shared = pages_shared<KIND>(P), skip = KIND == DECODE_OWN ? shared : 0;
  if (KIND == DECODE_16 && P.shared_len && tid == 0 && blockIdx.x == 0 && *P.shared_len < 0) report_invalid(P.err);

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
      const int arrivals = P.boxed ? (E4M3 ? 66 : 1) : 32;   // (e4m3: of two copying warps)
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
      const int len = clamped_len(P, n, skip);
      if (bad_len(P, n) && blockIdx.x == 0) report_invalid(P.err);
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
        const long long tiles = tiles_of<PAGED>(P, clamped_len(P, b == b0 ? n0 : P.lens[b], skip), T);
        if (lo < at + tiles * pairs) break;
        at += tiles * pairs;
      }
      b = min(b, P.B - 1);
      start_s[0] = b;
      start_s[1] = max(1, clamped_len(P, b == b0 ? n0 : P.lens[b], skip));
      scan_s[DEC_THREADS / 32] = lo - at;
    }
    // Requests without keys have no tile: their rows are written here.
    for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
      if (clamped_len(P, P.lens[b], skip) != 0) continue;
      for (int i = KIND == DECODE_OWN ? P.Hq * (P.D / 8) : tid; i < P.Hq * (P.D / 8); i += THREADS) {
        const int h = i / (P.D / 8), d = i % (P.D / 8);
        *reinterpret_cast<uint4*>(P.o + b * P.o_sb + h * P.o_sh + d * 16) = make_uint4(0, 0, 0, 0);
      }
      if (P.lse)
        for (int h = tid; h < P.Hq; h += THREADS) P.lse[(int64_t)b * P.Hq + h] = -INFINITY;
    }
    if (c >= runs) {         // (an exit counts for the dependent launch too)
      if (KIND == DECODE_OWN) end_behind_launch_before();
      return;
    }
    // Columns behind D meet zeros of Q and must be finite (boxes bring zeros).
    if (!P.boxed && P.D * cache_bytes(KIND) % 32 != 0) {
      char* ring = smem + decode_score_bytes(KIND, NT, T) + (E4M3 ? decode_query_bytes(NT, P.D) : 0);
      const int c16 = P.D * cache_bytes(KIND) / 16;
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
  const size_t fixed = decode_score_bytes(KIND, NT, T) + (E4M3 ? decode_query_bytes(NT, P.D) : 0);
  const uint32_t ring_k = smem_u32(smem + fixed);
  // (e4m3: the queries [32 columns][NT][lane] and their units [head], behind the scores)
  char* query_s = smem + decode_score_bytes(KIND, NT, T);
  float* unit_s = reinterpret_cast<float*>(query_s + (P.D + 31) / 32 * NT * 512);
  const uint32_t ring_v = ring_k + P.ring_k * stage;
  // (e4m3: the rows' scales behind the tiles)
  float* scale_k = reinterpret_cast<float*>(smem + fixed + (size_t)(P.ring_k + P.ring_v) * stage);
  float* scale_v = scale_k + P.ring_k * T;

  if (warp >= DEC_WARPS) {
    const bool is_v = warp > DEC_WARPS;
    uint64_t *full = is_v ? full_v : full_k, *empty = is_v ? empty_v : empty_k;
    const uint32_t ring = is_v ? ring_v : ring_k;
    const int slots = is_v ? P.ring_v : P.ring_k;
    const Run run{lo, total, total < gridDim.x ? total : gridDim.x, n_tiles};
    const uint32_t scale_ring = smem_u32(is_v ? scale_v : scale_k);
    if (E4M3 && (PAGED || P.boxed))
      produce_halves<PAGED>(P, T, HEADS, is_v, cur, run, ring_k, ring_v, smem_u32(scale_k), smem_u32(scale_v), full_k, full_v,
                            empty_k, empty_v, &abort_flag);
    else if (PAGED || P.boxed)
      produce_boxes<KIND, PAGED>(P, T, HEADS, is_v, skip, shared, cur, run, ring, slots, full, empty, &abort_flag);
    else
      produce_pieces<KIND>(P, T, HEADS, is_v, skip, shared, cur, run, ring, scale_ring, slots, full, empty, &abort_flag);
    return;
  }

  // ---- the computing warps
  const int ksteps = (P.D + 15) / 16;
  // Shares of D are whole chunks, so that a chunk's swizzle is a constant of the code.
  const int part = warp / MT;                        // in the first product (0 when a warp has two key tiles)
  const int kper = (P.chunks + PARTS - 1) / PARTS * CHUNK;
  const int k0 = part * kper, kn = max(0, min(kper, ksteps - k0));
  const int wkey = warp / WDS, wd = warp % WDS;    // group of keys, share of columns
  const int dper = E4M3 ? DT : (P.chunks + WDS - 1) / WDS * 4;   // (e4m3: a chunk)
  const int d0 = wd * dper, dn = max(0, min(dper, ksteps - d0));
  const int c2 = (lane % 4) * 2, hq = lane / 4;
  const uint32_t chunk_bytes = P.box_rows * 128;
  // Row r of a tile: boxes of box_rows rows, in each chunk after chunk.
  auto row_at = [&](int r) { return r / P.box_rows * (P.chunks * chunk_bytes) + r % P.box_rows * 128; };
  const int key0 = OWN ? warp * 32 : warp % MT * 16;   // first key of the first product
  const int kr = key0 + (lane & 15);
  const uint32_t k_at = ring_k + row_at(kr) + k0 / CHUNK * chunk_bytes + (((lane >> 4) ^ (lane & 7)) << 4);
  const uint32_t k_at2 = OWN ? k_at - row_at(kr) + row_at(kr + 16) : 0;
  // A matrix load brings 16 keys of 16 columns; of e4m3 values 32 keys of 16 columns.
  static_assert(!E4M3 || KSTEPS == 2, "32 keys a warp");
  const int vr = wkey * 32 + (E4M3 ? lane : (lane >> 4) * 8 + (lane & 7));
  const int v_unit = E4M3 ? 0 : (lane >> 3) & 1;
  const uint32_t v_x = d0 / CHUNK * chunk_bytes + ((v_unit ^ (lane & 7)) << 4);
  const uint32_t v_at = ring_v + row_at(vr) + v_x, v_at2 = E4M3 ? 0 : ring_v + row_at(vr + 16) + v_x;
  uint32_t qf[E4M3 ? 1 : 8][NT][2];                // (e4m3: from shared memory)
  float acc[DT][NT][4];
  float top[NT], sum[NT];                          // of head 8 n + lane / 4
  const uint32_t query_at = smem_u32(query_s) + k0 / 2 * NT * 512 + lane * 16;   // e4m3: of this warp's part
  float vtop[NT];                                  // e4m3: log2 of the unit of acc
  float q_unit[NT][2];                             // e4m3, bf16 queries: the units of heads c2 and c2 + 1
  int slot_k = 0, slot_v = 0;
  uint32_t lap_k = 0, lap_v = 0;
  bool alive = true;
  int buf = 0;

  for (int i0 = 0, turn = 0; i0 < n_tiles; turn ^= 1) {
    // ---- one pair's tiles of this run: [i0, i1)
    const int i1 = min(n_tiles, i0 + cur.tiles - cur.t);
    // One warp finds the pair after it; the others read that at the pair's end,
    // behind one barrier at least, so that all warps agree on every pair.
    if (warp == 0) {
      Place next = cur;
      next.t = next.tiles - 1;
      advance<PAGED>(P, pairs, next, T, skip);
      if (lane == 0) next_s[turn] = next;
    }
    const int hk = cur.u / P.head_tiles, ht = cur.u % P.head_tiles;
    const int hq0 = hk * P.group + ht * HEADS;
    const int rows = min(HEADS, P.group - ht * HEADS);
    if (E4M3) {
      // (the last pair's scores are formed: all warps are behind a barrier that follows them)
      for (int head = warp; head < HEADS; head += DEC_WARPS)
        bring_queries<F16>(P.q + cur.b * P.q_sb + (int64_t)(hq0 + head) * P.q_sh, head < rows, P.D, query_s + head / 8 * 512, NT * 512,
                           head % 8, unit_s + head);
      named_bar_sync(1, N);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        q_unit[n][0] = unit_s[n * 8 + c2];
        q_unit[n][1] = unit_s[n * 8 + c2 + 1];
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int head = n * 8 + hq;
      const char* src = P.q + cur.b * P.q_sb + (int64_t)(hq0 + head) * P.q_sh;
      if (!E4M3)
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
      vtop[n] = -INFINITY;
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
      if (E4M3 && OWN && left <= 0) {              // the tile's keys end before this warp's
        if (alive) alive = all_waited(smem_u32(full_k + slot_k), lap_k, P, &abort_flag);
        if (lane == 0) mbar_arrive(smem_u32(empty_k + slot_k));
        if (++slot_k == P.ring_k) {
          slot_k = 0;
          lap_k ^= 1u;
        }
        if (alive) alive = all_waited(smem_u32(full_v + slot_v), lap_v, P, &abort_flag);
        if (lane == 0) mbar_arrive(smem_u32(empty_v + slot_v));
        if (++slot_v == P.ring_v) {
          slot_v = 0;
          lap_v ^= 1u;
        }
        continue;
      }

      // ---- scores of 16 keys over this warp's part of D
      if (alive) alive = all_waited(smem_u32(full_k + slot_k), lap_k, P, &abort_flag);
      if (!E4M3 && i == i0) {                      // Q is here too: dealt out to the four lanes of a head
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
      if (E4M3) {
        // Both key tiles of a warp that has two, and the two steps of a matrix load apart: chains of
        // products that do not wait for each other.
        constexpr int Y = OWN ? 2 : 1;
        float s[Y][2][NT][4];
#pragma unroll
        for (int y = 0; y < Y; ++y)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int j = 0; j < 4; ++j) s[y][h][n][j] = 0.0f;
#pragma unroll
        for (int x = 0; x < (OWN ? 4 : 8); ++x) {
          if (2 * x >= kn) break;
          uint32_t q0[NT][2], q1[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 qx = ld_shared_v4(query_at + (x * NT + n) * 512);
            q0[n][0] = qx.x;
            q0[n][1] = qx.y;
            q1[n][0] = qx.z;
            q1[n][1] = qx.w;
          }
#pragma unroll
          for (int y = 0; y < Y; ++y) {
            const uint32_t a0 = (y ? k_at2 : k_at) + slot_k * stage;
            uint32_t c[4], lo[4], hi[4];
            ldm_x4((a0 + (x >> 2) * chunk_bytes) ^ ((x & 3) << 5), c);
#pragma unroll
            for (int j = 0; j < 4; ++j) widen_e4m3(c[j], lo[j], hi[j]);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16<true>(s[y][0][n], lo, q0[n]);
              mma16<true>(s[y][1][n], hi, q1[n]);
            }
          }
        }
        // times the keys' scales and the queries' units
#pragma unroll
        for (int y = 0; y < Y; ++y) {
          const float* sk = scale_k + slot_k * T + key0 + y * 16 + hq;
          const float s0 = sk[0], s8 = sk[8];
          float* dst = sc + (part * HEADS + c2) * SPITCH + key0 + y * 16 + hq;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float f[4] = {s0, s0, s8, s8};
            if (!F16) {
              f[0] *= q_unit[n][0];
              f[1] *= q_unit[n][1];
              f[2] *= q_unit[n][0];
              f[3] *= q_unit[n][1];
            }
            dst[n * 8 * SPITCH] = (s[y][0][n][0] + s[y][1][n][0]) * f[0];
            dst[(n * 8 + 1) * SPITCH] = (s[y][0][n][1] + s[y][1][n][1]) * f[1];
            dst[n * 8 * SPITCH + 8] = (s[y][0][n][2] + s[y][1][n][2]) * f[2];
            dst[(n * 8 + 1) * SPITCH + 8] = (s[y][0][n][3] + s[y][1][n][3]) * f[3];
          }
        }
      } else
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

      // (the values' scales come with them)
      if (E4M3 && alive) alive = all_waited(smem_u32(full_v + slot_v), lap_v, P, &abort_flag);

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
        if (F16 && !E4M3) most -= P_LIFT;
        const float now = fmaxf(top[n], most);
        const float base = now == -INFINITY ? 0.0f : now;
        fac[n] = ex2_approx(top[n] - base);
        if (!E4M3) moved |= now != top[n];
        top[n] = now;
        float add = 0.0f;
#pragma unroll
        for (int j = 0; j < 2 * KSTEPS; ++j) {
          x[j].x = ex2_approx(x[j].x - base);
          x[j].y = ex2_approx(x[j].y - base);
          add += x[j].x + x[j].y;
          if (!E4M3) split2<P16>(x[j].x, x[j].y, pf[j >> 1][n][j & 1], pr[j >> 1][n][j & 1]);
        }
        sum[n] = sum[n] * fac[n] + add;
        if (E4M3) {
          // Weights times the values' scales, in a unit of their own: the largest product so far
          // is 2^15, whatever the scales are (2^-120 of the largest weight is the smallest unit).
          const float* sv = scale_v + slot_v * T + wkey * 32 + c2;
          float big = 0.0f;
#pragma unroll
          for (int j = 0; j < 2 * KSTEPS; ++j) {
            const float2 w = *reinterpret_cast<const float2*>(sv + j * 8);
            x[j].x *= w.x;
            x[j].y *= w.y;
            big = fmax3(big, x[j].x, x[j].y);
          }
          big = fmaxf(big, __shfl_xor_sync(~0u, big, 1));
          big = fmaxf(big, __shfl_xor_sync(~0u, big, 2));
          const bool any = now != -INFINITY;
          const float unit = any ? fmaxf(vtop[n], now + fmaxf(__log2f(big), -105.0f) - P_LIFT) : vtop[n];
          const float lift = any ? ex2_approx(now - unit) : 0.0f;
          fac[n] = ex2_approx(vtop[n] - (unit == -INFINITY ? 0.0f : unit));
          moved |= unit != vtop[n];
          vtop[n] = unit;
#pragma unroll
          for (int j = 0; j < 2 * KSTEPS; ++j) {
            // An output of bf16 is rounded to 2^-8 of itself; one fp16 value of a weight, off by 2^-11, adds 1 % to
            // that error.  With two (L2 flushed before each): B128 Hkv16 D128 of up to 2048 keys 138 -> 145 us, one key head
            // and 16 heads of D256 53 -> 57.5, B1 D512 16.4 -> 17.2, B16 Hkv4 D1024 of 2000 58 -> 60, B32 Hkv8 D512 the same.
            if (TWO)
              split2<true>(x[j].x * lift, x[j].y * lift, pf[j >> 1][n][j & 1], pr[j >> 1][n][j & 1]);
            else
              pf[j >> 1][n][j & 1] = pack_f16(x[j].x * lift, x[j].y * lift);
          }
        }
      }
      if (__any_sync(~0u, moved) && (!E4M3 || i != i0)) {   // (the first tile's sums are zeros)
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
      if (!E4M3 && alive) alive = all_waited(smem_u32(full_v + slot_v), lap_v, P, &abort_flag);
      const bool tail = left < 16 * KSTEPS;        // rows behind the last key hold anything: zeros, not 0 * NaN
      if (E4M3) {
        // A matrix load leaves a lane two neighbouring columns of two keys: the codes of one
        // column are its bytes 0 and 2, those of the next 1 and 3.
#pragma unroll
        for (int s = 0; s < DT; s += 2) {            // (two column tiles: two chains of products)
          if (s >= dn) break;
          uint32_t c[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) ldm_x4_trans((v_at + slot_v * stage) ^ ((s + h) << 4), c[h]);
#pragma unroll
          for (int g = 0; g < KSTEPS; ++g) {
            uint32_t a[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              widen_e4m3(__byte_perm(c[h][2 * g], 0, 0x3120), a[h][0], a[h][1]);
              widen_e4m3(__byte_perm(c[h][2 * g + 1], 0, 0x3120), a[h][2], a[h][3]);
              if (tail) {
                const int k = g * 16 + c2;
                const uint32_t m0 = (k < left ? 0xffffu : 0u) | (k + 1 < left ? 0xffff0000u : 0u);
                const uint32_t m1 = (k + 8 < left ? 0xffffu : 0u) | (k + 9 < left ? 0xffff0000u : 0u);
                a[h][0] &= m0;
                a[h][1] &= m0;
                a[h][2] &= m1;
                a[h][3] &= m1;
              }
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma16<true>(acc[s][n], a[0], pf[g][n]);
              mma16<true>(acc[s + 1][n], a[1], pf[g][n]);
            }
            if (TWO)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                mma16<true>(acc[s][n], a[0], pr[g][n]);
                mma16<true>(acc[s + 1][n], a[1], pr[g][n]);
              }
          }
        }
      } else
#pragma unroll
      for (int s = 0; s < DT; s += 2) {              // (two column tiles: two chains of products)
        if (s >= dn) break;
#pragma unroll
        for (int g = 0; g < KSTEPS; ++g) {
          uint32_t a[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ldm_x4_trans(((g ? v_at2 : v_at) + slot_v * stage + (s >> 2) * chunk_bytes) ^ (((s + h) & 3) << 5), a[h]);
            if (tail) {
              const int k = g * 16 + c2;
              const uint32_t m0 = (k < left ? 0xffffu : 0u) | (k + 1 < left ? 0xffff0000u : 0u);
              const uint32_t m1 = (k + 8 < left ? 0xffffu : 0u) | (k + 9 < left ? 0xffff0000u : 0u);
              a[h][0] &= m0;
              a[h][1] &= m0;
              a[h][2] &= m1;
              a[h][3] &= m1;
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16<F16>(acc[s][n], a[0], pf[g][n]);
            mma16<F16>(acc[s + 1][n], a[1], pf[g][n]);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma16<F16>(acc[s][n], a[0], pr[g][n]);
            mma16<F16>(acc[s + 1][n], a[1], pr[g][n]);
          }
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
    // (own keys: normalised fp32 outputs in place of 16-bit ones)
    float* out32 = P.o32 + ((int64_t)cur.b * P.Hq + hq0) * P.D;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      sum[n] += __shfl_xor_sync(~0u, sum[n], 1);
      sum[n] += __shfl_xor_sync(~0u, sum[n], 2);
      if (E4M3) {                                  // acc in the unit of the sum from here on
        const float f = top[n] == -INFINITY ? 0.0f : ex2_approx(vtop[n] - top[n]);
        const float f0 = __shfl_sync(~0u, f, c2 * 4), f1 = __shfl_sync(~0u, f, c2 * 4 + 4);
#pragma unroll
        for (int s = 0; s < DT; ++s) {
          acc[s][n][0] *= f0;
          acc[s][n][1] *= f1;
          acc[s][n][2] *= f0;
          acc[s][n][3] *= f1;
        }
      }
    }
    if (GROUPS == 1) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float f0 = 1.0f, f1 = 1.0f;
        if (whole) {
          const float inv = sum[n] == 0.0f ? 0.0f : 1.0f / sum[n];
          f0 = __shfl_sync(~0u, inv, c2 * 4);
          f1 = __shfl_sync(~0u, inv, c2 * 4 + 4);
        }
        if (whole && KIND != DECODE_OWN) {
#pragma unroll
          for (int s = 0; s < DT; s += 2) {
            if (s >= dn) break;
            if (E4M3) {
              write_columns8<F16>(out + n * 8 * P.o_sh, P.o_sh, rows - n * 8, (d0 + s) * 16, acc[s][n], f0, f1);
              if (s + 1 < dn)
                write_columns8<F16>(out + n * 8 * P.o_sh, P.o_sh, rows - n * 8, (d0 + s + 1) * 16, acc[s + 1][n], f0, f1);
            } else {
              write_columns<F16>(out + n * 8 * P.o_sh, P.o_sh, rows - n * 8, (d0 + s) * 16, P.D, acc[s][n], acc[s + 1][n], f0, f1);
            }
          }
        } else if (E4M3) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int head = n * 8 + c2 + j;
            if (head >= rows) continue;
            float* to = part_o + head * P.D + d0 * 16 + 2 * hq;
#pragma unroll
            for (int s = 0; s < DT; ++s)
              if (s < dn) *reinterpret_cast<float2*>(to + s * 16) = make_float2(acc[s][n][j], acc[s][n][2 + j]);
          }
        } else {
          float* base = KIND == DECODE_OWN && whole ? out32 : part_o;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int head = n * 8 + c2 + (j & 1), d = d0 * 16 + (j >> 1) * 8;
            const int some = (P.D - d + 8) / 16;       // column tiles with these 8 columns
            if (head >= rows) continue;
            float* to = base + head * P.D + d + hq;
#pragma unroll
            for (int s = 0; s < DT; ++s)
              if (s < some) to[s * 16] = KIND == DECODE_OWN ? acc[s][n][j] * (j & 1 ? f1 : f0) : acc[s][n][j];
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
      constexpr int RP = WDS * DT * 16 + 4, ROUND = decode_score_bytes(KIND, NT, T) / decode_join_bytes(KIND, T);
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
            float* to = scores + (wkey * ROUND + row) * RP + d0 * 16 + (E4M3 ? 2 * hq + (j >> 1) : hq + (j >> 1) * 8);
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
            if (KIND == DECODE_OWN)
              *reinterpret_cast<float2*>(out32 + (int64_t)row * P.D + d) = make_float2(o.x * inv, o.y * inv);
            else
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
  if (KIND == DECODE_OWN) end_behind_launch_before();
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

template <int KIND, bool F16>
__global__ void __launch_bounds__(JOIN_WARPS * 32, 4) join_kernel(const __grid_constant__ DecodeParams P, int heads, int log_rows) {
  __shared__ float4 acc_s[JOIN_WARPS][32];
  __shared__ float2 ml_s[JOIN_WARPS];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tasks = (P.D + 127) / 128 << log_rows;
  if (KIND == DECODE_OWN) dependents_launch();     // (the merge waits for this kernel's end)
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
    if (KIND == DECODE_OWN) {
      if (col < P.D)
        *reinterpret_cast<float4*>(P.o32 + ((int64_t)m.z * P.Hq + hq) * P.D + col) =
            make_float4(s.a.x * inv, s.a.y * inv, s.a.z * inv, s.a.w * inv);
    } else if (col < P.D)
      *reinterpret_cast<uint2*>(P.o + m.z * P.o_sb + hq * P.o_sh + col * 2) =
          make_uint2(pack2<F16>(s.a.x * inv, s.a.y * inv), pack2<F16>(s.a.z * inv, s.a.w * inv));
    if (P.lse && col == 0)
      P.lse[(int64_t)m.z * P.Hq + hq] = s.l == 0.0f ? -INFINITY : (s.top + log2f(s.l)) * 0.69314718055994531f;
  }
}

// A launch that may begin when the one before it in the stream says so (dependents_launch) or ends.
template <class... Params, class... Args>
ffpa_status launch_dependent(void (*fn)(Params...), int grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fn, args...) == cudaSuccess) return FFPA_OK;
  cudaGetLastError();
  return FFPA_ERR_CUDA;
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

template <int KIND, bool F16, int NT, int T>
ffpa_status launch_decode_as(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  const auto fn = P.page_tiles ? &decode_kernel<KIND, F16, NT, T, true> : &decode_kernel<KIND, F16, NT, T, false>;
  const ffpa_status st = set_smem_attr_once(reinterpret_cast<const void*>(fn), dev, (int)pl.smem);
  if (st != FFPA_OK) return st;
  if (KIND == DECODE_OWN && P.shared_pages > 0) {
    // Beside the shared keys' launch before it, as SMs come free, and done after it (see the kernel's end).
    const ffpa_status own = launch_dependent(fn, grid, DEC_THREADS, pl.smem, stream, P);
    if (own != FFPA_OK) return own;
  } else {
    fn<<<grid, DEC_THREADS, pl.smem, stream>>>(P);
    if (cudaGetLastError() != cudaSuccess) return FFPA_ERR_CUDA;
  }
  const int heads = 8 * NT;
  int log_rows = 0;
  while ((1 << log_rows) < (P.group < heads ? P.group : heads)) ++log_rows;
  // A dependent launch: its blocks are set up while the first kernel runs out.
  return launch_dependent(join_kernel<KIND, F16>, 2 * grid, JOIN_WARPS * 32, 0, stream, P, heads, log_rows);
}

template <int KIND, bool F16, int T>
ffpa_status launch_decode_tile(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  return pl.nt == 1 ? launch_decode_as<KIND, F16, 1, T>(P, pl, grid, dev, stream)
                    : launch_decode_as<KIND, F16, 2, T>(P, pl, grid, dev, stream);
}

template <int KIND, bool F16>
ffpa_status launch_decode(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  switch (pl.tile) {
    case 16:   // (rows of more than 1 KB: never codes)
      return launch_decode_tile<KIND, F16, KIND == DECODE_E4M3 ? 32 : 16>(P, pl, grid, dev, stream);
    case 32: return launch_decode_tile<KIND, F16, 32>(P, pl, grid, dev, stream);
    case 64: return launch_decode_tile<KIND, F16, 64>(P, pl, grid, dev, stream);
    case 128: return launch_decode_tile<KIND, F16, 128>(P, pl, grid, dev, stream);
    default: return launch_decode_tile<KIND, F16, 256>(P, pl, grid, dev, stream);
  }
}


// ---- host: what the entry points share

// The checks that need no device (pointers may be anything).  Element sizes: queries and
// outputs 2 bytes, the cache's by its kind.
inline ffpa_status check_decode(int kind, ffpa_dtype dt, const DecodeShape& s, const float* scale, int enable_gqa, float* sc) {
  if (dt != FFPA_BF16 && dt != FFPA_FP16) return FFPA_ERR_DTYPE;
  if (s.B < 0 || s.Hq < 1 || s.Hkv < 1 || s.num_pages < 0 || s.page_size < 1 || s.max_pages < 0) return FFPA_ERR_INVALID;
  if (s.D < 64 || s.D > 1024 || s.D % (16 / cache_bytes(kind)) != 0) return FFPA_ERR_UNSUPPORTED;
  if (s.Hq % s.Hkv != 0 || (s.Hq != s.Hkv && !enable_gqa)) return FFPA_ERR_INVALID;
  if ((long long)s.max_pages * s.page_size > 0x7fff0000LL) return FFPA_ERR_INVALID;   // key numbers are int32
  *sc = scale ? *scale : 1.0f / std::sqrt(static_cast<float>(s.D));
  return std::isfinite(*sc) ? FFPA_OK : FFPA_ERR_INVALID;
}
inline ffpa_status check_decode_rows(int kind, const DecodeShape& s, const void* q, const void* k_cache, const void* v_cache,
                                     const void* o, const float* lse, const int64_t* q_str, const int64_t* o_str,
                                     const int32_t* block_table, int64_t table_str, const int32_t* seq_lens, const void* workspace) {
  if (!q || !o || !seq_lens || !workspace || !q_str || !s.k_str || !s.v_str || !o_str) return FFPA_ERR_INVALID;
  if (s.held() && (!k_cache || !v_cache || !block_table)) return FFPA_ERR_INVALID;
  if (!rows_ok(q_str, {s.B, s.Hq, s.D}) || !rows_ok(o_str, {s.B, s.Hq, s.D})) return FFPA_ERR_INVALID;
  const int unit = 16 / cache_bytes(kind);
  if (s.held() && (!rows_ok(s.k_str, {s.num_pages, s.page_size, s.Hkv, s.D}, unit) ||
                   !rows_ok(s.v_str, {s.num_pages, s.page_size, s.Hkv, s.D}, unit)))
    return FFPA_ERR_INVALID;
  if (s.held() && s.B > 1 && table_str < s.max_pages) return FFPA_ERR_INVALID;
  if (!on_boundary(q, 16) || !on_boundary(o, 16) || !on_boundary(lse, 4) || !on_boundary(seq_lens, 4) ||
      !on_boundary(workspace, 256))
    return FFPA_ERR_INVALID;
  if (s.held() && (!on_boundary(k_cache, 16) || !on_boundary(v_cache, 16) || !on_boundary(block_table, 4)))
    return FFPA_ERR_INVALID;
  return FFPA_OK;
}

// With a DeviceScope open: fills in what depends on the shape and the workspace and launches.
// The caller has set q, k, v, o, lse, table, lens, err, the strides of q, o and the table, the
// scales, and what belongs to own keys.
template <int KIND>
ffpa_status run_decode(DecodeParams& P, const DecodeShape& s, ffpa_dtype dt, float sc, int sms, int dev, char* ws,
                       const ffpa_options* options, cudaStream_t stream) {
  constexpr int CB = cache_bytes(KIND);
  const DecodePlan pl = decode_plan(s.D, s.Hq / s.Hkv, KIND);
  const int grid = (sms < DEC_SMS_MAX ? sms : DEC_SMS_MAX) * pl.ctas;
  const DecodeSpace sp = decode_space(grid, 8 * pl.nt, s.D);
  P.part = reinterpret_cast<float*>(ws + sp.part);
  P.part_ml = reinterpret_cast<float2*>(ws + sp.ml);
  P.cuts = reinterpret_cast<int4*>(ws + sp.cuts);
  if (s.held()) {
    P.k_sp = s.k_str[0] * CB;
    P.k_ss = s.k_str[1] * CB;
    P.k_sh = s.k_str[2] * CB;
    P.v_sp = s.v_str[0] * CB;
    P.v_ss = s.v_str[1] * CB;
    P.v_sh = s.v_str[2] * CB;
  }
  P.B = s.B;
  P.Hq = s.Hq;
  P.Hkv = s.Hkv;
  P.group = s.Hq / s.Hkv;
  P.D = s.D;
  P.head_tiles = pl.head_tiles;
  P.num_pages = s.num_pages;
  P.page_size = s.page_size;
  P.max_pages = s.held() ? s.max_pages : 0;   // without pages every request is empty
  P.chunks = pl.chunks;
  // Boxes of as many rows as divide a page, down to the 8 of the swizzle.  Where a
  // page's size is no multiple of 8 but fills enough of a tile, a tile is one box that
  // ends with its page (B32 Hkv8 D512 of 4096 keys, pages of 100: 321 us, in pieces
  // 454); smaller pages of that kind come in pieces.  "Enough" is where both cost the
  // same: a half (that case with pages of 12, of 32 keys a tile: 580 us, in pieces 455), and a
  // third of the tiles of 128 and 256 keys (B64 Hkv2 D64 of 3000 keys, pages of 100: 34 us, in
  // pieces 45; D128 of 2000 keys, pages of 36: 51, 45).
  const bool by_page = s.page_size % 8 != 0 && s.page_size > (pl.tile - 1) / (pl.tile >= 128 ? 3 : 2);
  P.boxed = s.held() && (s.page_size % 8 == 0 || by_page);
  P.page_tiles = by_page ? (s.page_size + pl.tile - 1) / pl.tile : 0;
  P.box_rows = pl.tile;
  P.box_chunks = s.D * CB % 128 == 0 ? pl.chunks : 1;
  if (P.boxed) {
    while (!by_page && s.page_size % P.box_rows != 0) P.box_rows /= 2;
    for (int i = 0; i < 2; ++i) {
      // (bytes; a dimension of one entry may have any stride, a tensor map takes multiples of 16)
      const int64_t* of = i ? s.v_str : s.k_str;
      const uint64_t one = (uint64_t)s.D * CB, row = s.page_size > 1 ? (uint64_t)of[1] * CB : one;
      const uint64_t head = s.Hkv > 1 ? (uint64_t)of[2] * CB : one, page = s.num_pages > 1 ? (uint64_t)of[0] * CB : one;
      CUtensorMap* map = i ? &P.map_v : &P.map_k;
      const void* base = i ? P.v : P.k;
      constexpr uint32_t wide = 128 / CB;
      ffpa_status st;
      if (P.box_chunks > 1) {
        const uint64_t dims[5] = {wide, (uint64_t)s.page_size, (uint64_t)pl.chunks, (uint64_t)s.Hkv, (uint64_t)s.num_pages};
        const uint64_t str[4] = {row, 128, head, page};
        const uint32_t box[5] = {wide, (uint32_t)P.box_rows, (uint32_t)pl.chunks, 1, 1};
        st = KIND == DECODE_E4M3 ? encode_codes(map, 5, base, dims, str, box, s.D) : encode_rows(map, dt, 5, base, dims, str, box);
      } else {
        const uint64_t dims[4] = {(uint64_t)s.D, (uint64_t)s.page_size, (uint64_t)s.Hkv, (uint64_t)s.num_pages};
        const uint64_t str[3] = {row, head, page};
        const uint32_t box[4] = {wide, (uint32_t)P.box_rows, 1, 1};
        st = KIND == DECODE_E4M3 ? encode_codes(map, 4, base, dims, str, box, s.D) : encode_rows(map, dt, 4, base, dims, str, box);
      }
      if (st != FFPA_OK) return st;
    }
  }
  P.ring_k = pl.ring_k;
  P.ring_v = pl.ring_v;
  P.timeout_ns = options && options->wait_timeout_ns ? options->wait_timeout_ns : 2000000000ull;
  P.drop = options && options->test_drop_first_copy ? 1 : 0;
  P.scale_log2 = sc * 1.4426950408889634f;
  return dt == FFPA_FP16 ? launch_decode<KIND, true>(P, pl, grid, dev, stream) : launch_decode<KIND, false>(P, pl, grid, dev, stream);
}

inline size_t decode_bytes(int Hq, int Hkv, int D) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 64 || D > 1024 || D % 8 != 0) return 0;
  const int nt = decode_nt(Hq / Hkv);
  return decode_space(DEC_SMS_MAX * decode_ctas(nt), 8 * nt, D).total;
}

// A whole entry point of one kind of cache (k_scale and v_scale, with strides over pages
// and heads, where it holds codes).
template <int KIND>
ffpa_status decode_entry(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse, ffpa_dtype dt,
                         const DecodeShape& s, const int64_t* q_str, const int64_t* o_str, const int32_t* block_table,
                         int64_t table_str, const int32_t* seq_lens, const float* k_scale, const float* v_scale,
                         const int64_t* ks_str, const int64_t* vs_str, const float* scale, int enable_gqa, void* workspace,
                         size_t workspace_bytes, ffpa_stream_t stream, const ffpa_options* options) {
  float sc = 0.0f;
  ffpa_status st = check_decode(KIND, dt, s, scale, enable_gqa, &sc);
  if (st != FFPA_OK) return st;
  if (s.B == 0) return FFPA_OK;
  st = check_decode_rows(KIND, s, q, k_cache, v_cache, o, lse, q_str, o_str, block_table, table_str, seq_lens, workspace);
  if (st != FFPA_OK) return st;
  const bool held = s.held(), scaled = held && KIND == DECODE_E4M3;
  if (scaled && (!k_scale || !v_scale || !ks_str || !vs_str || !on_boundary(k_scale, 4) || !on_boundary(v_scale, 4) ||
                 !scales_ok(ks_str, s.num_pages, s.Hkv, s.page_size) || !scales_ok(vs_str, s.num_pages, s.Hkv, s.page_size)))
    return FFPA_ERR_INVALID;
  if (workspace_bytes < decode_bytes(s.Hq, s.Hkv, s.D)) return FFPA_ERR_INVALID;
  if ((long long)s.B * s.Hkv * decode_plan(s.D, s.Hq / s.Hkv, KIND).head_tiles > 0x7fffffffLL) return FFPA_ERR_INVALID;
  int dev = 0;
  st = call_device({q, o, lse, seq_lens, workspace, held ? k_cache : nullptr, held ? v_cache : nullptr,
                    held ? (const void*)block_table : nullptr, scaled ? k_scale : nullptr, scaled ? v_scale : nullptr},
                   &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  DecodeParams P{};
  int sms = 0;
  if ((st = call_status(dev, options, &P.err, &sms)) != FFPA_OK) return st;
  P.q = static_cast<const char*>(q);
  P.k = static_cast<const char*>(k_cache);
  P.v = static_cast<const char*>(v_cache);
  P.o = static_cast<char*>(o);
  P.lse = lse;
  P.table = block_table;
  P.lens = seq_lens;
  P.q_sb = q_str[0] * 2;
  P.q_sh = q_str[1] * 2;
  P.o_sb = o_str[0] * 2;
  P.o_sh = o_str[1] * 2;
  P.table_str = table_str;
  if (scaled) {
    P.ks = k_scale;
    P.vs = v_scale;
    P.ks_sp = ks_str[0];
    P.ks_sh = ks_str[1];
    P.vs_sp = vs_str[0];
    P.vs_sh = vs_str[1];
    const int64_t odd = (s.num_pages > 1 ? P.ks_sp | P.vs_sp : 0) | (s.Hkv > 1 ? P.ks_sh | P.vs_sh : 0) | s.page_size;
    P.scale4 = odd % 4 == 0 && on_boundary(k_scale, 16) && on_boundary(v_scale, 16);
  }
  return run_decode<KIND>(P, s, dt, sc, sms, dev, static_cast<char*>(workspace), options, reinterpret_cast<cudaStream_t>(stream));
}

}  // namespace
}  // namespace ffpa
