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
//    cut into equal runs, one run per CTA (one CTA per SM): a long request is
//    shared by many CTAs and short ones share a CTA, whatever the mix, and the
//    host needs no lengths.  A pair that ends inside its CTA is written at
//    once; a pair cut between CTAs leaves fp32 partial sums with their maximum
//    and sum, which the second launch joins in the order of the CTAs.
//  - K and V tiles (T keys of D columns, about 33 KB) alternate in a ring of
//    shared-memory slots filled by 16-byte asynchronous copies: a row may lie in any page, so
//    page sizes, strides and tails need no special path.  Rows are 16 bytes
//    longer than D so that the matrix loads meet no bank conflict.
//  - The products run with keys (then columns of V) as the 16 rows of
//    mma.m16n8k16 and the heads as its 8 columns: K and V are the operands
//    read once, and 8 heads cost one instruction per 256 elements of K.  A warp
//    owns 64 columns of D in both products (WD warps; WK groups of them share
//    the keys when D is small), the scores are summed over the warps in shared
//    memory, and one pass keeps the running maximum and sum in fp32.
//    P is rounded to the input type, as in the forward kernels; the sum is
//    taken over the unrounded values.
#include "ffpa_paged.cuh"

namespace ffpa {
namespace {

constexpr int DEC_SLOTS_MAX = 8;
constexpr size_t DEC_SLOT_TARGET = 38 * 1024;

struct DecodeParams {
  const char *q, *k, *v;
  char* o;
  float* lse;
  const int32_t* table;
  const int32_t* lens;
  float* part;      // [2 grid][8 NT][D] unnormalised partial outputs
  float2* part_ml;  // [2 grid][8 NT] (maximum in log2 units, sum)
  int2* meta;       // [grid] (pair cut behind CTA c or -1, last CTA of that pair)
  int* err;
  int64_t q_sb, q_sh, o_sb, o_sh;       // bytes
  int64_t k_sp, k_ss, k_sh, v_sp, v_ss, v_sh;
  int64_t table_str;
  int B, Hq, Hkv, group, D, head_tiles;
  int num_pages, page_size, max_pages;
  int wd, wk, tile, pitch, slots;
  float scale_log2;
};

struct DecodePlan {
  int nt, wd, wk, tile, pitch, slots, head_tiles;
  size_t smem;
};

// Heads of one pass: 8 NT, as many as the accumulators have registers for
// (more than 8 warps leave 128 registers a thread).  A larger group is split
// over pairs that read the same keys (the second from L2).
int decode_nt(int group, int D) { return group <= 8 ? 1 : group <= 16 || D > 512 ? 2 : 4; }

size_t decode_fixed_smem(const DecodePlan& p) {
  const size_t heads = 8 * (size_t)p.nt;
  size_t s = p.wd * heads * (p.tile + 4) * 4;             // partial scores
  const size_t join = p.wk > 1 ? heads * (p.wd * 64 + 4) * 4 : 0;   // or the key groups' outputs
  if (join > s) s = join;
  s += heads * (p.tile + 8) * 2;                          // P
  s = (s + 15) & ~size_t(15);
  s += 2 * (size_t)p.tile * 16;                           // row offsets of two tiles
  s += heads * 12;                                        // maximum, sum, factor
  return (s + 127) & ~size_t(127);
}

DecodePlan decode_plan(int D, int group) {
  DecodePlan p;
  p.nt = decode_nt(group, D);
  p.head_tiles = (group + 8 * p.nt - 1) / (8 * p.nt);
  p.wd = (D + 63) / 64;
  p.wk = p.wd < 8 ? 8 / p.wd : 1;
  p.pitch = p.wd * 128 + 16;
  const int step = 16 * p.wk;
  p.tile = step;
  // At least one lane in two of the softmax step has a key from 32 keys on.
  while ((size_t)(p.tile + step) * p.pitch <= DEC_SLOT_TARGET && (p.tile + step) <= 32 * p.wd * p.wk) p.tile += step;
  const size_t budget = SMEM_LIMIT - 1024 - decode_fixed_smem(p);
  p.slots = static_cast<int>(budget / ((size_t)p.tile * p.pitch));
  if (p.slots > DEC_SLOTS_MAX) p.slots = DEC_SLOTS_MAX;
  p.smem = decode_fixed_smem(p) + (size_t)p.slots * p.tile * p.pitch;
  return p;
}

// A place on the line of tiles: tile t of `tiles` of pair u of request b.
struct Place {
  int b, u, t, tiles, len;
};

__device__ __forceinline__ int clamped_len(const DecodeParams& P, int b) {
  const long long cap = (long long)P.max_pages * P.page_size;
  const int n = P.lens[b];
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}

__device__ __forceinline__ void advance(const DecodeParams& P, int pairs, Place& p) {
  if (++p.t < p.tiles) return;
  p.t = 0;
  if (++p.u < pairs) return;
  p.u = 0;
  do {
    ++p.b;
    if (p.b >= P.B) {
      p.len = 0;
      p.tiles = 0;
      return;
    }
    p.len = clamped_len(P, p.b);
  } while (p.len == 0);
  p.tiles = (p.len + P.tile - 1) / P.tile;
}

template <bool F16, int NT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 1) decode_kernel(const DecodeParams P) {
  constexpr int HEADS = 8 * NT;
  extern __shared__ __align__(128) char smem[];
  const int tid = threadIdx.x, nthreads = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int T = P.tile, pitch = P.pitch, slots = P.slots;
  const int pairs = P.Hkv * P.head_tiles;

  // ---- this CTA's run of tiles
  __shared__ long long scan_s[17];
  __shared__ int start_s[2];
  long long total, lo, hi;
  Place cur;
  {
    const int per = (P.B + nthreads - 1) / nthreads;
    const int b0 = tid * per, b1 = min(P.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = P.lens[b];
      const int len = clamped_len(P, b);
      if (n != len && blockIdx.x == 0) report_invalid(P.err);
      mine += (len + T - 1) / T;
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
    for (int w = 0; w < nthreads / 32; ++w) {
      if (w < warp) before += scan_s[w];
      total += scan_s[w];
    }
    total *= pairs;
    long long at = (before + incl - mine) * pairs;   // first tile of request b0
    const long long runs = total < gridDim.x ? total : gridDim.x;
    const long long c = blockIdx.x;
    lo = c < runs ? c * total / runs : 0;
    hi = c < runs ? (c + 1) * total / runs : 0;
    if (c < runs && lo >= at && lo < at + mine * pairs) {
      int b = b0;
      long long tiles = 0;
      for (; b < b1; ++b) {
        tiles = (clamped_len(P, b) + T - 1) / T;
        if (lo < at + tiles * pairs) break;
        at += tiles * pairs;
      }
      start_s[0] = b;
      scan_s[16] = lo - at;
    }
    if (tid == 0) P.meta[blockIdx.x] = make_int2(-1, 0);
    __syncthreads();
    if (c < runs) {
      cur.b = start_s[0];
      cur.len = clamped_len(P, cur.b);
      cur.tiles = (cur.len + T - 1) / T;
      const long long r = scan_s[16];
      cur.u = (int)(r / cur.tiles);
      cur.t = (int)(r % cur.tiles);
    }
    // Requests without keys have no tile: their rows are written here.
    for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
      if (clamped_len(P, b) != 0) continue;
      for (int i = tid; i < P.Hq * (P.D / 8); i += nthreads) {
        const int h = i / (P.D / 8), d = i % (P.D / 8);
        *reinterpret_cast<uint4*>(P.o + b * P.o_sb + h * P.o_sh + d * 16) = make_uint4(0, 0, 0, 0);
      }
      if (P.lse)
        for (int h = tid; h < P.Hq; h += nthreads) P.lse[(int64_t)b * P.Hq + h] = -INFINITY;
    }
    if (c >= runs) return;
  }
  const long long runs = total < gridDim.x ? total : gridDim.x;
  const int n_tiles = (int)(hi - lo);

  // ---- shared memory
  float* part_s = reinterpret_cast<float*>(smem);                  // [wd][HEADS][T + 4]
  const int spitch = T + 4;
  size_t off = (size_t)P.wd * HEADS * spitch * 4;
  if (P.wk > 1) {
    const size_t join = (size_t)HEADS * (P.wd * 64 + 4) * 4;
    if (join > off) off = join;
  }
  char* p_s = smem + off;                                          // [HEADS][T + 8] 16-bit
  const int ppitch = (T + 8) * 2;
  off += (size_t)HEADS * ppitch;
  off = (off + 15) & ~size_t(15);
  longlong2* rows_s = reinterpret_cast<longlong2*>(smem + off);    // [2][T] byte offsets of K and V rows, or -1
  off += 2 * (size_t)T * 16;
  float* max_s = reinterpret_cast<float*>(smem + off);
  float* sum_s = max_s + HEADS;
  float* fac_s = sum_s + HEADS;
  off += HEADS * 12;
  off = (off + 127) & ~size_t(127);
  char* ring = smem + off;
  const int slot_bytes = T * pitch;

  for (int i = tid; i < HEADS * ppitch / 4; i += nthreads) reinterpret_cast<uint32_t*>(p_s)[i] = 0;
  for (int i = tid; i < HEADS; i += nthreads) fac_s[i] = 1.0f;
  // Columns past D are read by the matrix loads: zero once, never written again.
  if (P.D % 64 != 0) {
    const int pad = P.wd * 8 - P.D / 8;   // 16-byte pieces
    for (int i = tid; i < slots * T * pad; i += nthreads)
      *reinterpret_cast<uint4*>(ring + (i / pad) * pitch + P.D * 2 + (i % pad) * 16) = make_uint4(0, 0, 0, 0);
  }

  // ---- producer side: every thread copies its share of each half (K or V tile)
  const int cpr = P.D / 8;                         // 16-byte pieces of a row
  const int r0 = tid / cpr, c0 = tid % cpr, dr = nthreads / cpr, dc = nthreads % cpr;
  Place ahead = cur;        // tile whose rows are looked up next
  int looked = 0;           // tiles looked up
  int issued = 0;           // halves issued
  int page_next = -1;       // page of this thread's row in tile `ahead`
  bool row_next = false;
  int u_of[2] = {0, 0};     // pair of the two tiles in rows_s

  auto load_page = [&] {
    row_next = false;
    if (looked < n_tiles && tid < T) {
      const int key = ahead.t * T + tid;
      if (key < ahead.len) {
        row_next = true;
        page_next = P.table[ahead.b * P.table_str + key / P.page_size];
      }
    }
  };
  // Row offsets of tile `looked` into buffer looked & 1; then the pages of the next one are requested.
  auto look_up = [&] {
    if (looked < n_tiles) {
      if (tid < T) {
        longlong2 x = make_longlong2(-1, -1);
        if (row_next) {
          if (page_next >= 0 && page_next < P.num_pages) {
            const int in = (ahead.t * T + tid) % P.page_size;
            x.x = page_next * P.k_sp + in * P.k_ss;
            x.y = page_next * P.v_sp + in * P.v_ss;
          } else {
            report_invalid(P.err);
          }
        }
        rows_s[(looked & 1) * T + tid] = x;
      }
      u_of[looked & 1] = ahead.u;
      ++looked;
      advance(P, pairs, ahead);
      load_page();
    }
  };
  // The next half into its slot of the ring; past the run's end an empty group keeps the count.
  auto issue = [&] {
    const int tile = issued >> 1;
    if (tile < n_tiles) {
      const bool is_v = issued & 1;
      const uint32_t dst = smem_u32(ring + (issued % slots) * slot_bytes);
      const int hk = u_of[tile & 1] / P.head_tiles;
      const char* base = is_v ? P.v + hk * P.v_sh : P.k + hk * P.k_sh;
      const longlong2* rows = rows_s + (tile & 1) * T;
      int r = r0, c = c0;
      while (r < T) {
        const long long at = is_v ? rows[r].y : rows[r].x;
        copy16_async(dst + r * pitch + c * 16, at >= 0 ? base + at + c * 16 : base, at >= 0 ? 16 : 0);
        r += dr;
        c += dc;
        if (c >= cpr) {
          c -= cpr;
          ++r;
        }
      }
    }
    copy_commit();
    ++issued;
  };

  load_page();
  look_up();
  __syncthreads();
  for (int i = 0; i < slots; ++i) {
    issue();
    if ((issued & 1) == 0) {
      look_up();
      __syncthreads();
    }
  }

  // ---- consumer side
  const int wd = warp % P.wd, wkey = warp / P.wd;
  const int keys = T / P.wk, key0 = wkey * keys;         // this warp's keys of a tile
  uint32_t qf[4][NT][2];
  float acc[4][NT][4];
  int rows = 0, hq0 = 0, t0 = 0;

  // wait until at most `left` groups are in flight
  auto wait = [&](int left) {
    switch (left) {
      case 0: copy_wait<0>(); break;
      case 1: copy_wait<1>(); break;
      case 2: copy_wait<2>(); break;
      case 3: copy_wait<3>(); break;
      case 4: copy_wait<4>(); break;
      case 5: copy_wait<5>(); break;
      case 6: copy_wait<6>(); break;
      default: copy_wait<7>(); break;
    }
  };

  for (int i = 0; i < n_tiles; ++i) {
    if (i == 0 || cur.t == 0) {
      // A new pair: its queries into registers, sums cleared.
      const int hk = cur.u / P.head_tiles, ht = cur.u % P.head_tiles;
      hq0 = hk * P.group + ht * HEADS;
      rows = min(HEADS, P.group - ht * HEADS);
      t0 = cur.t;
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int head = n * 8 + lane / 4;
          const char* src = P.q + cur.b * P.q_sb + (int64_t)(hq0 + head) * P.q_sh;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int d = wd * 64 + s * 16 + j * 8 + (lane % 4) * 2;
            qf[s][n][j] = head < rows && d < P.D ? *reinterpret_cast<const uint32_t*>(src + d * 2) : 0u;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[s][n][j] = 0.0f;
        }
      for (int h = warp; h < HEADS; h += nthreads / 32)
        if (lane == 0) {
          max_s[h] = -INFINITY;
          sum_s[h] = 0.0f;
        }
    }
    const int half = 2 * i;
    wait(slots - 2);
    __syncthreads();           // K tile i has landed; every warp is done with V tile i - 1
    if (i > 0) {
      issue();
      if ((issued & 1) == 0) look_up();
    }
    {
      const uint32_t ks = smem_u32(ring + (half % slots) * slot_bytes);
      for (int g = 0; g < keys; g += 16) {
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[n][j] = 0.0f;
        const uint32_t a0 = ks + (key0 + g + ((lane >> 3) & 1) * 8 + (lane & 7)) * pitch + wd * 128 + (lane >> 4) * 16;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t a[4];
          ldm_x4(a0 + x * 32, a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<F16>(s[n], a, qf[x][n]);
        }
        float* dst = part_s + (wd * HEADS + (lane % 4) * 2) * spitch + key0 + g + lane / 4;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          dst[n * 8 * spitch] = s[n][0];
          dst[(n * 8 + 1) * spitch] = s[n][1];
          dst[n * 8 * spitch + 8] = s[n][2];
          dst[(n * 8 + 1) * spitch + 8] = s[n][3];
        }
      }
    }
    __syncthreads();           // the partial scores are complete; K tile i is free
    issue();
    if ((issued & 1) == 0) look_up();
    for (int h = warp; h < rows; h += nthreads / 32) {
      const int left = cur.len - cur.t * T;      // keys of this tile and beyond
      float x[8], top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = lane + 32 * j;
        x[j] = -INFINITY;
        if (key < T && key < left) {
          float sum = 0.0f;
          for (int w = 0; w < P.wd; ++w) sum += part_s[(w * HEADS + h) * spitch + key];
          x[j] = sum * P.scale_log2;
        }
        top = fmaxf(top, x[j]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
      const float old = max_s[h];
      const float now = fmaxf(old, top);
      const float base = now == -INFINITY ? 0.0f : now;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = lane + 32 * j;
        if (key < T) {
          const float e = ex2_approx(x[j] - base);
          sum += e;
          store16<F16>(p_s + h * ppitch + key * 2, e);
        }
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      __syncwarp();
      if (lane == 0) {
        const float f = ex2_approx(old - base);
        max_s[h] = now;
        sum_s[h] = sum_s[h] * f + sum;
        fac_s[h] = f;
      }
    }
    wait(slots - 1);
    __syncthreads();           // P is complete; V tile i has landed
    {
      const uint32_t vs = smem_u32(ring + ((half + 1) % slots) * slot_bytes);
      const uint32_t ps = smem_u32(p_s);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f0 = fac_s[n * 8 + (lane % 4) * 2], f1 = fac_s[n * 8 + (lane % 4) * 2 + 1];
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          acc[s][n][0] *= f0;
          acc[s][n][1] *= f1;
          acc[s][n][2] *= f0;
          acc[s][n][3] *= f1;
        }
      }
      for (int g = key0; g < key0 + keys; g += 16) {
        uint32_t b[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) ldm_x2(ps + (n * 8 + (lane & 7)) * ppitch + g * 2 + ((lane >> 3) & 1) * 16, b[n]);
        const uint32_t a0 = vs + (g + (lane >> 4) * 8 + (lane & 7)) * pitch + wd * 128 + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          uint32_t a[4];
          ldm_x4_trans(a0 + s * 32, a);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma16<F16>(acc[s][n], a, b[n]);
        }
      }
    }
    const bool done = cur.t == cur.tiles - 1;
    if (done || i == n_tiles - 1) {
      // ---- the pair's sums, whole or cut
      const bool whole = done && t0 == 0;
      const int64_t slot = 2 * (int64_t)blockIdx.x + (t0 == 0 ? 1 : 0);
      float* part = P.part + slot * HEADS * P.D;
      if (P.wk > 1) {
        // The key groups' outputs are added in their order (over the scores: PV does not read them).
        const int jpitch = P.wd * 64 + 4;
        for (int w = 0; w < P.wk; ++w) {
          if (wkey == w) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  float* dst = part_s + (n * 8 + (lane % 4) * 2 + (j & 1)) * jpitch + wd * 64 + s * 16 + lane / 4 + (j >> 1) * 8;
                  acc[s][n][j] = w == 0 ? acc[s][n][j] : *dst + acc[s][n][j];
                  if (w < P.wk - 1) *dst = acc[s][n][j];
                }
          }
          __syncthreads();
        }
      }
      if (wkey == P.wk - 1) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int head = n * 8 + (lane % 4) * 2 + (j & 1);
            if (head >= rows) continue;
            const float l = sum_s[head];
            const float inv = whole ? (l == 0.0f ? 0.0f : 1.0f / l) : 1.0f;
            char* out = P.o + cur.b * P.o_sb + (int64_t)(hq0 + head) * P.o_sh;
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const int d = wd * 64 + s * 16 + lane / 4 + (j >> 1) * 8;
              if (d >= P.D) continue;
              if (whole)
                store16<F16>(out + d * 2, acc[s][n][j] * inv);
              else
                part[(int64_t)head * P.D + d] = acc[s][n][j];
            }
          }
      }
      for (int h = tid; h < rows; h += nthreads) {
        if (whole) {
          if (P.lse)
            P.lse[(int64_t)cur.b * P.Hq + hq0 + h] =
                sum_s[h] == 0.0f ? -INFINITY : (max_s[h] + log2f(sum_s[h])) * 0.69314718055994531f;
        } else {
          P.part_ml[slot * HEADS + h] = make_float2(max_s[h], sum_s[h]);
        }
      }
      if (!done && t0 == 0 && tid == 0) {
        // The pair goes on in the next CTAs; its last tile says how far.
        const long long last = lo + i + (cur.tiles - 1 - cur.t);
        P.meta[blockIdx.x] = make_int2(cur.b * pairs + cur.u, (int)(((last + 1) * runs - 1) / total));
      }
      __syncthreads();         // the sums are read before the next pair clears them
    }
    advance(P, pairs, cur);
  }
  copy_wait<0>();
}

// Joins the partial sums of a pair cut between CTAs: block (c, row) the row of
// the pair that CTA c began, over CTAs c .. last, in that order.  Groups of
// threads take every n-th CTA's sums and are added in their order.
template <bool F16>
__global__ void __launch_bounds__(512) join_kernel(const DecodeParams P, int heads) {
  const int2 m = P.meta[blockIdx.x];
  if (m.x < 0) return;
  const int pairs = P.Hkv * P.head_tiles;
  const int b = m.x / pairs, u = m.x % pairs, row = blockIdx.y;
  const int hk = u / P.head_tiles, ht = u % P.head_tiles;
  if (row >= P.group - ht * heads) return;
  const int hq = hk * P.group + ht * heads + row;
  const int n = m.y - blockIdx.x + 1;
  const int cols = P.D / 4;                        // float4 columns
  const int groups = blockDim.x / cols;            // at least 2 (D <= 1024)
  const int g = threadIdx.x / cols, col = threadIdx.x % cols;
  __shared__ float4 acc_s[512];
  __shared__ float sum_sh[512];
  auto slot_of = [&](int i) { return i == 0 ? 2 * (int64_t)blockIdx.x + 1 : 2 * (int64_t)(blockIdx.x + i); };
  float top = -INFINITY;
  for (int i = 0; i < n; ++i) top = fmaxf(top, P.part_ml[slot_of(i) * heads + row].x);
  const float base = top == -INFINITY ? 0.0f : top;
  float4 a = make_float4(0, 0, 0, 0);
  float l = 0.0f;
  if (g < groups)
    for (int i = g; i < n; i += groups) {
      const float2 ml = P.part_ml[slot_of(i) * heads + row];
      const float w = ex2_approx(ml.x - base);
      const float4 x = *reinterpret_cast<const float4*>(P.part + (slot_of(i) * heads + row) * P.D + col * 4);
      a.x += w * x.x;
      a.y += w * x.y;
      a.z += w * x.z;
      a.w += w * x.w;
      l += w * ml.y;
    }
  acc_s[threadIdx.x] = a;
  sum_sh[threadIdx.x] = l;
  __syncthreads();
  if (g != 0) return;
  for (int w = 1; w < groups; ++w) {
    const float4 x = acc_s[w * cols + col];
    a.x += x.x;
    a.y += x.y;
    a.z += x.z;
    a.w += x.w;
    l += sum_sh[w * cols + col];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(P.o + b * P.o_sb + (int64_t)hq * P.o_sh + col * 8) =
      make_uint2(pack2<F16>(a.x * inv, a.y * inv), pack2<F16>(a.z * inv, a.w * inv));
  if (P.lse && col == 0) P.lse[(int64_t)b * P.Hq + hq] = l == 0.0f ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
}

// Workspace: partial outputs, their maxima and sums, the cut pairs.
struct DecodeSpace {
  size_t part, ml, meta, total;
};
DecodeSpace decode_space(int grid, int heads, int D) {
  DecodeSpace s;
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  s.part = 0;
  s.ml = up((size_t)2 * grid * heads * D * 4);
  s.meta = s.ml + up((size_t)2 * grid * heads * 8);
  s.total = s.meta + up((size_t)grid * 8);
  return s;
}

// CTAs of any sm_103 part; the workspace is sized for them without asking a device.
constexpr int DEC_GRID_MAX = 160;

template <bool F16, int NT, int WARPS>
ffpa_status launch_decode_as(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(&decode_kernel<F16, NT, WARPS>);
  const ffpa_status st = set_smem_attr_once(fn, dev, (int)pl.smem);
  if (st != FFPA_OK) return st;
  decode_kernel<F16, NT, WARPS><<<grid, pl.wd * pl.wk * 32, pl.smem, stream>>>(P);
  if (cudaGetLastError() != cudaSuccess) return FFPA_ERR_CUDA;
  const int heads = 8 * NT;
  const int rows = P.group < heads ? P.group : heads;
  join_kernel<F16><<<dim3(grid, rows), 512, 0, stream>>>(P, heads);
  return cudaGetLastError() == cudaSuccess ? FFPA_OK : FFPA_ERR_CUDA;
}

template <bool F16>
ffpa_status launch_decode(const DecodeParams& P, const DecodePlan& pl, int grid, int dev, cudaStream_t stream) {
  const bool wide = pl.wd * pl.wk > 8;
  if (pl.nt == 1)
    return wide ? launch_decode_as<F16, 1, 16>(P, pl, grid, dev, stream) : launch_decode_as<F16, 1, 8>(P, pl, grid, dev, stream);
  if (pl.nt == 2)
    return wide ? launch_decode_as<F16, 2, 16>(P, pl, grid, dev, stream) : launch_decode_as<F16, 2, 8>(P, pl, grid, dev, stream);
  return launch_decode_as<F16, 4, 8>(P, pl, grid, dev, stream);
}

}  // namespace
}  // namespace ffpa

extern "C" {

size_t ffpa_decode_paged_workspace_bytes(int Hq, int Hkv, int D) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || D < 64 || D > 1024 || D % 8 != 0) return 0;
  return ffpa::decode_space(ffpa::DEC_GRID_MAX, 8 * ffpa::decode_nt(Hq / Hkv, D), D).total;
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
  if (workspace_bytes < decode_space(DEC_GRID_MAX, 8 * pl.nt, D).total) return FFPA_ERR_INVALID;
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
  const int grid = sms < DEC_GRID_MAX ? sms : DEC_GRID_MAX;

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
  P.meta = reinterpret_cast<int2*>(ws + sp.meta);
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
  P.wd = pl.wd;
  P.wk = pl.wk;
  P.tile = pl.tile;
  P.pitch = pl.pitch;
  P.slots = pl.slots;
  P.scale_log2 = sc * 1.4426950408889634f;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FFPA_FP16 ? launch_decode<true>(P, pl, grid, dev, s) : launch_decode<false>(P, pl, grid, dev, s);
}

}  // extern "C"
