#pragma once
// RMS norm of query and key heads with the rotation by position: what the
// forward, the cache append and the backward share.
//
//   y = x * rsqrt(mean(x^2) + eps) * w           (x when there is no weight)
//   pair i of the first rot columns, angle t = position * inv_freq[i]:
//     (a, b) -> rope_scale * (a cos t - b sin t, b cos t + a sin t)
//   pairs (i, rot/2 + i), or (2i, 2i+1) when interleaved; later columns stay.
//
// A row (one head of one token) belongs to LPR lanes.  A lane holds ITER
// chunks of 2 VEC values: two VEC-wide vectors that hold VEC whole pairs, so
// that a rotation never leaves its lane, or two behind the rotated columns.
//
// Angles are taken in turns, as 64-bit fixed-point fractions: position times
// frequency wraps there as the angle does, so that far positions need neither
// a table nor 64-bit floating point per angle (off by 2^-34 turns, by the position times
// the frequency's rounding to 2^-65 turns, and by that to a double, 2^-52 of the angle).
#include "ffpa_paged.cuh"

namespace ffpa {

struct RopeTensor {
  const char* x;       // input rows
  char* y;             // output rows
  int64_t xs[3], ys[3];   // byte strides (b, h, n)
  const void* w;       // norm weight [D], or NULL
  int H;
};

struct RopeParams {
  RopeTensor t[2];     // queries, keys
  const char* pos;
  int64_t pos_s[2];    // byte strides (b, n)
  const double* inv_freq;
  int pos64, rot, w32, B, N, D;
  float eps, rope_scale;
  int heads_per[2];    // heads of one work item
  unsigned items[2];   // work items of queries and of keys
  int chunks[2];       // head chunks of a token
  // append (keys go to pages, values are copied): slots == NULL otherwise
  const int64_t* slots;
  int64_t n_slots, slot_page;
  char *kc, *vc;
  const char* v;
  int64_t vs[2], kcs[3], vcs[3];   // byte strides (h, n); (page, slot, h)
  unsigned items_v;    // and of values
  int* err;
  // backward
  const char* g[2];    // gradients of the outputs
  int64_t gs[2][3];
  float* part[2];      // per-block weight gradients
  void* dw[2];
  int blocks[2];
};

// The vector width that the pairs' halves and the row's end allow.
inline int rope_vec(int D, int rot) { return D % 16 == 0 && rot % 16 == 0 ? 8 : 4; }
// Heads that share a token's cosines and sines: 8 where the rows fill their
// lanes (a power of two of chunks) and the memory is the bound, 16 where lanes
// idle and the arithmetic weighs more (T8192 D512: 110 us with 8 and 118 with
// 16; T8192 D320: 61 and 55; T16384 D120: 60 and 54); fewer where that would leave
// SMs without work.
inline int rope_heads(int D, int rot, int64_t tokens, int H, int sms) {
  const int n = D / (2 * rope_vec(D, rot));
  int per = (n & (n - 1)) == 0 ? 8 : 16;
  while (per > 1 && tokens * ((H + per - 1) / per) < (int64_t)sms * 32) per /= 2;
  return per;
}

template <int VEC>
struct RopeChunk {
  int a, b;      // columns of the two vectors
  bool pair;     // rotated
  bool live;
};

// Chunk j of a row: a vector of the first half of the rotated columns and the
// one as far into their second half, then so for the columns behind them: the
// lanes of a row read neighbouring vectors.  A vector holds whole pairs when
// they are interleaved; else the two vectors hold each other's.
template <int VEC>
__device__ __forceinline__ RopeChunk<VEC> rope_chunk(int j, int D, int rot) {
  RopeChunk<VEC> c;
  const int np = rot / (2 * VEC);
  c.live = j < D / (2 * VEC);
  c.pair = j < np;
  c.a = c.pair ? j * VEC : rot + (j - np) * VEC;
  c.b = c.a + (c.pair ? rot : D - rot) / 2;
  return c;
}
// Number (of a frequency) of pair i of a chunk.
template <int VEC, bool INTER>
__device__ __forceinline__ int pair_number(const RopeChunk<VEC>& c, int i) {
  return !INTER ? c.a + i : i < VEC / 2 ? c.a / 2 + i : c.b / 2 + i - VEC / 2;
}

template <int VEC>
struct alignas(VEC * 2) Raw {
  uint32_t u[VEC / 2];
};

// The two vectors of a chunk as a thread keeps them in its own place of shared
// memory: vector v of chunk k at [k][v][thread].
template <int VEC>
__device__ __forceinline__ Raw<VEC> own_load(const char* at) {
  return *reinterpret_cast<const Raw<VEC>*>(at);
}

template <bool F16, int VEC>
__device__ __forceinline__ void widen(const Raw<VEC>& r, float2* x) {
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) x[i] = unpack2<F16>(r.u[i]);
}
template <bool F16, int VEC>
__device__ __forceinline__ Raw<VEC> narrow(const float2* x) {
  Raw<VEC> r;
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i) r.u[i] = pack2<F16>(x[i].x, x[i].y);
  return r;
}

template <bool F16>
__device__ __forceinline__ float one_weight(const void* w, int w32, int d) {
  return w32 ? static_cast<const float*>(w)[d] : unpack2<F16>(static_cast<const uint16_t*>(w)[d]).x;
}
// VEC weights from column col on.
template <bool F16, int VEC>
__device__ __forceinline__ void load_weight(const void* w, int w32, int col, float2* x) {
#pragma unroll
  for (int i = 0; i < VEC / 2; ++i)
    x[i] = make_float2(one_weight<F16>(w, w32, col + 2 * i), one_weight<F16>(w, w32, col + 2 * i + 1));
}

// A frequency in turns per position, as a fraction of 2^64 (whole turns drop out).
__device__ __forceinline__ long long freq_turns(double inv_freq) {
  double f = inv_freq * 0.15915494309189534561;   // 1 / (2 pi)
  f -= rint(f);
  return __double2ll_rn(f * 18446744073709551616.0);
}
// The call's frequencies in turns, once per block (rot / 2 <= 512 of them):
// that of pair i of chunk j at [i][j], so that the lanes of a row read neighbours.
template <int VEC, bool INTER>
__device__ __forceinline__ void load_freqs(const RopeParams& P, long long* freq_s) {
  const int np = P.rot / (2 * VEC);
  for (int x = threadIdx.x; x < P.rot / 2; x += blockDim.x) {
    const int i = x / np, j = x - i * np;
    freq_s[x] = freq_turns(P.inv_freq[pair_number<VEC, INTER>(rope_chunk<VEC>(j, P.D, P.rot), i)]);
  }
  __syncthreads();
}
// Cosine and sine of position times frequency, times scale.  The angle in turns goes
// to the nearest quarter (its two highest bits) and the rest, u quarters with |u| <= 1/2,
// to fp32 from 2^-34 turns on.  On it two polynomials in w = u^2 (minimax fits by Remez exchange
// of sin(pi u / 2) / u and (cos(pi u / 2) - 1) / w, off by 2^-28 and 2^-34) leave both
// functions off by at most 2^-22 of themselves, however small.  (The hardware's, off by
// 2^-21 of one, lost small sines and cosines; with them T8192 D512 took 107.6 us in place of
// 109.9, its backward 88.2 in place of 90.4.)
__device__ __forceinline__ void turn(long long pos, long long freq, float scale, float& c, float& s) {
  const unsigned long long t = static_cast<unsigned long long>(pos) * static_cast<unsigned long long>(freq);
  const unsigned hi = static_cast<unsigned>(t >> 32), lo = static_cast<unsigned>(t), quarter = hi + 0x20000000u;
  const float u = static_cast<float>(static_cast<int>(__funnelshift_l(lo, hi, 2))) * 0x1p-32f, w = u * u;
  float sn = fmaf(w, -0x1.2d9278p-8f, 0x1.465e90p-4f), cs = fmaf(w, 0x1.d9f6ecp-11f, -0x1.55c662p-6f);
  sn = fmaf(w, sn, -0x1.4abbb8p-1f);
  cs = fmaf(w, cs, 0x1.03c1dep-2f);
  sn = fmaf(w, sn, 0x1.921fb6p+0f);
  cs = fmaf(w, cs, -0x1.3bd3ccp+0f);
  sn = u * sn * scale;
  cs = fmaf(w, cs, 1.0f) * scale;
  const bool odd = quarter & 0x40000000u;          // a quarter on: (c, s) -> (-s, c)
  c = __uint_as_float(__float_as_uint(odd ? sn : cs) ^ ((quarter + 0x40000000u) & 0x80000000u));
  s = __uint_as_float(__float_as_uint(odd ? cs : sn) ^ (quarter & 0x80000000u));
}

__device__ __forceinline__ long long position_of(const RopeParams& P, int b, int n) {
  const char* p = P.pos + b * P.pos_s[0] + n * P.pos_s[1];
  return P.pos64 ? *reinterpret_cast<const long long*>(p) : *reinterpret_cast<const int*>(p);
}

// Two fp32 values in one instruction.
__device__ __forceinline__ uint64_t pair2(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 both2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair2(a)), "l"(pair2(b)), "l"(pair2(c)));
  return both2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair2(a)), "l"(pair2(b)));
  return both2(r);
}

// A chunk in fp32 is VEC twos of neighbouring columns, those of the first
// vector, then of the second.  The other halves of the pairs in two i: two
// i +- VEC / 2, or the same two swapped when interleaved.
template <int VEC, bool INTER>
__device__ __forceinline__ float2 partner(const float2* x, int i) {
  return INTER ? make_float2(x[i].y, x[i].x) : x[i < VEC / 2 ? i + VEC / 2 : i - VEC / 2];
}
// The pair that value j (0, 1) of two i belongs to, and whether as its b.
template <int VEC, bool INTER>
__device__ __forceinline__ constexpr int pair_of(int i, int j) { return INTER ? i : 2 * (i % (VEC / 2)) + j; }
template <int VEC, bool INTER>
__device__ __forceinline__ constexpr bool second_of(int i, int j) { return INTER ? j == 1 : i >= VEC / 2; }

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) x += __shfl_xor_sync(~0u, x, d);
  return x;
}

// Host: the checks of ffpa_rope and the parameters that the passes share.
ffpa_status rope_params(const ffpa_rope* r, ffpa_dtype dt, int B, int Hq, int Hkv, int N, int D, RopeParams* P);

}  // namespace ffpa
