#pragma once
// RMS norm of query and key heads with the rotation by position, forward, and
// the same with keys and values going to their slots of a paged cache, as 16-bit
// values (ffpa_rope.cu) or as e4m3 codes (ffpa_append_fp8.cu).
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
//  - e4m3: a row's lanes hold it in fp32 when its largest value is known (one
//    more maximum over the lanes), so it is still read and written once.  Bound by a row's chain
//    (copy, products, maximum, division, codes), with too few rows on their way to cover it: issue slots are 59 to 61 % busy and
//    the memory at 72 to 78 % of its rate.  T16001 Hq16 Hkv4 D256, half the head rotated, 75 us, 4.8 TB/s; T5000 of 32 heads
//    of D128 as they are 39.5 us, 5.2 TB/s; T16384 of 8 and 8 heads D128 42 us, D320 (T8192) 73.
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

template <int LPR>
__device__ __forceinline__ float row_max_of(float x) {
#pragma unroll
  for (int d = LPR / 2; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, d));
  return x;
}

// 2 VEC values as codes.
template <int VEC>
__device__ __forceinline__ void store_codes(char* to, const float2* y, float f) {
  uint32_t c[VEC / 4];
#pragma unroll
  for (int i = 0; i < VEC / 4; ++i)
    c[i] = pack_e4m3x4(y[2 * i].x * f, y[2 * i].y * f, y[2 * i + 1].x * f, y[2 * i + 1].y * f);
  if (VEC == 8)
    *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[VEC / 4 - 1]);
  else
    *reinterpret_cast<uint32_t*>(to) = c[0];
}

template <bool E4M3, bool F16, int VEC, int LPR, int ITER, bool INTER>
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
    float* dst_scale = nullptr;
    int64_t scale_h = 0;
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
      if (E4M3) {
        scale_h = it.which == 2 ? P.v_scale_s[1] : P.k_scale_s[1];
        dst_scale = it.which == 2 ? P.v_scale + page * P.v_scale_s[0] + slot : P.k_scale + page * P.k_scale_s[0] + slot;
        dst_scale += it.h0 * scale_h;
      }
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
    const bool codes = E4M3 && __any_sync(~0u, it.which > 0);   // (rows of a warp may be of both kinds)
    const bool turned = it.which < 2 && (!E4M3 || norm || P.rot > 0);   // (e4m3: else rows are as they came)
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
      if (E4M3 && codes) {
        // Codes do not depend on the row's norm: it goes into the scale alone (but in the smallest rows).
        float2 y[ITER][VEC];
        float top = 0.0f;
        if (on) {
#pragma unroll
          for (int k = 0; k < ITER; ++k)
            if (ch[k].live) {
              float2 x[VEC];
              widen<F16, VEC>(ra[k], x);
              widen<F16, VEC>(rb[k], x + VEC / 2);
              if (turned) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[k][i] = mul2(x[i], f0[k][i]);
                if (ch[k].pair) {
#pragma unroll
                  for (int i = 0; i < VEC; ++i) y[k][i] = fma2(partner<VEC, INTER>(x, i), f1[k][i], y[k][i]);
                }
              } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[k][i] = x[i];
              }
#pragma unroll
              for (int i = 0; i < VEC; ++i) top = fmax3(top, fabsf(y[k][i].x), fabsf(y[k][i].y));
            }
        }
        top = row_max_of<LPR>(top);
        if (!on) continue;
        const float r = norm ? rsqrtf(sum * inv_d + P.eps) : 1.0f;
        if (it.which == 0) {                       // (queries beside keys in a warp)
#pragma unroll
          for (int k = 0; k < ITER; ++k)
            if (ch[k].live) {
#pragma unroll
              for (int i = 0; i < VEC; ++i) y[k][i] = mul2(y[k][i], make_float2(r, r));
              *reinterpret_cast<Raw<VEC>*>(dst + ch[k].a * 2) = narrow<F16, VEC>(y[k]);
              *reinterpret_cast<Raw<VEC>*>(dst + ch[k].b * 2) = narrow<F16, VEC>(y[k] + VEC / 2);
            }
        } else {
          constexpr float least = 0x1p-117f;
          const float whole = top * r;
          float f = 448.0f / top, scale = whole * (1.0f / 448.0f);
          // Rows whose factor or scale would leave the normal range, zeros and those that the norm makes NaN
          // among them: the norm's factor goes into the row first, and the smallest scale is a normal number
          // whose inverse is finite.  (A NaN spreads through the norm; an infinity has the norm's factor 0.)
          if (top < least || !(whole >= least)) {
            if (top != 0.0f) {
#pragma unroll
              for (int k = 0; k < ITER; ++k)
#pragma unroll
                for (int i = 0; i < VEC; ++i) y[k][i] = mul2(y[k][i], make_float2(r, r));
            }
            f = top == 0.0f ? 1.0f : 448.0f / fmaxf(whole, least);
            scale = whole > 0.0f ? fmaxf(whole, least) * (1.0f / 448.0f) : r == r ? 1.0f : r;
          }
#pragma unroll
          for (int k = 0; k < ITER; ++k)
            if (ch[k].live) {
              store_codes<VEC>(dst + ch[k].a, y[k], f);
              store_codes<VEC>(dst + ch[k].b, y[k] + VEC / 2, f);
            }
          if (lane == 0) *dst_scale = scale;
          dst_scale += scale_h;
        }
        dst += dst_h;
        continue;
      }
      if (!on) continue;
      const float r = norm ? rsqrtf(sum * inv_d + P.eps) : 1.0f;
      const float2 r2 = make_float2(r, r);
#pragma unroll
      for (int k = 0; k < ITER; ++k)
        if (ch[k].live) {
          if (turned) {
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

template <bool E4M3, bool F16, int VEC, int LPR, int ITER>
ffpa_status launch_rope_as(const RopeParams& P, bool inter, int sms, int dev, cudaStream_t stream) {
  const int64_t all = P.items[0] + P.items[1] + P.items_v;
  const int64_t per = ROPE_THREADS / LPR;
  int64_t grid = (all + per - 1) / per;
  // As many blocks as are resident, so that the frequencies are formed once
  // and no last wave is left over.
  const int64_t resident = (int64_t)sms * rope_blocks<VEC, ITER>();
  if (grid > resident) grid = resident;
  const int smem = ROPE_DEPTH * rope_row_bytes<VEC, ITER>() + 2 * P.D * 4;
  auto fn = inter ? &rope_kernel<E4M3, F16, VEC, LPR, ITER, true> : &rope_kernel<E4M3, F16, VEC, LPR, ITER, false>;
  const ffpa_status st = set_smem_attr_once(reinterpret_cast<const void*>(fn), dev, smem);
  if (st != FFPA_OK) return st;
  fn<<<(int)grid, ROPE_THREADS, smem, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? FFPA_OK : FFPA_ERR_CUDA;
}

template <bool E4M3, bool F16>
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
    if (n <= 4) return launch_rope_as<E4M3, F16, 8, 4, 1>(P, inter, sms, dev, stream);
    if (n <= 8) return launch_rope_as<E4M3, F16, 8, 8, 1>(P, inter, sms, dev, stream);
    if (n <= 16) return launch_rope_as<E4M3, F16, 8, 16, 1>(P, inter, sms, dev, stream);
    if (n <= 32) return launch_rope_as<E4M3, F16, 8, 32, 1>(P, inter, sms, dev, stream);
    return launch_rope_as<E4M3, F16, 8, 32, 2>(P, inter, sms, dev, stream);
  }
  const int n = P.D / 8;
  if (n <= 16) return launch_rope_as<E4M3, F16, 4, 16, 1>(P, inter, sms, dev, stream);
  if (n <= 32) return launch_rope_as<E4M3, F16, 4, 32, 1>(P, inter, sms, dev, stream);
  if (n <= 64) return launch_rope_as<E4M3, F16, 4, 32, 2>(P, inter, sms, dev, stream);
  return launch_rope_as<E4M3, F16, 4, 32, 4>(P, inter, sms, dev, stream);
}


// The append's entry points (scales and their strides where the cache holds codes).
template <bool E4M3>
ffpa_status append_entry(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                         float* k_scale, float* v_scale, ffpa_dtype dt, int T, int Hq, int Hkv, int D, int num_pages,
                         int page_size, const int64_t* q_str, const int64_t* k_str, const int64_t* v_str,
                         const int64_t* qo_str, const int64_t* kc_str, const int64_t* vc_str, const int64_t* ks_str,
                         const int64_t* vs_str, const int64_t* slots, const ffpa_rope* rope, ffpa_stream_t stream,
                         const ffpa_options* options) {
  RopeParams P{};
  ffpa_status st = rope_params(rope, dt, 1, Hq, Hkv, T, D, &P);
  if (st != FFPA_OK) return st;
  if (E4M3 && D % 16 != 0) return FFPA_ERR_UNSUPPORTED;   // rows of whole 16-byte pieces
  if (num_pages < 1 || page_size < 1) return FFPA_ERR_INVALID;
  if (T == 0) return FFPA_OK;
  if (!k || !v || !k_cache || !v_cache || !slots || !k_str || !v_str || !kc_str || !vc_str) return FFPA_ERR_INVALID;
  if (q && (!q_out || !q_str || !qo_str)) return FFPA_ERR_INVALID;
  const int unit = E4M3 ? 16 : 8, bytes = E4M3 ? 1 : 2;
  if (!rows_ok(k_str, {T, Hkv, D}) || !rows_ok(v_str, {T, Hkv, D}) ||
      !rows_ok(kc_str, {num_pages, page_size, Hkv, D}, unit) || !rows_ok(vc_str, {num_pages, page_size, Hkv, D}, unit))
    return FFPA_ERR_INVALID;
  if (E4M3 && (!k_scale || !v_scale || !ks_str || !vs_str || !on_boundary(k_scale, 4) || !on_boundary(v_scale, 4) ||
               !scales_ok(ks_str, num_pages, Hkv, page_size) || !scales_ok(vs_str, num_pages, Hkv, page_size)))
    return FFPA_ERR_INVALID;
  if (q && (!rows_ok(q_str, {T, Hq, D}) || !rows_ok(qo_str, {T, Hq, D}))) return FFPA_ERR_INVALID;
  if (!on_boundary(q, 16) || !on_boundary(k, 16) || !on_boundary(v, 16) || !on_boundary(q_out, 16) ||
      !on_boundary(k_cache, 16) || !on_boundary(v_cache, 16) || !on_boundary(slots, 8))
    return FFPA_ERR_INVALID;
  int dev = 0;
  const bool turns = rope->rot_dim > 0;
  st = call_device({k, v, q, q ? q_out : nullptr, k_cache, v_cache, slots, k_scale, v_scale, turns ? rope->positions : nullptr,
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
    P.kcs[j] = kc_str[j] * bytes;
    P.vcs[j] = vc_str[j] * bytes;
  }
  if (E4M3) {
    P.k_scale = k_scale;
    P.v_scale = v_scale;
    for (int j = 0; j < 2; ++j) {
      P.k_scale_s[j] = ks_str[j];
      P.v_scale_s[j] = vs_str[j];
    }
  }
  P.slots = slots;
  P.n_slots = (int64_t)num_pages * page_size;
  P.slot_page = page_size;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return dt == FFPA_FP16 ? launch_rope<E4M3, true>(P, rope->interleaved != 0, sms, dev, s)
                         : launch_rope<E4M3, false>(P, rope->interleaved != 0, sms, dev, s);
}

}  // namespace
}  // namespace ffpa
