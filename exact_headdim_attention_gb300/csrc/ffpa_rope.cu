// RMS norm of query and key heads with the rotation by position, forward, and
// the same with keys and values going to their slots of a paged cache.
//
// Each row is read once and written once: the memory's bandwidth is the bound.
// A work item is a few heads of one token, so that the cosines and sines of
// that token (one sincospif per pair) are shared by its heads.
#include "ffpa_rope.cuh"

namespace ffpa {
namespace {

constexpr int ROPE_THREADS = 256;

template <bool F16, int VEC, int LPR, int ITER, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(const RopeParams P) {
  const int lane = threadIdx.x % LPR;
  const int64_t group = (int64_t)blockIdx.x * (ROPE_THREADS / LPR) + threadIdx.x / LPR;
  const int64_t all = P.items[0] + P.items[1] + P.items_v;
  // Whole warps stay in the loop: the lanes of a row talk through shuffles.
  const int64_t warp_first = group - (threadIdx.x % 32) / LPR;
  const int64_t stride = (int64_t)gridDim.x * (ROPE_THREADS / LPR);
  RopeChunk<VEC> ch[ITER];
  long long freq[ITER][VEC];
#pragma unroll
  for (int k = 0; k < ITER; ++k) {
    ch[k] = rope_chunk<VEC, INTER>(lane + k * LPR, P.D, P.rot);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      freq[k][i] = ch[k].live && ch[k].pair ? freq_turns(P.inv_freq[(lane + k * LPR) * VEC + i]) : 0;
  }
  for (int64_t first = warp_first; first < all; first += stride) {
    const int64_t item = first + (threadIdx.x % 32) / LPR;
    const bool in = item < all;
    const int which = item < P.items[0] ? 0 : item < P.items[0] + P.items[1] ? 1 : 2;
    const int64_t local = !in ? 0 : which == 0 ? item : which == 1 ? item - P.items[0] : item - P.items[0] - P.items[1];
    const int wt = which == 2 ? 1 : which;
    const RopeTensor& t = P.t[wt];
    const int64_t token = local / P.chunks[wt];
    const int h0 = (int)(local % P.chunks[wt]) * P.heads_per[wt];
    const int h1 = in ? min(t.H, h0 + P.heads_per[wt]) : h0;
    const int b = (int)(token / P.N), n = (int)(token % P.N);
    // The slot of a cached row; a negative one is padding and is not stored.
    int64_t page = 0, slot = -1;
    if (which > 0 && P.slots && in) {
      slot = P.slots[n];
      if (slot >= P.n_slots) {
        report_invalid(P.err);
        slot = -1;
      }
      if (slot >= 0) {
        page = slot / P.slot_page;
        slot -= page * P.slot_page;
      }
    }
    if (which == 2) {
      if (slot >= 0)
        for (int h = h0; h < h1; ++h) {
          const uint4* src = reinterpret_cast<const uint4*>(P.v + h * P.vs[0] + n * P.vs[1]);
          uint4* dst = reinterpret_cast<uint4*>(P.vc + page * P.vcs[0] + slot * P.vcs[1] + h * P.vcs[2]);
          for (int i = lane; i < P.D / 8; i += LPR) dst[i] = src[i];
        }
    }
    float cs[ITER][VEC], sn[ITER][VEC], w[ITER][2 * VEC];
    if (which < 2 && in) {
      const long long pos = P.rot ? position_of(P, b, n) : 0;
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        if (!ch[k].live) continue;
        if (ch[k].pair) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) turn(pos, freq[k][i], P.rope_scale, cs[k][i], sn[k][i]);
        }
        if (t.w) {
          load_weight<F16, VEC>(t.w, P.w32, ch[k].a, w[k]);
          load_weight<F16, VEC>(t.w, P.w32, ch[k].b, w[k] + VEC);
        }
      }
    }
    const int heads = P.heads_per[0] > P.heads_per[1] ? P.heads_per[0] : P.heads_per[1];
    for (int i = 0; i < heads; ++i) {
      const int h = h0 + i;
      const bool on = which < 2 && h < h1;
      float x[ITER][2 * VEC];
      float sq = 0.0f;
      if (on) {
        const char* src = t.x + b * t.xs[0] + h * t.xs[1] + n * t.xs[2];
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
          if (!ch[k].live) continue;
          widen<F16, VEC>(*reinterpret_cast<const Raw<VEC>*>(src + ch[k].a * 2), x[k]);
          widen<F16, VEC>(*reinterpret_cast<const Raw<VEC>*>(src + ch[k].b * 2), x[k] + VEC);
#pragma unroll
          for (int j = 0; j < 2 * VEC; ++j) sq += x[k][j] * x[k][j];
        }
      }
      sq = row_sum<LPR>(sq);
      if (!on) continue;
      const float r = rsqrtf(sq / P.D + P.eps);
      char* dst = t.y + b * t.ys[0] + h * t.ys[1] + n * t.ys[2];
      if (which == 1 && P.slots) {
        if (slot < 0) continue;
        dst = P.kc + page * P.kcs[0] + slot * P.kcs[1] + h * P.kcs[2];
      }
#pragma unroll
      for (int k = 0; k < ITER; ++k) {
        if (!ch[k].live) continue;
        if (t.w) {
#pragma unroll
          for (int j = 0; j < 2 * VEC; ++j) x[k][j] *= r * w[k][j];
        }
        if (ch[k].pair) rotate<VEC, INTER, false>(x[k], cs[k], sn[k]);
        *reinterpret_cast<Raw<VEC>*>(dst + ch[k].a * 2) = narrow<F16, VEC>(x[k]);
        *reinterpret_cast<Raw<VEC>*>(dst + ch[k].b * 2) = narrow<F16, VEC>(x[k] + VEC);
      }
    }
  }
}

template <bool F16, int VEC, int LPR, int ITER>
ffpa_status launch_rope_as(const RopeParams& P, bool inter, int sms, cudaStream_t stream) {
  const int64_t all = P.items[0] + P.items[1] + P.items_v;
  const int64_t per = ROPE_THREADS / LPR;
  int64_t grid = (all + per - 1) / per;
  if (grid > (int64_t)sms * 16) grid = (int64_t)sms * 16;
  if (inter)
    rope_kernel<F16, VEC, LPR, ITER, true><<<(int)grid, ROPE_THREADS, 0, stream>>>(P);
  else
    rope_kernel<F16, VEC, LPR, ITER, false><<<(int)grid, ROPE_THREADS, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? FFPA_OK : FFPA_ERR_CUDA;
}

template <bool F16>
ffpa_status launch_rope(RopeParams& P, bool inter, int sms, cudaStream_t stream) {
  const int64_t tokens = (int64_t)P.B * P.N;
  // Heads of an item: as many as leave every SM some 32 rows in work.
  for (int i = 0; i < 2; ++i) {
    int per = 8;
    while (per > 1 && tokens * ((P.t[i].H + per - 1) / per) < (int64_t)sms * 32) per /= 2;
    P.heads_per[i] = per;
    P.chunks[i] = (P.t[i].H + per - 1) / per;
    P.items[i] = P.t[i].x ? tokens * P.chunks[i] : 0;
  }
  P.items_v = P.slots ? tokens * P.chunks[1] : 0;
  if (rope_vec(P.D, P.rot) == 8) {
    const int n = P.D / 16;
    if (n <= 4) return launch_rope_as<F16, 8, 4, 1>(P, inter, sms, stream);
    if (n <= 8) return launch_rope_as<F16, 8, 8, 1>(P, inter, sms, stream);
    if (n <= 16) return launch_rope_as<F16, 8, 16, 1>(P, inter, sms, stream);
    if (n <= 32) return launch_rope_as<F16, 8, 32, 1>(P, inter, sms, stream);
    return launch_rope_as<F16, 8, 32, 2>(P, inter, sms, stream);
  }
  const int n = P.D / 8;
  if (n <= 16) return launch_rope_as<F16, 4, 16, 1>(P, inter, sms, stream);
  if (n <= 32) return launch_rope_as<F16, 4, 32, 1>(P, inter, sms, stream);
  if (n <= 64) return launch_rope_as<F16, 4, 32, 2>(P, inter, sms, stream);
  return launch_rope_as<F16, 4, 32, 4>(P, inter, sms, stream);
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
  if ((int64_t)B * N > 0x7fffffffLL) return FFPA_ERR_INVALID;
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
  return dt == FFPA_FP16 ? launch_rope<true>(P, rope->interleaved != 0, sms, s)
                         : launch_rope<false>(P, rope->interleaved != 0, sms, s);
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
  return dt == FFPA_FP16 ? launch_rope<true>(P, rope->interleaved != 0, sms, s)
                         : launch_rope<false>(P, rope->interleaved != 0, sms, s);
}

}  // extern "C"
