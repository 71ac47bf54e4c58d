// RMS norm of query and key heads with the rotation by position, forward, and
// the same with keys and values going to a paged cache of 16-bit values.
#include "ffpa_rope_fwd.cuh"

namespace ffpa {

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
  return dt == FFPA_FP16 ? launch_rope<false, true>(P, rope->interleaved != 0, sms, dev, s)
                         : launch_rope<false, false>(P, rope->interleaved != 0, sms, dev, s);
}

ffpa_status ffpa_kv_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                           ffpa_dtype dt, int T, int Hq, int Hkv, int D, int num_pages, int page_size,
                           const int64_t q_str[3], const int64_t k_str[3], const int64_t v_str[3],
                           const int64_t qo_str[3], const int64_t kc_str[4], const int64_t vc_str[4],
                           const int64_t* slots, const ffpa_rope* rope, ffpa_stream_t stream,
                           const ffpa_options* options) {
  using namespace ffpa;
  return append_entry<false>(q, k, v, q_out, k_cache, v_cache, nullptr, nullptr, dt, T, Hq, Hkv, D, num_pages, page_size, q_str,
                             k_str, v_str, qo_str, kc_str, vc_str, nullptr, nullptr, slots, rope, stream, options);
}

}  // extern "C"
