// Keys (normed and rotated) and values into a paged cache of e4m3 codes with a
// scale for each row: the kernel of ffpa_rope_fwd.cuh.
#include "ffpa_rope_fwd.cuh"

extern "C" {

ffpa_status ffpa_kv_append_fp8(const void* q, const void* k, const void* v, void* q_out, void* k_cache, void* v_cache,
                               float* k_scale, float* v_scale, ffpa_dtype dt, int T, int Hq, int Hkv, int D,
                               int num_pages, int page_size, const int64_t q_str[3], const int64_t k_str[3],
                               const int64_t v_str[3], const int64_t qo_str[3], const int64_t kc_str[4],
                               const int64_t vc_str[4], const int64_t ks_str[3], const int64_t vs_str[3],
                               const int64_t* slots, const ffpa_rope* rope, ffpa_stream_t stream,
                               const ffpa_options* options) {
  using namespace ffpa;
  return append_entry<true>(q, k, v, q_out, k_cache, v_cache, k_scale, v_scale, dt, T, Hq, Hkv, D, num_pages, page_size, q_str,
                            k_str, v_str, qo_str, kc_str, vc_str, ks_str, vs_str, slots, rope, stream, options);
}

}  // extern "C"
