// Attention of one new token per request over a paged cache of e4m3 codes with a
// scale for each key and value row: the kernels of ffpa_decode.cuh, with the
// codes widened to fp16 (which holds every one) on their way into the products.
#include "ffpa_decode.cuh"

extern "C" {

size_t ffpa_decode_paged_fp8_workspace_bytes(int Hq, int Hkv, int D) {
  return D % 16 == 0 ? ffpa::decode_bytes(Hq, Hkv, D) : 0;
}

ffpa_status ffpa_decode_paged_fp8(const void* q, const void* k_cache, const void* v_cache, const float* k_scale,
                                  const float* v_scale, void* o, float* lse, ffpa_dtype dt, int B, int Hq, int Hkv,
                                  int D, int num_pages, int page_size, int max_pages, const int64_t q_str[3],
                                  const int64_t k_str[4], const int64_t v_str[4], const int64_t ks_str[3],
                                  const int64_t vs_str[3], const int64_t o_str[3], const int32_t* block_table,
                                  int64_t table_str, const int32_t* seq_lens, const float* scale, int enable_gqa,
                                  void* workspace, size_t workspace_bytes, ffpa_stream_t stream,
                                  const ffpa_options* options) {
  using namespace ffpa;
  const DecodeShape s{B, Hq, Hkv, D, num_pages, page_size, max_pages, k_str, v_str};
  return decode_entry<DECODE_E4M3>(q, k_cache, v_cache, o, lse, dt, s, q_str, o_str, block_table, table_str, seq_lens,
                                   k_scale, v_scale, ks_str, vs_str, scale, enable_gqa, workspace, workspace_bytes, stream,
                                   options);
}

}  // extern "C"
