// The entry of decode attention behind shared pages; its kernels are not here yet and every call is refused.
#include "ffpa_paged.cuh"
extern "C" {
size_t ffpa_decode_shared_workspace_bytes(int B, int Hq, int Hkv, int D) { return 0; }
ffpa_status ffpa_decode_shared(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                               ffpa_dtype dt, int B, int Hq, int Hkv, int D, int num_pages, int page_size,
                               int max_pages, int n_shared, const int64_t q_str[3], const int64_t k_str[4],
                               const int64_t v_str[4], const int64_t o_str[3], const int32_t* shared_pages,
                               const int32_t* shared_len, const int32_t* block_table, int64_t table_str,
                               const int32_t* seq_lens, const float* scale, int enable_gqa, void* workspace,
                               size_t workspace_bytes, ffpa_stream_t stream, const ffpa_options* options) {
  return FFPA_ERR_UNSUPPORTED;
}
}
