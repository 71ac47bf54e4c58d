// Attention of one new token per request over a paged cache of 16-bit values.
#include "ffpa_decode.cuh"

namespace ffpa {

ffpa_status run_decode_16(DecodeParams& P, const DecodeShape& s, ffpa_dtype dt, float sc, int sms, int dev, char* ws,
                          const ffpa_options* options, cudaStream_t stream) {
  return run_decode<DECODE_16>(P, s, dt, sc, sms, dev, ws, options, stream);
}

}  // namespace ffpa

extern "C" {

size_t ffpa_decode_paged_workspace_bytes(int Hq, int Hkv, int D) { return ffpa::decode_bytes(Hq, Hkv, D); }

ffpa_status ffpa_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                              ffpa_dtype dt, int B, int Hq, int Hkv, int D, int num_pages, int page_size,
                              int max_pages, const int64_t q_str[3], const int64_t k_str[4],
                              const int64_t v_str[4], const int64_t o_str[3], const int32_t* block_table,
                              int64_t table_str, const int32_t* seq_lens, const float* scale, int enable_gqa,
                              void* workspace, size_t workspace_bytes, ffpa_stream_t stream,
                              const ffpa_options* options) {
  using namespace ffpa;
  const DecodeShape s{B, Hq, Hkv, D, num_pages, page_size, max_pages, k_str, v_str};
  return decode_entry<DECODE_16>(q, k_cache, v_cache, o, lse, dt, s, q_str, o_str, block_table, table_str, seq_lens, nullptr,
                                 nullptr, nullptr, nullptr, scale, enable_gqa, workspace, workspace_bytes, stream, options);
}

}  // extern "C"
