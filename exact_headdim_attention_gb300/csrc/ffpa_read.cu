// The cached keys and values of a batch as packed 16-bit rows, from pages of
// 16-bit values or of e4m3 codes with a scale for each row.
//
// Every row is read and written once: the memory's bandwidth is the bound.  A block
// takes some tokens of keys or of values; it looks up their requests and pages first,
// then all its threads move 16-byte pieces, FLIGHT of them on their way a thread, in
// the order of the output.  24 contexts of up to 8192 keys, Hkv8 D512, codes: 297 us, 6.4 TB/s of bytes read and
// written; 40 of up to 3000, Hkv16 D128, 16 bits: 157 us, 6.4 TB/s.
#include "ffpa_paged.cuh"

namespace ffpa {
namespace {

constexpr int READ_THREADS = 256;
constexpr int READ_TOKENS = 32;     // of a block, at most
constexpr int READ_FLIGHT = 4;

struct ReadSide {
  const char* cache;
  const float* scale;
  char* out;
  int64_t sp, ss, sh;               // bytes (page, slot, head)
  int64_t scale_p, scale_h;         // elements
  int64_t ot, oh;                   // bytes (token, head)
};

struct ReadParams {
  ReadSide side[2];                 // keys, values
  const int32_t *table, *cu;
  int* err;
  int64_t table_str;
  int T, B, Hkv, D, num_pages, page_size, max_pages, tokens;
};

// Two codes times a scale, rounded once.
template <bool F16>
__device__ __forceinline__ uint32_t scaled2(uint32_t h2, float scale) {
  const float2 x = unpack2<true>(h2);
  return pack2<F16>(x.x * scale, x.y * scale);
}

template <bool E4M3, bool F16>
__global__ void __launch_bounds__(READ_THREADS) read_kernel(const __grid_constant__ ReadParams P) {
  const ReadSide& S = P.side[blockIdx.y];
  __shared__ long long from_s[READ_TOKENS];      // byte offset of the row; -1: zeros, -2: not written
  __shared__ long long scale_s[READ_TOKENS];
  const int t0 = blockIdx.x * P.tokens, n = min(P.tokens, P.T - t0);
  const long long cap = (long long)P.max_pages * P.page_size;
  for (int i = threadIdx.x; i < n; i += READ_THREADS) {
    const int t = t0 + i;
    // The last request that begins at or before t and is not empty, if it reaches t.
    int lo = 0, hi = P.B;                        // cu[lo] <= t < cu[hi], if at all
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (P.cu[mid] <= t)
        lo = mid;
      else
        hi = mid;
    }
    const long long j = (long long)t - P.cu[lo];
    from_s[i] = -2;
    if (j >= 0 && t < P.cu[lo + 1] && j < cap) {
      const int page = P.table[lo * P.table_str + (int)j / P.page_size], at = (int)j % P.page_size;
      if (page >= 0 && page < P.num_pages) {
        from_s[i] = page * S.sp + at * S.ss;
        scale_s[i] = E4M3 ? page * S.scale_p + at : 0;
      } else {
        from_s[i] = -1;
        report_invalid(P.err);
      }
    }
  }
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int b = threadIdx.x; b < P.B; b += READ_THREADS) {
      const int a = P.cu[b], e = P.cu[b + 1];
      if (a < 0 || e < a || e > P.T || (long long)e - a > cap) report_invalid(P.err);
    }
  __syncthreads();
  constexpr int PIECE = E4M3 ? 16 : 8;           // values of 16 bytes
  const unsigned per_head = P.D / PIECE, per_token = per_head * P.Hkv, all = n * per_token;
  for (unsigned u0 = threadIdx.x; u0 < all; u0 += READ_THREADS * READ_FLIGHT) {
    uint4 x[READ_FLIGHT];
    float scale[READ_FLIGHT];
    char* to[READ_FLIGHT];
#pragma unroll
    for (int f = 0; f < READ_FLIGHT; ++f) {
      const unsigned u = u0 + f * READ_THREADS;
      to[f] = nullptr;
      x[f] = make_uint4(0, 0, 0, 0);
      scale[f] = 0.0f;
      if (u >= all) continue;
      const unsigned i = u / per_token, w = u - i * per_token, h = w / per_head, c = w - h * per_head;
      const long long from = from_s[i];
      if (from == -2) continue;
      to[f] = S.out + (t0 + i) * S.ot + h * S.oh + c * (PIECE * 2);
      if (from < 0) continue;
      x[f] = __ldcs(reinterpret_cast<const uint4*>(S.cache + from + h * S.sh + c * 16));
      if (E4M3) scale[f] = S.scale[scale_s[i] + h * S.scale_h];
    }
#pragma unroll
    for (int f = 0; f < READ_FLIGHT; ++f) {
      if (!to[f]) continue;
      if (!E4M3) {
        *reinterpret_cast<uint4*>(to[f]) = x[f];
      } else {
        const uint32_t c[4] = {x[f].x, x[f].y, x[f].z, x[f].w};
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t a, b;
          widen_e4m3(c[k], a, b);
          y[2 * k] = scaled2<F16>(a, scale[f]);
          y[2 * k + 1] = scaled2<F16>(b, scale[f]);
        }
        reinterpret_cast<uint4*>(to[f])[0] = make_uint4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<uint4*>(to[f])[1] = make_uint4(y[4], y[5], y[6], y[7]);
      }
    }
  }
}

}  // namespace
}  // namespace ffpa

extern "C" {

ffpa_status ffpa_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, void* k,
                         void* v, ffpa_dtype dt, int T, int B, int Hkv, int D, int num_pages, int page_size,
                         int max_pages, const int64_t kc_str[4], const int64_t vc_str[4], const int64_t ks_str[3],
                         const int64_t vs_str[3], const int64_t k_str[3], const int64_t v_str[3],
                         const int32_t* block_table, int64_t table_str, const int32_t* cu_seqlens,
                         ffpa_stream_t stream, const ffpa_options* options) {
  using namespace ffpa;
  if (dt != FFPA_BF16 && dt != FFPA_FP16) return FFPA_ERR_DTYPE;
  if (T < 0 || B < 0 || Hkv < 1 || num_pages < 0 || page_size < 1 || max_pages < 0) return FFPA_ERR_INVALID;
  const bool codes = k_scale || v_scale;
  if (codes && (!k_scale || !v_scale)) return FFPA_ERR_INVALID;
  if (D < 64 || D > 1024 || D % (codes ? 16 : 8) != 0) return FFPA_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size > 0x7fff0000LL) return FFPA_ERR_INVALID;   // key numbers are int32
  if (T == 0 || B == 0) return FFPA_OK;
  if (!k || !v || !cu_seqlens || !k_str || !v_str || !kc_str || !vc_str) return FFPA_ERR_INVALID;
  const bool held = num_pages > 0 && max_pages > 0;
  if (held && (!k_cache || !v_cache || !block_table)) return FFPA_ERR_INVALID;
  const int unit = codes ? 16 : 8;
  if (!rows_ok(k_str, {T, Hkv, D}) || !rows_ok(v_str, {T, Hkv, D})) return FFPA_ERR_INVALID;
  if (held && (!rows_ok(kc_str, {num_pages, page_size, Hkv, D}, unit) || !rows_ok(vc_str, {num_pages, page_size, Hkv, D}, unit)))
    return FFPA_ERR_INVALID;
  if (held && B > 1 && table_str < max_pages) return FFPA_ERR_INVALID;
  if (!on_boundary(k, 16) || !on_boundary(v, 16) || !on_boundary(cu_seqlens, 4)) return FFPA_ERR_INVALID;
  if (held && (!on_boundary(k_cache, 16) || !on_boundary(v_cache, 16) || !on_boundary(block_table, 4))) return FFPA_ERR_INVALID;
  if (held && codes && (!ks_str || !vs_str || !on_boundary(k_scale, 4) || !on_boundary(v_scale, 4) ||
                        !scales_ok(ks_str, num_pages, Hkv, page_size) || !scales_ok(vs_str, num_pages, Hkv, page_size)))
    return FFPA_ERR_INVALID;
  if ((long long)Hkv * D > 0x7fffffffLL / 64) return FFPA_ERR_INVALID;   // a block's pieces in 31 bits
  int dev = 0;
  ffpa_status st = call_device({k, v, cu_seqlens, held ? k_cache : nullptr, held ? v_cache : nullptr,
                                held ? (const void*)block_table : nullptr, held ? k_scale : nullptr, held ? v_scale : nullptr},
                               &dev);
  if (st != FFPA_OK) return st;
  DeviceScope scope(dev);
  if (!scope.ok()) return FFPA_ERR_CUDA;
  ReadParams P{};
  int sms = 0;
  if ((st = call_status(dev, options, &P.err, &sms)) != FFPA_OK) return st;
  const int bytes = codes ? 1 : 2;
  for (int i = 0; i < 2; ++i) {
    ReadSide& S = P.side[i];
    S.cache = static_cast<const char*>(i ? v_cache : k_cache);
    S.scale = i ? v_scale : k_scale;
    S.out = static_cast<char*>(i ? v : k);
    const int64_t *c = i ? vc_str : kc_str, *o = i ? v_str : k_str, *f = i ? vs_str : ks_str;
    if (held) {
      S.sp = c[0] * bytes;
      S.ss = c[1] * bytes;
      S.sh = c[2] * bytes;
      if (codes) {
        S.scale_p = f[0];
        S.scale_h = f[1];
      }
    }
    S.ot = o[0] * 2;
    S.oh = o[1] * 2;
  }
  P.table = block_table;
  P.table_str = table_str;
  P.cu = cu_seqlens;
  P.T = T;
  P.B = B;
  P.Hkv = Hkv;
  P.D = D;
  P.num_pages = num_pages;
  P.page_size = page_size;
  P.max_pages = held ? max_pages : 0;
  // Four blocks an SM at least, where there are tokens for them.
  P.tokens = T / (sms * 2);
  if (P.tokens < 1) P.tokens = 1;
  if (P.tokens > READ_TOKENS) P.tokens = READ_TOKENS;
  const dim3 grid((T + P.tokens - 1) / P.tokens, 2);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (codes)
    (dt == FFPA_FP16 ? read_kernel<true, true> : read_kernel<true, false>)<<<grid, READ_THREADS, 0, s>>>(P);
  else
    read_kernel<false, false><<<grid, READ_THREADS, 0, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? FFPA_OK : FFPA_ERR_CUDA;
}

}  // extern "C"
