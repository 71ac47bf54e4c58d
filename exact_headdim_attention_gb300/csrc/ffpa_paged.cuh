#pragma once
// Shared by the operators around a paged key/value cache (ffpa_decode.cu,
// ffpa_rope.cu, ffpa_rope_bwd.cu, ffpa_pages.cu): the host checks they have
// in common with the attention entry points, and small device helpers.
#include <initializer_list>

#include "ffpa_common.cuh"

namespace ffpa {

// ---- host (defined in ffpa_api.cu, next to the attention entry points)

// Every non-null pointer is memory of one device; that device in *dev.
ffpa_status call_device(std::initializer_list<const void*> ptrs, int* dev);
// With a DeviceScope of `dev` open: the arch check, the word that the call's
// kernels report to (the options' or the device's fallback word) and the
// number of SMs.
ffpa_status call_status(int dev, const ffpa_options* options, int** err, int* sms);

// Tensor map of 64-column boxes of 16-bit rows with the 128-byte swizzle; byte
// strides of dims 1 .. rank - 1, zeros outside.
ffpa_status encode_rows(CUtensorMap* map, ffpa_dtype dt, int rank, const void* base, const uint64_t* dims,
                        const uint64_t* stride_bytes, const uint32_t* box);

inline bool on_boundary(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// As for the attention inputs: unit last stride, every other stride of a
// dimension longer than 1 positive and a multiple of 16 bytes.
inline bool rows_ok(const int64_t* str, std::initializer_list<int64_t> sizes) {
  int i = 0;
  const int rank = static_cast<int>(sizes.size());
  for (int64_t n : sizes) {
    if (i == rank - 1) return str[i] == 1;
    if (n > 1 && (str[i] <= 0 || str[i] % 8 != 0)) return false;
    ++i;
  }
  return true;
}

// ---- device

// Records the first kind of bad index a call meets (the word keeps a
// non-zero value that is already there).
__device__ __forceinline__ void report_invalid(int* err) { atomicCAS(err, 0, static_cast<int>(FFPA_ERR_INVALID)); }

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return F16 ? pack_f16(a, b) : pack_bf16(a, b);
}
template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if (F16) {
    __half2 h;
    memcpy(&h, &u, 4);
    return __half22float2(h);
  }
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
// Two non-negative values, each as a value of the type below it and the rest,
// which is positive where the value is (so that an infinite factor of both stays
// infinite): off by 2^-16, fp16 2^-21, of the value.
template <bool F16>
__device__ __forceinline__ void split2(float a, float b, uint32_t& most, uint32_t& rest) {
  float2 m;
  if (F16) {
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(most) : "f"(b), "f"(a));
    m = unpack2<F16>(most);
  } else {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    most = __byte_perm(x, y, 0x7632);
    m = make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u));
  }
  constexpr float more = 1.0f + 0x1p-23f;
  rest = pack2<F16>(fmaf(a, more, -m.x), fmaf(b, more, -m.y));
}
template <bool F16>
__device__ __forceinline__ void store16(void* p, float x) {
  if (F16)
    *static_cast<__half*>(p) = __float2half_rn(x);
  else
    *static_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(x);
}

// 16 bytes from global to shared memory; bytes = 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes));
}
// N (8 or 16) bytes, for the copying thread's own use.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src));
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src));
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// An arrival of this thread on `bar` once its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void ldm_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// C [16 x 8] += A [16 x 16] B [16 x 8], 16-bit operands, fp32 accumulators.
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ void fetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// Transposes an 8 x 8 matrix of 16-bit values, of which lane i holds row i / 4,
// columns i % 4 * 2 and the next.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Dependent launch: let the next kernel of the stream start its blocks, and
// wait (in that kernel) until this one's memory is visible.
__device__ __forceinline__ void dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace ffpa
