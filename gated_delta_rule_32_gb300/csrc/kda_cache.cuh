// kda_cache.cuh -- what the kernels of the paged 8-bit cache share: the
// cache's layout, code conversions and the argument structs.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kda_common.cuh"

namespace kda_cache {

constexpr int kMaxRequests = 16384;

__host__ __device__ constexpr float code_top(int code) { return code == KDA_I8 ? 127.0f : 448.0f; }

inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128; }
inline bool head_dim_ok(int d) { return d == 64 || d == 128; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return a && b && na && nb && x < y + nb && y < x + na;
}

// Whether all addresses are multiples of n (a power of two).
template <class... Ptr>
inline bool aligned(size_t n, Ptr... ptr) {
  return (((uintptr_t)ptr | ...) & (n - 1)) == 0;
}

__device__ __forceinline__ void report(int32_t* dev_status, kda_status s) {
  if (dev_status) atomicExch(dev_status, (int32_t)s);
}

// One byte's value.
template <int CODE>
__device__ __forceinline__ float decode1(uint8_t b) {
  if (CODE == KDA_I8) return (float)(int8_t)b;
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}

// The nearest code of x, |x| <= top, ties to even.
template <int CODE>
__device__ __forceinline__ uint32_t encode1(float x) {
  if (CODE == KDA_I8) return (uint32_t)__float2int_rn(x) & 0xffu;
  return (uint32_t)__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

}  // namespace kda_cache
