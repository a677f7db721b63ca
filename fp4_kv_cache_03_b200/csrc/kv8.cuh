// The paged 8-bit cache: E4M3 codes [page][kv head][128][D] with one scale 2^e per 16 tokens
// and head, e + 127 in a byte.  A power of two, so that a block whose scale has to grow keeps
// its older codes exactly (only codes that become subnormal round), and so that attention can
// fold the scales into its fp32 exponents.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace csa2 {

constexpr int kKv8Block = 16;
constexpr int kKv8Blocks = kPageRows / kKv8Block;      // scales per page and head
constexpr int kKv8MinExp = -60, kKv8MaxExp = 60, kKv8Bias = 127;

__device__ __forceinline__ int kv8_exp(uint32_t byte) {
  return max(kKv8MinExp, min(kKv8MaxExp, (int)byte - kKv8Bias));
}
// 2^e for |e| <= 126
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// the least e with amax <= 448 * 2^e (448 = 1.75 * 2^8 is the largest E4M3 value), from the
// bits of amax; a subnormal amax gives something at or below -134, infinity 120
__device__ __forceinline__ int kv8_least_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3x2(__half2 v) {
  return (uint32_t)__nv_cvt_halfraw2_to_fp8x2(__half2_raw(v), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ __half2 e4m3x2_half2(uint32_t two) {
  return __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
}
__device__ __forceinline__ float2 e4m3x2_value(uint32_t two) { return __half22float2(e4m3x2_half2(two)); }

// host checks of a cache argument
inline csa2_status_t kv8_check(const csa2_kv8_t& c) {
  if (c.num_pages < 1 || c.H_kv < 1 || c.D < 1) return CSA2_ERR_INVALID_ARG;
  if (c.D > 128 || c.D % 16 || c.H_kv > 1024 || (int64_t)c.num_pages * c.H_kv >= (1ll << 31))
    return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}
inline bool kv8_pointers_ok(const csa2_kv8_t& c) {
  return c.k && c.v && c.k_exp && c.v_exp &&
         !((reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v)) & 15) &&
         !((reinterpret_cast<uintptr_t>(c.k_exp) | reinterpret_cast<uintptr_t>(c.v_exp)) & 7);
}

}  // namespace csa2
