// sv_cache_device.cuh -- device helpers of the cache-side kernels: element
// conversion, page lookup and the 8-bit rounding.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "sv_cache.h"
#include "sv_device.cuh"

namespace sv {

constexpr unsigned int kFlagInvalidPage = 128u;

__device__ __forceinline__ void raise_flag(Ctrl* ctrl, unsigned int flag) {
  if (ctrl) atomicOr(&ctrl->flags, flag);
}

// Quotient of a position (0 <= n < 2^31) by the page size.
__device__ __forceinline__ int page_of(const CacheView& c, int n) {
  if (c.div_page.m == 0u) return n;  // pages of one token
  return static_cast<int>(__umulhi(static_cast<unsigned int>(n), c.div_page.m) >> c.div_page.shift);
}

// Page and place of a sequence's position; false (and the flag) when there is none.
__device__ __forceinline__ bool find_place(const CacheView& c, int b, long long pos, int& page,
                                           int& place, Ctrl* ctrl) {
  if (pos >= static_cast<long long>(c.max_pages) * c.page_size || pos > 0x7fffffffll) {
    raise_flag(ctrl, kFlagCapacity);
    return false;
  }
  const int n = static_cast<int>(pos);
  const int pi = page_of(c, n);
  page = __ldg(c.table + static_cast<long long>(b) * c.table_stride + pi);
  place = n - pi * c.page_size;
  if (static_cast<unsigned int>(page) >= static_cast<unsigned int>(c.num_pages)) {
    raise_flag(ctrl, kFlagInvalidPage);
    return false;
  }
  return true;
}

__device__ __forceinline__ int quotient(int n, const UDiv& d) {
  return d.m == 0u ? n : static_cast<int>(__umulhi(static_cast<unsigned int>(n), d.m) >> d.shift);
}

__device__ __forceinline__ float elem_f32(float v) { return v; }
__device__ __forceinline__ float elem_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float elem_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float elem_f32(__nv_fp8_e4m3 v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(v.__x, __NV_E4M3)));
}
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Eight elements at p (16-byte aligned for 2- and 4-byte types, 8-byte for codes).
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  const float4 b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float (&f)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void load8(const __nv_fp8_e4m3* p, float (&f)[8]) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  const uint32_t w[2] = {a.x, a.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t two =
        static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1)));
    const float2 v = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(two, __NV_E4M3)));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Two e4m3 codes, rounded to nearest, ties to even, saturating.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace sv
