// Element access and the bounds' number format, shared by the paged-cache kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace thin {

struct e4m3 {
  uint8_t b;
};

__device__ __forceinline__ float e4m3_to_f(uint32_t b) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)b, __NV_E4M3)));
}
template <typename T> __device__ __forceinline__ float elem_f(T x);
template <> __device__ __forceinline__ float elem_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float elem_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float elem_f<__half>(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float elem_f<e4m3>(e4m3 x) { return e4m3_to_f(x.b); }
template <typename T> __device__ __forceinline__ T elem_of(float x);
template <> __device__ __forceinline__ float elem_of<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 elem_of<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half elem_of<__half>(float x) { return __float2half_rn(x); }

// Eight neighbouring elements (16-byte aligned where they are two bytes or more).
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 u = ((const float4*)p)[0], v = ((const float4*)p)[1];
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
  } else if constexpr (sizeof(T) == 1) {
    const uint2 u = *(const uint2*)p;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = e4m3_to_f(((i < 4 ? u.x : u.y) >> (8 * (i & 3))) & 0xFF);
  } else {
    const uint4 u = *(const uint4*)p;
    const T* e = (const T*)&u;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = elem_f<T>(e[i]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  if constexpr (sizeof(T) == 4) {
    ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 u;
    T* e = (T*)&u;
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = elem_of<T>(x[i]);
    *(uint4*)p = u;
  }
}

// Bounds are whole numbers times 2^x: the least x in [-40, 48] with 127 * 2^x >= m.  m = f 2^(e),
// f in [1, 2): 127 * 2^(e - 6) = 1.984375 * 2^e covers f <= 1.984375.
constexpr int kBoundMin = -40, kBoundMax = 48;
__device__ __forceinline__ int bound_exponent(float m) {
  const uint32_t u = __float_as_uint(m);
  const int e = (int)(u >> 23) - 127;
  return min(max((u & 0x7FFFFFu) <= 0x7E0000u ? e - 6 : e - 5, kBoundMin), kBoundMax);
}
__device__ __forceinline__ float pow2f(int x) { return __uint_as_float((uint32_t)(x + 127) << 23); }

}  // namespace thin
