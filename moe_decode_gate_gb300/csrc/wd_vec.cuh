// wd_vec.cuh - eight consecutive elements of a row, as the kernels load, convert and store them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace wd {

template <typename T>
struct alignas(16) Eight {
  T v[8];
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Eight inputs as floats, and the bits of the largest magnitude as a float (NaN above Inf).
template <typename T>
struct Widen;
template <>
struct Widen<float> {
  static __device__ __forceinline__ uint32_t run(const Eight<float>& x, float (&f)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      f[k] = x.v[k];
      top = max(top, __float_as_uint(f[k]) & 0x7FFFFFFFu);
    }
    return top;
  }
};
template <typename T>
__device__ __forceinline__ uint32_t top_half(const Eight<T>& x) {
  const uint4 w = *reinterpret_cast<const uint4*>(&x);
  const uint32_t m = max_u16x2(max_u16x2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                               max_u16x2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
  return max(m & 0xFFFFu, m >> 16);
}
template <>
struct Widen<__nv_bfloat16> {
  static __device__ __forceinline__ uint32_t run(const Eight<__nv_bfloat16>& x, float (&f)[8]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
    return top_half(x) << 16;
  }
};
template <>
struct Widen<__half> {
  static __device__ __forceinline__ uint32_t run(const Eight<__half>& x, float (&f)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&x);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 p = __half22float2(h[k]);
      f[2 * k] = p.x;
      f[2 * k + 1] = p.y;
    }
    const uint32_t top = top_half(x);
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)top))) & 0x7FFFFFFFu;
  }
};

template <typename T>
__device__ __forceinline__ Eight<T> narrow(const float (&f)[8]);
template <>
__device__ __forceinline__ Eight<float> narrow(const float (&f)[8]) {
  Eight<float> y;
#pragma unroll
  for (int k = 0; k < 8; ++k) y.v[k] = f[k];
  return y;
}
template <>
__device__ __forceinline__ Eight<__nv_bfloat16> narrow(const float (&f)[8]) {
  Eight<__nv_bfloat16> y;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    reinterpret_cast<__nv_bfloat162*>(&y)[k] = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
  return y;
}
template <>
__device__ __forceinline__ Eight<__half> narrow(const float (&f)[8]) {
  Eight<__half> y;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    reinterpret_cast<__half2*>(&y)[k] = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
  return y;
}

}  // namespace wd
