// wd_norm.cu - residual addition and root-mean-square norm, to the input's type
// or to MXFP8 (declared in include/wd_step.h).
//
// A row stands in the registers of kTpr threads (a warp, or a CTA) from its one reading to
// its one writing: r = x + residual, the sum of squares over the threads, y. Bytes bound it: x and
// residual in, r and y out, and nothing else but the weights, which stay in L2.
//
// Rows of whole, aligned vectors give a thread 8 elements at a time; four neighbouring lanes then hold a
// block of 32, whose largest magnitude is two shuffles away. Any other row (odd H, odd strides) is
// taken one element to a lane, so that a warp's access stays contiguous, and a block is a warp.
#include <float.h>

#include "wd_device.cuh"
#include "wd_step.cuh"
#include "wd_vec.cuh"

namespace wd {
namespace {

constexpr int kMinThreads = 128;  // of a CTA: short rows share one

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ void narrow_to(float* p, float x) { *p = x; }
__device__ __forceinline__ void narrow_to(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void narrow_to(__half* p, float x) { *p = __float2half_rn(x); }

// Two values -> two E4M3 codes (round to nearest even, saturating), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

// The exponent of a block whose largest magnitude has these bits; `bad` if one is not finite.
__device__ __forceinline__ int block_exponent(uint32_t top, bool& bad) {
  bad = top >= 0x7F800000u;
  const int ex = (int)(top >> 23);  // floor(log2) + 127, 0 for what lies below 2^-126
  return top == 0 || bad ? 0 : (ex <= 8 ? -127 : ex - 135);
}

// 2^e for e in [-127, 127], the lowest a subnormal.
__device__ __forceinline__ float exp2_of(int e) {
  return e < -126 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

// The sum over the kTpr threads of a row, the same bits in each of them.
template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if (kTpr <= 32) return v;
  constexpr int kWarps = kTpr / 32;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) v += part[i];
  return v;
}

// kPer: groups of 8 elements of a thread; kVec: they are consecutive and aligned.
template <typename T, int kTpr, int kPer, bool kVec>
__global__ void __launch_bounds__(kTpr < kMinThreads ? kMinThreads : kTpr)
    rms_norm(const NormArgs a) {
  constexpr int kThreads = kTpr < kMinThreads ? kMinThreads : kTpr;
  __shared__ float part[2][kThreads / 32];
  const int t = threadIdx.x % kTpr;
  const long long row = (long long)blockIdx.x * (kThreads / kTpr) + threadIdx.x / kTpr;
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  if (row >= a.rows) return;  // a whole warp's row, or none: rows of several warps have a CTA each
  const long long token = a.heads == 1 ? row : row / a.heads;
  const int head = a.heads == 1 ? 0 : (int)(row - token * a.heads);
  const T* x = static_cast<const T*>(a.x) + token * a.x_token + head * a.x_head;
  const T* res = static_cast<const T*>(a.residual) + token * a.residual_token + head * a.residual_head;
  const long long at = row * a.H;
  // element k of group i of this thread
  const auto index = [&](int i, int k) { return kVec ? 8 * (i * kTpr + t) + k : (8 * i + k) * kTpr + t; };
  float r[kPer][8];
  float sum = 0.f;
  if constexpr (kVec) {
    Eight<T> in[kPer], more[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (index(i, 0) < a.H) in[i] = *reinterpret_cast<const Eight<T>*>(x + index(i, 0));
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (index(i, 0) < a.H) more[i] = *reinterpret_cast<const Eight<T>*>(res + index(i, 0));
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool here = index(i, 0) < a.H;
      if (here) Widen<T>::run(in[i], r[i]);
      if (here && a.residual) {
        float f[8];
        Widen<T>::run(more[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[i][k] += f[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (!here) r[i][k] = 0.f;
        sum += r[i][k] * r[i][k];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = index(i, k);
        r[i][k] = j < a.H ? widen(x[j]) : 0.f;
        if (a.residual && j < a.H) r[i][k] += widen(res[j]);
      }
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += r[i][k] * r[i][k];
  }
  sum = row_sum<kTpr>(sum, part[0]);
  if (a.residual_out) {
    T* to = static_cast<T*>(a.residual_out) + at;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (kVec) {
        if (index(i, 0) < a.H) *reinterpret_cast<Eight<T>*>(to + index(i, 0)) = narrow<T>(r[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (index(i, k) < a.H) narrow_to(to + index(i, k), r[i][k]);
      }
    }
  }
  float rstd = rsqrtf(sum / a.H + a.eps);
  if (!(sum <= FLT_MAX)) {
    // Squares beyond FP32: once more with r 2^-72 (2^128 2^-72 squared, 2^14 times, is below 2^127); eps is
    // then below the last bit. A row that holds what is not finite comes out as NaN.
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[i][k] *= 0x1p-72f;
        sum += r[i][k] * r[i][k];
      }
    sum = row_sum<kTpr>(sum, part[1]);
    rstd = sum <= FLT_MAX ? rsqrtf(sum / a.H) : __uint_as_float(0x7FC00000u);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (kVec) {
      const int j = index(i, 0);
      const bool here = j < a.H;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 1.f;
      if (here && a.weight) {
        if (a.weight_fp32)
          Widen<float>::run(*reinterpret_cast<const Eight<float>*>(static_cast<const float*>(a.weight) + j), w);
        else
          Widen<T>::run(*reinterpret_cast<const Eight<T>*>(static_cast<const T*>(a.weight) + j), w);
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        r[i][k] = r[i][k] * rstd * w[k];
        top = max(top, __float_as_uint(r[i][k]) & 0x7FFFFFFFu);
      }
      if (a.y && here) *reinterpret_cast<Eight<T>*>(static_cast<T*>(a.y) + at + j) = narrow<T>(r[i]);
      if (a.codes) {
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        bool bad;
        const int e = block_exponent(top, bad);
        const float inv = exp2_of(-e);
        uint2 c;
        c.x = e4m3x2_of(r[i][0] * inv, r[i][1] * inv) | e4m3x2_of(r[i][2] * inv, r[i][3] * inv) << 16;
        c.y = e4m3x2_of(r[i][4] * inv, r[i][5] * inv) | e4m3x2_of(r[i][6] * inv, r[i][7] * inv) << 16;
        if (bad) c = make_uint2(0u, 0u);
        if (here) {
          *reinterpret_cast<uint2*>(a.codes + at + j) = c;
          if ((t & 3) == 0) a.scales[(at + j) >> 5] = (uint8_t)(bad ? 255 : e + 127);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = index(i, k);
        const bool here = j < a.H;
        float w = 1.f;
        if (here && a.weight)
          w = a.weight_fp32 ? static_cast<const float*>(a.weight)[j] : widen(static_cast<const T*>(a.weight)[j]);
        const float y = r[i][k] * rstd * w;
        if (a.y && here) narrow_to(static_cast<T*>(a.y) + at + j, y);
        if (a.codes) {
          const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(y) & 0x7FFFFFFFu);
          bool bad;
          const int e = block_exponent(top, bad);
          if (here) {
            a.codes[at + j] = bad ? 0 : (uint8_t)e4m3x2_of(y * exp2_of(-e), 0.f);
            if ((t & 31) == 0) a.scales[(at + j) >> 5] = (uint8_t)(bad ? 255 : e + 127);
          }
        }
      }
    }
  }
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

template <typename T, int kTpr, int kPer>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  constexpr int kThreads = kTpr < kMinThreads ? kMinThreads : kTpr;
  constexpr int kRows = kThreads / kTpr;
  constexpr int kUnit = 16 / sizeof(T);  // elements to 16 bytes
  const bool vec = a.H % 8 == 0 && aligned(a.x, 16) && aligned(a.residual, 16) && aligned(a.weight, 16) &&
                   aligned(a.residual_out, 16) && aligned(a.y, 16) && aligned(a.codes, 8) &&
                   a.x_token % kUnit == 0 && a.x_head % kUnit == 0 && a.residual_token % kUnit == 0 &&
                   a.residual_head % kUnit == 0;
  const int ctas = (int)(((long long)a.rows + kRows - 1) / kRows);
  return launch_dependent(vec ? rms_norm<T, kTpr, kPer, true> : rms_norm<T, kTpr, kPer, false>, ctas, kThreads,
                          0, s, a);
}

// Rows up to 512 elements have a warp, longer ones a CTA of so many threads that each holds
// 8 to 16 elements, 32 at the longest.
template <typename T>
cudaError_t run_type(const NormArgs& a, cudaStream_t s) {
  if (a.H <= 256) return run<T, 32, 1>(a, s);
  if (a.H <= 512) return run<T, 32, 2>(a, s);
  if (a.H <= 1024) return run<T, 128, 1>(a, s);
  if (a.H <= 2048) return run<T, 256, 1>(a, s);
  if (a.H <= 4096) return run<T, 512, 1>(a, s);
  if (a.H <= 8192) return run<T, 512, 2>(a, s);
  return run<T, 512, 4>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, wd_dtype dtype, cudaStream_t s) {
  switch (dtype) {
    case WD_BF16: return run_type<__nv_bfloat16>(a, s);
    case WD_FP16: return run_type<__half>(a, s);
    default: return run_type<float>(a, s);
  }
}

}  // namespace wd
