// wd_norm.cu - residual addition and root-mean-square norm, to the input's type
// or to MXFP8 (declared in include/wd_step.h).
//
// A row stands in the registers of its threads (8 or 16 lanes, a warp, or a CTA) from its one reading to
// its one writing: r = x + residual, the sum of squares over the threads, y. Bytes bound it: x and
// residual in, r and y out, and nothing else but the weights, which stay in L2.
//
// A thread takes eight elements at a time, of 16 aligned bytes (32 in FP32). Where H is a multiple of eight and all is
// aligned, four neighbouring lanes hold a block of 32, whose largest magnitude is two shuffles away. Where rows begin
// anywhere but all tensors alike (odd H), the eights begin at the first aligned place, and the up to 14 elements around them
// are taken by a lane each. What is left (tensors of unlike alignment, MXFP8 of unaligned rows) is taken one element
// to a lane, so that a warp's access stays contiguous, and a block is a warp.
// Measured (BF16, with residual): 16384 x 2048 41.5 us, 6.5 TB/s, 0.95 of the copy rate; 2048 x 16384 50.7 us (0.78: few CTAs
// of many warps that wait for each other); 16376 x 2049 45.3 us (0.87: the weights are then taken one by one, 3.7 us of
// it), 100,764 x 333 53.8 (0.73); 16384 x 2048 into MXFP8 43.3 us (0.80), 2048 x 16384 52.8 (0.66). FP32 up to 4096 elements
// 0.84 to 0.97, 1024 x 16384 62 us (0.64). Without residual 32 heads of 128 of 8192 tokens 23.3 us (0.85), 16384 x 2048 27.8
// (0.71), 8192 x 4096 30.7 (0.64: half as much on its way), 4096 x 8192 32.8 (0.60). One row of 2048: 1.4 us. Tried: groups of rows after
// each other in a CTA that stays (registers for two, 10 to 50 % slower), CTAs of 1024 threads (2048 x 16384 64.8), eight
// eights in one warp (51.8 for 8192 x 2048 of FP32).
#include <float.h>

#include "wd_device.cuh"
#include "wd_step.cuh"
#include "wd_vec.cuh"

namespace wd {
namespace {

constexpr int kThreads = 128;  // of a CTA whose rows are a warp's or less
enum Mode { kAligned, kShifted, kSingle };

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

// The sum over the threads of a row (kTpr lanes; 0: the CTA), the same bits in each of them.
template <int kTpr>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int off = kTpr ? kTpr / 2 : 16; off > 0; off /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
  if (kTpr) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(lane < (int)(blockDim.x >> 5) ? part[lane] : 0.f);
}

// Rows of kTpr lanes (0: a CTA), kPer eights to a thread.
template <typename T, int kTpr, int kPer, Mode kMode>
__global__ void __launch_bounds__(kTpr ? kThreads : 512) rms_norm(const NormArgs a) {
  __shared__ float part[2][32];
  const int tpr = kTpr ? kTpr : blockDim.x;
  const int t = kTpr ? threadIdx.x % (kTpr ? kTpr : 1) : threadIdx.x;
  const long long row = kTpr ? (long long)blockIdx.x * (kThreads / (kTpr ? kTpr : 1)) + threadIdx.x / (kTpr ? kTpr : 1)
                             : (long long)blockIdx.x;
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  const bool live = !kTpr || row < a.rows;  // (lanes of no row take part in their warp's sums)
  const unsigned token = a.heads == 1 ? (unsigned)row : (unsigned)row / (unsigned)a.heads;  // rows are below 2^31
  const int head = a.heads == 1 ? 0 : (int)((unsigned)row - token * (unsigned)a.heads);
  const T* x = static_cast<const T*>(a.x) + token * a.x_token + head * a.x_head;
  const T* res = static_cast<const T*>(a.residual) + token * a.residual_token + head * a.residual_head;
  const long long at = row * a.H;
  constexpr int kUnit = 16 / sizeof(T);
  // kShifted: the eights' elements are [begin, stop), and lane t has loose element `loose` of those around them
  const int begin =
      kMode == kShifted ? min(a.H, (int)((kUnit - reinterpret_cast<uintptr_t>(x) / sizeof(T) % kUnit) % kUnit)) : 0;
  const int stop = kMode == kShifted ? begin + (a.H - begin) / 8 * 8 : a.H;
  const int loose = t < begin ? t : stop + t - begin;
  const bool loosed = kMode == kShifted && live && loose < a.H;
  // the first element of eight i, or single element (i, k)
  const auto eight = [&](int i) { return begin + 8 * (i * tpr + t); };
  const auto single = [&](int i, int k) { return (8 * i + k) * tpr + t; };
  float r[kPer][8], rl = 0.f;
  // A thread with one eight asks for its weights with the row (one row of 2048 1.6 -> 1.5 us, 200 of 4096 to MXFP8 2.7 -> 2.5);
  // with more, their registers cost more than the wait (2048 x 16384 50.7 -> 62 us).
  constexpr bool kEarly = kMode == kAligned && kPer == 1;
  const bool early = kEarly && a.weight && !a.weight_fp32;
  Eight<T> wt[1];
  float sum = 0.f;
  if constexpr (kMode != kSingle) {
    Eight<T> in[kPer], more[kPer];
    if (early && live && eight(0) < stop)
      wt[0] = *reinterpret_cast<const Eight<T>*>(static_cast<const T*>(a.weight) + eight(0));
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (live && eight(i) < stop) in[i] = *reinterpret_cast<const Eight<T>*>(x + eight(i));
    if (loosed) rl = widen(x[loose]);
    if (a.residual) {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (live && eight(i) < stop) more[i] = *reinterpret_cast<const Eight<T>*>(res + eight(i));
      if (loosed) rl += widen(res[loose]);
    }
    sum = rl * rl;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool here = live && eight(i) < stop;
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
        const int j = single(i, k);
        r[i][k] = live && j < a.H ? widen(x[j]) : 0.f;
        if (a.residual && live && j < a.H) r[i][k] += widen(res[j]);
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
      if constexpr (kMode != kSingle) {
        if (live && eight(i) < stop) *reinterpret_cast<Eight<T>*>(to + eight(i)) = narrow<T>(r[i]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (live && single(i, k) < a.H) narrow_to(to + single(i, k), r[i][k]);
      }
    }
    if (loosed) narrow_to(to + loose, rl);
  }
  const float mean = sum / a.H + a.eps;
  float rstd = rsqrtf(mean);
  // Squares, or their mean and eps, beyond FP32: once more with r 2^-72 and eps 2^-144 (2^128 2^-72 squared, 2^14
  // times, is below 2^127). A row that holds what is not finite comes out as NaN.
  const bool beyond = !(mean <= FLT_MAX);
  if (kTpr && kTpr < 32 ? __any_sync(0xFFFFFFFFu, beyond) : beyond) {
    if (beyond) rl *= 0x1p-72f;
    float small = rl * rl;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (beyond) r[i][k] *= 0x1p-72f;
        small += r[i][k] * r[i][k];
      }
    small = row_sum<kTpr>(small, part[1]);
    if (beyond) rstd = small <= FLT_MAX ? rsqrtf(fmaf(a.eps, 0x1p-144f, small / a.H)) : __uint_as_float(0x7FC00000u);
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (kMode != kSingle) {
      const int j = eight(i);
      const bool here = live && j < stop;
      float w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = 1.f;
      if (here && a.weight) {
        if (kMode == kAligned || (begin == 0 && a.weight_aligned)) {
          if (a.weight_fp32)
            Widen<float>::run(*reinterpret_cast<const Eight<float>*>(static_cast<const float*>(a.weight) + j), w);
          else if (early)
            Widen<T>::run(wt[0], w);
          else
            Widen<T>::run(*reinterpret_cast<const Eight<T>*>(static_cast<const T*>(a.weight) + j), w);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            w[k] = a.weight_fp32 ? static_cast<const float*>(a.weight)[j + k]
                                 : widen(static_cast<const T*>(a.weight)[j + k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r[i][k] = r[i][k] * rstd * w[k];
      if (a.y && here) *reinterpret_cast<Eight<T>*>(static_cast<T*>(a.y) + at + j) = narrow<T>(r[i]);
      if (kMode == kAligned && a.codes) {
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(r[i][k]) & 0x7FFFFFFFu);
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
        const int j = single(i, k);
        const bool here = live && j < a.H;
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
  if (loosed && a.y) {
    float w = 1.f;
    if (a.weight)
      w = a.weight_fp32 ? static_cast<const float*>(a.weight)[loose] : widen(static_cast<const T*>(a.weight)[loose]);
    narrow_to(static_cast<T*>(a.y) + at + loose, rl * rstd * w);
  }
}

bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int eights_of(int H, Mode mode) { return mode == kShifted ? (H / 8 ? H / 8 : 1) : (H + 7) / 8; }

template <typename T, int kTpr, int kPer, Mode kMode>
cudaError_t run(const NormArgs& a, cudaStream_t s) {
  const int rows = kTpr ? kThreads / (kTpr ? kTpr : 1) : 1;  // of a CTA
  const int eights = eights_of(a.H, kMode);
  const int threads = kTpr ? kThreads : ((eights + kPer - 1) / kPer + 31) / 32 * 32;
  return launch_dependent(rms_norm<T, kTpr, kPer, kMode>, (int)(((long long)a.rows + rows - 1) / rows), threads, 0, s, a);
}

// How many eights a thread has. Few rows want all the threads that they can have: one eight each, up to 512 threads. Many rows
// fill the GPU, and then each thread wants much on its way and each row few warps that wait for each other: two
// eights where there is no residual and rows are up to 32 lanes (32 heads of 64 elements 34.4 -> 23.5 us), up to four to a warp's
// lane for up to 1024 elements, and four beyond that (16 bits, aligned; 4096 x 8192 with residual 48.2 -> 45.6 us, 8192 x
// 4096 without 35.5 -> 30.1) or two (FP32, whose four cost registers: 49.5 against 46.4 us for 4096 x 4096; rows that begin
// anywhere: 51.6 against 45.0 for 22369 x 1500, with one 47.9).
template <typename T, Mode kMode>
cudaError_t run_mode(const NormArgs& a, cudaStream_t s) {
  const int eights = eights_of(a.H, kMode);
  const bool many = a.rows >= 152 * 8;
  if constexpr (kMode == kAligned) {
    if (!a.residual && a.rows >= 152 * 64) {
      if (eights == 8) return run<T, 4, 2, kMode>(a, s);
      if (eights > 8 && eights <= 16) return run<T, 8, 2, kMode>(a, s);
      if (eights > 16 && eights <= 32) return run<T, 16, 2, kMode>(a, s);
    }
  }
  if constexpr (kMode == kAligned) {
    if (eights <= 8) return run<T, 8, 1, kMode>(a, s);
  }
  if constexpr (kMode != kSingle) {
    if (eights <= 16) return run<T, 16, 1, kMode>(a, s);  // (as many lanes as there may be loose elements)
    if (eights <= 32) return run<T, 32, 1, kMode>(a, s);
  }
  if (eights <= 64) return run<T, 32, 2, kMode>(a, s);
  if constexpr (kMode == kAligned) {
    if (eights <= 96) return run<T, 32, 3, kMode>(a, s);
  }
  if constexpr (kMode != kSingle) {
    if (eights <= 128) return run<T, 32, 4, kMode>(a, s);
  }
  if (kMode == kAligned && sizeof(T) == 2 && many) return run<T, 0, 4, kMode>(a, s);
  if (eights <= 512 && !many) return run<T, 0, 1, kMode>(a, s);
  if (eights <= 1024) return run<T, 0, 2, kMode>(a, s);
  return run<T, 0, 4, kMode>(a, s);
}

template <typename T>
cudaError_t run_type(const NormArgs& a, cudaStream_t s) {
  constexpr int kUnit = 16 / sizeof(T);  // elements to 16 bytes
  const auto place = [](const void* p) { return (long long)(reinterpret_cast<uintptr_t>(p) / sizeof(T) % kUnit); };
  const bool vec = a.H % 8 == 0 && aligned(a.x, 16) && aligned(a.residual, 16) && aligned(a.weight, 16) &&
                   aligned(a.residual_out, 16) && aligned(a.y, 16) && aligned(a.codes, 8) &&
                   a.x_token % kUnit == 0 && a.x_head % kUnit == 0 && a.residual_token % kUnit == 0 &&
                   a.residual_head % kUnit == 0;
  if (vec) return run_mode<T, kAligned>(a, s);
  NormArgs b = a;
  b.weight_aligned = aligned(a.weight, 16);
  // rows that begin at the same place of 16 bytes in every tensor, whichever place that is
  const long long per_token = (long long)a.heads * a.H;
  const auto alike = [&](const void* p, long long token, long long head) {
    return !p || (place(p) == place(a.x) && (token - a.x_token) % kUnit == 0 && (a.heads == 1 || (head - a.x_head) % kUnit == 0));
  };
  if (!a.codes && alike(a.residual, a.residual_token, a.residual_head) && alike(a.residual_out, per_token, a.H) &&
      alike(a.y, per_token, a.H))
    return run_mode<T, kShifted>(b, s);
  return run_mode<T, kSingle>(b, s);
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
