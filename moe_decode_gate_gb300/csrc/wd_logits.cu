// wd_logits.cu - penalties, biases, temperature and masks on logits (declared
// in include/wd_step.h).
//
// One pass: a CTA takes a slice of one row's vocabulary, counts in shared memory how often the row's
// history names each of its tokens (every CTA of a row reads the whole history, which is
// small beside the logits and comes from L2), notes which bias is the last for each, and then
// streams its logits through: counts, biases and mask are looked up beside them. Nothing is
// written but the result, no counts live from call to call, and counting whole numbers gives the same sums
// in any order. Bytes bound it where rows are many, the history's scan where they are few.
#include "wd_device.cuh"
#include "wd_step.cuh"
#include "wd_vec.cuh"

namespace wd {
namespace {

constexpr int kThreads = 256;
constexpr int kFour = 4;               // elements of an access
constexpr int kMinSlice = 1024;        // tokens of a CTA: one access to a thread
constexpr int kMaxSlice = 4096;        // two arrays of it are 32 KB: seven CTAs to an SM
constexpr int kCtasWanted = 4 * 152;   // for which slices are made smaller
constexpr uint32_t kPrompt = 1u << 31;  // of a count: the prompt has the token
constexpr uint32_t kAnswer = kPrompt - 1;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }

template <typename T>
struct alignas(sizeof(T) * kFour) Four {
  T v[kFour];
};

// What a row's tokens go through.
struct Row {
  float repetition, presence, frequency, scale;
  const float* bias;      // the values of the row's biases
  const int32_t* mask;    // its words
  bool counts, biases;    // whether the slice has some
};

// Token `at` of the slice. count: how often its history has each; named: 1 + the last bias of each.
__device__ __forceinline__ float adjusted(const Row& r, const uint32_t* count, const int32_t* named, float l, int at,
                                          bool allowed) {
  if (r.counts) {
    const uint32_t c = count[at];
    if (c) {
      l = l > 0.f ? l / r.repetition : l * r.repetition;
      const uint32_t n = c & kAnswer;
      if (n) l -= (float)n * r.frequency + r.presence;
    }
  }
  if (r.biases) {
    const int e = named[at];
    if (e) l += r.bias[e - 1];
  }
  l *= r.scale;
  return allowed ? l : -INFINITY;
}

// Slice `blockIdx.x % slices` of row `blockIdx.x / slices`. kVec: input and output of a row reach
// the alignment of four elements at the same token.
template <typename T, typename U, bool kVec>
__global__ void __launch_bounds__(kThreads) adjust_logits(const LogitsArgs a, int slices, int slice) {
  extern __shared__ uint32_t shared[];
  const int b = blockIdx.x / slices, part = blockIdx.x % slices;
  const T* in = static_cast<const T*>(a.logits) + b * a.stride;
  U* out = static_cast<U*>(a.out) + b * a.out_stride;
  // tokens [from, to): slices begin where four elements are aligned, the first with what is before that
  const int lead = kVec ? (int)((kFour - (reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kFour) % kFour) : 0;
  const int from = part == 0 ? 0 : lead + part * slice;
  const int to = part == slices - 1 ? a.V : min(a.V, lead + (part + 1) * slice);
  const int n = to - from;
  uint32_t* count = shared;
  int32_t* named = reinterpret_cast<int32_t*>(shared + (a.history.tokens ? slice + kFour : 0));
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  if (n <= 0) return;
  Row r;
  r.repetition = a.repetition ? a.repetition[b] : 1.f;
  r.presence = a.presence ? a.presence[b] : 0.f;
  r.frequency = a.frequency ? a.frequency[b] : 0.f;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  r.scale = t > 0.f ? 1.f / t : 1.f;
  r.mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
  // the row's history, if it has one and its penalties are any
  const int32_t* tokens = nullptr;
  int length = 0, prompt = 0;
  if (a.history.tokens && (r.repetition != 1.f || r.presence != 0.f || r.frequency != 0.f)) {
    const int s = a.history.seqs ? a.history.seqs[b] : b;
    if ((unsigned)s < (unsigned)a.history.slots) {
      tokens = a.history.tokens + s * a.history.stride;
      length = max(0, min(a.history.lengths[s], a.history.columns));
      prompt = a.history.prompt_lengths ? max(0, min(a.history.prompt_lengths[s], length)) : 0;
    }
  }
  int bias_from = 0, bias_to = 0;
  if (a.bias_start) {
    bias_from = a.bias_start[b];
    bias_to = a.bias_start[b + 1];
    if (bias_from < 0 || bias_to > a.biases) bias_to = bias_from;
  }
  r.counts = length > 0;
  r.biases = bias_to > bias_from;
  r.bias = a.bias_values + bias_from;
  if (r.counts || r.biases) {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      if (r.counts) count[i] = 0;
      if (r.biases) named[i] = 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < length; i += kThreads) {
      const unsigned at = (unsigned)tokens[i] - (unsigned)from;
      if (at < (unsigned)n) {
        if (i < prompt)
          atomicOr(&count[at], kPrompt);
        else
          atomicAdd(&count[at], 1u);
      }
    }
    for (int i = bias_from + threadIdx.x; i < bias_to; i += kThreads) {
      const unsigned at = (unsigned)a.bias_ids[i] - (unsigned)from;
      if (at < (unsigned)n) atomicMax(&named[at], i - bias_from + 1);
    }
    __syncthreads();
  }
  const auto bit = [&](int v) { return !r.mask || (r.mask[v >> 5] >> (v & 31)) & 1; };
  if constexpr (kVec) {
    const int head = part == 0 ? min(lead, n) : 0;
    const int fours = (n - head) / kFour;
    for (int i = threadIdx.x; i < fours; i += kThreads) {
      const int at = head + kFour * i, v = from + at;
      const Four<T> x = *reinterpret_cast<const Four<T>*>(in + v);
      uint32_t bits = 15u;
      if (r.mask) {
        const uint32_t w = r.mask[v >> 5];
        const uint32_t next = (v & 31) > 32 - kFour ? r.mask[(v >> 5) + 1] : 0u;
        bits = __funnelshift_r(w, next, v & 31);
      }
      Four<U> y;
#pragma unroll
      for (int k = 0; k < kFour; ++k) put(&y.v[k], adjusted(r, count, named, to_float(x.v[k]), at + k, bits >> k & 1));
      *reinterpret_cast<Four<U>*>(out + v) = y;
    }
    // what is before and behind the aligned ones: at most three each
    const int rest = n - head - kFour * fours;
    if ((int)threadIdx.x < head + rest) {
      const int at = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + kFour * fours;
      put(&out[from + at], adjusted(r, count, named, to_float(in[from + at]), at, bit(from + at)));
    }
  } else {
    for (int at = threadIdx.x; at < n; at += kThreads)
      put(&out[from + at], adjusted(r, count, named, to_float(in[from + at]), at, bit(from + at)));
  }
}

template <typename T, typename U>
cudaError_t run(const LogitsArgs& a, cudaStream_t s) {
  const auto place = [](const void* p, size_t size) { return (long long)(reinterpret_cast<uintptr_t>(p) / size % kFour); };
  const auto same = [](long long x, long long y) { return ((x - y) % kFour) == 0; };
  const bool vec = same(place(a.logits, sizeof(T)), place(a.out, sizeof(U))) && (a.B == 1 || same(a.stride, a.out_stride));
  // Large slices where the rows fill the GPU (each reads the history once more), smaller ones where they do not.
  int slice = kMaxSlice;
  while (slice > kMinSlice && (long long)a.B * ((a.V + slice - 1) / slice) < kCtasWanted) slice /= 2;
  const int slices = (a.V + slice - 1) / slice;
  const long long ctas = (long long)a.B * slices;
  const int arrays = (a.history.tokens ? 1 : 0) + (a.bias_start ? 1 : 0);
  const int bytes = arrays * 4 * (slice + kFour);
  const auto kernel = vec ? adjust_logits<T, U, true> : adjust_logits<T, U, false>;
  return launch_dependent(kernel, (int)ctas, kThreads, bytes, s, a, slices, slice);
}

template <typename T>
cudaError_t run_type(const LogitsArgs& a, wd_dtype dtype, wd_dtype out_dtype, cudaStream_t s) {
  return out_dtype == WD_FP32 && dtype != WD_FP32 ? run<T, float>(a, s) : run<T, T>(a, s);
}

}  // namespace

cudaError_t launch_adjust_logits(const LogitsArgs& a, wd_dtype dtype, wd_dtype out_dtype, cudaStream_t s) {
  switch (dtype) {
    case WD_BF16: return run_type<__nv_bfloat16>(a, dtype, out_dtype, s);
    case WD_FP16: return run_type<__half>(a, dtype, out_dtype, s);
    default: return run_type<float>(a, dtype, out_dtype, s);
  }
}

}  // namespace wd
