// wd_logits.cu - penalties, biases, temperature and masks on logits (declared
// in include/wd_step.h).
//
// One pass: a CTA takes a slice of one row's vocabulary, with its logits and their bits of the mask in registers. While
// they are on their way it counts in shared memory how often the row's history names each of its
// tokens (every CTA of a row reads the whole history, which is small beside the logits and comes from
// L2) and notes which bias is the last for each. Nothing is written but the result, no counts live from call to call,
// and counting whole numbers gives the same sums in any order. Bytes bound it where rows are many, the
// history's scan where they are few.
#include "wd_device.cuh"
#include "wd_step.cuh"
#include "wd_vec.cuh"

namespace wd {
namespace {

constexpr int kThreads = 256;
constexpr int kFour = 4;                     // elements of an access
constexpr int kUnit = kThreads * kFour;      // tokens of a slice: this, twice or four times
constexpr int kCtasWanted = 4 * 152;         // for which slices are made smaller
constexpr uint32_t kPrompt = 1u << 31;       // of a count: the prompt has the token
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
  float repetition, presence, frequency;
  float relief, scale;  // 1 / repetition, 1 / temperature
  const float* bias;    // the values of the row's biases
  const int32_t* mask;  // its words, null: all allowed
};

// A logit with its token's count.
__device__ __forceinline__ float penalised(const Row& r, float l, uint32_t count) {
  const float turned = l * (l > 0.f ? r.relief : r.repetition);
  const uint32_t n = count & kAnswer;
  const float less = n ? fmaf((float)n, r.frequency, r.presence) : 0.f;
  return count ? turned - less : l;
}
// ... and with 1 + its last bias, 0 for none.
__device__ __forceinline__ float biased(const Row& r, float l, uint32_t named) {
  return named ? l + r.bias[named - 1] : l;
}

// The tokens of a row's history that are in [from, from + n), counted at `count`.
__device__ __forceinline__ void count_tokens(const int32_t* tokens, int length, int prompt, int from, int n, uint32_t* count) {
  const auto one = [&](int token, int i) {
    const unsigned at = (unsigned)token - (unsigned)from;
    if (at < (unsigned)n) {
      if (i >= prompt)
        atomicAdd(&count[at], 1u);
      else if (!(count[at] & kPrompt))
        atomicOr(&count[at], kPrompt);
    }
  };
  // up to the first aligned one, then four to an access and four accesses on their way at a time
  const int head = min(length, (int)((4 - (reinterpret_cast<uintptr_t>(tokens) >> 2) % 4) % 4));
  const int fours = (length - head) / 4;
  const int4* aligned = reinterpret_cast<const int4*>(tokens + head);
  for (int i = threadIdx.x; i < fours; i += 4 * kThreads) {
    int4 t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      t[j] = i + j * kThreads < fours ? aligned[i + j * kThreads] : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int at = head + 4 * (i + j * kThreads);
      one(t[j].x, at);
      one(t[j].y, at + 1);
      one(t[j].z, at + 2);
      one(t[j].w, at + 3);
    }
  }
  const int rest = length - head - 4 * fours;
  if ((int)threadIdx.x < head + rest) {
    const int i = (int)threadIdx.x < head ? threadIdx.x : threadIdx.x + 4 * fours;
    one(tokens[i], i);
  }
}

// Slice `blockIdx.x % slices` of row `blockIdx.x / slices`, kPer fours of tokens to a thread. kVec: input and output of a
// row reach the alignment of four elements at the same token; slices begin there. The first one has what is
// before that, too, and the one of the last four what is behind it.
template <typename T, typename U, int kPer, bool kVec>
__global__ void __launch_bounds__(kThreads) adjust_logits(const LogitsArgs a, int slices) {
  constexpr int kSlice = kPer * kUnit;
  constexpr int kPlaces = kSlice + 2 * kFour;  // of an array in shared memory: place 4 is the slice's first four
  extern __shared__ uint4 shared[];
  const int b = blockIdx.x / slices, part = blockIdx.x % slices;
  const T* in = static_cast<const T*>(a.logits) + b * a.stride;
  U* out = static_cast<U*>(a.out) + b * a.out_stride;
  const int lead =
      kVec ? min(a.V, (int)((kFour - (reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kFour) % kFour)) : 0;
  const int last = lead + (a.V - lead) / kFour * kFour;  // behind the row's last four
  const int begin = lead + part * kSlice, end = min(begin + kSlice, last);
  const int closing = min((last - lead) / kSlice, slices - 1);  // the slice that the tokens behind the last four go to
  const int from = part == 0 ? 0 : begin, to = part == closing ? a.V : end;
  uint32_t* count = reinterpret_cast<uint32_t*>(shared);
  int32_t* named = reinterpret_cast<int32_t*>(count + (a.history.tokens ? kPlaces : 0));
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  if (to <= from) return;
  Row r;
  r.mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
  // this thread's logits, and four bits of the mask for each access
  Four<T> x[kPer];
  uint32_t allowed = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int v = begin + kFour * (threadIdx.x + j * kThreads);
    if (v >= end) continue;
    if constexpr (kVec) {
      x[j] = *reinterpret_cast<const Four<T>*>(in + v);
    } else {
#pragma unroll
      for (int k = 0; k < kFour; ++k) x[j].v[k] = in[v + k];
    }
  }
  if (r.mask) {
    allowed = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = begin + kFour * (threadIdx.x + j * kThreads);
      if (v >= end) continue;
      const uint32_t word = r.mask[v >> 5];
      const uint32_t next = (v & 31) > 32 - kFour ? r.mask[(v >> 5) + 1] : 0u;
      allowed |= (__funnelshift_r(word, next, v & 31) & 15u) << (kFour * j);
    }
  }
  r.repetition = a.repetition ? a.repetition[b] : 1.f;
  r.presence = a.presence ? a.presence[b] : 0.f;
  r.frequency = a.frequency ? a.frequency[b] : 0.f;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  r.scale = t > 0.f ? 1.f / t : 1.f;
  r.relief = 1.f / r.repetition;
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
  r.bias = a.bias_values + bias_from;
  const bool counts = length > 0, biases = bias_to > bias_from;
  if (counts || biases) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < kPlaces / kFour; i += kThreads) {
      if (counts) reinterpret_cast<uint4*>(count)[i] = zero;
      if (biases) reinterpret_cast<uint4*>(named)[i] = zero;
    }
    __syncthreads();
    const int place = kFour - (begin - from);  // of token `from`
    if (counts) count_tokens(tokens, length, prompt, from, to - from, count + place);
    for (int i = bias_from + threadIdx.x; i < bias_to; i += kThreads) {
      const unsigned at = (unsigned)a.bias_ids[i] - (unsigned)from;
      if (at < (unsigned)(to - from)) atomicMax(&named[place + at], i - bias_from + 1);
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int f = threadIdx.x + j * kThreads, v = begin + kFour * f;
    if (v >= end) continue;
    float l[kFour];
#pragma unroll
    for (int k = 0; k < kFour; ++k) l[k] = to_float(x[j].v[k]);
    if (counts) {
      const uint4 c = reinterpret_cast<const uint4*>(count)[f + 1];
      if (c.x | c.y | c.z | c.w) {
        l[0] = penalised(r, l[0], c.x);
        l[1] = penalised(r, l[1], c.y);
        l[2] = penalised(r, l[2], c.z);
        l[3] = penalised(r, l[3], c.w);
      }
    }
    if (biases) {
      const uint4 e = reinterpret_cast<const uint4*>(named)[f + 1];
      if (e.x | e.y | e.z | e.w) {
        l[0] = biased(r, l[0], e.x);
        l[1] = biased(r, l[1], e.y);
        l[2] = biased(r, l[2], e.z);
        l[3] = biased(r, l[3], e.w);
      }
    }
    Four<U> y;
#pragma unroll
    for (int k = 0; k < kFour; ++k) put(&y.v[k], allowed >> (kFour * j + k) & 1 ? l[k] * r.scale : -INFINITY);
    if constexpr (kVec) {
      *reinterpret_cast<Four<U>*>(out + v) = y;
    } else {
#pragma unroll
      for (int k = 0; k < kFour; ++k) out[v + k] = y.v[k];
    }
  }
  // the loose tokens, at most three before the first four and three behind the last
  const int before = begin - from > 0 ? min(begin, to) - from : 0, behind = max(0, to - max(end, begin));
  if ((int)threadIdx.x < before + behind) {
    const int v = (int)threadIdx.x < before ? from + threadIdx.x : max(end, begin) + threadIdx.x - before;
    const int at = kFour + v - begin;
    const float l = biased(r, penalised(r, to_float(in[v]), counts ? count[at] : 0u), biases ? named[at] : 0u);
    put(&out[v], !r.mask || (r.mask[v >> 5] >> (v & 31) & 1) ? l * r.scale : -INFINITY);
  }
}

template <typename T, typename U, int kPer>
cudaError_t run_slices(const LogitsArgs& a, bool vec, cudaStream_t s) {
  const int slices = (a.V + kPer * kUnit - 1) / (kPer * kUnit);
  const int arrays = (a.history.tokens ? 1 : 0) + (a.bias_start ? 1 : 0);
  return launch_dependent(vec ? adjust_logits<T, U, kPer, true> : adjust_logits<T, U, kPer, false>, a.B * slices, kThreads,
                          arrays * 4 * (kPer * kUnit + 2 * kFour), s, a, slices);
}

template <typename T, typename U>
cudaError_t run(const LogitsArgs& a, cudaStream_t s) {
  const auto place = [](const void* p, size_t size) { return (long long)(reinterpret_cast<uintptr_t>(p) / size % kFour); };
  const auto same = [](long long x, long long y) { return ((x - y) % kFour) == 0; };
  const bool vec = same(place(a.logits, sizeof(T)), place(a.out, sizeof(U))) && (a.B == 1 || same(a.stride, a.out_stride));
  // Large slices where the rows fill the GPU (each reads the history once more), smaller ones where they do not.
  const auto ctas = [&](int per) { return (long long)a.B * ((a.V + per * kUnit - 1) / (per * kUnit)); };
  if (ctas(4) >= kCtasWanted) return run_slices<T, U, 4>(a, vec, s);
  if (ctas(2) >= kCtasWanted) return run_slices<T, U, 2>(a, vec, s);
  return run_slices<T, U, 1>(a, vec, s);
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
