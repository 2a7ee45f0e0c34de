// wd_route.cu - routing of tokens to experts (declared in include/wd_step.h).
//
// A warp takes a token. Its lanes hold the experts in order: a group of experts (there are 1 to 32)
// has 32 / groups lanes, rounded down to a power of two, and each of them kV consecutive ones, so that
// a group's value is a few shuffles within its lanes. K times the warp's largest key is found by one
// redux over keys whose integer order is their order, and struck out.
//
// Keys are exact where no bias and no sums of groups are asked for: they are the logits. Those of 16 bits
// share a word with their expert's index, so that one redux gives both, the lowest index first of equal keys; a lane
// sorts its words once and only its first one is looked at. Other keys need a second redux for the index.
// Keys of scores and biases carry FP32's errors (margin below); a token of which two keys that the choice
// hangs on are nearer than that is chosen again from keys in 64 bits: those of the K and
// of what is as near to the last of them, one to a lane, or all of them where groups are in doubt.
//
// Bounded by the instructions of a token, not by its bytes.
#include "wd_device.cuh"
#include "wd_step.cuh"
#include "wd_vec.cuh"

namespace wd {
namespace {

constexpr int kWarps = 4;  // tokens of a CTA
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// Integers in the order of the numbers; 0 stands below -inf. NaN is not asked for, -0 is 0.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t u) {
  return __uint_as_float(u ^ ((u & 0x80000000u) ? 0x80000000u : 0xFFFFFFFFu));
}
__device__ __forceinline__ unsigned long long order_of(double x) {
  const long long u = __double_as_longlong(x + 0.0);
  return (unsigned long long)(u ^ ((u >> 63) | (long long)0x8000000000000000ull));
}

__device__ __forceinline__ float warp_max(float v) {
  return value_of(__reduce_max_sync(kAll, order_of(v)));
}
__device__ __forceinline__ float warp_min(float v) { return -warp_max(-v); }
__device__ __forceinline__ uint32_t largest(uint32_t v) { return __reduce_max_sync(kAll, v); }
__device__ __forceinline__ unsigned long long largest(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(kAll, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return (unsigned long long)hi << 32 | lo;
}

// The same of 16-bit numbers, given as floats.
__device__ __forceinline__ uint32_t half_order(float x, __nv_bfloat16) { return order_of(x) >> 16; }
__device__ __forceinline__ float half_value(uint32_t u, __nv_bfloat16) {
  return __uint_as_float((u << 16) ^ ((u & 0x8000u) ? 0x80000000u : 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t half_order(float x, __half) {
  const uint32_t u = __half_as_ushort(__float2half_rn(x + 0.f));
  return (u ^ ((u & 0x8000u) ? 0xFFFFu : 0x8000u)) & 0xFFFFu;
}
__device__ __forceinline__ float half_value(uint32_t u, __half) {
  return __half2float(__ushort_as_half((unsigned short)(u ^ ((u & 0x8000u) ? 0x8000u : 0xFFFFu))));
}
__device__ __forceinline__ uint32_t half_order(float, float) { return 0; }  // (no 16 bits, not used)

// Where the experts of a lane begin, and how many it has.
struct Span {
  int first, n;
};
struct Lanes {
  int shift;      // log2 of per_group
  int per_group;  // lanes of a group
  int per_lane;   // experts of a lane
  int size;       // experts of a group
};
Lanes lanes_of(int E, int groups) {
  int up = 1, shift = 5;
  while (up < groups) up *= 2, --shift;
  const int per_group = 32 / up, size = E / groups;
  return Lanes{shift, per_group, (size + per_group - 1) / per_group, size};
}

// The value of a group from its lanes' two largest keys, in each of its lanes. A masked second
// key takes no part.
template <typename F>
__device__ __forceinline__ F group_value(F a, F b, int lanes, int best) {
  for (int off = 1; off < lanes; off *= 2) {
    const F c = __shfl_xor_sync(kAll, a, off), d = __shfl_xor_sync(kAll, b, off);
    const F low = a < c ? a : c;
    a = a < c ? c : a;
    b = b < d ? d : b;
    b = b < low ? low : b;
  }
  return best == 2 && b > -INFINITY ? a + b : a;
}

// Whether this lane's group is among the `top` largest, ties to the lowest index.
template <typename F>
__device__ __forceinline__ bool group_chosen(F value, int group, int groups, int lanes, int top) {
  int before = 0;
  for (int g = 0; g < groups; ++g) {
    const F other = __shfl_sync(kAll, value, g * lanes);
    before += other > value || (other == value && g < group);
  }
  return before < top;
}

// The `n` largest keys of the warp, largest first: entry r in lane r % 32, place r / 32 of `ids`. Keys are
// struck out of k. With a margin, goes on until the next key is further than that below the last one: returns how many it
// took, kMany if that is more than 64; `near`: whether two neighbours of the order are nearer than the margin.
constexpr int kMany = 65;

template <int kV, typename Key>
__device__ __forceinline__ int take(Key (&k)[kV], const Span& mine, int n, int lane, float margin, bool& near,
                                    int (&ids)[2]) {
  Key last = 0;
  for (int r = 0;; ++r) {
    if (r >= n && !(margin > 0.f)) return r;
    Key top = k[0];
#pragma unroll
    for (int i = 1; i < kV; ++i) top = top < k[i] ? k[i] : top;
    const Key all = largest(top);
    if (margin > 0.f && r > 0) {
      const bool close = all && value_of((uint32_t)last) - value_of((uint32_t)all) < margin;
      if (r >= n && (!close || r == 64)) return close ? kMany : r;
      near |= close;
    }
    last = all;
    int at = 1 << 20;  // of this lane's experts that have the key, the first
#pragma unroll
    for (int i = kV - 1; i >= 0; --i)
      if (k[i] == all) at = mine.first + i;
    const int id = __reduce_min_sync(kAll, at);
#pragma unroll
    for (int i = 0; i < kV; ++i)
      if (mine.first + i == id) k[i] = 0;
    if (lane == r) ids[0] = id;
    if (lane + 32 == r) ids[1] = id;
  }
}

// Descending order of a lane's words (Batcher's bitonic sort: its loops are plain enough to be unrolled at any kV).
template <int kV>
__device__ __forceinline__ void sort_down(uint32_t (&k)[kV]) {
#pragma unroll
  for (int run = 2; run <= kV; run *= 2)
#pragma unroll
    for (int apart = run / 2; apart > 0; apart /= 2)
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        if (i & apart) continue;
        const uint32_t a = k[i], b = k[i + apart];
        const bool down = (i & run) == 0;
        k[i] = down ? max(a, b) : min(a, b);
        k[i + apart] = down ? min(a, b) : max(a, b);
      }
}

// The K largest words, as take(): of words that hold key and index no two are equal.
template <int kV>
__device__ __forceinline__ void take_words(uint32_t (&k)[kV], int K, int lane, uint32_t (&words)[2]) {
  sort_down<kV>(k);
  const auto next = [&] {  // the largest of all, taken from the lane that has it
    const uint32_t all = largest(k[0]);
    const bool taken = k[0] == all;
#pragma unroll
    for (int i = 0; i < kV; ++i) k[i] = taken ? (i + 1 < kV ? k[i + 1] : 0u) : k[i];
    return all;
  };
#pragma unroll(kV <= 8 ? 4 : 1)
  for (int r = 0; r < min(K, 32); ++r) {
    const uint32_t all = next();
    words[0] = lane == r ? all : words[0];
  }
  for (int r = 32; r < K; ++r) {
    const uint32_t all = next();
    words[1] = lane + 32 == r ? all : words[1];
  }
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// For keys, which are compared as they are: __expf is off by |x| units relative to itself, s (1 - s) of which reaches the
// sigmoid s, at most one unit of 1; the quotient by two.
__device__ __forceinline__ float sigmoid_key(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// exp(x - top), where top is at least x; 1 for the largest even if infinite, 0 for masked ones.
__device__ __forceinline__ float exp_below(float x, float top) {
  return x == -INFINITY ? 0.f : x == top ? 1.f : expf(x - top);
}

// The score's key in 64 bits of an expert whose logit is l. `top`: the token's largest logit, `sum`: of exp(l - top).
__device__ __forceinline__ double exact_key(const RouteArgs& a, float l, int id, float top, double sum) {
  if (!(l > -INFINITY)) return -(double)INFINITY;
  const double score = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : l == top ? 1.0 / sum : exp((double)l - (double)top) / sum;
  const double key = score + (a.bias ? (double)a.bias[id] : 0.0);
  return key == key ? key : -(double)INFINITY;
}

// The sum of exp(l - top) over all experts, in 64 bits; not needed for sigmoids.
template <typename T>
__device__ __forceinline__ double exact_sum(const RouteArgs& a, const T* x, const Span& mine, float top) {
  if (a.sigmoid) return 1.0;
  double sum = 0.0;
  for (int i = 0; i < mine.n; ++i) {
    const float l = to_float(x[mine.first + i]);
    if (l > -INFINITY) sum += l == top ? 1.0 : exp((double)l - (double)top);
  }
  for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(kAll, sum, off);
  return sum;
}

// The order of the `n` <= 64 candidates that take() found, from keys in 64 bits. Rare, so it is kept out of the way
// of the other registers.
template <typename T>
__device__ __noinline__ void order_again(const RouteArgs& a, const T* x, const Span mine, int lane, float top, int n,
                                         int (&ids)[2]) {
  const double sum = exact_sum(a, x, mine, top);
  unsigned long long key[2];
  int rank[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    key[e] = 0;
    if (lane + 32 * e < n) key[e] = order_of(exact_key(a, to_float(x[ids[e]]), ids[e], top, sum));
  }
  for (int r = 0; r < n; ++r) {
    const unsigned long long other = __shfl_sync(kAll, key[r >> 5], r & 31);
    const int id = __shfl_sync(kAll, ids[r >> 5], r & 31);
#pragma unroll
    for (int e = 0; e < 2; ++e) rank[e] += other > key[e] || (other == key[e] && id < ids[e]);
  }
  int sorted[2] = {0, 0};
  for (int r = 0; r < n; ++r) {
    const int to = __shfl_sync(kAll, rank[r >> 5], r & 31);
    const int id = __shfl_sync(kAll, ids[r >> 5], r & 31);
    if (to == lane) sorted[0] = id;
    if (to == lane + 32) sorted[1] = id;
  }
  ids[0] = sorted[0];
  ids[1] = sorted[1];
}

// The token's whole choice from keys in 64 bits.
template <typename T, int kV>
__device__ __noinline__ void choose_again(const RouteArgs& a, const T* x, const Span mine, const Lanes lanes, int lane,
                                          float top, int (&ids)[2]) {
  const int group = lane >> lanes.shift;
  const double sum = exact_sum(a, x, mine, top);
  unsigned long long k[kV];
  double best = -INFINITY, second = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < kV; ++i) {
    k[i] = 0;
    if (i >= mine.n) continue;
    const float l = to_float(x[mine.first + i]);
    const double key = exact_key(a, l, mine.first + i, top, sum);
    second = second > key ? second : best < key ? best : key;
    best = best < key ? key : best;
    // where nothing is added, keys are ordered by the logits
    k[i] = order_of(a.bias ? key : (double)(l > -INFINITY ? l : -INFINITY));
  }
  if (a.groups > 1) {
    const double value = group_value(best, second, lanes.per_group, a.group_best);
    const bool chosen = group_chosen(group < a.groups ? value : -(double)INFINITY, group, a.groups, lanes.per_group, a.top_groups);
    if (!chosen)
#pragma unroll
      for (int i = 0; i < kV; ++i) k[i] = 0;
  }
  bool none;
  take<kV>(k, mine, a.K, lane, 0.f, none, ids);
}

// kWords: logits of 16 bits, and no bias.
template <typename T, int kV, bool kVec, bool kWords>
__global__ void __launch_bounds__(32 * kWarps) route(const __grid_constant__ RouteArgs a, const Lanes lanes) {
  const int lane = threadIdx.x & 31;
  const int token = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int group = lane >> lanes.shift, j = lane & (lanes.per_group - 1);
  Span mine{group * lanes.size + j * lanes.per_lane, 0};
  if (group < a.groups) mine.n = max(0, min(lanes.per_lane, lanes.size - j * lanes.per_lane));
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  if (token >= a.tokens) return;
  const T* x = static_cast<const T*>(a.logits) + (long long)token * a.stride;
  float l[kV];
  if constexpr (kVec) {  // every lane has kV experts
    struct alignas(sizeof(T) * kV < 16 ? sizeof(T) * kV : 16) Pack {
      T v[kV];
    };
    const Pack p = *reinterpret_cast<const Pack*>(x + mine.first);
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = to_float(p.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kV; ++i) l[i] = i < mine.n ? to_float(x[mine.first + i]) : -INFINITY;
  }
  const bool sums = a.groups > 1 && a.group_best == 2;
  const bool inexact = a.bias || sums;  // keys that are not the logits
  float top = -INFINITY, sum = 0.f;     // of a softmax over all experts: the largest logit, the sum of exp(l - top)
  float s[kV];                          // scores, then keys
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    if (!(l[i] == l[i])) l[i] = -INFINITY;
    s[i] = l[i];
  }
  if (!a.sigmoid && (inexact || !a.renormalise)) {
#pragma unroll
    for (int i = 0; i < kV; ++i) top = fmaxf(top, l[i]);
    top = warp_max(top);
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      s[i] = exp_below(l[i], top);
      sum += s[i];
    }
    sum = warp_sum(sum);
  }
  const float unit = a.sigmoid ? 1.f : sum > 0.f ? 1.f / sum : 0.f;  // the largest score there may be
  float margin = 0.f;
  if (inexact) {
    float most = 0.f;  // largest magnitude of a key
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      if (l[i] > -INFINITY) {
        s[i] = a.sigmoid ? sigmoid_key(l[i]) : s[i] * unit;
        if (a.bias) s[i] += a.bias[mine.first + i];
        if (!(s[i] == s[i])) s[i] = -INFINITY;
        if (fabsf(s[i]) < INFINITY) most = fmaxf(most, fabsf(s[i]));
      } else {
        s[i] = -INFINITY;
      }
    }
    // In units of 2^-24, a softmax' score is off by 2 (expf), 1 (its argument), 2 (quotient), 1 (the product by it) and the
    // sum of all of them, kV + 5 roundings at most; a sigmoid's by less than 12 of 1; a key by half a unit of its own more.
    // Two keys are compared.
    most = warp_max(most);
    margin = 0x1p-23f * (a.sigmoid ? 12 : kV + 12) * unit + 0x1p-23f * most;
  }
  bool again = false, chosen = true;
  if (a.groups > 1) {
    float best = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const float key = inexact ? s[i] : l[i];
      second = fmaxf(second, fminf(best, key));
      best = fmaxf(best, key);
    }
    float value = group_value(best, second, lanes.per_group, a.group_best);
    if (group >= a.groups) value = -INFINITY;
    chosen = group_chosen(value, group, a.groups, lanes.per_group, a.top_groups);  // (all lanes take part)
    if (group >= a.groups) chosen = false;
    if (inexact) {
      const float in = warp_min(chosen ? value : INFINITY);
      const float out = warp_max(chosen ? -INFINITY : value);
      again = in - out < 2.f * margin;
    }
  }
  uint32_t k[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    // without a bias the choice goes by the logits even where the groups' goes by sums of scores
    if (!chosen || (!kVec && i >= mine.n))
      k[i] = 0;
    else if (kWords)
      k[i] = half_order(l[i], T{}) << 16 | (0xFFFFu - (mine.first + i));
    else
      k[i] = order_of(a.bias ? s[i] : l[i]);
  }
  int ids[2] = {0, 0};
  float y[2] = {-INFINITY, -INFINITY}, w[2] = {0.f, 0.f};  // logits and weights of the chosen
  if constexpr (kWords) {
    uint32_t words[2] = {0, 0};
    take_words<kV>(k, a.K, lane, words);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < a.K) {
        ids[e] = 0xFFFF - (words[e] & 0xFFFFu);
        y[e] = half_value(words[e] >> 16, T{});
      }
  } else {
    bool near = false;
    const int n = take<kV>(k, mine, a.K, lane, a.bias ? margin : 0.f, near, ids);
    if (n == kMany) again = true;
    if (near && !again) {
      int mended[2] = {ids[0], ids[1]};  // (its own, so that ids stay in registers)
      order_again<T>(a, x, mine, lane, top, n, mended);
      ids[0] = mended[0];
      ids[1] = mended[1];
    }
  }
  if (again) {
    int mended[2] = {0, 0};
    choose_again<T, kV>(a, x, mine, lanes, lane, top, mended);
    ids[0] = mended[0];
    ids[1] = mended[1];
  }
  const int halves = a.K > 32 ? 2 : 1;
  if (!kWords || again) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < a.K) {
        y[e] = to_float(x[ids[e]]);
        if (!(y[e] == y[e])) y[e] = -INFINITY;
      }
  }
  const float high = warp_max(fmaxf(y[0], y[1]));
  float total = 0.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (e >= halves) break;
    if (a.renormalise)  // scaled alike: far below 0 a sigmoid is an exponential, to all of FP32's bits
      w[e] = a.sigmoid && high > -40.f ? (y[e] > -INFINITY ? sigmoid(y[e]) : 0.f) : exp_below(y[e], high);
    else
      w[e] = y[e] > -INFINITY ? (a.sigmoid ? sigmoid(y[e]) : exp_below(y[e], top) * unit) : 0.f;
    total += w[e];
  }
  if (a.renormalise) {
    total = warp_sum(total);
    const float f = total > 0.f ? a.scale / total : 0.f;
    w[0] *= f;
    w[1] *= f;
  } else {
    w[0] *= a.scale;
    w[1] *= a.scale;
  }
  const long long at = (long long)token * a.K + lane;
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 32 * e < a.K) {
      a.ids[at + 32 * e] = ids[e];
      a.weights[at + 32 * e] = w[e];
    }
}

template <typename T, int kV>
cudaError_t run(const RouteArgs& a, const Lanes lanes, cudaStream_t s) {
  constexpr int kBytes = sizeof(T) * kV < 16 ? sizeof(T) * kV : 16;
  const bool vec = lanes.per_lane == kV && a.groups * lanes.per_group == 32 && a.E == 32 * kV &&
                   reinterpret_cast<uintptr_t>(a.logits) % kBytes == 0 && a.stride * (long long)sizeof(T) % kBytes == 0;
  const int ctas = (a.tokens + kWarps - 1) / kWarps;
  constexpr bool kWords = sizeof(T) == 2;
  constexpr bool kPacks = kV <= 16;  // (1024 experts are rare enough for single loads)
  const auto kernel = kWords && !a.bias ? (vec ? route<T, kV, kPacks, kWords> : route<T, kV, false, kWords>)
                                        : (vec ? route<T, kV, kPacks, false> : route<T, kV, false, false>);
  return launch_dependent(kernel, ctas, 32 * kWarps, 0, s, a, lanes);
}

template <typename T>
cudaError_t run_type(const RouteArgs& a, cudaStream_t s) {
  const Lanes lanes = lanes_of(a.E, a.groups);
  if (lanes.per_lane <= 1) return run<T, 1>(a, lanes, s);
  if (lanes.per_lane <= 2) return run<T, 2>(a, lanes, s);
  if (lanes.per_lane <= 4) return run<T, 4>(a, lanes, s);
  if (lanes.per_lane <= 8) return run<T, 8>(a, lanes, s);
  if (lanes.per_lane <= 16) return run<T, 16>(a, lanes, s);
  return run<T, 32>(a, lanes, s);
}

}  // namespace

bool route_supported(int E, int groups) {
  return E <= WD_ROUTE_MAX_EXPERTS && groups <= 32 && E % groups == 0 && lanes_of(E, groups).per_lane <= 32;
}

cudaError_t launch_route(const RouteArgs& a, wd_dtype dtype, cudaStream_t s) {
  switch (dtype) {
    case WD_BF16: return run_type<__nv_bfloat16>(a, s);
    case WD_FP16: return run_type<__half>(a, s);
    default: return run_type<float>(a, s);
  }
}

}  // namespace wd
