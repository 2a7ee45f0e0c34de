// wd_route.cu - routing of tokens to experts (declared in include/wd_step.h).
//
// A warp takes a token. Its lanes hold the experts in order: a group of experts (there are 1 to 32)
// has 32 / groups lanes, rounded down to a power of two, and each of them kV consecutive ones, so that
// a group's value is a few shuffles within its lanes. K times the warp's largest key is found by one
// redux over keys whose integer order is their order, and struck out.
//
// A lane sorts its keys once, and of them only the first is looked at.
//
// Keys are exact where no bias and no sums of groups are asked for: they are the logits. Those of 16 bits
// share a word with their expert's index, so that one redux gives both, the lowest index first of equal keys. Keys
// of 32 bits share one with their place in the lane, which takes their last few bits. Keys of scores and biases carry FP32's errors
// besides. A token of which two keys that the choice hangs on are nearer than that is looked at again with keys in
// 64 bits, of those experts alone that are in doubt, one to a lane: the best of each group, the K and what is
// as near to the last of them. (With all keys in 64 bits one token takes 12 us at 496 experts, and the call waits for it.)
//
// Bounded by the instructions of a token, most of them for the half-rate pipe that compares and selects, not by
// its bytes. Measured: 16384 tokens of 128 experts, 8 of them, BF16 7.3 us (FP32 11.0); of 256 in 8 groups with a bias
// 19.9 us; of 512 13.5 us, of 1000 30.9; 32 tokens of 128 1.9 us. Tried: a warp that goes from token to token with the biases
// in registers (27 -> 30.7 us of the groups then, 7.0 -> 7.8), lanes' lists moved up in registers (15.8 against 13.5 us at 512
// experts, the same at 128).
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
  int per_lane;   // experts of a lane, a power of two; the last lanes of a group have fewer or none
  int size;       // experts of a group
  bool packs, bias_packs;  // logits and biases of a lane that has all its experts may be loaded as vectors
};
Lanes lanes_of(int E, int groups) {
  int up = 1, shift = 5, per_lane = 1;
  while (up < groups) up *= 2, --shift;
  const int per_group = 32 / up, size = E / groups;
  while (per_lane * per_group < size) per_lane *= 2;
  return Lanes{shift, per_group, per_lane, size, false, false};
}

// The two largest keys of a group from its lanes' two largest, in each of its lanes.
template <typename F>
__device__ __forceinline__ void two_of_group(F& a, F& b, int lanes) {
  for (int off = 1; off < lanes; off *= 2) {
    const F c = __shfl_xor_sync(kAll, a, off), d = __shfl_xor_sync(kAll, b, off);
    const F low = a < c ? a : c;
    a = a < c ? c : a;
    b = b < d ? d : b;
    b = b < low ? low : b;
  }
}
// ... and its value. A masked second key takes no part.
__device__ __forceinline__ double group_value(double a, double b, int lanes, int best) {
  two_of_group(a, b, lanes);
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

// The `n` largest keys of 64 bits, largest first, the lowest index first of equal ones: entry r in lane r % 32, place r / 32
// of `ids`. Keys are struck out of k.
template <int kV>
__device__ __forceinline__ void take_exact(unsigned long long (&k)[kV], const Span& mine, int n, int lane, int (&ids)[2]) {
  for (int r = 0; r < n; ++r) {
    unsigned long long top = k[0];
#pragma unroll
    for (int i = 1; i < kV; ++i) top = top < k[i] ? k[i] : top;
    const unsigned long long all = largest(top);
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

// A lane's words in descending order, of which the first is looked at: the others stand in shared memory (the columns of a
// warp's `rows` of 32), where taking one is a load of the next instead of a move of all.
template <int kV>
struct Sorted {
  uint32_t head;
  const uint32_t* next;
  // (of lanes that are not `open` none is taken)
  __device__ __forceinline__ Sorted(uint32_t (&k)[kV], uint32_t* rows, int lane, bool open) {
    sort_down<kV>(k);
    head = open ? k[0] : 0;
    next = rows + lane;
#pragma unroll
    for (int i = 1; i < kV; ++i) rows[32 * (i - 1) + lane] = k[i];
    rows[32 * (kV - 1) + lane] = 0;  // (a lane reads its own column alone)
  }
  __device__ __forceinline__ void take(bool mine) {
    if (mine) {
      head = *next;
      next += 32;
    }
  }
};

// The K largest words, to taken[0] .. taken[K - 1]: of words that hold key and index no two are equal.
template <int kV>
__device__ __forceinline__ void take_words(Sorted<kV>& sorted, int K, uint32_t* taken) {
#pragma unroll 2
  for (int r = 0; r < K; ++r) {
    const uint32_t all = largest(sorted.head);
    const bool mine = all && sorted.head == all;  // (nothing is open while groups are in doubt)
    if (mine) taken[r] = all;
    sorted.take(mine);
  }
  __syncwarp();
}

// Takes the largest word of key and place in the lane, and its expert, to taken[r] and ids[r] (0 if there is none).
template <int kV>
__device__ __forceinline__ void take_place(Sorted<kV>& sorted, const Span& mine, int lane, int r, uint32_t* taken,
                                           uint32_t* ids) {
  const uint32_t all = largest(sorted.head);
  const int winner = __ffs(__ballot_sync(kAll, sorted.head == all)) - 1;  // (words of two lanes may be the same)
  const bool take = lane == winner;
  if (take) {
    taken[r] = all;
    ids[r] = mine.first + (kV - 1 - (int)(all & (kV - 1)));
  }
  sorted.take(take && all);
}

// Whether the key of word b may be before that of its neighbour a: the two words are the same but for the place or, where keys
// are off by `off` and `part` of themselves, nearer than that. Masked ones are like nothing else, infinite ones far from all
// that are not.
template <int kV>
__device__ __forceinline__ bool too_near(uint32_t a, uint32_t b, float off, float part) {
  if (!b) return false;
  constexpr uint32_t kKey = ~(uint32_t)(kV - 1);  // without the place, which may lift b as far as a's next step
  if ((a ^ b) < (uint32_t)kV) return true;
  const float x = value_of(a & kKey), y = value_of(b & kKey);
  return off > 0.f && b > order_of(-INFINITY) && !(x - y >= fmaf(part, fmaxf(fabsf(x), fabsf(y)), off));
}

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// For keys, which are compared as they are: the exponential is off by 4 + 1.5 |x| units of 2^-24 relative to itself, s (1 - s)
// of which reaches the sigmoid s, little more than one unit of 1; the sum and the reciprocal by three.
__device__ __forceinline__ float sigmoid_key(float x) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

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

// The order of `n` <= 64 experts, from keys in 64 bits. Rare, so it is kept out of the way
// of the other registers.
template <typename T>
__device__ __noinline__ void order_again(const RouteArgs& a, const T* x, const Span mine, int lane, float top, int n,
                                         int (&ids)[2]) {
  const double sum = a.bias ? exact_sum(a, x, mine, top) : 1.0;
  unsigned long long key[2];
  int rank[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    key[e] = 0;
    if (lane + 32 * e < n) {
      const float l = to_float(x[ids[e]]);
      key[e] = order_of(a.bias ? exact_key(a, l, ids[e], top, sum) : (double)(l > -INFINITY ? l : -INFINITY));
    }
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

// Whether this lane's group is chosen, from the keys in 64 bits of those experts that may be the best of a group: whose
// key is not below `least` (NaN where biases are infinite: all of the group). False in `sure` if those are more than 64. Rare, too.
template <typename T, int kV>
__device__ __noinline__ bool groups_again(const RouteArgs& a, const T* x, const Span mine, const Lanes lanes, int lane,
                                          float top, const float (&keys)[kV], float least, uint32_t* list, bool& sure) {
  const int group = lane >> lanes.shift;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    const bool may = i < mine.n && keys[i] > -INFINITY && !(keys[i] < least);
    const uint32_t who = __ballot_sync(kAll, may);
    const int at = n + __popc(who & ((1u << lane) - 1));
    if (may && at < 64) list[at] = mine.first + i;
    n += __popc(who);
  }
  __syncwarp();
  sure = n <= 64;
  if (!sure) return false;
  const double sum = exact_sum(a, x, mine, top);
  double key[2] = {0.0, 0.0};
  int id[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 2; ++e)
    if (lane + 32 * e < n) {
      id[e] = list[lane + 32 * e];
      key[e] = exact_key(a, to_float(x[id[e]]), id[e], top, sum);
    }
  __syncwarp();
  double best = -INFINITY, second = -INFINITY;
  for (int r = 0; r < n; ++r) {
    const double k = __shfl_sync(kAll, r < 32 ? key[0] : key[1], r & 31);
    const int of = __shfl_sync(kAll, r < 32 ? id[0] : id[1], r & 31) / lanes.size;
    if (of != group) continue;
    second = second > k ? second : best < k ? best : k;
    best = best < k ? k : best;
  }
  const double value = a.group_best == 2 && second > -INFINITY ? best + second : best;
  const bool chosen = group_chosen(group < a.groups ? value : -(double)INFINITY, group, a.groups, lanes.per_group, a.top_groups);
  return chosen && group < a.groups;
}

// The choice of a token's experts from all their keys in 64 bits, in the chosen groups.
template <typename T, int kV>
__device__ __noinline__ void choose_again(const RouteArgs& a, const T* x, const Span mine, const Lanes lanes, int lane,
                                          float top, bool groups_too, bool chosen, int (&ids)[2]) {
  const int group = lane >> lanes.shift;
  const bool scores = a.bias || groups_too;  // else the logits are the keys
  const double sum = scores ? exact_sum(a, x, mine, top) : 1.0;
  unsigned long long k[kV];
  double best = -INFINITY, second = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < kV; ++i) {
    k[i] = 0;
    if (i >= mine.n) continue;
    const float l = to_float(x[mine.first + i]);
    const double logit = l > -INFINITY ? l : -INFINITY;
    const double key = scores ? exact_key(a, l, mine.first + i, top, sum) : logit;
    second = second > key ? second : best < key ? best : key;
    best = best < key ? key : best;
    // where nothing is added, keys are ordered by the logits
    k[i] = order_of(a.bias ? key : logit);
  }
  if (groups_too) {
    const double value = group_value(best, second, lanes.per_group, a.group_best);
    chosen = group_chosen(group < a.groups ? value : -(double)INFINITY, group, a.groups, lanes.per_group, a.top_groups);
  }
  if (!chosen)
#pragma unroll
    for (int i = 0; i < kV; ++i) k[i] = 0;
  take_exact<kV>(k, mine, a.K, lane, ids);
}

// kWords: logits of 16 bits, and no bias.
template <typename T, int kV, bool kVec, bool kWords>
__global__ void __launch_bounds__(32 * kWarps) route(const __grid_constant__ RouteArgs a, const Lanes lanes) {
  const int lane = threadIdx.x & 31;
  const int token = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int group = lane >> lanes.shift, j = lane & (lanes.per_group - 1);
  Span mine{group * lanes.size + j * lanes.per_lane, 0};
  if (group < a.groups) mine.n = max(0, min(lanes.per_lane, lanes.size - j * lanes.per_lane));
  __shared__ uint32_t shared[kWarps][32 * kV + (kWords ? 64 : 131)];
  uint32_t* rows = shared[threadIdx.x >> 5];
  uint32_t* taken = rows + 32 * kV;  // the words that were taken, in order, and behind them the experts of them
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  if (token >= a.tokens) return;
  const T* x = static_cast<const T*>(a.logits) + (long long)token * a.stride;
  float l[kV];
  if (kVec || (lanes.packs && mine.n == kV)) {  // (kVec: every lane has kV experts)
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
    l[i] = fmaxf(l[i], -INFINITY);  // (NaN is the other of two)
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
  // In units of 2^-24, a softmax' score is off by 4 (expf), 1 (its argument), 2 (quotient and product) and the sum, itself by
  // 4, 3 (the arguments) and kV + 5 roundings at most; a sigmoid's by less than 12 of 1; a key by one of its own
  // more, and its word, once the place is cleared, by less than 2 kV: one way, so that the difference of two
  // words is off by 2 kV and not by twice that. Two keys are compared.
  float off = 0.f;
  constexpr float kPart = 0x1p-23f * (1 + kV);
  if (inexact) {
    off = 0x1p-23f * (a.sigmoid ? 12 : kV + 20) * unit;
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < kV; ++i) s[i] = sigmoid_key(l[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kV; ++i) s[i] *= unit;
    }
    if (!kWords && a.bias) {
      if (lanes.bias_packs && (kVec || mine.n == kV)) {
        struct alignas(4 * kV < 16 ? 4 * kV : 16) Pack {
          float v[kV];
        };
        const Pack p = *reinterpret_cast<const Pack*>(a.bias + mine.first);
#pragma unroll
        for (int i = 0; i < kV; ++i) s[i] = fmaxf(s[i] + p.v[i], -INFINITY);
      } else {
#pragma unroll
        for (int i = 0; i < kV; ++i)
          if (i < mine.n) s[i] = fmaxf(s[i] + a.bias[mine.first + i], -INFINITY);
      }
    }
#pragma unroll
    for (int i = 0; i < kV; ++i) s[i] = l[i] > -INFINITY ? s[i] : -INFINITY;
  }
  bool again = false, groups_too = false, chosen = true;  // what is chosen again with all keys
  if (a.groups > 1) {
    float best = -INFINITY, second = -INFINITY;
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const float key = inexact ? s[i] : l[i];
      second = fmaxf(second, fminf(best, key));
      best = fmaxf(best, key);
    }
    two_of_group(best, second, lanes.per_group);
    float value = a.group_best == 2 && second > -INFINITY ? best + second : best;
    if (group >= a.groups) value = -INFINITY;
    chosen = group_chosen(value, group, a.groups, lanes.per_group, a.top_groups);  // (all lanes take part)
    if (group >= a.groups) chosen = false;
    if (inexact) {  // sums of two keys each
      const float in = warp_min(chosen ? value : INFINITY);
      const float out = warp_max(chosen ? -INFINITY : value);
      const float most = warp_max(fmaxf(best > -INFINITY ? fabsf(best) : 0.f, second > -INFINITY ? fabsf(second) : 0.f));
      const float margin = 2.f * fmaf(kPart, most, off);
      // (keys of which two may leave FP32 in a sum are always looked at again)
      if (in - out < margin || !(most < 0x1p126f)) {
        float keys[kV];  // (their own, so that s stays in registers)
#pragma unroll
        for (int i = 0; i < kV; ++i) keys[i] = s[i];
        const float low = a.group_best == 2 && second > -INFINITY ? second : best;
        bool sure;
        chosen = groups_again<T, kV>(a, x, mine, lanes, lane, top, keys, low - margin, taken, sure);
        again = groups_too = !sure;
      }
    }
  }
  uint32_t k[kV];
#pragma unroll
  for (int i = 0; i < kV; ++i) {
    // without a bias the choice goes by the logits even where the groups' goes by sums of scores
    if (kWords)
      k[i] = half_order(l[i], T{}) << 16 | (0xFFFFu - (mine.first + i));
    else
      k[i] = (order_of(a.bias ? s[i] : l[i]) & ~(uint32_t)(kV - 1)) | (kV - 1 - i);
    if (!kVec && i >= mine.n) k[i] = 0;
  }
  Sorted<kV> sorted(k, rows, lane, chosen);
  int ids[2] = {0, 0};
  float y[2] = {-INFINITY, -INFINITY}, w[2] = {0.f, 0.f};  // logits and weights of the chosen
  if constexpr (kWords) {
    take_words<kV>(sorted, a.K, taken);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < a.K) {
        const uint32_t word = taken[lane + 32 * e];
        ids[e] = 0xFFFF - (word & 0xFFFFu);
        y[e] = half_value(word >> 16, T{});
      }
  } else {
    uint32_t* order = taken + 66;
    const float part = kPart, apart = a.bias ? off : 0.f;
    for (int r = 0; r <= a.K; ++r) take_place<kV>(sorted, mine, lane, r, taken, order);
    __syncwarp();
    bool near = false;  // two neighbours among the K and the one behind them
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (lane + 32 * e < a.K) near |= too_near<kV>(taken[lane + 32 * e], taken[lane + 32 * e + 1], apart, part);
    if (__any_sync(kAll, near)) {
      // as many more as are too near to the K-th
      int n = a.K;
      while (n <= 64 && too_near<kV>(taken[n - 1], taken[n], apart, part)) {
        ++n;
        if (n <= 64) take_place<kV>(sorted, mine, lane, n, taken, order);
        __syncwarp();
      }
      if (n > 64) {
        again = true;
      } else if (!again) {
        int mended[2] = {0, 0};  // (its own, so that ids stay in registers)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (lane + 32 * e < n) mended[e] = order[lane + 32 * e];
        order_again<T>(a, x, mine, lane, top, n, mended);
        ids[0] = mended[0];
        ids[1] = mended[1];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (lane + 32 * e < a.K) ids[e] = order[lane + 32 * e];
    }
  }
  if (again) {
    int mended[2] = {0, 0};
    choose_again<T, kV>(a, x, mine, lanes, lane, top, groups_too, chosen, mended);
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
    float f = total > 0.f ? a.scale / total : 0.f;
    if (isinf(f)) {  // a large scale over a small sum
      w[0] /= total;
      w[1] /= total;
      f = a.scale;
    }
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
cudaError_t run(const RouteArgs& a, Lanes lanes, cudaStream_t s) {
  constexpr int kBytes = sizeof(T) * kV < 16 ? sizeof(T) * kV : 16, kBiasBytes = 4 * kV < 16 ? 4 * kV : 16;
  const bool one = a.groups == 1;  // (else groups begin at places of their own)
  lanes.packs = reinterpret_cast<uintptr_t>(a.logits) % kBytes == 0 && a.stride * (long long)sizeof(T) % kBytes == 0 &&
                (one || lanes.size * sizeof(T) % kBytes == 0);
  lanes.bias_packs = reinterpret_cast<uintptr_t>(a.bias) % kBiasBytes == 0 && (one || lanes.size * 4 % kBiasBytes == 0);
  // experts that fill the lanes get an instance of their own (1024 are rare enough without)
  const bool vec = kV <= 16 && lanes.packs && a.E == 32 * kV;
  constexpr bool kWords = sizeof(T) == 2, kPacks = kV <= 16;
  const auto kernel = kWords && !a.bias ? (vec ? route<T, kV, kPacks, kWords> : route<T, kV, false, kWords>)
                                        : (vec ? route<T, kV, kPacks, false> : route<T, kV, false, false>);
  return launch_dependent(kernel, (a.tokens + kWarps - 1) / kWarps, 32 * kWarps, 0, s, a, lanes);
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
