// wd_logits.cu - penalties, biases, temperature and masks on logits (declared
// in include/wd_step.h).
//
// One pass: a CTA takes a slice of one row's vocabulary. While its first logits are on their way it counts in shared
// memory how often the row's history names each of the slice's tokens (every CTA of a row reads the whole
// history, which is small beside the logits and comes from L2) and notes which bias is each one's. Then it
// streams its logits through, the next ones always on their way. Nothing is written but the result, no counts
// live from call to call, and counting whole numbers gives the same sums in any order.
//
// Measured (BF16 to FP32): 64 rows of 131,072 with histories of 300 to 8192, biases, masks and temperatures 16.9 us, of
// which the logits alone take 6.4 (50 MB, in part from L2), masks 0.5, and the histories 8: their counting and what their
// tokens go through is half of the 540 instructions that a warp has for 16 tokens a lane. One row of 32,768
// 2.8 us. Seven rows of 100,003 with a history of up to 32,768 11.9 us: all CTAs of a row read its history at the same time, so
// that time grows with it (one row of 131,072: 8.6 us with 32,768 tokens so far, 26.7 with 131,072, 195 with 1,048,576).
// Tried: the CTAs of a cluster sharing the history and counting in each other's shared memory (its two barriers cost more
// than the reading: 24.4 against 21.1 us then); one slice after the other in smaller slices (19 to 24); five CTAs to an
// SM for four (no faster); eight accesses to the history at a time (13.0 for the long ones); sums and biases behind one
// pointer that is chosen for each token (19.1).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "wd_device.cuh"
#include "wd_step.cuh"

namespace wd {
namespace {

constexpr int kThreads = 256;
constexpr int kFour = 4;                     // elements of an access
constexpr int kUnit = kThreads * kFour;      // tokens that the threads take with one access each
constexpr int kCtasWanted = 4 * 152;         // for which slices are made smaller

// What shared memory has of a token. Narrow: one word, in its upper half the bias (1 + its index in the row, 0: none), below it
// a bit for the prompt and 15 for the count. Wide, for longer histories or more biases: a word for each half, in two
// arrays. A token of several biases has the half's highest bit, and below it 1 + the place of their sum, or ones if the places
// are all taken. The host knows how many biases there are in all, not those of a row, and goes by that: 109 rows of 131,072 with 300
// biases each take 14.6 us, 110 rows (33,000 biases, wide) 19.0.
constexpr int kNarrowHistory = 32767, kNarrowBiases = 32767;
constexpr int kSums = 512;
template <bool kWide>
struct Layout {
  static constexpr uint32_t kPrompt = kWide ? 1u << 31 : 1u << 15;
  static constexpr int kBiasShift = kWide ? 0 : 16;
  static constexpr uint32_t kSeveral = kWide ? 1u << 31 : 1u << 15;  // above the bias
};

// Four elements as whole words: as elements of 16 bits the compiler takes them apart and puts them together again.
template <typename T>
struct Four {
  uint32_t w[sizeof(T)];
};

template <typename T, bool kVec>
__device__ __forceinline__ Four<T> get_four(const T* p) {
  Four<T> x;
  if constexpr (sizeof(T) == 4) {
    if (kVec) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      x.w[0] = v.x, x.w[1] = v.y, x.w[2] = v.z, x.w[3] = v.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) x.w[k] = reinterpret_cast<const uint32_t*>(p)[k];
    }
  } else {
    if (kVec) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      x.w[0] = v.x, x.w[1] = v.y;
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      x.w[0] = h[0] | (uint32_t)h[1] << 16;
      x.w[1] = h[2] | (uint32_t)h[3] << 16;
    }
  }
  return x;
}

__device__ __forceinline__ void floats_of(const Four<float>& x, float (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = __uint_as_float(x.w[k]);
}
__device__ __forceinline__ void floats_of(const Four<__nv_bfloat16>& x, float (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    f[2 * k] = __uint_as_float(x.w[k] << 16);
    f[2 * k + 1] = __uint_as_float(x.w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void floats_of(const Four<__half>& x, float (&f)[4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x.w[k]));
    f[2 * k] = p.x;
    f[2 * k + 1] = p.y;
  }
}

__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ float get(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float get(const __half* p) { return __half2float(*p); }

template <bool kVec>
__device__ __forceinline__ void put_four(float* p, const float (&f)[4]) {
  if (kVec) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) p[k] = f[k];
  }
}
template <bool kVec, typename U>
__device__ __forceinline__ void put_four(U* p, const float (&f)[4]) {
  if (kVec) {
    uint2 v;
    if constexpr (std::is_same<U, __half>::value) {
      const __half2 lo = __floats2half2_rn(f[0], f[1]), hi = __floats2half2_rn(f[2], f[3]);
      v = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(f[0], f[1]), hi = __floats2bfloat162_rn(f[2], f[3]);
      v = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    *reinterpret_cast<uint2*>(p) = v;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) put(p + k, f[k]);
  }
}

// What a row's tokens go through.
struct Row {
  float repetition, presence, frequency;
  float relief, scale;  // 1 / repetition, 1 / temperature
  const float* bias;    // the values of the row's biases
};

// The sum of row b's biases of a token, in the order in which they stand.
__device__ __forceinline__ float sum_of_biases(const LogitsArgs& a, int b, int token) {
  float sum = 0.f;
#pragma unroll 1
  for (int i = a.bias_start[b], to = a.bias_start[b + 1]; i < to; ++i)
    if (a.bias_ids[i] == token) sum += a.bias_values[i];
  return sum;
}

// The same for a token of each lane of a warp. A lane reads every 32nd bias and hands it to the others: for 300 biases that
// takes 4 us where lanes that read them all took 11.
__device__ __forceinline__ float sums_of_biases(const LogitsArgs& a, int from, int to, int token) {
  float sum = 0.f;
  int id = -1;
  float value = 0.f;
  const unsigned n = to - from;  // (places are counted from `from`, unsigned: those behind the last bias may pass 2^31)
  const auto ask = [&](unsigned i) {
    id = i < n ? a.bias_ids[from + (int)i] : -1;
    value = i < n ? a.bias_values[from + (int)i] : 0.f;
  };
  ask(threadIdx.x & 31);
#pragma unroll 1
  for (unsigned at = 0; at < n; at += 32) {
    const int ids = id;
    const float values = value;
    if (n - at > 32) ask(at + 32 + (threadIdx.x & 31));
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      const int other = __shfl_sync(~0u, ids, k);
      const float its = __shfl_sync(~0u, values, k);
      sum = other == token ? sum + its : sum;
    }
  }
  return sum;
}

// The logit of a token with its prompt bit and count, and its bias unless it has several.
template <bool kWide>
__device__ __forceinline__ float penalised(const Row& r, float l, uint32_t count, uint32_t named) {
  if (!kWide) {
    named = count >> 16;
    count &= 0xFFFFu;
  }
  const float turned = l * (l > 0.f ? r.relief : r.repetition);
  const uint32_t n = count & (Layout<kWide>::kPrompt - 1);
  const float less = n ? fmaf((float)n, r.frequency, r.presence) : 0.f;
  l = count ? turned - less : l;
  return named ? l + r.bias[named - 1] : l;
}

// Tokens `first` .. `first` + 3 of a history of `columns`; -1 behind its end.
__device__ __forceinline__ int4 four_tokens(const int32_t* tokens, bool aligned, int first, int columns) {
  int4 v = make_int4(-1, -1, -1, -1);
  if (aligned && first + 4 <= columns) {
    v = *reinterpret_cast<const int4*>(tokens + first);
  } else {
    if (first < columns) v.x = tokens[first];
    if (first + 1 < columns) v.y = tokens[first + 1];
    if (first + 2 < columns) v.z = tokens[first + 2];
    if (first + 3 < columns) v.w = tokens[first + 3];
  }
  return v;
}

// Marks a token as the prompt's, or counts it, if it is one of the n of the slice; `words`: the shared address of the first
// one's. Without a branch: most accesses of a warp have a token for most slices.
__device__ __forceinline__ void mark(uint32_t words, uint32_t at, int n, uint32_t bit) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lo.u32 p, %1, %2;\n\t@p red.shared.or.b32 [%0], %3;\n\t}"
               :: "r"(words + 4 * at), "r"(at), "r"(n), "r"(bit) : "memory");
}
__device__ __forceinline__ void add(uint32_t words, uint32_t at, int n) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lo.u32 p, %1, %2;\n\t@p red.shared.add.u32 [%0], 1;\n\t}"
               :: "r"(words + 4 * at), "r"(at), "r"(n) : "memory");
}

// Slice blockIdx.x of row blockIdx.y: `chunks` times kPer fours of tokens to a thread. kVec: input and output of a row reach
// the alignment of four elements at the same token; slices begin there. The first one has what is
// before that, too, and the one of the last four what is behind it.
template <typename T, typename U, int kPer, bool kVec, bool kWide>
__global__ void __launch_bounds__(kThreads, 4) adjust_logits(const LogitsArgs a, int chunks) {
  constexpr int kChunk = kPer * kUnit;
  constexpr int kBatch = 4;  // accesses of a thread to the history that are on their way at a time
  constexpr uint32_t kSeveral = Layout<kWide>::kSeveral << Layout<kWide>::kBiasShift;
  static_assert(kSeveral == 1u << 31, "the highest bit of its word");
  constexpr uint32_t kIndex = kSeveral - (1u << Layout<kWide>::kBiasShift);  // the bits of an index
  extern __shared__ uint4 shared[];
  __shared__ float sums[kSums];  // of the slice's tokens of several biases
  __shared__ int places_taken;
  const int slice = chunks * kChunk, places = slice + 2 * kFour;  // place 4 of an array is the slice's first four
  const int b = blockIdx.y, part = blockIdx.x;
  const T* in = static_cast<const T*>(a.logits) + b * a.stride;
  U* out = static_cast<U*>(a.out) + b * a.out_stride;
  const int lead =
      kVec ? min(a.V, (int)((kFour - (reinterpret_cast<uintptr_t>(in) / sizeof(T)) % kFour) % kFour)) : 0;
  const int last = lead + (a.V - lead) / kFour * kFour;  // behind the row's last four
  const int begin = lead + part * slice, end = min(begin + slice, last);
  const int before = part == 0 ? lead : 0;  // loose tokens that are this slice's
  const int behind = begin <= last && last < begin + slice ? a.V - last : 0;
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  // A chunk's logits of this thread, and the words of the mask that hold the bits of each access (nothing is done
  // with them yet: a use waits for what it needs, and the loads behind it wait, too).
  struct Chunk {
    Four<T> x[kPer];
    uint32_t word[kPer], next[kPer];
  };
  const int32_t* mask = a.mask ? a.mask + b * a.mask_stride : nullptr;
  const bool astride = lead % kFour;  // some fours' bits are in two words
  const int shift = (begin + kFour * threadIdx.x) & 31;  // kUnit tokens are whole words: the same for all accesses
  const auto fetch = [&](int at) {  // the chunk that begins at token `at`
    Chunk c;
    const int mine = at + kFour * threadIdx.x;
    if (end - at >= kChunk) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) c.x[j] = get_four<T, kVec>(in + mine + j * kUnit);
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (mine + j * kUnit < end) c.x[j] = get_four<T, kVec>(in + mine + j * kUnit);
    }
    if (mask) {
      const int32_t* words = mask + (mine >> 5);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (mine + j * kUnit < end) c.word[j] = words[j * (kUnit / 32)];
      if (astride) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (mine + j * kUnit < end && shift > 32 - kFour) c.next[j] = words[j * (kUnit / 32) + 1];
      }
    }
    return c;
  };
  Chunk next = fetch(begin);
  Row r;
  r.repetition = a.repetition ? a.repetition[b] : 1.f;
  r.presence = a.presence ? a.presence[b] : 0.f;
  r.frequency = a.frequency ? a.frequency[b] : 0.f;
  const float t = a.temperature ? a.temperature[b] : 1.f;
  int slot = -1, bias_from = 0, bias_to = 0;
  if (a.history.tokens) slot = a.history.seqs ? a.history.seqs[b] : b;
  if (a.bias_start) {
    bias_from = a.bias_start[b];
    bias_to = a.bias_start[b + 1];
    if (bias_from < 0 || bias_to > a.biases || bias_to < bias_from) bias_from = bias_to = 0;
  }
  const unsigned listed = bias_to - bias_from;  // the row's biases (bias_from + a place behind them may pass 2^31)
  r.bias = a.bias_values + bias_from;
  // the row's history, if it has one and its penalties are any
  const bool penalties = r.repetition != 1.f || r.presence != 0.f || r.frequency != 0.f;
  const bool counts = penalties && (unsigned)slot < (unsigned)a.history.slots, biases = listed > 0;
  if (counts || biases) {
    const int from = begin - before, n = max(0, end - begin) + before + behind;  // the slice's tokens
    const uint32_t words = (uint32_t)__cvta_generic_to_shared(shared) + 4 * (kFour - before);  // of token `from`
    int4 tokens[kBatch];
    const int32_t* history = nullptr;
    int length = 0, prompt = 0;
    const int columns = a.history.columns;
    const auto ask = [&](int base) {
      const bool aligned = reinterpret_cast<uintptr_t>(history) % 16 == 0;
      if (aligned && base + 4 * kBatch * kThreads <= columns) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          tokens[j] = reinterpret_cast<const int4*>(history + base)[threadIdx.x + j * kThreads];
      } else {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          tokens[j] = four_tokens(history, aligned, base + 4 * (threadIdx.x + j * kThreads), columns);
      }
    };
    if (counts) {
      history = a.history.tokens + slot * a.history.stride;
      ask(0);  // beside the lengths
      length = max(0, min(a.history.lengths[slot], columns));
      prompt = a.history.prompt_lengths ? max(0, min(a.history.prompt_lengths[slot], length)) : 0;
    }
    int id = -1;  // this thread's first bias
    if (threadIdx.x < listed) id = a.bias_ids[bias_from + (int)threadIdx.x];
    const int fours = places / kFour * (kWide ? 2 : 1);
    for (int i = threadIdx.x; i < fours; i += kThreads) shared[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) places_taken = 0;
    __syncthreads();
    uint32_t* named = reinterpret_cast<uint32_t*>(shared) + kFour - before + (kWide ? places : 0);
    const auto add_up = [&] {  // the biases of the tokens that have several, all of which are noted
      const int several = min(places_taken, kSums);
      if (!several) return;
      for (int first = threadIdx.x & ~31; first < several; first += kThreads) {  // whole warps
        const int i = first + (threadIdx.x & 31);
        const int token = i < several ? __float_as_int(sums[i]) : -1;
        const float sum = sums_of_biases(a, bias_from, bias_to, token);
        if (i < several) {
          named[token - from] = kSeveral | (uint32_t)(i + 1) << Layout<kWide>::kBiasShift;
          sums[i] = sum;
        }
      }
      __syncthreads();
    };
    if (biases) {
      for (unsigned i = threadIdx.x;;) {
        const uint32_t at = (uint32_t)id - (uint32_t)from;
        if (id >= 0 && at < (uint32_t)n && atomicMax(&named[at], (i + 1) << Layout<kWide>::kBiasShift) &&
            !(atomicOr(&named[at], kSeveral) & kSeveral)) {  // the second one of its token
          const int place = atomicAdd(&places_taken, 1);
          if (place < kSums) sums[place] = __int_as_float(id);
          else atomicOr(&named[at], kIndex);
        }
        i += kThreads;
        if (i >= listed) break;
        id = a.bias_ids[bias_from + (int)i];
      }
      if (!kWide) {  // before the lower halves change
        __syncthreads();
        add_up();
      }
    }
    for (int base = 0; base < length;) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = base + 4 * (threadIdx.x + j * kThreads);
        if (i >= length) break;
        const uint32_t at[4] = {(uint32_t)tokens[j].x - (uint32_t)from, (uint32_t)tokens[j].y - (uint32_t)from,
                                (uint32_t)tokens[j].z - (uint32_t)from, (uint32_t)tokens[j].w - (uint32_t)from};
        if (i + 4 <= prompt) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mark(words, at[k], n, Layout<kWide>::kPrompt);
        } else if (i >= prompt && i + 4 <= length) {
#pragma unroll
          for (int k = 0; k < 4; ++k) add(words, at[k], n);
        } else {  // what holds the end of one of the two
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (i + k < prompt) mark(words, at[k], n, Layout<kWide>::kPrompt);
            else if (i + k < length) add(words, at[k], n);
          }
        }
      }
      base += 4 * kBatch * kThreads;
      if (base < length) ask(base);
    }
    __syncthreads();
    if (kWide && biases) add_up();
  }
  r.scale = t > 0.f ? 1.f / t : 1.f;
  r.relief = 1.f / r.repetition;
  // A slice with tokens of several biases is taken one by one: what their sums ask of registers would cost
  // the others (64 x 131,072 FP32 13.3 against 12.5 us). Rows with such tokens in every slice pay for it (64 x 131,072 BF16 with 150
  // tokens named twice each 35.8 us, with the sums in the main loop 20; with 300 distinct ones 9.6).
  if (biases && places_taken) {
    const int from = begin - before, n = max(0, end - begin) + before + behind;
#pragma unroll 1
    for (int v = from + threadIdx.x; v < from + n; v += kThreads) {
      const uint32_t* word = reinterpret_cast<const uint32_t*>(shared) + kFour + v - begin;
      const uint32_t named = word[kWide ? places : 0], place = named & kIndex;
      float l = get(in + v);
      if (named & kSeveral)
        l = penalised<kWide>(r, l, kWide ? word[0] : word[0] & 0xFFFFu, 0u) +
            (place == kIndex ? sum_of_biases(a, b, v) : sums[(place >> Layout<kWide>::kBiasShift) - 1]);
      else
        l = penalised<kWide>(r, l, word[0], named);
      put(&out[v], !mask || (mask[v >> 5] >> (v & 31) & 1) ? l * r.scale : -INFINITY);
    }
    return;
  }
  const uint4* noted = shared + 1 + threadIdx.x;
  for (int at = begin; at < end; at += kChunk, noted += kPer * kThreads) {
    const Chunk c = next;
    if (at + kChunk < end) next = fetch(at + kChunk);
    const int mine = at + kFour * threadIdx.x;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (mine + j * kUnit >= end) break;
      float l[kFour];
      floats_of(c.x[j], l);
      if (counts || biases) {
        const uint4 w = noted[j * kThreads];
        uint4 e = make_uint4(0, 0, 0, 0);
        if (kWide) e = noted[places / kFour + j * kThreads];
        if (w.x | w.y | w.z | w.w | e.x | e.y | e.z | e.w) {
          l[0] = penalised<kWide>(r, l[0], w.x, e.x);
          l[1] = penalised<kWide>(r, l[1], w.y, e.y);
          l[2] = penalised<kWide>(r, l[2], w.z, e.z);
          l[3] = penalised<kWide>(r, l[3], w.w, e.w);
        }
      }
#pragma unroll
      for (int k = 0; k < kFour; ++k) l[k] *= r.scale;
      if (mask) {
        const uint32_t allowed = astride ? __funnelshift_r(c.word[j], c.next[j], shift) : c.word[j] >> shift;
#pragma unroll
        for (int k = 0; k < kFour; ++k) l[k] = allowed & (1u << k) ? l[k] : -INFINITY;
      }
      put_four<kVec>(out + mine + j * kUnit, l);
    }
  }
  // the loose tokens, at most three before the first four and three behind the last
  if ((int)threadIdx.x < before + behind) {
    const int v = (int)threadIdx.x < before ? threadIdx.x : last + threadIdx.x - before;
    const uint32_t* word = reinterpret_cast<const uint32_t*>(shared) + kFour + v - begin;
    float l = get(in + v);
    if (counts || biases) l = penalised<kWide>(r, l, word[0], kWide ? word[places] : 0u);
    put(&out[v], !mask || (mask[v >> 5] >> (v & 31) & 1) ? l * r.scale : -INFINITY);
  }
}

template <typename T, typename U, int kPer>
cudaError_t run_slices(const LogitsArgs& a, int chunks, cudaStream_t s) {
  const auto place = [](const void* p, size_t size) { return (long long)(reinterpret_cast<uintptr_t>(p) / size % kFour); };
  const auto same = [](long long x, long long y) { return ((x - y) % kFour) == 0; };
  const bool vec = same(place(a.logits, sizeof(T)), place(a.out, sizeof(U))) && (a.B == 1 || same(a.stride, a.out_stride));
  const bool noted = a.history.tokens || a.bias_start;
  const bool wide = noted && (a.history.columns > kNarrowHistory || a.biases > kNarrowBiases);
  const int slice = chunks * kPer * kUnit;
  const auto kernel = vec ? (wide ? adjust_logits<T, U, kPer, true, true> : adjust_logits<T, U, kPer, true, false>)
                          : (wide ? adjust_logits<T, U, kPer, false, true> : adjust_logits<T, U, kPer, false, false>);
  const int bytes = noted ? 4 * (slice + 2 * kFour) * (wide ? 2 : 1) : 0;
  if (bytes > 48 * 1024) {
    const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), bytes);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(kernel, dim3((unsigned)((a.V + slice - 1) / slice), (unsigned)a.B), kThreads, bytes, s, a, chunks);
}

template <typename T, typename U>
cudaError_t run(const LogitsArgs& a, cudaStream_t s) {
  // Large slices where the rows fill the GPU (each reads the history once more; 64 x 131,072 in slices of 4096 took 27.4
  // us where those of 8192 took 23.6), smaller ones where they do not.
  const auto enough = [&](int slice) { return (long long)a.B * ((a.V + slice - 1) / slice) >= kCtasWanted; };
  if (enough(8 * kUnit)) return run_slices<T, U, 4>(a, 2, s);
  if (enough(4 * kUnit)) return run_slices<T, U, 4>(a, 1, s);
  if (enough(2 * kUnit)) return run_slices<T, U, 1>(a, 2, s);
  return run_slices<T, U, 1>(a, 1, s);
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
