// wd_kv_append_rotated.cu - queries and keys rotated by their positions; keys and
// values quantised to MXFP4 into the pages (declared in include/wd_kv.h).
//
// A pair (x1, x2) of a head's channels becomes (x1 c - x2 s, x2 c + x1 s), c and s from the row of the
// table that the token's position names. Products and sums are rounded to FP32 one by one, not
// contracted: the codes of a key are then the same whatever kernel computes them, and
// its quantising sees the FP32 values (they are not rounded to the key's type on the way).
//
// One launch, two kinds of CTA. The first ones take keys and values, 8 channels of one token, head and side
// to a thread as in wd_kv_append.cu; a key's thread reads its partner's channels too, half a rotation away.
// The others take queries, which are most of the bytes: a thread has the 8 + 8 channels
// of 8 pairs (16 neighbours where pairs are neighbours), so that each cosine and sine is read once for both.
// The table's rows of a CTA's tokens stand in shared memory, and a thread's next token is on its way
// while it turns one.
//
// To read and write: q in and out, k and v in, 4.25 bits a channel of them out, the table's rows. Measured: eight prompts,
// 15,841 tokens of 32 query and 4 key heads of 128 in BF16 with the values back, 335 MB, 58.9 us, 5.7 TB/s, 0.84 of the copy
// rate; one token of 32 sequences 3.0 us. Tried: the table's rows from L1 for each token (70.9), 3, 4 and 6 CTAs to
// an SM for 5 (67.5, 61.7, 59.8), 8 and 32 tokens to a CTA (61.0, 59.1), first all keys and then all queries (63.9).
#include "wd_device.cuh"
#include "wd_kv_quant.cuh"

namespace wd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a CTA

// Eight channels as whole words: as elements of 16 bits the compiler takes them apart and puts them together again.
template <typename T>
struct Words {
  uint32_t w[2 * sizeof(T)];
};

template <typename T, bool kVec>
__device__ __forceinline__ Words<T> fetch(const T* src) {
  Words<T> x;
  if (kVec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(src)[i];
      x.w[4 * i] = v.x, x.w[4 * i + 1] = v.y, x.w[4 * i + 2] = v.z, x.w[4 * i + 3] = v.w;
    }
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x.w[k] = reinterpret_cast<const uint32_t*>(src)[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x.w[k] = reinterpret_cast<const uint16_t*>(src)[2 * k] | (uint32_t)reinterpret_cast<const uint16_t*>(src)[2 * k + 1] << 16;
  }
  return x;
}

template <typename T, bool kVec>
__device__ __forceinline__ void put(T* dst, const Words<T>& x) {
  if (kVec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      reinterpret_cast<uint4*>(dst)[i] = make_uint4(x.w[4 * i], x.w[4 * i + 1], x.w[4 * i + 2], x.w[4 * i + 3]);
  } else if (sizeof(T) == 4) {
#pragma unroll
    for (int k = 0; k < 8; ++k) reinterpret_cast<uint32_t*>(dst)[k] = x.w[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      reinterpret_cast<uint16_t*>(dst)[2 * k] = (uint16_t)x.w[k];
      reinterpret_cast<uint16_t*>(dst)[2 * k + 1] = (uint16_t)(x.w[k] >> 16);
    }
  }
}

__device__ __forceinline__ void floats_of(const Words<float>& x, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(x.w[k]);
}
__device__ __forceinline__ void floats_of(const Words<__nv_bfloat16>& x, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f[2 * k] = __uint_as_float(x.w[k] << 16);
    f[2 * k + 1] = __uint_as_float(x.w[k] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void floats_of(const Words<__half>& x, float (&f)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&x.w[k]));
    f[2 * k] = p.x;
    f[2 * k + 1] = p.y;
  }
}
__device__ __forceinline__ void words_of(const float (&f)[8], Words<float>& x) {
#pragma unroll
  for (int k = 0; k < 8; ++k) x.w[k] = __float_as_uint(f[k]);
}
__device__ __forceinline__ void words_of(const float (&f)[8], Words<__nv_bfloat16>& x) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
    x.w[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
}
__device__ __forceinline__ void words_of(const float (&f)[8], Words<__half>& x) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __half2 p = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
    x.w[k] = *reinterpret_cast<const uint32_t*>(&p);
  }
}

// A pair's first and second channel: products and sums rounded one by one, never contracted (as pairs in packed
// instructions, mul.rn.f32x2 and add.rn.f32x2, they are).
__device__ __forceinline__ void turn(float& x1, float& x2, float c, float s) {
  const float a = x1, b = x2;
  x1 = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  x2 = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Four neighbouring pairs, with their cosines and sines.
__device__ __forceinline__ void turn_neighbours(float (&f)[8], const float4 c, const float4 s) {
  turn(f[0], f[1], c.x, s.x);
  turn(f[2], f[3], c.y, s.y);
  turn(f[4], f[5], c.z, s.z);
  turn(f[6], f[7], c.w, s.w);
}

// Four pairs that are a run of first channels at x1 and one of second channels at x2.
__device__ __forceinline__ void turn_runs(float* x1, float* x2, const float4 c, const float4 s) {
  turn(x1[0], x2[0], c.x, s.x);
  turn(x1[1], x2[1], c.y, s.y);
  turn(x1[2], x2[2], c.z, s.z);
  turn(x1[3], x2[3], c.w, s.w);
}

// The token's place, none if the table has no row for its position.
template <int D>
__device__ __forceinline__ Place rotated_place(const KvRotateArgs& a, int token) {
  Place p = find_place<D>(a.kv.cache, a.kv.batch, a.kv.layer, token);
  if (p.pos >= a.positions) {
    atomicOr(a.kv.cache.flag, WD_KV_FLAG_BAD_INDEX);
    p.group = nullptr;
    p.pos = -1;
  }
  return p;
}

// Channels 8e .. 8e + 7 of one token, head and side (v: values, else keys): the largest magnitude of
// their block from the row's `lanes` (`top`: the bits of these eight's), codes and scales to the token's place,
// and what they stand for to `out` if `back`.
template <typename T, int D, bool kVec>
__device__ __forceinline__ void store_eight(const float (&f)[8], uint32_t top, unsigned lanes, int e, bool v, const Place* at,
                                            long long head_at, bool back, T* out) {
  using G = KvGroup<D>;
  const int block = e >> 2, t8 = e & 3;
  top = max(top, __shfl_xor_sync(lanes, top, 1));
  top = max(top, __shfl_xor_sync(lanes, top, 2));
  const bool bad = top >= 0x7F800000u;
  // floor(log2(top)) - 2, at least -127; a subnormal's floor(log2) is below -126
  const int ex = (int)(top >> 23);
  const int exp2 = top == 0 || bad ? 0 : (ex <= 2 ? -127 : ex - 129);
  const float inv = power_of_two(-exp2);
  float y[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] = f[k] * inv;
  const uint32_t word = bad ? 0u : e2m1x8_of(y);
  // the scales of the row's blocks side by side
  uint32_t scales = (bad ? 255u : (uint32_t)(exp2 + 127)) << (8 * (block & 3));
  scales |= __shfl_xor_sync(lanes, scales, 4);
  if (G::kBlocks >= 4) scales |= __shfl_xor_sync(lanes, scales, 8);
  // V: blocks c and c ^ 1 swap halves, so that the even one has channels 4g .. of both for
  // g = 2 t8 and the odd one for g = 2 t8 + 1
  const uint32_t other = __shfl_xor_sync(lanes, word, 4);
  const Place p = *at;
  if (p.group) {
    uint8_t* g = p.group + head_at;
    uint8_t* scale_to = g + (v ? G::kVScale : G::kKScale) + p.t * G::kBlocks + block;
    if (!v) {
      *reinterpret_cast<uint32_t*>(g + G::k_word(p.t, block, t8)) = word;
    } else {
      const uint32_t both = block & 1 ? __byte_perm(other, word, 0x7632)
                                      : __byte_perm(word, other, 0x5410);
      *reinterpret_cast<uint32_t*>(g + G::v_half(p.t, block & ~1, 2 * t8 + (block & 1))) = both;
    }
    if ((e & 15) == 0) {
      if (G::kBlocks == 2)
        *reinterpret_cast<uint16_t*>(scale_to) = (uint16_t)scales;
      else
        *reinterpret_cast<uint32_t*>(scale_to) = scales;
    }
    if (back) {
      const float unit = bad ? __uint_as_float(0x7FC00000u) : power_of_two(exp2);
      e2m1x8_values(word, y);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] *= unit;
      Words<T> z;
      words_of(y, z);
      put<T, kVec>(out, z);
    }
  }
}

// The places of tokens [base, base + n), and the rows of the table at their positions: of eight pairs e, cosines 0 to 3
// and 4 to 7 and sines alike are float4 e of the row's first, second, third and fourth quarter, so that a warp
// reads each without bank conflicts.
template <int D>
__device__ __forceinline__ void stage(const KvRotateArgs& a, int base, int n, int rot, Place* place, float4* turns) {
  if ((int)threadIdx.x < n) place[threadIdx.x] = rotated_place<D>(a, base + threadIdx.x);
  __syncthreads();
  const int eights = rot / 16, fours = rot / 4;
  for (int i = threadIdx.x; i < n * fours; i += kThreads) {
    const int token = i / fours, f = i - token * fours;
    const int pos = place[token].pos;
    if (pos < 0) continue;
    const int quarter = (f & 1) + (f >= 2 * eights ? 2 : 0), e = (f >= 2 * eights ? f - 2 * eights : f) >> 1;
    turns[token * fours + quarter * eights + e] = reinterpret_cast<const float4*>(a.cos_sin + (long long)pos * rot)[f];
  }
  __syncthreads();
}

// kWhole: all channels are turned, in runs (rot = D, not paired); else as the arguments say.

// Queries of tokens [base, base + n).
template <typename T, int D, bool kVec, bool kWhole>
__device__ __forceinline__ void queries(const KvRotateArgs& a, int base, int n, Place* place, float4* turns) {
  constexpr int kPerRow = D / 16;  // threads to a token and head
  constexpr int kRowsOfThreads = kThreads / kPerRow;
  const int rot = kWhole ? D : a.rot;
  const bool paired = !kWhole && a.paired;
  const int half = rot / 2, eights = rot / 16, fours = rot / 4;
  const int e = threadIdx.x % kPerRow, row0 = threadIdx.x / kPerRow;
  const bool turned = kWhole || 16 * e < rot;  // else 16 channels that stay as they are
  // this thread's two runs of 8 channels
  const int c0 = turned && !paired ? 8 * e : 16 * e;
  const int apart = turned && !paired ? half : 8;
  const int at_once = max(1, kRowsOfThreads / a.q_heads);  // tokens
  const int token0 = row0 / a.q_heads;                     // (0 if there are more heads than threads for them)
  const long long src_step = at_once * a.q_token, dst_step = (long long)at_once * a.q_heads * D;
  bool staged = false;
  for (int h = row0 - token0 * a.q_heads; h < a.q_heads || !staged; h += kRowsOfThreads) {
    const bool here = h < a.q_heads && token0 < at_once;
    const T* src = static_cast<const T*>(a.q) + (base + token0) * a.q_token + h * a.q_head + c0;
    Words<T> next0, next1;
    if (here && token0 < n) {  // on their way while the places are found
      next0 = fetch<T, kVec>(src);
      next1 = fetch<T, kVec>(src + apart);
    }
    if (!staged) {
      stage<D>(a, base, n, rot, place, turns);
      staged = true;
    }
    if (!here) continue;
    T* dst = static_cast<T*>(a.q_out) + ((long long)(base + token0) * a.q_heads + h) * D + c0;
    const float4* row = turns + token0 * fours + e;
    for (int token = token0; token < n; token += at_once) {
      const bool write = place[token].pos >= 0;
      float f[8], g[8];
      if (turned) {
        floats_of(next0, f);
        floats_of(next1, g);
      } else if (write) {
        put<T, kVec>(dst, next0);
        put<T, kVec>(dst + apart, next1);
      }
      src += src_step;
      if (token + at_once < n) {
        next0 = fetch<T, kVec>(src);
        next1 = fetch<T, kVec>(src + apart);
      }
      if (turned && write) {
        const float4 ca = row[0], cb = row[eights], sa = row[2 * eights], sb = row[3 * eights];
        if (paired) {
          turn_neighbours(f, ca, sa);
          turn_neighbours(g, cb, sb);
        } else {
          turn_runs(f, g, ca, sa);
          turn_runs(f + 4, g + 4, cb, sb);
        }
        Words<T> x;
        words_of(f, x);
        put<T, kVec>(dst, x);
        words_of(g, x);
        put<T, kVec>(dst + apart, x);
      }
      dst += dst_step;
      row += at_once * fours;
    }
  }
}

// Keys and values of tokens [base, base + n).
template <typename T, int D, bool kVec, bool kWhole>
__device__ __forceinline__ void keys_and_values(const KvRotateArgs& a, int base, int n, Place* place, float4* turns) {
  constexpr int kPerRow = D / 8;  // threads to a token, head and side
  constexpr int kRowsOfThreads = kThreads / kPerRow;
  const KvView& c = a.kv.cache;
  const int rows = 2 * c.kv_heads;  // of a token: the heads' K, then the heads' V
  const int rot = kWhole ? D : a.rot;
  const bool paired = !kWhole && a.paired;
  const int half = rot / 2, eights = rot / 16, fours = rot / 4;
  const int e = threadIdx.x % kPerRow;  // channels 8e .. 8e + 7
  const int row0 = threadIdx.x / kPerRow;
  const int at_once = max(1, kRowsOfThreads / rows);  // tokens
  const int token0 = row0 / rows;
  // a row's lanes are all here, or none: kPerRow divides the warp or is a warp
  const unsigned lanes = kPerRow >= 32 ? 0xFFFFFFFFu
                                       : ((1u << (kPerRow % 32)) - 1u) << (threadIdx.x & 31 & ~(kPerRow - 1));
  const bool lower = 8 * e < half;  // of the two halves that a rotation pairs
  const uint32_t sign = lower ? 0x80000000u : 0u;
  bool staged = false;
  for (int hs = row0 - token0 * rows; hs < rows || !staged; hs += kRowsOfThreads) {
    const bool here = hs < rows && token0 < at_once;
    const bool v = hs >= c.kv_heads;
    const int head = v ? hs - c.kv_heads : hs;
    const bool turned = !v && (kWhole || 8 * e < rot), partnered = turned && !paired;
    const long long stride = v ? a.kv.v_token : a.kv.k_token;
    const T* src = static_cast<const T*>(v ? a.kv.v : a.kv.k) + (base + token0) * stride +
                   head * (v ? a.kv.v_head : a.kv.k_head) + 8 * e;
    const int partner = lower ? half : -half;
    Words<T> next, next_partner;
    if (here && token0 < n) {  // on their way while the places are found
      next = fetch<T, kVec>(src);
      if (partnered) next_partner = fetch<T, kVec>(src + partner);
    }
    if (!staged) {
      stage<D>(a, base, n, rot, place, turns);
      staged = true;
    }
    if (!here) continue;
    const long long head_at = (long long)head * c.head_bytes;
    T* out = static_cast<T*>(v ? a.kv.v_out : a.kv.k_out) + ((long long)(base + token0) * c.kv_heads + head) * D + 8 * e;
    for (int token = token0; token < n; token += at_once) {
      float f[8], g[8];
      floats_of(next, f);
      if (partnered) floats_of(next_partner, g);
      src += at_once * stride;
      if (token + at_once < n) {
        next = fetch<T, kVec>(src);
        if (partnered) next_partner = fetch<T, kVec>(src + partner);
      }
      if (turned && place[token].pos >= 0) {
        const float4* row = turns + token * fours;
        if (paired) {
          row += (e & 1) * eights + (e >> 1);
          turn_neighbours(f, row[0], row[2 * eights]);
        } else {
          row += lower ? e : e - eights;
          const float4 ca = row[0], cb = row[eights], sa = row[2 * eights], sb = row[3 * eights];
          const float co[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
          const float si[8] = {sa.x, sa.y, sa.z, sa.w, sb.x, sb.y, sb.z, sb.w};
#pragma unroll
          for (int k = 0; k < 8; ++k)  // x1 c - x2 s, or x2 c + x1 s
            f[k] = __fadd_rn(__fmul_rn(f[k], co[k]),
                             __fmul_rn(g[k], __uint_as_float(__float_as_uint(si[k]) ^ sign)));
        }
      }
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(f[k]) & 0x7FFFFFFFu);
      store_eight<T, D, kVec>(f, top, lanes, e, v, &place[token], head_at, a.kv.k_out != nullptr, out);
      out += (long long)at_once * c.kv_heads * D;
    }
  }
}

// CTAs of kv_tokens tokens' keys and values and of q_tokens' queries by turns (the first have more to compute, the others
// more to move), and the rest of either behind them.
template <typename T, int D, bool kVec, bool kWhole>
__global__ void __launch_bounds__(kThreads, 5)
    kv_append_rotated(const KvRotateArgs a, int kv_ctas, int kv_tokens, int q_ctas, int q_tokens) {
  __shared__ Place place[kMaxTokens];
  extern __shared__ float4 turns[];
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  const int i = blockIdx.x, both = 2 * min(kv_ctas, q_ctas);
  if (i < both ? i % 2 == 0 : kv_ctas > q_ctas) {
    const int base = (i < both ? i / 2 : i - both / 2) * kv_tokens;
    keys_and_values<T, D, kVec, kWhole>(a, base, min(kv_tokens, a.kv.batch.tokens - base), place, turns);
  } else {
    const int base = (i < both ? i / 2 : i - both / 2) * q_tokens;
    queries<T, D, kVec, kWhole>(a, base, min(q_tokens, a.kv.batch.tokens - base), place, turns);
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Tokens of a CTA: few are spread over the SMs, a pass of the threads to each CTA at least; many get kMaxTokens.
int tokens_of(int tokens, int rows, int per_row) {
  const int one_pass = (kThreads / per_row + rows - 1) / rows;
  int n = (tokens + 8 * kKvSms - 1) / (8 * kKvSms);
  n = n < one_pass ? one_pass : n;
  return n > kMaxTokens ? kMaxTokens : n;
}

template <typename T, int D>
cudaError_t run(const KvRotateArgs& a, cudaStream_t s) {
  const KvAppendArgs& kv = a.kv;
  const int tokens = kv.batch.tokens;
  const int kv_tokens = tokens_of(tokens, 2 * kv.cache.kv_heads, D / 8);
  const int kv_ctas = (tokens + kv_tokens - 1) / kv_tokens;
  const int q_tokens = a.q ? tokens_of(tokens, a.q_heads, D / 16) : 1;
  const int q_ctas = a.q ? (tokens + q_tokens - 1) / q_tokens : 0;
  constexpr long long u = 16 / sizeof(T);  // elements to 16 bytes
  const bool vec = aligned16(kv.k) && aligned16(kv.v) && aligned16(kv.k_out) && aligned16(kv.v_out) && aligned16(a.q) &&
                   aligned16(a.q_out) && kv.k_token % u == 0 && kv.k_head % u == 0 && kv.v_token % u == 0 &&
                   kv.v_head % u == 0 && a.q_token % u == 0 && a.q_head % u == 0;
  const auto kernel = !vec ? kv_append_rotated<T, D, false, false>
                      : a.rot == D && !a.paired ? kv_append_rotated<T, D, true, true>
                                                : kv_append_rotated<T, D, true, false>;
  return launch_dependent(kernel, kv_ctas + q_ctas, kThreads, 4 * a.rot * (q_tokens > kv_tokens ? q_tokens : kv_tokens), s,
                          a, kv_ctas, kv_tokens, q_ctas, q_tokens);
}

template <typename T>
cudaError_t run_dim(const KvRotateArgs& a, cudaStream_t s) {
  switch (a.kv.cache.head_dim) {
    case 64: return run<T, 64>(a, s);
    case 128: return run<T, 128>(a, s);
    default: return run<T, 256>(a, s);
  }
}

}  // namespace

cudaError_t launch_kv_append_rotated(const KvRotateArgs& a, cudaStream_t s) {
  switch (a.kv.dtype) {
    case WD_KV_BF16: return run_dim<__nv_bfloat16>(a, s);
    case WD_KV_FP16: return run_dim<__half>(a, s);
    default: return run_dim<float>(a, s);
  }
}

}  // namespace wd
