// wd_kv_append.cu - quantise new keys and values to MXFP4 and write them into
// the pages of their sequences (declared in include/wd_kv.h).
//
// A thread takes 8 consecutive channels of one token, head and side (K or V):
// one 16-byte load of 16-bit inputs.  Four neighbouring lanes hold a block of 32
// channels, so its largest magnitude is two shuffles away.  The 8 codes are one
// 32-bit word of the K layout; in the V layout they are two 16-bit halves in
// different places, and a third shuffle pairs them with those of the neighbouring block to
// one 32-bit word per lane.
//
// To read and write: 2 * 2 * head_dim bytes in and head_dim + head_dim / 16 out
// per token and head (BF16), the values back (if asked for) as much as the input.
// Measured: 147 MB of prompts (BF16, head_dim 128, values back) 36.8 us, 4.0 TB/s, 0.59
// of the copy rate: the pipe that compares, permutes and converts is 57 % busy and the
// issue slots 64 %, the loads of a thread's few blocks do not hide the rest, and 8 CTAs to an SM
// leave 32 registers, which every instance spills beyond (28 bytes of stores and 40 of loads here,
// 68 and 88 for FP32).  One token of 32 sequences: 2.9 us.  Tried: loads ahead, other numbers of tokens to a CTA (37 to 41 us).
#include "wd_device.cuh"
#include "wd_kv.cuh"

namespace wd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;  // tokens of a CTA

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

// Eight values -> eight E2M1 codes (round to nearest even, saturating), the first in the low bits.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// ... and back.
__device__ __forceinline__ void e2m1x8_values(uint32_t w, float (&f)[8]) {
  uint32_t r[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&r[k]));
    f[2 * k] = p.x;
    f[2 * k + 1] = p.y;
  }
}

// 2^e for e in [-127, 127], the lowest a subnormal.
__device__ __forceinline__ float power_of_two(int e) {
  return e < -126 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

struct Place {
  uint8_t* group;  // K head 0's group of the token, null to skip it
  int t;           // token within the group
};

// Where a token of the batch goes.
template <int D>
__device__ __forceinline__ Place find_place(const KvAppendArgs& a, int token) {
  const KvView& c = a.cache;
  Place p{nullptr, 0};
  int b = token;  // the last entry that starts at or before this token
  if (a.batch.q_start) {
    int lo = 0, hi = a.batch.entries;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.batch.q_start[mid] <= token) lo = mid + 1; else hi = mid;
    }
    b = lo - 1;
  }
  if (b < 0 || b >= a.batch.entries) return p;
  int first, n;
  kv_tokens(c, a.batch, b, first, n);
  const int s = kv_slot(c, a.batch, b);
  if (s < 0 || token >= first + n) return p;
  const int pos = kv_length(c, s) - n + token - first;
  if (pos < 0) {
    atomicOr(c.flag, WD_KV_FLAG_BAD_INDEX);
    return p;
  }
  const int id = c.table[(long long)s * c.columns + (pos >> c.page_shift)];
  if ((unsigned)id >= (unsigned)c.num_pages) {
    atomicOr(c.flag, WD_KV_FLAG_BAD_INDEX);
    return p;
  }
  p.group = kv_group(c, id, a.layer, 0, pos, KvGroup<D>::kBytes);
  p.t = pos & 15;
  return p;
}

// per_cta: tokens of a CTA.  A thread stays with one head and side (or a few, if there are more than
// the CTA has rows of threads) and goes from token to token.
template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(kThreads, 8) kv_append(const KvAppendArgs a, int per_cta) {
  using G = KvGroup<D>;
  constexpr int kPerRow = D / 8;  // threads to a token, head and side
  constexpr int kRowsOfThreads = kThreads / kPerRow;
  __shared__ Place place[kMaxTokens];
  const KvView& c = a.cache;
  const int rows = 2 * c.kv_heads;  // of a token: the heads' K, then the heads' V
  const int base = blockIdx.x * per_cta;
  const int n = min(per_cta, a.batch.tokens - base);
  const int e = threadIdx.x % kPerRow;  // channels 8e .. 8e + 7
  const int block = e >> 2, t8 = e & 3;
  const int row0 = threadIdx.x / kPerRow;
  const int at_once = max(1, kRowsOfThreads / rows);  // tokens
  const int token0 = row0 / rows;  // (0 if there are more rows than threads for them)
  // a row's lanes are all here, or none: kPerRow divides the warp or is a warp
  const unsigned lanes = kPerRow >= 32
                             ? 0xFFFFFFFFu
                             : ((1u << (kPerRow % 32)) - 1u) << (threadIdx.x & 31 & ~(kPerRow - 1));
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();
  const auto fetch = [&](const T* src) {
    Eight<T> x;
    if (kVec) {
      x = *reinterpret_cast<const Eight<T>*>(src);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) x.v[k] = src[k];
    }
    return x;
  };
  bool placed = false;
  for (int hs = row0 - token0 * rows; hs < rows || !placed; hs += kRowsOfThreads) {
    const bool here = hs < rows && token0 < at_once;
    const bool v = hs >= c.kv_heads;
    const int head = v ? hs - c.kv_heads : hs;
    const long long stride = v ? a.v_token : a.k_token;
    const T* src = static_cast<const T*>(v ? a.v : a.k) + (base + token0) * stride +
                   head * (v ? a.v_head : a.k_head) + 8 * e;
    Eight<T> next;
    if (here && token0 < n) next = fetch(src);  // on its way while the places are found
    if (!placed) {
      if ((int)threadIdx.x < n) place[threadIdx.x] = find_place<D>(a, base + threadIdx.x);
      __syncthreads();
      placed = true;
    }
    if (!here) continue;
    const long long head_at = (long long)head * c.head_bytes;
    T* out = static_cast<T*>(v ? a.v_out : a.k_out) +
             ((long long)(base + token0) * c.kv_heads + head) * D + 8 * e;
    for (int token = token0; token < n; token += at_once) {
      const Eight<T> x = next;
      src += at_once * stride;
      if (token + at_once < n) next = fetch(src);
      float f[8];
      uint32_t top = Widen<T>::run(x, f);
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
      const Place p = place[token];
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
        if (a.k_out) {
          const float unit = bad ? __uint_as_float(0x7FC00000u) : power_of_two(exp2);
          e2m1x8_values(word, y);
#pragma unroll
          for (int k = 0; k < 8; ++k) y[k] *= unit;
          const Eight<T> z = narrow<T>(y);
          if (kVec) {
            *reinterpret_cast<Eight<T>*>(out) = z;
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) out[k] = z.v[k];
          }
        }
      }
      out += (long long)at_once * c.kv_heads * D;
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int D>
cudaError_t run(const KvAppendArgs& a, cudaStream_t s) {
  // Few tokens are spread over the SMs, a pass of the threads to each CTA at least; many get CTAs of
  // kMaxTokens.
  const int rows = 2 * a.cache.kv_heads;
  const int one_pass = (kThreads / (D / 8) + rows - 1) / rows;
  int per_cta = (a.batch.tokens + 8 * kKvSms - 1) / (8 * kKvSms);
  per_cta = per_cta < one_pass ? one_pass : per_cta;
  per_cta = per_cta > kMaxTokens ? kMaxTokens : per_cta;
  const int ctas = (a.batch.tokens + per_cta - 1) / per_cta;
  constexpr long long u = 16 / sizeof(T);  // elements to 16 bytes
  const bool vec = aligned16(a.k) && aligned16(a.v) && aligned16(a.k_out) && aligned16(a.v_out) &&
                   a.k_token % u == 0 && a.k_head % u == 0 && a.v_token % u == 0 &&
                   a.v_head % u == 0;
  return kv_launch(vec ? kv_append<T, D, true> : kv_append<T, D, false>, ctas, kThreads, 0, s, a,
                   per_cta);
}

template <typename T>
cudaError_t run_dim(const KvAppendArgs& a, cudaStream_t s) {
  switch (a.cache.head_dim) {
    case 64: return run<T, 64>(a, s);
    case 128: return run<T, 128>(a, s);
    default: return run<T, 256>(a, s);
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  switch (a.dtype) {
    case WD_KV_BF16: return run_dim<__nv_bfloat16>(a, s);
    case WD_KV_FP16: return run_dim<__half>(a, s);
    default: return run_dim<float>(a, s);
  }
}

}  // namespace wd
