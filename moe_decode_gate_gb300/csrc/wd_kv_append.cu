// wd_kv_append.cu - quantise new keys and values to MXFP4 and write them into
// the pages of their sequences (declared in include/wd_kv.h).
//
// A thread takes 8 consecutive channels of one token, head and side (K or V):
// one 16-byte load of 16-bit inputs.  Four neighbouring lanes hold a block of 32
// channels, so its largest magnitude is two shuffles away.  The 8 codes are one
// 32-bit word of the K layout or two 16-bit halves of the V layout.
//
// Bound by memory: 2 * 2 * head_dim bytes in and head_dim + head_dim / 16 out
// per token and head (BF16), the values back (if asked for) as much as the input.
#include "wd_kv.cuh"

namespace wd {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;  // tokens whose places a CTA looks up at a time

template <typename T>
__device__ __forceinline__ float to_float(T v);
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float(float v) { return v; }

template <typename T>
struct alignas(16) Eight {
  T v[8];
};

// Two values -> two E2M1 codes (round to nearest even, saturating), x in the
// low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2(float x, float y) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(r)
      : "f"(x), "f"(y));
  return r;
}

// E2M1 code -> value
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  const float a = m < 2u ? 0.5f * (float)m
                         : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return (code & 8u) ? -a : a;
}

// 2^e for e in [-127, 127], the lowest a subnormal.
__device__ __forceinline__ float power_of_two(int e) {
  return e < -126 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)(e + 127) << 23);
}

struct Place {
  uint8_t* group;  // K head 0's group of the token, null to skip it
  int t;           // token within the group
};

template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(kThreads) kv_append(const KvAppendArgs a) {
  using G = KvGroup<D>;
  __shared__ Place place[kTokens];
  const KvView& c = a.cache;
  const int per_head = D / 8;  // threads to a token, head and side
  const int per_token = 2 * c.kv_heads * per_head;
  for (long long base = (long long)blockIdx.x * kTokens; base < a.batch.tokens;
       base += (long long)gridDim.x * kTokens) {
    if (threadIdx.x < kTokens) {
      const long long token = base + threadIdx.x;
      Place p{nullptr, 0};
      if (token < a.batch.tokens) {
        // the last entry that starts at or before this token
        int b = (int)token;
        if (a.batch.q_start) {
          int lo = 0, hi = a.batch.entries;
          while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (a.batch.q_start[mid] <= token) lo = mid + 1; else hi = mid;
          }
          b = lo - 1;
        }
        if (b >= 0 && b < a.batch.entries) {
          int first, n;
          kv_tokens(c, a.batch, b, first, n);
          const int s = kv_slot(c, a.batch, b);
          if (s >= 0 && token < (long long)first + n) {
            const int pos = kv_length(c, s) - n + (int)(token - first);
            if (pos < 0) {
              atomicOr(c.flag, WD_KV_FLAG_BAD_INDEX);
            } else {
              const int id = c.table[(long long)s * c.columns + (pos >> c.page_shift)];
              if ((unsigned)id < (unsigned)c.num_pages) {
                p.group = kv_group(c, id, a.layer, 0, pos, G::kBytes);
                p.t = pos & 15;
              } else {
                atomicOr(c.flag, WD_KV_FLAG_BAD_INDEX);
              }
            }
          }
        }
      }
      place[threadIdx.x] = p;
    }
    __syncthreads();
    const int here = (int)min((long long)kTokens, a.batch.tokens - base);
    for (int i = threadIdx.x; i < here * per_token; i += kThreads) {
      const int token = i / per_token, r = i % per_token;
      const int head = r / (2 * per_head);
      const int side = (r / per_head) & 1;  // 0: K, 1: V
      const int e = r % per_head;           // channels 8e .. 8e + 7
      const T* src = static_cast<const T*>(side ? a.v : a.k) +
                     (base + token) * (side ? a.v_token : a.k_token) +
                     head * (side ? a.v_head : a.k_head) + 8 * e;
      Eight<T> x;
      if (kVec) {
        x = *reinterpret_cast<const Eight<T>*>(src);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x.v[k] = src[k];
      }
      float f[8];
      uint32_t top = 0;  // largest magnitude's bits: order as the values do, NaN above Inf
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[k] = to_float(x.v[k]);
        top = max(top, __float_as_uint(f[k]) & 0x7FFFFFFFu);
      }
      // per_token is a multiple of 4, so the four lanes of a block are active together
      const unsigned quad = 0xFu << (threadIdx.x & 28);
      top = max(top, __shfl_xor_sync(quad, top, 1));
      top = max(top, __shfl_xor_sync(quad, top, 2));
      const bool bad = top >= 0x7F800000u;
      // floor(log2(top)) - 2, at least -127; a subnormal's floor(log2) is below -126
      const int ex = (int)(top >> 23);
      const int exp2 = top == 0 ? 0 : (ex <= 2 ? -127 : ex - 129);
      const uint32_t scale = bad ? 255u : (uint32_t)(exp2 + 127);
      const float inv = power_of_two(-exp2);
      uint32_t word = 0;
      if (!bad) {
#pragma unroll
        for (int k = 0; k < 4; ++k) word |= e2m1x2(f[2 * k] * inv, f[2 * k + 1] * inv) << (8 * k);
      }
      const Place p = place[token];
      if (p.group) {
        uint8_t* g = p.group + (long long)head * c.head_bytes;
        const int block = e >> 2, t8 = e & 3;
        if (side == 0) {
          *reinterpret_cast<uint32_t*>(g + G::k_word(p.t, block, t8)) = word;
        } else {
          *reinterpret_cast<uint16_t*>(g + G::v_half(p.t, block, 2 * t8)) = (uint16_t)word;
          *reinterpret_cast<uint16_t*>(g + G::v_half(p.t, block, 2 * t8 + 1)) =
              (uint16_t)(word >> 16);
        }
        if (t8 == 0)
          g[(side ? G::kVScale : G::kKScale) + p.t * G::kBlocks + block] = (uint8_t)scale;
      }
      if (a.k_out && p.group) {
        const float unit = bad ? __uint_as_float(0x7FC00000u) : power_of_two(exp2);
        Eight<T> y;
#pragma unroll
        for (int k = 0; k < 8; ++k) y.v[k] = from_float<T>(e2m1_value(word >> (4 * k)) * unit);
        T* out = static_cast<T*>(side ? a.v_out : a.k_out) +
                 ((base + token) * c.kv_heads + head) * D + 8 * e;
        if (kVec) {
          *reinterpret_cast<Eight<T>*>(out) = y;
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) out[k] = y.v[k];
        }
      }
    }
    __syncthreads();
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T, int D>
cudaError_t run(const KvAppendArgs& a, cudaStream_t s) {
  const int ctas = (a.batch.tokens + kTokens - 1) / kTokens;
  constexpr long long u = 16 / sizeof(T);  // elements to 16 bytes
  const bool vec = aligned16(a.k) && aligned16(a.v) && aligned16(a.k_out) && aligned16(a.v_out) &&
                   a.k_token % u == 0 && a.k_head % u == 0 && a.v_token % u == 0 &&
                   a.v_head % u == 0;
  if (vec)
    kv_append<T, D, true><<<ctas, kThreads, 0, s>>>(a);
  else
    kv_append<T, D, false><<<ctas, kThreads, 0, s>>>(a);
  return cudaGetLastError();
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
