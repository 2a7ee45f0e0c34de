// wd_kv_attention.cuh - what the two attention kernels of the 4-bit cache share: conversions, the
// batch's entries, the keys that a tile of query rows sees, and the store of a finished row.
#pragma once

#include <float.h>

#include "wd_device.cuh"
#include "wd_kv.cuh"
#include "wd_mma.cuh"

namespace wd {

constexpr int kStep = 32;      // keys of a step: two groups
constexpr int kCached = 256;   // entries whose slot and length are kept in shared memory
constexpr float kBias = 8.f;   // P = 2^kBias at the reference m ...
constexpr float kSlack = 6.f;  // ... which may fall this far behind the maximum (log2)
// Sums of K with queries of up to 2^15, each scaled by its block's 2^(s - 127), are kept 2^26 times smaller: 256
// products of up to 6 x 2^15 then stay within FP32 for any s.
constexpr int kKeyShift = 26;
constexpr uint32_t kAll = 0xFFFFFFFFu;
// How far the values of a key that some rows of a tile do not see may raise V's reference: what those rows see
// stays within FP32 beside it (2^-134 of it at worst), and so does what lies above (up to 2^104, added one by one).
constexpr uint32_t kSharedMost = 150;

// A piece of an item, and where the item's output goes.
struct Part {
  long long slot0;  // the place of the item's first piece among all pieces
  int pieces;       // of the item; 0: nothing to do
  int tile, head, first, n;
};

// Four E2M1 pairs (the bytes of w, low half first) -> four f16x2, exactly.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t& r0, uint32_t& r1, uint32_t& r2,
                                       uint32_t& r3) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
      : "r"(w));
}

// Two E8M0 scale bytes (the low 16 bits of w) -> BF16 2^(s-127), NaN for 255, exactly.
__device__ __forceinline__ uint32_t e8m0x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.bf16x2.ue8m0x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 8x8 transpose of 16-bit elements across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

template <int N>
struct Words {
  uint32_t v[N];
};
// N words of shared memory (N * 4 bytes aligned, up to 16).
template <int N>
__device__ __forceinline__ Words<N> lds(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 4) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    r.v[0] = x.x; r.v[1] = x.y; r.v[2] = x.z; r.v[3] = x.w;
  } else if constexpr (N == 2) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    r.v[0] = x.x; r.v[1] = x.y;
  } else {
    static_assert(N == 1, "");
    r.v[0] = *reinterpret_cast<const uint32_t*>(p);
  }
  return r;
}

// The scale bytes of one token: 2 (in the low half of a word), 4 or 8.
template <int CB>
__device__ __forceinline__ Words<(CB + 3) / 4> lds_scales(const uint8_t* p) {
  if constexpr (CB == 2) {
    Words<1> r;
    r.v[0] = *reinterpret_cast<const uint16_t*>(p);
    return r;
  } else {
    return lds<CB / 4>(p);
  }
}

// x / d with inv = 1.f / d: the quotient in FP32 is at most one off where x is small, and put right; the
// compiler's own division takes three times as long, and a piece is found by several in a row.
struct Divisor {
  unsigned d;
  float inv;
  __device__ __forceinline__ explicit Divisor(unsigned by) : d(by), inv(1.f / (float)by) {}
  __device__ __forceinline__ unsigned of(unsigned x) const {
    if (x >= 1u << 22) return x / d;
    unsigned q = (unsigned)((float)x * inv);
    const int r = (int)(x - q * d);
    q += r >= (int)d ? 1u : 0u;
    q -= r < 0 ? 1u : 0u;
    return q;
  }
};

// What of the sequence one entry of the batch works on.
struct Entry {
  int slot, len, first, n;
};
__device__ __forceinline__ Entry load_entry(const KvAttentionArgs& a, int b,
                                            const int2* cached = nullptr) {
  Entry e;
  if (cached && b < kCached) {
    e.slot = cached[b].x;
    e.len = cached[b].y;
  } else {
    e.slot = kv_slot(a.cache, a.batch, b);
    e.len = e.slot < 0 ? 0 : kv_length(a.cache, e.slot);
  }
  kv_tokens(a.cache, a.batch, b, e.first, e.n);
  return e;
}
template <int kRows>
__device__ __forceinline__ int tiles_of(const Entry& e, int group) {
  return (e.n * group + kRows - 1) / kRows;
}

// Steps that each of an entry's tiles is given: what the tile that sees the most needs, at least
// one (a tile that sees nothing is written too).  The tiles of a causal chunk see unlike numbers
// of keys; they are taken from both ends in turn, so that what is given and not needed
// spreads over the warps.
template <int kRows>
__device__ __forceinline__ int steps_of(const Entry& e, int group, int window) {
  if (e.len <= 0) return 1;
  int steps = (e.len - 1) / kStep + 1;
  if (window > 0) {
    if (e.n == 1) {
      steps -= max(0, e.len - window) / kStep;
    } else {
      const int tokens = min(e.n - 1, (kRows - 1) / group + 1);  // between a tile's ends
      const long long keys = (long long)window + tokens;
      steps = (int)min((long long)steps, (keys + kStep - 2) / kStep + 1);
    }
  }
  return steps;
}

// The keys that a tile sees: from those of step `first` up to `end`.
struct Span {
  int first, end;
};
template <int kRows>
__device__ __forceinline__ Span tile_span(const Entry& e, int tile, int group, int window) {
  int i0 = 0, i1 = e.n - 1;
  if (e.n > 1) {
    i0 = tile * kRows / group;
    i1 = min(i1, (tile * kRows + kRows - 1) / group);
  }
  Span s;
  s.first = window > 0 ? max(0, e.len - e.n + i0 - window + 1) / kStep : 0;
  s.end = e.len - e.n + i1 + 1;
  return s;
}

// Eight 16-bit values of a query row, from wherever they lie.
__device__ __forceinline__ Words<4> load8(const KvAttentionArgs& a, long long off, bool vec) {
  const uint16_t* s = static_cast<const uint16_t*>(a.q) + off;
  Words<4> w;
  if (vec) {
    const uint4 v = *reinterpret_cast<const uint4*>(s);
    w.v[0] = v.x; w.v[1] = v.y; w.v[2] = v.z; w.v[3] = v.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) w.v[k] = s[2 * k] | ((uint32_t)s[2 * k + 1] << 16);
  }
  return w;
}
__device__ __forceinline__ void widen8(const Words<4>& w, bool half, float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = half ? __half22float2(*reinterpret_cast<const __half2*>(&w.v[k]))
                          : make_float2(__uint_as_float(w.v[k] << 16),
                                        __uint_as_float(w.v[k] & 0xFFFF0000u));
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}

// Four channels of a finished row: y / sum, and with the first of them the row's lse.
template <int D, int kRows>
__device__ __forceinline__ void store_row(const KvAttentionArgs& a, const Part& p, int row, int ch,
                                          const float4& y, float top, float sum) {
  const int group = a.q_heads / a.cache.kv_heads;
  const int flat = p.tile * kRows + row;
  if (flat >= p.n * group) return;
  const int token = p.n > 1 ? flat / group : 0;
  const long long at =
      (long long)(p.first + token) * a.q_heads + p.head * group + flat - token * group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const float v[4] = {y.x * inv, y.y * inv, y.z * inv, y.w * inv};
  uint16_t* to = static_cast<uint16_t*>(a.out) + at * D + ch;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (a.half)
      reinterpret_cast<__half*>(to)[q] = __float2half_rn(v[q]);
    else
      reinterpret_cast<__nv_bfloat16*>(to)[q] = __float2bfloat16_rn(v[q]);
  }
  if (a.lse && ch == 0)
    a.lse[at] = sum == 0.f ? -INFINITY : (top - kBias) * 0.6931471805599453f + logf(sum);
}

// Scaling of a query row whose largest magnitude has these bits: 2^k brings it into
// [2^14, 2^15) (subnormals are scaled as if 2^-126), in two factors.
struct RowScale {
  float up, up2;
  bool bad;  // holds an infinity or NaN
};
__device__ __forceinline__ RowScale row_scale(uint32_t bits) {
  RowScale r;
  r.bad = bits >= 0x7F800000u;
  const int k = r.bad || bits == 0u ? 0 : 14 - (max((int)(bits >> 23), 1) - 127);
  r.up = exp2_int(k / 2);
  r.up2 = exp2_int(k - k / 2);
  return r;
}
// 2^kFactorShift times what the row's sums are multiplied by, a number that FP32 holds for all queries (scale up
// to 1): a row with an infinity or NaN has no finite logit; never 0, so that -inf stays -inf.
constexpr int kFactorShift = kKeyShift / 2;
__device__ __forceinline__ float row_factor(const RowScale& r, float scale) {
  constexpr float kUp = (float)(1 << kFactorShift);
  return r.bad ? __uint_as_float(0x7FC00000u)
               : fminf(fmaxf(scale * 1.4426950408889634f / r.up * kUp / r.up2, 1.2e-38f), FLT_MAX);
}
// Of a row whose sums are 2^kKeyShift times smaller and have all of `scale` but a power of two, `unit`, in them.
// (|q| unit beyond 2^114 has to do with 2^127.)
__device__ __forceinline__ float power_factor(const RowScale& r, float unit) {
  constexpr float kUp = (float)(1 << (kKeyShift / 2));
  return r.bad ? __uint_as_float(0x7FC00000u)
               : fminf(fmaxf(unit / r.up * kUp / r.up2 * kUp, 0x1p-126f), 0x1p127f);
}
// ... for sums that are 2^kKeyShift times smaller (where |q| scale is beyond 2^114 FP32's largest has to do).
__device__ __forceinline__ float shifted_factor(float factor) {
  const float f = factor * (float)(1 << (kKeyShift - kFactorShift));
  return f > FLT_MAX ? FLT_MAX : f;
}
__device__ __forceinline__ uint4 row_fragment(const float (&x)[8], const RowScale& r) {
  uint4 f;
  f.x = pack_half2(x[0] * r.up * r.up2, x[1] * r.up * r.up2);
  f.y = pack_half2(x[2] * r.up * r.up2, x[3] * r.up * r.up2);
  f.z = pack_half2(x[4] * r.up * r.up2, x[5] * r.up * r.up2);
  f.w = pack_half2(x[6] * r.up * r.up2, x[7] * r.up * r.up2);
  return f;
}

// The kernel for many query rows to a key head (wd_kv_attention_rows.cu).
bool kv_attention_rows_supported(const KvAttentionArgs& a);
cudaError_t launch_kv_attention_rows(const KvAttentionArgs& a, cudaStream_t s);

}  // namespace wd
