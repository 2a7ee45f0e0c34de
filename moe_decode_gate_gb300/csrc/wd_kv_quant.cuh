// wd_kv_quant.cuh - what the kernels that write into the 4-bit cache share: the
// conversions of eight channels to MXFP4 and back, and where a token goes.
#pragma once

#include "wd_kv.cuh"
#include "wd_vec.cuh"

namespace wd {

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
  int pos;         // its position in the sequence, negative if it has none
};

// Where a token of the batch goes.
template <int D>
__device__ __forceinline__ Place find_place(const KvView& c, const KvBatch& batch, int layer, int token) {
  Place p{nullptr, 0, -1};
  int b = token;  // the last entry that starts at or before this token
  if (batch.q_start) {
    int lo = 0, hi = batch.entries;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (batch.q_start[mid] <= token) lo = mid + 1; else hi = mid;
    }
    b = lo - 1;
  }
  if (b < 0 || b >= batch.entries) return p;
  int first, n;
  kv_tokens(c, batch, b, first, n);
  const int s = kv_slot(c, batch, b);
  if (s < 0 || token >= first + n) return p;
  const int pos = kv_length(c, s) - n + token - first;
  if (pos < 0) {
    atomicOr(c.flag, WD_KV_FLAG_BAD_INDEX);
    return p;
  }
  p.pos = pos;
  const int id = c.table[(long long)s * c.columns + (pos >> c.page_shift)];
  if ((unsigned)id >= (unsigned)c.num_pages) {
    atomicOr(c.flag, WD_KV_FLAG_BAD_INDEX);
    return p;
  }
  p.group = kv_group(c, id, layer, 0, pos, KvGroup<D>::kBytes);
  p.t = pos & 15;
  return p;
}

}  // namespace wd
