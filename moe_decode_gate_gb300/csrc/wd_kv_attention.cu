// wd_kv_attention.cu - attention over the 4-bit cache (declared in include/wd_kv.h).
//
// Work.  An item is (entry, tile of 8 * NT query rows, key head); the rows of a tile are the
// heads that share the key head and, behind them, further new tokens.  An item is cut into steps
// of 32 keys, and all steps of the call, in order, are dealt out evenly over a grid of as many
// CTAs as fit the GPU: a CTA takes a contiguous range of steps and its eight warps take turns in
// it.  The lengths are known to the device alone, so every CTA derives the whole division from
// them; a captured graph can be replayed while the sequences grow.  A CTA that has all of an
// item writes its output; else it leaves a partial result (maximum, sum, output) in the
// workspace, and the CTA that arrives last joins the parts in their order.
//
// A step.  Each warp streams its steps' groups (2176 bytes per 16 keys at head_dim 128) with
// bulk copies into a ring of its own.  With K as the left operand, S^T = K Q^T and O^T = V^T P^T
// are m16n8k16 products whose 16 rows are keys or channels and whose 8 columns are query rows,
// so eight query heads fill a tile, where a 16-row query tile would be half empty.  The groups are stored in
// fragment order: one 16-byte shared-memory read per lane brings 32 codes, which the hardware
// conversion turns into FP16 (exactly) in place.
//   - K: the sums over a block of 32 channels are scaled by the block's 2^(s-127) in FP32.
//   - Queries are FP16 x 2^k with k per row (exact for BF16 and FP16 within 2^31 of the row's
//     largest magnitude), 2^-k folded into the softmax scale.
//   - P = 2^14 exp2(x - max) is rounded to FP16 once (11 bits; below 2^-28 of the largest it
//     loses bits, below 2^-39 it is zero); the row sums are of the unrounded values, in FP32.
//   - V: the scales lie along the channels that are the product's rows, so each of P's
//     columns is multiplied by 2^(s - r + 1) for every block, with r the largest scale that the warp
//     has met for that block of channels: exact while s >= r - 15. A step that holds other
//     scales (or NaN) adds its products one by one in FP32 instead.
#include "wd_kv.cuh"
#include "wd_mma.cuh"

namespace wd {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStep = 32;     // keys of a warp's step: two groups
constexpr int kPad = 36;      // floats to a row of the merge buffer
constexpr uint32_t kAll = 0xFFFFFFFFu;

template <int D, int NT>
struct Shape {
  using G = KvGroup<D>;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * G::kBytes;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kCtasPerSm = D <= 128 && NT == 1 ? 2 : 1;
  // shared memory, in bytes from its start
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kWarps * kStages * kStageBytes;  // fragments [NT][blocks][32] uint4
  static constexpr int kMerge = kQ + NT * G::kBlocks * 512;          // float [kWarps][kRows][kPad]
  static constexpr int kStats = kMerge + kWarps * kRows * kPad * 4;  // float m, l [kWarps][kRows] each
  static constexpr int kRowInfo = kStats + 2 * kWarps * kRows * 4;   // factor, lo, hi, max, sum [kRows]
  static constexpr int kBars = kRowInfo + 5 * kRows * 4;             // uint64 [kWarps][kStages]
  static constexpr int kScan = kBars + kWarps * kStages * 8;         // long long [16]
  static constexpr int kPrefix = kScan + 16 * 8;                     // long long [entries + 1]
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

// What of the sequence one entry of the batch works on.
struct Entry {
  int slot, len, first, n;
};
__device__ __forceinline__ Entry load_entry(const KvAttentionArgs& a, int b) {
  Entry e;
  e.slot = kv_slot(a.cache, a.batch, b);
  e.len = e.slot < 0 ? 0 : kv_length(a.cache, e.slot);
  kv_tokens(a.cache, a.batch, b, e.first, e.n);
  return e;
}

// The steps of keys that a tile of query rows sees: at least one, so that a tile that sees
// nothing is written too.
struct Span {
  int first, steps;  // in steps of kStep keys
  int end;           // keys from here on are not seen
};
template <int kRows>
__device__ __forceinline__ Span tile_span(const Entry& e, int tile, int group, int window) {
  const int i0 = tile * kRows / group;
  const int i1 = min(e.n - 1, (tile * kRows + kRows - 1) / group);
  const int hi = e.len - e.n + i1;
  const int lo = window > 0 ? max(0, e.len - e.n + i0 - window + 1) : 0;
  Span s;
  s.first = lo / kStep;
  s.steps = hi < 0 ? 1 : max(1, hi / kStep + 1 - s.first);
  s.end = hi + 1;
  return s;
}

// A place in the order of all steps.
struct Place {
  int entry, tile, head, step;
  Span span;
};
template <int kRows>
__device__ __forceinline__ Place locate(const KvAttentionArgs& a, const long long* prefix,
                                        long long p, int group, Entry& e) {
  int lo = 0, hi = a.batch.entries;  // the last entry whose steps begin at or before p
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= p) lo = mid; else hi = mid;
  }
  Place at;
  at.entry = lo;
  e = load_entry(a, lo);
  long long rest = p - prefix[lo];
  const int heads = a.cache.kv_heads;
  // (the last tile and head are also where it ends if someone rewrites the lengths meanwhile)
  const int tiles = max(1, (e.n * group + kRows - 1) / kRows);
  for (at.tile = 0;; ++at.tile) {
    at.span = tile_span<kRows>(e, at.tile, group, a.window);
    const long long cost = (long long)at.span.steps * heads;
    if (rest < cost || at.tile + 1 == tiles) break;
    rest -= cost;
  }
  at.head = min((int)((uint32_t)rest / (uint32_t)at.span.steps), heads - 1);
  at.step = (int)((uint32_t)rest % (uint32_t)at.span.steps);
  return at;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kCtasPerSm)
    kv_attention(const KvAttentionArgs a) {
  using G = KvGroup<D>;
  using L = Shape<D, NT>;
  constexpr int CB = G::kBlocks, SB = G::kSlabBlocks, NS = G::kSlabs, NW = (CB + 3) / 4;
  constexpr int kRows = L::kRows, kStages = L::kStages;
  constexpr bool kQInRegs = NT == 1;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tq = lane & 3;
  const KvView& cache = a.cache;
  const int heads = cache.kv_heads, group = a.q_heads / heads;
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* m_sh = reinterpret_cast<float*>(smem + L::kStats);
  float* l_sh = m_sh + kWarps * kRows;
  float* factor_sh = reinterpret_cast<float*>(smem + L::kRowInfo);
  int* lo_sh = reinterpret_cast<int*>(factor_sh + kRows);
  int* hi_sh = lo_sh + kRows;
  float* max_sh = reinterpret_cast<float*>(hi_sh + kRows);
  float* sum_sh = max_sh + kRows;
  long long* scan = reinterpret_cast<long long*>(smem + L::kScan);
  long long* prefix = reinterpret_cast<long long*>(smem + L::kPrefix);
  uint8_t* ring = smem + L::kRing + warp * kStages * L::kStageBytes;
  const uint32_t bar = smem_u32(smem + L::kBars) + warp * kStages * 8;
  __shared__ int last_sh;

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    mbar_init_fence();
  }
  // prefix[b] = steps of the entries before b
  long long before = 0;
  for (int base = 0; base < a.batch.entries; base += kThreads) {
    const int b = base + threadIdx.x;
    long long cost = 0;
    if (b < a.batch.entries) {
      const Entry e = load_entry(a, b);
      const int tiles = (e.n * group + kRows - 1) / kRows;
      for (int t = 0; t < tiles; ++t) cost += tile_span<kRows>(e, t, group, a.window).steps;
      cost *= heads;
    }
    long long incl = cost;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long t = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += t;
    }
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long below = before, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) below += scan[w];
      all += scan[w];
    }
    if (b < a.batch.entries) prefix[b] = below + incl - cost;
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) prefix[a.batch.entries] = before;
  __syncthreads();
  const long long total = before;
  // steps to a CTA: a whole number for each of its warps
  const long long quota = (total + (long long)gridDim.x * kWarps - 1) /
                          ((long long)gridDim.x * kWarps) * kWarps;
  const long long begin = blockIdx.x * quota, end = min(total, begin + quota);
  if (begin >= end) return;

  // The warp's steps are begin + warp, + kWarps, ...: its k-th step's groups are worked out by
  // lane k % 32, 32 steps at a time, and copied into stage k % kStages.
  const uint8_t *src0 = nullptr, *src1 = nullptr;
  const auto plan = [&](int k0) {
    const long long p = begin + warp + (long long)kWarps * (k0 + lane);
    src0 = src1 = nullptr;
    if (p >= end) return;
    Entry e;
    const Place at = locate<kRows>(a, prefix, p, group, e);
    const int pos = (at.span.first + at.step) * kStep;
    if (pos < at.span.end)
      src0 = kv_group(cache, kv_page(cache, e.slot, pos >> cache.page_shift), a.layer, at.head,
                      pos, G::kBytes);
    if (pos + 16 < at.span.end)
      src1 = kv_group(cache, kv_page(cache, e.slot, (pos + 16) >> cache.page_shift), a.layer,
                      at.head, pos + 16, G::kBytes);
  };
  const auto issue = [&](int stage) {
    const uint32_t to = smem_u32(ring) + stage * L::kStageBytes;
    mbar_arrive_expect_tx(bar + 8 * stage, (src0 ? G::kBytes : 0) + (src1 ? G::kBytes : 0));
    if (src0) bulk_g2s_nohint(to, src0, G::kBytes, bar + 8 * stage);
    if (src1) bulk_g2s_nohint(to + G::kBytes, src1, G::kBytes, bar + 8 * stage);
  };
  plan(0);
  if (lane < kStages && begin + warp + (long long)kWarps * lane < end) issue(lane);
  __syncwarp();

  int k = 0, stage = 0;
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out
  Entry entry;
  for (long long p0 = begin; p0 < end;) {
    const Place at = locate<kRows>(a, prefix, p0, group, entry);
    const long long item = p0 - at.step;                      // the item's first step
    const long long p1 = min(end, item + at.span.steps);      // the segment is [p0, p1)

    // the tile's queries, as fragments: channel 32c + 8t + 4j + 2r + {0,1} of row 8nt + g is
    // register r of product j in lane 4g + t
    __syncthreads();
    for (int row = warp; row < kRows; row += kWarps) {
      const int flat = at.tile * kRows + row;
      const bool real = flat < entry.n * group;
      const int i = flat / group;
      uint32_t bits = 0;
      float x[D / 32];
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        float lo = 0.f, hi = 0.f;
        if (real) {
          const long long off = (entry.first + i) * a.q_token +
                                (at.head * group + flat % group) * a.q_head + 64 * q + 2 * lane;
          if (a.half) {
            const __half* s = static_cast<const __half*>(a.q) + off;
            lo = __half2float(s[0]);
            hi = __half2float(s[1]);
          } else {
            const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(a.q) + off;
            lo = __bfloat162float(s[0]);
            hi = __bfloat162float(s[1]);
          }
        }
        x[2 * q] = lo;
        x[2 * q + 1] = hi;
        bits = max(bits, max(__float_as_uint(lo) & 0x7FFFFFFFu, __float_as_uint(hi) & 0x7FFFFFFFu));
      }
      bits = __reduce_max_sync(kAll, bits);
      // 2^k brings the largest magnitude into [2^14, 2^15); subnormals are scaled as if 2^-126
      const bool bad = bits >= 0x7F800000u;
      const int k2 = bad || bits == 0u ? 0 : 14 - (max((int)(bits >> 23), 1) - 127);
      const float up = exp2_int(k2 / 2), up2 = exp2_int(k2 - k2 / 2);
#pragma unroll
      for (int q = 0; q < D / 64; ++q) {
        const int ch = 64 * q + 2 * lane;
        const int c = ch >> 5, t = (ch & 31) >> 3, r = (ch & 7) >> 1;
        *reinterpret_cast<uint32_t*>(smem + L::kQ + (((row >> 3) * CB + c) * 32 + (row & 7) * 4 + t) * 16 +
                                     r * 4) = pack_half2(x[2 * q] * up * up2, x[2 * q + 1] * up * up2);
      }
      if (lane == 0) {
        const int pos = entry.len - entry.n + i;
        // a row with an infinity or NaN has no finite logit
        factor_sh[row] = bad ? __uint_as_float(0x7FC00000u)
                             : a.scale * 1.4426950408889634f / up / up2;
        lo_sh[row] = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
        hi_sh[row] = real ? pos : at.span.end - 1;  // no row: nothing to hide, never stored
      }
    }
    __syncthreads();

    uint4 qf[kQInRegs ? CB : 1];
    if constexpr (kQInRegs) {
#pragma unroll
      for (int c = 0; c < CB; ++c)
        qf[c] = *reinterpret_cast<const uint4*>(smem + L::kQ + (c * 32 + lane) * 16);
    }
    float factor[NT][2];
    int seen_lo = 0, seen_hi = 0x7FFFFFFF;  // keys that every row of the tile sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 8 * nt + 2 * tq + e;
        factor[nt][e] = factor_sh[row];
        seen_lo = max(seen_lo, lo_sh[row]);
        seen_hi = min(seen_hi, hi_sh[row]);
      }
    seen_lo = max(seen_lo, __shfl_xor_sync(kAll, seen_lo, 1));
    seen_lo = max(seen_lo, __shfl_xor_sync(kAll, seen_lo, 2));
    seen_hi = min(seen_hi, __shfl_xor_sync(kAll, seen_hi, 1));
    seen_hi = min(seen_hi, __shfl_xor_sync(kAll, seen_hi, 2));

    float o[CB][2][NT][4];
    float m[NT][2], l[NT][2];
    uint32_t ref[NW];  // the largest V scale met, a byte to a block, at least 16
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][j][nt][e] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }
#pragma unroll
    for (int w = 0; w < NW; ++w) ref[w] = 0x10101010u;

    for (; begin + warp + (long long)kWarps * k < p1; ++k) {
      const int j0 = (at.span.first + (int)(begin + warp + (long long)kWarps * k - item)) * kStep;
      if (!dead && !mbar_wait(bar + 8 * stage, phase)) {
        dead = true;
        if (lane == 0) atomicOr(cache.flag, WD_KV_FLAG_TIMEOUT);
      }
      dead = __any_sync(kAll, dead);
      if (dead) break;
      const uint8_t* buf = ring + stage * L::kStageBytes;

      // ---- S^T = K Q^T
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
      Words<NW> ks[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          ks[u][h] = lds_scales<CB>(buf + u * G::kBytes + G::kKScale + (8 * h + g) * CB);
#pragma unroll
      for (int sl = 0; sl < NS; ++sl) {
        Words<SB> kw[2][2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            kw[u][h] = lds<SB>(buf + u * G::kBytes + sl * G::kSlabBytes + (8 * h + g) * 16 * SB +
                               tq * 4 * SB);
#pragma unroll
        for (int c = 0; c < SB; ++c) {
          const int cb = sl * SB + c;
          uint4 q[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            q[nt] = kQInRegs ? qf[kQInRegs ? cb : 0]
                             : *reinterpret_cast<const uint4*>(
                                   smem + L::kQ + ((nt * CB + cb) * 32 + lane) * 16);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
            e2m1x8(kw[u][0].v[c], a0, a2, b0, b2);
            e2m1x8(kw[u][1].v[c], a1, a3, b1, b3);
            const float s0 = __uint_as_float(((ks[u][0].v[cb / 4] >> (8 * (cb % 4))) & 0xFFu) << 23);
            const float s1 = __uint_as_float(((ks[u][1].v[cb / 4] >> (8 * (cb % 4))) & 0xFFu) << 23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float t[4];
              mma_f16_zero(t, a0, a1, a2, a3, q[nt].x, q[nt].y);
              mma_f16_acc(t, b0, b1, b2, b3, q[nt].z, q[nt].w);
              s[u][nt][0] = fmaf(t[0], s0, s[u][nt][0]);
              s[u][nt][1] = fmaf(t[1], s0, s[u][nt][1]);
              s[u][nt][2] = fmaf(t[2], s1, s[u][nt][2]);
              s[u][nt][3] = fmaf(t[3], s1, s[u][nt][3]);
            }
          }
        }
      }

      // ---- the scales of token j0 + lane: are all of them in range?
      const bool inside = j0 + lane < at.span.end;
      bool slow = false;
      {
        const uint8_t* sc = buf + (lane >> 4) * G::kBytes + (lane & 15) * CB;
        const Words<NW> kt = lds_scales<CB>(sc + G::kKScale);
        Words<NW> vt = lds_scales<CB>(sc + G::kVScale);
        bool odd = false, nan_k = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          if (CB == 2) vt.v[w] |= ref[w] & 0xFFFF0000u;
          nan_k |= (((kt.v[w] & 0x7F7F7F7Fu) + 0x01010101u) & kt.v[w] & 0x80808080u) != 0u;
          const uint32_t t0 = ((ref[w] & 0x00FF00FFu) | 0x80008000u) - (vt.v[w] & 0x00FF00FFu);
          const uint32_t t1 =
              (((ref[w] >> 8) & 0x00FF00FFu) | 0x80008000u) - ((vt.v[w] >> 8) & 0x00FF00FFu);
          odd |= ((t0 | t1) & 0x7FF07FF0u) != 0u;
        }
        if (__any_sync(kAll, inside && (odd || nan_k))) {
          const uint32_t nan_tokens = __ballot_sync(kAll, inside && nan_k);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (nan_tokens >> (16 * u + 8 * (e >> 1) + g) & 1u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) s[u][nt][e] = __uint_as_float(0x7FC00000u);
          // raise the reference scales, and what stands on them
          uint32_t bad = 0;
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            const uint32_t sh = 8 * (c % 4), mine = (vt.v[c / 4] >> sh) & 0xFFu;
            const uint32_t old = (ref[c / 4] >> sh) & 0xFFu;
            const uint32_t top =
                max(old, __reduce_max_sync(kAll, inside && mine != 255u ? mine : 0u));
            if (top != old) {
              const float down = exp2_fast((float)(int)old - (float)(int)top);
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[c][j][nt][e] *= down;
              ref[c / 4] = (ref[c / 4] & ~(0xFFu << sh)) | (top << sh);
            }
            bad |= inside && (mine > top || mine + 15u < top) ? 1u : 0u;
          }
          slow = __any_sync(kAll, bad != 0u);
        }
        // keys behind the end get a scale in range; their probabilities are zero
        if (j0 + kStep > at.span.end) {
          if (!inside) {
            uint8_t* to = ring + stage * L::kStageBytes + (lane >> 4) * G::kBytes + G::kVScale +
                          (lane & 15) * CB;
            if constexpr (CB == 2) {
              *reinterpret_cast<uint16_t*>(to) = (uint16_t)ref[0];
            } else {
#pragma unroll
              for (int w = 0; w < NW; ++w) reinterpret_cast<uint32_t*>(to)[w] = ref[w];
            }
          }
          __syncwarp();
        }
      }

      // ---- softmax
      const bool whole = j0 >= seen_lo && j0 + kStep - 1 <= seen_hi;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x = s[u][nt][2 * h + e] * factor[nt][e];
              if (!whole) {
                const int row = 8 * nt + 2 * tq + e, key = j0 + 16 * u + 8 * h + g;
                if (key < lo_sh[row] || key > hi_sh[row]) x = -INFINITY;
              }
              s[u][nt][2 * h + e] = x;
              t = fmaxf(t, x);
            }
          top[nt][e] = t;
        }
      bool grow = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = top[nt][e];
          t = fmaxf(t, __shfl_xor_sync(kAll, t, 4));
          t = fmaxf(t, __shfl_xor_sync(kAll, t, 8));
          t = fmaxf(t, __shfl_xor_sync(kAll, t, 16));
          top[nt][e] = fmaxf(m[nt][e], t);
          grow |= t > m[nt][e];
        }
      if (__any_sync(kAll, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // both -inf: nothing stands yet, and 0 is kept
            const float keep =
                m[nt][e] == -INFINITY ? 0.f : exp2_fast(m[nt][e] - top[nt][e]);
            m[nt][e] = top[nt][e];
            l[nt][e] *= keep;
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                o[c][j][nt][e] *= keep;
                o[c][j][nt][2 + e] *= keep;
              }
          }
      }
      uint32_t p[2][2][NT];  // P^T fragments: tokens 16u + 8h + 2tq + {0, 1} of column g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float z0 = m[nt][0] == -INFINITY ? 0.f : 14.f - m[nt][0];
        const float z1 = m[nt][1] == -INFINITY ? 0.f : 14.f - m[nt][1];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = exp2_fast(s[u][nt][2 * h] + z0);
            const float p1_ = exp2_fast(s[u][nt][2 * h + 1] + z1);
            l[nt][0] += p0;
            l[nt][1] += p1_;
            p[u][h][nt] = transpose8(pack_half2(p0, p1_));
          }
      }

      // ---- O^T += V^T P^T
      if (!slow) {
        uint32_t low[NW];  // 4 * (reference - 16), a byte to a block
#pragma unroll
        for (int w = 0; w < NW; ++w) low[w] = 4u * (ref[w] - 0x10101010u);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // FP16 2^(s - ref + 1) of tokens (2tq, 2tq + 1) of each half: the exponent field is
          // s - ref + 16, here four times that in the byte it belongs in
          uint32_t d[2][2][NW];  // [half][pair of blocks' word ...]
          uint32_t f01[2][NW], f23[2][NW];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint8_t* sc = buf + u * G::kBytes + G::kVScale + (8 * h + 2 * tq) * CB;
            if constexpr (CB == 2) {
              const uint32_t both = *reinterpret_cast<const uint32_t*>(sc);
              const uint32_t l2 = 4u * (((ref[0] & 0xFFFFu) | (ref[0] << 16)) - 0x10101010u);
              f01[h][0] = 4u * both - l2;
            } else {
              const Words<NW> w0 = lds<NW>(sc), w1 = lds<NW>(sc + CB);
#pragma unroll
              for (int w = 0; w < NW; ++w) {
                d[h][0][w] = 4u * w0.v[w] - low[w];
                d[h][1][w] = 4u * w1.v[w] - low[w];
                f01[h][w] = __byte_perm(d[h][0][w], d[h][1][w], 0x5410);
                f23[h][w] = __byte_perm(d[h][0][w], d[h][1][w], 0x7632);
              }
            }
          }
#pragma unroll
          for (int sl = 0; sl < NS; ++sl) {
            const uint8_t* vb = buf + u * G::kBytes + G::kCodeBytes + sl * G::kSlabBytes +
                                g * 16 * SB + tq * 4 * SB;
            const Words<SB> v0 = lds<SB>(vb), v1 = lds<SB>(vb + 128 * SB);
#pragma unroll
            for (int cp = 0; cp < SB / 2; ++cp) {  // blocks 2cp, 2cp + 1
              // codes of two tokens side by side: channels n = 0, 2 (x) and 1, 3 (y)
              const uint32_t e0 = v0.v[cp], f0 = v0.v[SB / 2 + cp];
              const uint32_t e1 = v1.v[cp], f1 = v1.v[SB / 2 + cp];
              const uint32_t x0 = (e0 & 0x0F0F0F0Fu) | ((f0 << 4) & 0xF0F0F0F0u);
              const uint32_t y0 = ((e0 >> 4) & 0x0F0F0F0Fu) | (f0 & 0xF0F0F0F0u);
              const uint32_t x1 = (e1 & 0x0F0F0F0Fu) | ((f1 << 4) & 0xF0F0F0F0u);
              const uint32_t y1 = ((e1 >> 4) & 0x0F0F0F0Fu) | (f1 & 0xF0F0F0F0u);
              uint32_t a0[4], a1[4], a2[4], a3[4];
              e2m1x8(x0, a0[0], a0[1], a0[2], a0[3]);
              e2m1x8(y0, a1[0], a1[1], a1[2], a1[3]);
              e2m1x8(x1, a2[0], a2[1], a2[2], a2[3]);
              e2m1x8(y1, a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
              for (int cc = 0; cc < 2; ++cc) {
                const int cb = sl * SB + 2 * cp + cc;
                uint32_t sc[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t f = (cb % 4) < 2 ? f01[h][cb / 4] : f23[h][cb / 4];
                  sc[h] = (cb & 1 ? f : f << 8) & 0xFF00FF00u;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const uint32_t b0 = mul_half2(p[u][0][nt], sc[0]);
                  const uint32_t b1 = mul_half2(p[u][1][nt], sc[1]);
#pragma unroll
                  for (int j = 0; j < 2; ++j)
                    mma_f16_acc(o[cb][j][nt], a0[2 * cc + j], a1[2 * cc + j], a2[2 * cc + j],
                                a3[2 * cc + j], b0, b1);
                }
              }
            }
          }
        }
      } else {
        // scales that one FP16 exponent range does not hold, or NaN: product by product
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            for (int t = 0; t < 8; ++t) {
              const int token = 16 * u + 8 * h + t, key = j0 + token;
              if (key >= at.span.end) break;
              const uint8_t* grp = buf + u * G::kBytes;
              float pr[NT][2];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t w = __shfl_sync(kAll, p[u][h][nt], (2 * tq + e) * 4 + (t >> 1));
                  const __half2 both = *reinterpret_cast<const __half2*>(&w);
                  const int row = 8 * nt + 2 * tq + e;
                  const bool seen = key >= lo_sh[row] && key <= hi_sh[row];
                  // what is not seen adds nothing, not even 0 * NaN
                  pr[nt][e] = !seen ? -1.f : (t & 1 ? __high2float(both) : __low2float(both));
                }
#pragma unroll
              for (int c = 0; c < CB; ++c) {
                const uint32_t sv = grp[G::kVScale + (8 * h + t) * CB + c];
                const int rc = (int)((ref[c / 4] >> (8 * (c % 4))) & 0xFFu);
                const float unit = sv == 255u ? __uint_as_float(0x7FC00000u)
                                              : exp2f((float)((int)sv - rc + 1));
                uint32_t v[4];
                e2m1x8(*reinterpret_cast<const uint16_t*>(grp + G::v_half(8 * h + t, c, g)), v[0],
                       v[1], v[2], v[3]);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v[j]));
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                      if (pr[nt][e] >= 0.f || pr[nt][e] != pr[nt][e]) {
                        o[c][j][nt][e] += pr[nt][e] * (x.x * unit);
                        o[c][j][nt][2 + e] += pr[nt][e] * (x.y * unit);
                      }
                }
              }
            }
      }

      // ---- refill the stage
      __syncwarp();
      const int next = k + kStages;
      if ((next & 31) == 0) plan(next);
      if (lane == (next & 31) && begin + warp + (long long)kWarps * next < end) issue(stage);
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float t = l[nt][e];
        t += __shfl_xor_sync(kAll, t, 4);
        t += __shfl_xor_sync(kAll, t, 8);
        t += __shfl_xor_sync(kAll, t, 16);
        if (g == 0) {
          m_sh[warp * kRows + 8 * nt + 2 * tq + e] = m[nt][e];
          l_sh[warp * kRows + 8 * nt + 2 * tq + e] = t;
        }
      }
    __syncthreads();
    if (threadIdx.x < kRows) {
      const int row = threadIdx.x;
      float top = -INFINITY, sum = 0.f;
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_sh[w * kRows + row]);
      for (int w = 0; w < kWarps; ++w) {
        const float f = top == -INFINITY ? 0.f : exp2_fast(m_sh[w * kRows + row] - top);
        // a warp whose keys were all NaN has no maximum but a NaN sum
        const float lw = l_sh[w * kRows + row];
        sum += lw != lw ? lw : lw * f;
        m_sh[w * kRows + row] = f;
      }
      max_sh[row] = top;
      sum_sh[row] = sum;
    }
    __syncthreads();
    const bool alone = p0 == item && p1 == item + at.span.steps;
    const int first_cta = (int)(item / quota);
    const int last_cta = (int)((item + at.span.steps - 1) / quota);
    const long long slot_floats = (long long)kKvMaxRows * (D + 2);
    float* part = a.partial + (2 * (long long)blockIdx.x + (p0 > begin ? 1 : 0)) * slot_floats;
    const auto store_out = [&](int row, int ch, float y) {
      const int flat = at.tile * kRows + row;
      if (flat >= entry.n * group) return;
      const long long o_at = ((long long)(entry.first + flat / group) * a.q_heads + at.head * group +
                              flat % group) * D + ch;
      if (a.half)
        static_cast<__half*>(a.out)[o_at] = __float2half_rn(y);
      else
        static_cast<__nv_bfloat16*>(a.out)[o_at] = __float2bfloat16_rn(y);
    };
    const auto store_lse = [&](int row, float top, float sum) {
      const int flat = at.tile * kRows + row;
      if (!a.lse || flat >= entry.n * group) return;
      a.lse[(long long)(entry.first + flat / group) * a.q_heads + at.head * group + flat % group] =
          sum == 0.f ? -INFINITY : (top - 14.f) * 0.6931471805599453f + logf(sum);
    };
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      const float unit = exp2f((float)((int)((ref[c / 4] >> (8 * (c % 4))) & 0xFFu) - 128));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * nt + 2 * tq + e;
          const float f = m_sh[warp * kRows + row] * unit;
          float* to = merge + (warp * kRows + row) * kPad + 4 * g;
          *reinterpret_cast<float4*>(to) =
              make_float4(o[c][0][nt][e] * f, o[c][0][nt][2 + e] * f, o[c][1][nt][e] * f,
                          o[c][1][nt][2 + e] * f);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < kRows * 32; i += kThreads) {
        const int row = i >> 5, ch = i & 31;
        float y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) y += merge[(w * kRows + row) * kPad + ch];
        if (alone)
          store_out(row, 32 * c + ch, sum_sh[row] == 0.f ? 0.f : y / sum_sh[row]);
        else
          part[row * D + 32 * c + ch] = y;
      }
      __syncthreads();
    }
    if (alone) {
      if (threadIdx.x < kRows) store_lse(threadIdx.x, max_sh[threadIdx.x], sum_sh[threadIdx.x]);
    } else {
      if (threadIdx.x < kRows) {
        part[kRows * D + threadIdx.x] = max_sh[threadIdx.x];
        part[kRows * D + kRows + threadIdx.x] = sum_sh[threadIdx.x];
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0)
        last_sh = atomicAdd(a.counters + first_cta, 1u) == (uint32_t)(last_cta - first_cta);
      __syncthreads();
      if (last_sh) {
        // every part is there: join them in their order
        __threadfence();
        if (threadIdx.x == 0) a.counters[first_cta] = 0;
        const auto part_of = [&](int x) {
          return a.partial + (2 * (long long)x + (item > x * quota ? 1 : 0)) * slot_floats;
        };
        if (threadIdx.x < kRows) {
          float top = -INFINITY, sum = 0.f;
          for (int x = first_cta; x <= last_cta; ++x)
            top = fmaxf(top, __ldcg(part_of(x) + kRows * D + threadIdx.x));
          for (int x = first_cta; x <= last_cta; ++x) {
            const float mx = __ldcg(part_of(x) + kRows * D + threadIdx.x);
            const float lx = __ldcg(part_of(x) + kRows * D + kRows + threadIdx.x);
            sum += lx != lx ? lx : lx * (top == -INFINITY ? 0.f : exp2_fast(mx - top));
          }
          max_sh[threadIdx.x] = top;
          sum_sh[threadIdx.x] = sum;
          store_lse(threadIdx.x, top, sum);
        }
        __syncthreads();
        for (int i = threadIdx.x; i < kRows * D; i += kThreads) {
          const int row = i / D;
          const float top = max_sh[row];
          float y = 0.f;
          for (int x = first_cta; x <= last_cta; ++x) {
            const float mx = __ldcg(part_of(x) + kRows * D + row);
            y += __ldcg(part_of(x) + i) * (top == -INFINITY ? 0.f : exp2_fast(mx - top));
          }
          store_out(row, i % D, sum_sh[row] == 0.f ? 0.f : y / sum_sh[row]);
        }
      }
    }
    p0 = p1;
  }
  if (dead) {
    // give up, but not before the copies in flight have landed (or as long again has passed)
    for (int s = 0; s < kStages; ++s) mbar_wait(bar + 8 * s, s >= stage ? phase : phase ^ 1u);
  }
}

template <int D, int NT>
cudaError_t run(const KvAttentionArgs& a, cudaStream_t s) {
  using L = Shape<D, NT>;
  const int bytes = L::kPrefix + 8 * (a.batch.entries + 1);
  const void* fn = reinterpret_cast<const void*>(kv_attention<D, NT>);
  cudaError_t e = ensure_dynamic_smem(fn, bytes);
  if (e != cudaSuccess) return e;
  const int sms = kKvMaxCtas / 2;
  kv_attention<D, NT><<<sms * L::kCtasPerSm, kThreads, bytes, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t s) {
  const int rows = (int)((long long)a.max_q * (a.q_heads / a.cache.kv_heads) > 32
                             ? 32 : a.max_q * (a.q_heads / a.cache.kv_heads));
  switch (a.cache.head_dim) {
    case 64: return rows <= 8 ? run<64, 1>(a, s) : rows <= 16 ? run<64, 2>(a, s) : run<64, 4>(a, s);
    case 128:
      return rows <= 8 ? run<128, 1>(a, s) : rows <= 16 ? run<128, 2>(a, s) : run<128, 4>(a, s);
    default: return rows <= 8 ? run<256, 1>(a, s) : run<256, 2>(a, s);
  }
}

}  // namespace wd
