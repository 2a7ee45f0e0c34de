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
//   - P = 2^8 exp2(x - m) is rounded to FP16 once; the row sums are of the unrounded values, in
//     FP32.  m follows the running maximum only when that has grown by more than 2^6, so that
//     hardly any step has to rescale what stands on it: P stays below 2^14 and has its 11 bits
//     down to 2^-22 of 2^m (2^-16 of the largest at worst) and an error of 2^-33 of 2^m below.
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
constexpr int kCached = 256;  // entries whose slot and length are kept in shared memory
constexpr float kBias = 8.f;  // P = 2^kBias at the reference m ...
constexpr float kSlack = 6.f; // ... which may fall this far behind the maximum (log2)
constexpr uint32_t kAll = 0xFFFFFFFFu;

template <int D, int NT>
struct Shape {
  using G = KvGroup<D>;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * G::kBytes;
  static constexpr int kStages = D == 64 ? 4 : 2;
  static constexpr int kCtasPerSm = D <= 128 && NT == 1 ? 2 : 1;
  // the warps' outputs are joined through shared memory, in one round where it has room for all
  static constexpr int kRounds = D == 256 ? 2 * NT : D == 128 && NT == 4 ? 2 : 1;
  static constexpr int kRoundBlocks = G::kBlocks / kRounds;
  static constexpr int kMergeRow = 32 * kRoundBlocks + 4;  // floats
  // shared memory, in bytes from its start
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kWarps * kStages * kStageBytes;  // fragments [NT][blocks][32] uint4
  static constexpr int kQBytes = NT * G::kBlocks * 512;                // twice: this segment's, the next's
  static constexpr int kMerge = kQ + 2 * kQBytes;  // float [kWarps][kRows][kMergeRow]
  static constexpr int kStats = kMerge + kWarps * kRows * kMergeRow * 4;  // float m, l [kWarps][kRows]
  static constexpr int kRowInfo = kStats + 2 * kWarps * kRows * 4;   // twice: factor, lo, hi [kRows]
  static constexpr int kBars = kRowInfo + 2 * 3 * kRows * 4;         // uint64 [kWarps][kStages]
  static constexpr int kScan = kBars + kWarps * kStages * 8;         // long long [kWarps], int [kWarps][8]
  static constexpr int kPrefix = kScan + kWarps * 8 + kWarps * 32;   // long long [entries + 1]
  static constexpr int shared_bytes(int entries) {  // ... and int2 [min(entries, kCached)]
    return kPrefix + 8 * (entries + 1) + 8 * (entries < kCached ? entries : kCached);
  }
  static_assert(kPrefix + 8 * (WD_KV_MAX_ENTRIES + 1) + 8 * kCached <= 227 * 1024, "shared memory");
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

// What of the sequence one entry of the batch works on.
struct Entry {
  int slot, len, first, n;
};

// The steps of keys that a tile of query rows sees: at least one, so that a tile that sees
// nothing is written too.
struct Span {
  int first, steps;  // in steps of kStep keys
  int end;           // keys from here on are not seen
};
template <int kRows>
__device__ __forceinline__ Span tile_span(const Entry& e, int tile, int group, int window) {
  int i0 = 0, i1 = e.n - 1;
  if (e.n > 1) {
    i0 = tile * kRows / group;
    i1 = min(i1, (tile * kRows + kRows - 1) / group);
  }
  const int hi = e.len - e.n + i1;
  const int lo = window > 0 ? max(0, e.len - e.n + i0 - window + 1) : 0;
  Span s;
  s.first = lo / kStep;
  s.steps = hi < 0 ? 1 : max(1, hi / kStep + 1 - s.first);
  s.end = hi + 1;
  return s;
}
template <int kRows>
__device__ __forceinline__ int tiles_of(const Entry& e, int group) {
  return (e.n * group + kRows - 1) / kRows;
}

// All steps of the call in a row: entries, their tiles, the key heads, the item's steps (rounded
// up to a multiple of `pad`).
struct Order {
  const long long* prefix;  // steps of the entries before each entry
  const int2* cached;       // slot and length of the first kCached entries
  int pad, group;
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
struct Place {
  int entry, tile, head, step;
  Span span;
  int padded;  // steps with the padding
};
template <int kRows>
__device__ __forceinline__ Place locate(const KvAttentionArgs& a, const Order& o, long long p,
                                        Entry& e) {
  int lo = 0, hi = a.batch.entries;  // the last entry whose steps begin at or before p
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (o.prefix[mid] <= p) lo = mid; else hi = mid;
  }
  Place at;
  at.entry = lo;
  e = load_entry(a, lo, o.cached);
  long long rest = p - o.prefix[lo];
  const int heads = a.cache.kv_heads;
  // (the last tile and head are also where it ends if someone rewrites the lengths meanwhile)
  const int tiles = max(1, tiles_of<kRows>(e, o.group));
  for (at.tile = 0;; ++at.tile) {
    at.span = tile_span<kRows>(e, at.tile, o.group, a.window);
    at.padded = (at.span.steps + o.pad - 1) / o.pad * o.pad;
    const long long cost = (long long)at.padded * heads;
    if (rest < cost || at.tile + 1 == tiles) break;
    rest -= cost;
  }
  at.head = min((int)((uint32_t)rest / (uint32_t)at.padded), heads - 1);
  at.step = (int)((uint32_t)rest % (uint32_t)at.padded);
  return at;
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

// Part of an item that one CTA has done, and where the whole item's output goes.
struct Part {
  long long item;           // the item's first step
  int first_cta, last_cta;  // that have parts of it
  int tile, head, first, n;
};
// Where CTA x leaves its part: it has at most two, the first if the item began before it.
__device__ __forceinline__ float* part_at(const KvAttentionArgs& a, const Part& p, int x,
                                          int quota) {
  const long long slot = 2 * (long long)x + (p.item > (long long)x * quota ? 1 : 0);
  return a.partial + slot * kKvMaxRows * (a.cache.head_dim + 2);
}

// Four channels of a finished row: y / sum, and with the first of them the row's lse.
template <int D, int kRows>
__device__ __forceinline__ void store_row(const KvAttentionArgs& a, const Part& p, int row, int ch,
                                          const float4& y, float top, float sum) {
  const int group = a.q_heads / a.cache.kv_heads;
  const int flat = p.tile * kRows + row;
  if (flat >= p.n * group) return;
  const long long at =
      (long long)(p.first + flat / group) * a.q_heads + p.head * group + flat % group;
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
  long long* scan = reinterpret_cast<long long*>(smem + L::kScan);
  int* scan2 = reinterpret_cast<int*>(scan + kWarps);
  long long* prefix = reinterpret_cast<long long*>(smem + L::kPrefix);
  int2* cached = reinterpret_cast<int2*>(prefix + a.batch.entries + 1);
  uint8_t* ring = smem + L::kRing + warp * kStages * L::kStageBytes;
  const uint32_t bar = smem_u32(smem + L::kBars) + warp * kStages * 8;
  __shared__ Part parts_sh[2];
  __shared__ int last_sh[2];

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    mbar_init_fence();
  }
  // The division of the work.  Where there are no more items than CTAs, each item gets CTAs of
  // its own (its steps are padded to a multiple of a CTA's), so that a CTA has one item to do;
  // else the CTAs' ranges cross the items' bounds and are all of the same length.  A CTA takes at
  // least kLeast rounds of its warps where an item has as many: fewer would only add parts to
  // join, and a join through memory costs as much as two rounds.
  constexpr int kLeast = 3;
  constexpr int kTries = kWarps;
  Order order{prefix, cached, 1, group};
  Entry own{-1, 0, 0, 0};
  if ((int)threadIdx.x < a.batch.entries) own = load_entry(a, threadIdx.x);
  long long total = 0;
  int longest = 0, items = 0;
  {
    long long steps_here = 0;
    for (int b = threadIdx.x; b < a.batch.entries; b += kThreads) {
      const Entry e = b < kThreads ? own : load_entry(a, b);
      if (b < kCached) cached[b] = make_int2(e.slot, e.len);
      const int tiles = tiles_of<kRows>(e, group);
      for (int t = 0; t < tiles; ++t) {
        const int steps = tile_span<kRows>(e, t, group, a.window).steps;
        steps_here += steps;
        longest = max(longest, steps);
      }
      items += tiles * heads;
    }
    steps_here *= heads;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) steps_here += __shfl_xor_sync(kAll, steps_here, off);
    longest = __reduce_max_sync(kAll, longest);
    items = __reduce_add_sync(kAll, min(items, 1 << 24));
    if (lane == 0) {
      scan[warp] = steps_here;
      scan2[8 + 2 * warp] = longest;
      scan2[9 + 2 * warp] = items;
    }
    __syncthreads();
    items = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      total += scan[w];
      longest = max(longest, scan2[8 + 2 * w]);
      items += min(scan2[9 + 2 * w], 1 << 24);
    }
  }
  const long long rounds = (total + (long long)gridDim.x * kWarps - 1) /
                           ((long long)gridDim.x * kWarps);
  int quota = (int)max(rounds, 1ll) * kWarps;
  if (items <= (int)gridDim.x) {
    // the shortest of some quotas at which the CTAs suffice
    const int lowest = max(quota, min(kLeast, (longest + kWarps - 1) / kWarps) * kWarps);
    const auto try_quota = [&](int i) {  // times 16, 17, 18, 20, 24, 32, 48, 64 sixteenths
      const int by = i < 3 ? 16 + i : i < 5 ? 12 + 4 * (i - 1) : i < 6 ? 32 : 16 * (i - 3);
      return (int)((((long long)lowest * by >> 4) + kWarps - 1) >> 3 << 3);
    };
    if (longest <= lowest) {  // no item needs two CTAs
      order.pad = quota = lowest;
    } else {
      const unsigned q = try_quota(warp);  // a warp to each
      int need = 0;
      for (int b = lane; b < a.batch.entries; b += 32) {
        const Entry e = load_entry(a, b, cached);
        const int tiles = tiles_of<kRows>(e, group);
        for (int t = 0; t < tiles; ++t)
          need += (int)((unsigned)tile_span<kRows>(e, t, group, a.window).steps + q - 1) / q;
      }
      need = __reduce_add_sync(kAll, need);
      if (lane == 0) scan2[warp] = need;
      __syncthreads();
#pragma unroll
      for (int i = kTries - 1; i >= 0; --i)
        if ((long long)scan2[i] * heads <= (long long)gridDim.x) order.pad = quota = try_quota(i);
    }
  }
  // prefix[b] = steps, with the padding, of the entries before b
  total = 0;
  for (int base = 0; base < a.batch.entries; base += kThreads) {
    const int b = base + threadIdx.x;
    long long cost = 0;
    if (b < a.batch.entries) {
      const Entry e = b < kThreads ? own : load_entry(a, b);
      const int tiles = tiles_of<kRows>(e, group);
      for (int t = 0; t < tiles; ++t)
        cost += (tile_span<kRows>(e, t, group, a.window).steps + order.pad - 1) / order.pad * order.pad;
      cost *= heads;
    }
    long long incl = cost;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long t = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += t;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    long long below = total, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) below += scan[w];
      all += scan[w];
    }
    if (b < a.batch.entries) prefix[b] = below + incl - cost;
    total += all;
  }
  if (threadIdx.x == 0) prefix[a.batch.entries] = total;
  __syncthreads();
  const long long begin = (long long)blockIdx.x * quota;
  if (begin >= total) return;
  const int mine = (int)min(total - begin, (long long)quota);  // steps of this CTA

  // The warp's steps are warp, warp + kWarps, ... of the CTA's: its k-th step's groups are
  // worked out by lane k % 32, 32 steps at a time, and copied into stage k % kStages.
  const uint8_t *src0 = nullptr, *src1 = nullptr;
  uint32_t bytes0 = 0;
  const auto plan = [&](int k0) {
    const int r = warp + kWarps * (k0 + lane);
    src0 = src1 = nullptr;
    bytes0 = 0;
    if (r >= mine) return;
    Entry e;
    const Place at = locate<kRows>(a, order, begin + r, e);
    const int pos = (at.span.first + at.step) * kStep;
    if (at.step >= at.span.steps || pos >= at.span.end) return;
    src0 = kv_group(cache, kv_page(cache, e.slot, pos >> cache.page_shift), a.layer, at.head, pos,
                    G::kBytes);
    bytes0 = G::kBytes;
    if (pos + 16 < at.span.end) {
      if (cache.page_size >= kStep)  // the step lies within a page, its groups side by side
        bytes0 = 2 * G::kBytes;
      else
        src1 = kv_group(cache, kv_page(cache, e.slot, (pos + 16) >> cache.page_shift), a.layer,
                        at.head, pos + 16, G::kBytes);
    }
  };
  const uint32_t ring_at = smem_u32(ring);
  const auto issue = [&](int stage) {
    const uint32_t to = ring_at + stage * L::kStageBytes, full = bar + 8 * stage;
    mbar_arrive_expect_tx(full, bytes0 + (src1 ? G::kBytes : 0));
    if (bytes0) bulk_g2s_nohint(to, src0, bytes0, full);
    if (src1) bulk_g2s_nohint(to + G::kBytes, src1, G::kBytes, full);
  };

  const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.q_token % 8 == 0 &&
                   a.q_head % 8 == 0;
  int r = warp;  // the warp's next step, of the CTA's
  int k = 0, stage = 0;
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out
  // refill the stage that the k-th step has used, and go on to the next
  const auto issue_next = [&]() {
    __syncwarp();
    const int next = k + kStages;
    if ((next & 31) == 0) plan(next);
    if (lane == (next & 31) && warp + kWarps * next < mine) issue(stage);
    __syncwarp();
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  };
  // A tile's queries as fragments: channel 32c + 8t + 4j + 2i + {0,1} of row 8nt + g is register
  // i of product j in lane 4g + t.  Four lanes to a block of 32 channels.
  constexpr int kQueryPasses = (kRows * (D / 8) + kThreads - 1) / kThreads;
  Words<4> query[kQueryPasses];
  const auto fetch_queries = [&](const Place& at, const Entry& entry) {
    const int rows = entry.n * group - at.tile * kRows;  // of the tile's, those that are real
#pragma unroll
    for (int pass = 0; pass < kQueryPasses; ++pass) {
      const int i = threadIdx.x + pass * kThreads;
      const int row = i / (D / 8), e8 = i % (D / 8);
      const int flat = at.tile * kRows + row;
      query[pass] = Words<4>{{0u, 0u, 0u, 0u}};
      if (row < kRows && row < rows)
        query[pass] = load8(a, (entry.first + flat / group) * a.q_token +
                                   (at.head * group + flat % group) * a.q_head + 8 * e8, vec);
    }
  };
  const auto put_queries = [&](const Place& at, const Entry& entry, int which) {
    const int rows = entry.n * group - at.tile * kRows;
    float* factor_sh = reinterpret_cast<float*>(smem + L::kRowInfo) + which * 3 * kRows;
    int* lo_sh = reinterpret_cast<int*>(factor_sh + kRows);
    int* hi_sh = lo_sh + kRows;
#pragma unroll
    for (int pass = 0; pass < kQueryPasses; ++pass) {
      const int i = threadIdx.x + pass * kThreads;
      const int row = i / (D / 8), e8 = i % (D / 8);
      if (row >= kRows) break;  // (whole warps)
      float x[8];
      widen8(query[pass], a.half, x);
      uint32_t bits = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) bits = max(bits, __float_as_uint(x[q]) & 0x7FFFFFFFu);
#pragma unroll
      for (int off = 1; off < D / 8; off <<= 1)
        bits = max(bits, __shfl_xor_sync(kAll, bits, off));
      // 2^k brings the largest magnitude into [2^14, 2^15); subnormals are scaled as if 2^-126
      const bool bad = bits >= 0x7F800000u;
      const int k2 = bad || bits == 0u ? 0 : 14 - (max((int)(bits >> 23), 1) - 127);
      const float up = exp2_int(k2 / 2), up2 = exp2_int(k2 - k2 / 2);
      uint4 f;
      f.x = pack_half2(x[0] * up * up2, x[1] * up * up2);
      f.y = pack_half2(x[2] * up * up2, x[3] * up * up2);
      f.z = pack_half2(x[4] * up * up2, x[5] * up * up2);
      f.w = pack_half2(x[6] * up * up2, x[7] * up * up2);
      *reinterpret_cast<uint4*>(smem + L::kQ + which * L::kQBytes +
                                (((row >> 3) * CB + (e8 >> 2)) * 32 + (row & 7) * 4 + (e8 & 3)) * 16) = f;
      if (e8 == 0) {
        const int pos = entry.len - entry.n + (at.tile * kRows + row) / group;
        // a row with an infinity or NaN has no finite logit; never 0, so that -inf stays -inf
        factor_sh[row] = bad ? __uint_as_float(0x7FC00000u)
                             : fmaxf(a.scale * 1.4426950408889634f / up / up2, 1.2e-38f);
        const bool real = row < rows;  // no row: nothing to hide, never stored
        lo_sh[row] = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
        hi_sh[row] = real ? pos : at.span.end - 1;
      }
    }
  };
  Entry entry;
  Place at = locate<kRows>(a, order, begin, entry);
  fetch_queries(at, entry);
  plan(0);
  if (lane < kStages && warp + kWarps * lane < mine) issue(lane);
  __syncwarp();
  put_queries(at, entry, 0);
  __syncthreads();
  int pending = 0;  // parts of items that other CTAs have parts of: at most the first and the last
  for (int r0 = 0, which = 0; r0 < mine; which ^= 1) {
    const int r1 = min(mine, r0 + at.padded - at.step);  // the segment is [r0, r1)
    const uint8_t* q_sh = smem + L::kQ + which * L::kQBytes;
    const float* factor_sh = reinterpret_cast<const float*>(smem + L::kRowInfo) + which * 3 * kRows;
    const int* lo_sh = reinterpret_cast<const int*>(factor_sh + kRows);
    const int* hi_sh = lo_sh + kRows;

    uint4 qf[kQInRegs ? CB : 1];
    if constexpr (kQInRegs) {
#pragma unroll
      for (int c = 0; c < CB; ++c)
        qf[c] = *reinterpret_cast<const uint4*>(q_sh + (c * 32 + lane) * 16);
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

    for (; r < r1; r += kWarps, ++k) {
      const int step = at.step + r - r0;
      if (step >= at.span.steps) break;  // padding: the CTA has no other item
      const int j0 = (at.span.first + step) * kStep;
      if (dead) break;
      const bool landed = mbar_wait(bar + 8 * stage, phase);
      const uint8_t* buf = ring + stage * L::kStageBytes;

      // ---- S^T = K Q^T
      float s[2][NT][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][nt][e] = 0.f;
      uint32_t kf[2][2][CB / 2];  // the scales of keys 16u + 8h + g, BF16, two blocks to a word
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const Words<NW> w = lds_scales<CB>(buf + u * G::kBytes + G::kKScale + (8 * h + g) * CB);
#pragma unroll
          for (int c = 0; c < CB / 2; ++c) kf[u][h][c] = e8m0x2(w.v[c / 2] >> (16 * (c & 1)));
        }
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
                                   q_sh + ((nt * CB + cb) * 32 + lane) * 16);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
            e2m1x8(kw[u][0].v[c], a0, a2, b0, b2);
            e2m1x8(kw[u][1].v[c], a1, a3, b1, b3);
            const float s0 = __uint_as_float(cb & 1 ? kf[u][0][cb / 2] & 0xFFFF0000u
                                                    : kf[u][0][cb / 2] << 16);
            const float s1 = __uint_as_float(cb & 1 ? kf[u][1][cb / 2] & 0xFFFF0000u
                                                    : kf[u][1][cb / 2] << 16);
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

      // ---- does anything change: a larger logit, a V scale out of range, keys behind the end?
      const bool whole = j0 >= seen_lo && j0 + kStep - 1 <= seen_hi;
      float top[NT][2];
      bool odd = !landed;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float t = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& x = s[u][nt][2 * h + e];
              if (!whole) {
                const int row = 8 * nt + 2 * tq + e, key = j0 + 16 * u + 8 * h + g;
                if (key < lo_sh[row] || key > hi_sh[row]) x = -INFINITY;
              }
              t = fmaxf(t, x);
            }
          top[nt][e] = t * factor[nt][e];
          odd |= top[nt][e] > m[nt][e] + kSlack;
        }
      // the V scales of key j0 + lane: all within [r - 15, r]?
      const bool inside = j0 + lane < at.span.end;
      Words<NW> vt = lds_scales<CB>(buf + (lane >> 4) * G::kBytes + G::kVScale + (lane & 15) * CB);
      const auto out_of_range = [&]() {
        bool bad = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const uint32_t v = CB == 2 ? vt.v[w] | (ref[w] & 0xFFFF0000u) : vt.v[w];
          const uint32_t t0 = ((ref[w] & 0x00FF00FFu) | 0x80008000u) - (v & 0x00FF00FFu);
          const uint32_t t1 = (((ref[w] >> 8) & 0x00FF00FFu) | 0x80008000u) - ((v >> 8) & 0x00FF00FFu);
          bad |= ((t0 | t1) & 0x7FF07FF0u) != 0u;
        }
        return bad;
      };
      odd |= inside ? out_of_range() : true;
      bool slow = false;
      if (__any_sync(kAll, odd)) {
        if (__any_sync(kAll, !landed)) {
          dead = true;
          if (lane == 0) atomicOr(cache.flag, WD_KV_FLAG_TIMEOUT);
          break;
        }
        // the maxima, and what stands on them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = fmaxf(m[nt][e], top[nt][e]);
            t = fmaxf(t, __shfl_xor_sync(kAll, t, 4));
            t = fmaxf(t, __shfl_xor_sync(kAll, t, 8));
            t = fmaxf(t, __shfl_xor_sync(kAll, t, 16));
            if (t <= m[nt][e] + kSlack) t = m[nt][e];
            // both -inf: nothing stands yet
            const float keep = m[nt][e] == -INFINITY ? 0.f : exp2_fast(m[nt][e] - t);
            // (a NaN that stands there stays: a sum of NaN is not forgotten)
            l[nt][e] = m[nt][e] == -INFINITY ? l[nt][e] : l[nt][e] * keep;
            m[nt][e] = t;
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                o[c][j][nt][e] *= keep;
                o[c][j][nt][2 + e] *= keep;
              }
          }
        // the largest V scales, and what stands on them
        if (__any_sync(kAll, inside && out_of_range())) {
          bool bad = false;
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            const uint32_t sh = 8 * (c % 4), mine_c = (vt.v[c / 4] >> sh) & 0xFFu;
            const uint32_t old = (ref[c / 4] >> sh) & 0xFFu;
            const uint32_t most =
                max(old, __reduce_max_sync(kAll, inside && mine_c != 255u ? mine_c : 0u));
            if (most != old) {
              const float down = exp2_fast((float)(int)old - (float)(int)most);
#pragma unroll
              for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int e = 0; e < 4; ++e) o[c][j][nt][e] *= down;
              ref[c / 4] = (ref[c / 4] & ~(0xFFu << sh)) | (most << sh);
            }
            bad |= inside && (mine_c > most || mine_c + 15u < most);
          }
          slow = __any_sync(kAll, bad);
        }
        // keys behind the end get scales in range; their probabilities are zero
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

      // ---- P = 2^kBias exp2(x - m)
      uint32_t p[2][2][NT];  // P^T fragments: tokens 16u + 8h + 2tq + {0, 1} of column g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float z0 = m[nt][0] == -INFINITY ? 0.f : kBias - m[nt][0];
        const float z1 = m[nt][1] == -INFINITY ? 0.f : kBias - m[nt][1];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float p0 = exp2_fast(fmaf(s[u][nt][2 * h], factor[nt][0], z0));
            const float p1 = exp2_fast(fmaf(s[u][nt][2 * h + 1], factor[nt][1], z1));
            l[nt][0] += p0;
            l[nt][1] += p1;
            p[u][h][nt] = transpose8(pack_half2(p0, p1));
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

      issue_next();
    }

    // ---- join the warps
    if (r0 > 0) __syncthreads();  // the segment before has been read
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
    const auto write_round = [&](int round) {
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const int cr = c - round * L::kRoundBlocks;
        if (cr < 0 || cr >= L::kRoundBlocks) continue;
        const float unit = exp2_int((int)((ref[c / 4] >> (8 * (c % 4))) & 0xFFu) - 128);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(
                merge + (warp * kRows + 8 * nt + 2 * tq + e) * L::kMergeRow + 32 * cr + 4 * g) =
                make_float4(o[c][0][nt][e] * unit, o[c][0][nt][2 + e] * unit,
                            o[c][1][nt][e] * unit, o[c][1][nt][2 + e] * unit);
      }
    };
    write_round(0);
    Part part;
    part.item = begin + r0 - at.step;
    part.first_cta = (int)(part.item / quota);
    part.last_cta = (int)((part.item + at.padded - 1) / quota);
    part.tile = at.tile;
    part.head = at.head;
    part.first = entry.first;
    part.n = entry.n;
    const bool alone = at.step == 0 && r1 - r0 == at.padded;
    float* to = part_at(a, part, blockIdx.x, quota);
    if (!alone) {
      if (threadIdx.x == 0) parts_sh[pending] = part;
      ++pending;
    }
    // what comes next, while the slower warps finish
    if (r1 < mine) {
      at = locate<kRows>(a, order, begin + r1, entry);
      fetch_queries(at, entry);
      put_queries(at, entry, which ^ 1);
    }
#pragma unroll
    for (int round = 0; round < L::kRounds; ++round) {
      if (round > 0) {
        __syncthreads();
        write_round(round);
      }
      __syncthreads();
      constexpr int kQuads = 8 * L::kRoundBlocks;  // four channels each, of a row
      for (int i = threadIdx.x; i < kRows * kQuads; i += kThreads) {
        const int row = i / kQuads, ch = 4 * (i % kQuads);
        float mw[kWarps], top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          mw[w] = m_sh[w * kRows + row];
          top = fmaxf(top, mw[w]);
        }
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = top == -INFINITY ? 0.f : exp2_fast(mw[w] - top);
          const float lw = l_sh[w * kRows + row];
          // a warp whose keys were all NaN has no maximum, but a NaN sum
          sum += lw != lw ? lw : lw * f;
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * kRows + row) * L::kMergeRow + ch);
          y.x = fmaf(v.x, f, y.x);
          y.y = fmaf(v.y, f, y.y);
          y.z = fmaf(v.z, f, y.z);
          y.w = fmaf(v.w, f, y.w);
        }
        const int at_ch = 32 * round * L::kRoundBlocks + ch;
        if (alone) {
          store_row<D, kRows>(a, part, row, at_ch, y, top, sum);
        } else {
          __stcg(reinterpret_cast<float4*>(to + row * D + at_ch), y);
          if (at_ch == 0) {
            __stcg(to + kRows * D + row, top);
            __stcg(to + kRows * D + kRows + row, sum);
          }
        }
      }
    }
    r0 = r1;
  }
  if (pending > 0) {
    // the CTA that arrives last at an item joins its parts, in their order
    __syncthreads();
    if (threadIdx.x < pending) {
      __threadfence();
      const Part part = parts_sh[threadIdx.x];
      const uint32_t others = (uint32_t)(part.last_cta - part.first_cta);
      const bool last = atomicAdd(a.counters + part.first_cta, 1u) == others;
      if (last) a.counters[part.first_cta] = 0;
      __threadfence();
      last_sh[threadIdx.x] = last;
    }
    __syncthreads();
    for (int which = 0; which < pending; ++which) {
      if (!last_sh[which]) continue;
      const Part part = parts_sh[which];
      const int parts = part.last_cta - part.first_cta + 1;
      for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
        const int row = i / (D / 4), ch = 4 * (i % (D / 4));
        float top = -INFINITY, sum = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 8;  // parts on their way at a time
        for (int x0 = 0; x0 < parts; x0 += kBatch) {
          float mx[kBatch], lx[kBatch];
          float4 v[kBatch];
#pragma unroll
          for (int x = 0; x < kBatch; ++x) {
            mx[x] = -INFINITY;
            lx[x] = 0.f;
            v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (x0 + x < parts) {
              const float* from = part_at(a, part, part.first_cta + x0 + x, quota);
              mx[x] = __ldcg(from + kRows * D + row);
              lx[x] = __ldcg(from + kRows * D + kRows + row);
              v[x] = __ldcg(reinterpret_cast<const float4*>(from + row * D + ch));
            }
          }
          float next = top;
#pragma unroll
          for (int x = 0; x < kBatch; ++x) next = fmaxf(next, mx[x]);
          const float keep = top == -INFINITY ? 0.f : exp2_fast(top - next);
          if (x0 > 0) {
            sum = sum != sum ? sum : sum * keep;
            y.x *= keep;
            y.y *= keep;
            y.z *= keep;
            y.w *= keep;
          }
          top = next;
#pragma unroll
          for (int x = 0; x < kBatch; ++x) {
            const float f = top == -INFINITY ? 0.f : exp2_fast(mx[x] - top);
            sum += lx[x] != lx[x] ? lx[x] : lx[x] * f;
            y.x = fmaf(v[x].x, f, y.x);
            y.y = fmaf(v[x].y, f, y.y);
            y.z = fmaf(v[x].z, f, y.z);
            y.w = fmaf(v[x].w, f, y.w);
          }
        }
        store_row<D, kRows>(a, part, row, ch, y, top, sum);
      }
    }
  }
  if (dead) {
    // give up, but not before the copies in flight have landed (or as long again has passed)
    for (int s = 0; s < kStages; ++s) mbar_wait(bar + 8 * s, s >= stage ? phase : phase ^ 1u);
  }
}

template <int D, int NT>
cudaError_t run(const KvAttentionArgs& a, cudaStream_t s) {
  using L = Shape<D, NT>;
  const int bytes = L::shared_bytes(a.batch.entries);
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
