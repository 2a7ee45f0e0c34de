// wd_kv_attention.cu - attention over the 4-bit cache (declared in include/wd_kv.h).
//
// Work.  An item is (entry, tile of 8 * NT query rows, key head); the rows of a tile are the
// heads that share the key head and, behind them, further new tokens.  An item is cut into pieces
// of q steps of 32 keys, a warp to a piece, and the pieces of the call, in order, are dealt out
// to the warps of as many CTAs as fit the GPU (twelve or eight pieces to a CTA, in several passes if
// they are many).  The lengths are known to the device alone, so every CTA derives q and the whole
// division from them; a captured graph can be replayed while the sequences grow.  A warp that
// has all of an item writes its output; the pieces of one CTA meet in shared memory; and where an
// item has pieces in several CTAs, each leaves a partial result (maximum, sum, output) in
// the workspace, and the CTA that arrives last joins them in their order.
//
// A step.  Each warp streams its steps' groups (2176 bytes per 16 keys at head_dim 128) with
// bulk copies into a ring of its own.  With K as the left operand, S^T = K Q^T and O^T = V^T P^T
// are m16n8k16 products whose 16 rows are keys or channels and whose 8 columns are query rows,
// so eight query heads fill a tile, where a 16-row query tile would be half empty.  The groups are
// stored in fragment order: one 16-byte shared-memory read per lane brings 32 codes, which the
// hardware conversion turns into FP16 (exactly) in place.
//   - K: the sums over a block of 32 channels are scaled by the block's 2^(s-127) in FP32, with it by what the
//     softmax scale x log2 e is of a power of two, and by 2^-26, so that no finite keys leave FP32
//     here.  The rows' own factors are then powers of two: a logit and the maximum are exact products, and
//     their difference is right however large they are.
//   - Queries are FP16 x 2^k with k per row (exact for BF16 and FP16 within 2^31 of the row's
//     largest magnitude), 2^-k folded into the softmax scale.
//   - P = 2^8 exp2(x - m) is rounded to FP16 once; the row sums are of the unrounded values, in
//     FP32.  m follows the running maximum only when that has grown by more than 2^6, so that
//     hardly any step has to rescale what stands on it: P stays below 2^14 and has its 11 bits
//     down to 2^-22 of 2^m (2^-16 of the largest at worst) and an error of 2^-33 of 2^m below.
//   - V: the scales lie along the channels that are the product's rows, so each of P's
//     columns is multiplied by 2^(s - r + 1) for every block, with r the largest scale that the warp
//     has met for that block of channels (keys that some rows do not see raise it to 2^23 at most, and
//     what no row sees does not): 2^(s - r + 1) is a normal FP16 number while s >= r - 15, and a product that
//     is not one, of P below 1 (2^-8 of the reference), is off by 2^-25 at most.  A step that holds other
//     scales (or NaN) adds its products one by one in FP32 instead.
//
// What bounds it.  A key head's 32 keys cost 4352 bytes and, in each warp, about 620 instructions,
// half of them on the pipe that converts codes, permutes and compares; so neither the memory (50 %
// busy) nor that pipe (53 %) nor the tensor cores (23 %) is full, and twelve warps to an SM do
// not hide each other's latencies.  Measured (BF16, head_dim 128, 8 query heads to a key
// head): 4 sequences of up to 131,072 keys, 4 key heads 57.6 us, 4.35 TB/s, 0.64 of the copy rate;
// 32 sequences of up to 8192 21.4 us; one of 517 9.4 us, of which 5 us find the work
// and read the first page, 1.5 us are the launch and the rest is one step and the join.
#include "wd_kv_attention.cuh"

namespace wd {
namespace {

template <int D, int NT>
struct Shape {
  using G = KvGroup<D>;
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * G::kBytes;
  static constexpr int kStages = 2;
  // (12 warps of 168 registers: 4 x 131k keys 60.8 us, two CTAs of 8 warps of 128 68.6; 10 warps
  // at NT = 2 and head_dim 128: 35.2 us, 8 warps 32.6)
  static constexpr int kWarps = D <= 128 && NT == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtasPerSm = D == 64 && NT == 2 ? 2 : 1;
  // One tile of queries fits the registers; more are shared by the CTA's warps, whose
  // pieces are then always of one item.
  static constexpr bool kShared = NT > 1;
  // groups of a step whose products run side by side, as far as the registers go (4 x 131k keys:
  // one 58.2 us, two 56.1)
  static constexpr int kTogether = NT == 1 || (NT == 2 && D <= 128) ? 2 : 1;
  // the warps' outputs are joined through shared memory, in one round where it has room for all
  static constexpr int kRounds = D == 256 ? 2 * NT : D == 128 && NT == 4 ? 2 : 1;
  static constexpr int kRoundBlocks = G::kBlocks / kRounds;
  static constexpr int kMergeRow = 32 * kRoundBlocks + 4;  // floats
  // shared memory, in bytes from its start
  static constexpr int kRing = 0;
  static constexpr int kQ = kRing + kWarps * kStages * kStageBytes;  // fragments [NT][blocks][32] uint4
  static constexpr int kMerge = kQ + (kShared ? NT * G::kBlocks * 512 : 0);  // float [kWarps][kRows][kMergeRow]
  static constexpr int kStats = kMerge + kWarps * kRows * kMergeRow * 4;  // float m, l [kWarps][kRows]
  static constexpr int kRowInfo = kStats + 2 * kWarps * kRows * 4;  // factor, lo, hi [kRows], of each warp or all
  static constexpr int kParts = kRowInfo + (kShared ? 1 : kWarps) * 3 * kRows * 4;  // Part [kWarps]
  // a step's scales as the products want them, per warp: float of each key and block,
  // FP16 factor of each pair of keys and block
  static constexpr int kScaleBytes = 32 * G::kBlocks * 4 + 16 * G::kBlocks * 4;
  static constexpr int kScales = kParts + kWarps * (int)sizeof(Part);
  static constexpr int kBars = kScales + kWarps * kScaleBytes;  // uint64 [kWarps][kStages]
  static constexpr int kScan = kBars + kWarps * kStages * 8;         // long long [kWarps]
  static constexpr int kScan2 = kScan + kWarps * 8;                  // int [2 * kWarps]
  static constexpr int kPrefix = kScan2 + 2 * kWarps * 4;              // long long [entries]
  static constexpr int shared_bytes(int entries) {  // ... and int2 [min(entries, kCached)]
    return kPrefix + 8 * entries + 8 * (entries < kCached ? entries : kCached);
  }
  static_assert(kScales % 16 == 0 && kBars % 8 == 0, "alignment");
  static_assert(kPrefix + 8 * WD_KV_MAX_ENTRIES + 8 * kCached <= 227 * 1024, "shared memory");
};

// Where CTA `unit` leaves its part of an item: it has at most two, that of an item that began
// before it and that of one that goes on behind it.
template <int D, int NT>
__device__ __forceinline__ float* part_at(const KvAttentionArgs& a, const Part& p, int unit) {
  using L = Shape<D, NT>;
  const long long slot = 2 * (long long)unit + (p.slot0 >= (long long)unit * L::kWarps ? 1 : 0);
  return a.partial + slot * L::kRows * (D + 2);
}

// The i-th of the lengths of a piece that are tried, a warp to each: around what fills one pass
// (`fair`), and at last what leaves an item to one CTA and to one warp.
template <int kWarps>
__device__ __forceinline__ int steps_choice(int i, int fair, int longest) {
  if (i == kWarps - 1) return longest;
  if (i == kWarps - 2) return (longest + kWarps - 1) / kWarps;
  if (fair < kWarps - 3) return 1 + i;
  constexpr uint64_t kBy = kWarps == 12 ? 0x2820181614131110ull : 0x0000282018141210ull;  // sixteenths
  const int by = i < 8 ? (int)(kBy >> (8 * i)) & 0xFF : i == 8 ? 8 : 12;
  return max(1, (int)(((long long)fair * by + 15) >> 4));
}

// S^T of one group of 16 keys: s[nt] has keys g (0, 1) and 8 + g (2, 3) of columns 2tq, 2tq + 1.
// `scales`: the group's keys' block scales, times a.key_scale.
template <int D, int NT>
__device__ __forceinline__ void scores(const uint8_t* buf, const uint8_t* scales, const uint4* qf,
                                       const uint8_t* q_sh, int lane, float (&s)[NT][4]) {
  using G = KvGroup<D>;
  constexpr int CB = G::kBlocks, SB = G::kSlabBlocks, NS = G::kSlabs;
  const int g = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
  for (int sl = 0; sl < NS; ++sl) {
    Words<SB> kw[2], kf[2];  // codes and scales of keys 8h + g
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      kw[h] = lds<SB>(buf + sl * G::kSlabBytes + (8 * h + g) * 16 * SB + tq * 4 * SB);
      kf[h] = lds<SB>(scales + ((8 * h + g) * CB + sl * SB) * 4);
    }
#pragma unroll
    for (int c = 0; c < SB; ++c) {
      const int cb = sl * SB + c;
      uint32_t a0, a1, a2, a3, b0, b1, b2, b3;
      e2m1x8(kw[0].v[c], a0, a2, b0, b2);
      e2m1x8(kw[1].v[c], a1, a3, b1, b3);
      const float s0 = __uint_as_float(kf[0].v[c]), s1 = __uint_as_float(kf[1].v[c]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4 q = Shape<D, NT>::kShared ? *reinterpret_cast<const uint4*>(
                                                    q_sh + ((nt * CB + cb) * 32 + lane) * 16)
                                              : qf[Shape<D, NT>::kShared ? 0 : cb];
        float t[4];
        mma_f16_zero(t, a0, a1, a2, a3, q.x, q.y);
        mma_f16_acc(t, b0, b1, b2, b3, q.z, q.w);
        s[nt][0] = fmaf(t[0], s0, s[nt][0]);
        s[nt][1] = fmaf(t[1], s0, s[nt][1]);
        s[nt][2] = fmaf(t[2], s1, s[nt][2]);
        s[nt][3] = fmaf(t[3], s1, s[nt][3]);
      }
    }
  }
}

// O^T += V^T P^T of one group: p[h] has tokens 8h + 2tq + {0, 1} of column g; `factors`: the group's
// pairs of tokens' block factors, FP16.
template <int D, int NT>
__device__ __forceinline__ void values(const uint8_t* buf, const uint8_t* factors,
                                       const uint32_t (&p)[2][NT], int lane,
                                       float (&o)[KvGroup<D>::kBlocks][2][NT][4]) {
  using G = KvGroup<D>;
  constexpr int CB = G::kBlocks, SB = G::kSlabBlocks, NS = G::kSlabs;
  const int g = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int sl = 0; sl < NS; ++sl) {
    const uint8_t* vb = buf + G::kCodeBytes + sl * G::kSlabBytes + g * 16 * SB + tq * 4 * SB;
    const Words<SB> v0 = lds<SB>(vb), v1 = lds<SB>(vb + 128 * SB);
    const Words<SB> f0 = lds<SB>(factors + (tq * CB + sl * SB) * 4);
    const Words<SB> f1 = lds<SB>(factors + ((4 + tq) * CB + sl * SB) * 4);
#pragma unroll
    for (int cp = 0; cp < SB / 2; ++cp) {  // blocks 2cp, 2cp + 1
      // codes of two tokens side by side: channels n = 0, 2 (x) and 1, 3 (y)
      const uint32_t l0 = v0.v[cp], h0 = v0.v[SB / 2 + cp];
      const uint32_t l1 = v1.v[cp], h1 = v1.v[SB / 2 + cp];
      const uint32_t x0 = (l0 & 0x0F0F0F0Fu) | ((h0 << 4) & 0xF0F0F0F0u);
      const uint32_t y0 = ((l0 >> 4) & 0x0F0F0F0Fu) | (h0 & 0xF0F0F0F0u);
      const uint32_t x1 = (l1 & 0x0F0F0F0Fu) | ((h1 << 4) & 0xF0F0F0F0u);
      const uint32_t y1 = ((l1 >> 4) & 0x0F0F0F0Fu) | (h1 & 0xF0F0F0F0u);
      uint32_t a0[4], a1[4], a2[4], a3[4];
      e2m1x8(x0, a0[0], a0[1], a0[2], a0[3]);
      e2m1x8(y0, a1[0], a1[1], a1[2], a1[3]);
      e2m1x8(x1, a2[0], a2[1], a2[2], a2[3]);
      e2m1x8(y1, a3[0], a3[1], a3[2], a3[3]);
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int cb = sl * SB + 2 * cp + cc;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = mul_half2(p[0][nt], f0.v[2 * cp + cc]);
          const uint32_t b1 = mul_half2(p[1][nt], f1.v[2 * cp + cc]);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            mma_f16_acc(o[cb][j][nt], a0[2 * cc + j], a1[2 * cc + j], a2[2 * cc + j],
                        a3[2 * cc + j], b0, b1);
        }
      }
    }
  }
}

// The same, product by product in FP32, for scales that one FP16 exponent range does not hold, or
// NaN.  `key0`: the group's first key, `end`: the first that no row sees.
template <int D, int NT>
__device__ __forceinline__ void values_singly(const uint8_t* buf, const uint32_t (&p)[2][NT],
                                              const uint32_t (&ref)[(KvGroup<D>::kBlocks + 3) / 4],
                                              int key0, int end, const int* lo, const int* hi, int lane,
                                              float (&o)[KvGroup<D>::kBlocks][2][NT][4]) {
  using G = KvGroup<D>;
  constexpr int CB = G::kBlocks;
  const int g = lane >> 2, tq = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    for (int t = 0; t < 8; ++t) {
      const int key = key0 + 8 * h + t;
      if (key >= end) break;
      float pr[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t w = __shfl_sync(kAll, p[h][nt], (2 * tq + e) * 4 + (t >> 1));
          const __half2 both = *reinterpret_cast<const __half2*>(&w);
          const int row = 8 * nt + 2 * tq + e;
          const bool seen = key >= lo[row] && key <= hi[row];
          // what is not seen adds nothing, not even 0 * NaN
          pr[nt][e] = !seen ? -1.f : (t & 1 ? __high2float(both) : __low2float(both));
        }
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const uint32_t sv = buf[G::kVScale + (8 * h + t) * CB + c];
        const int rc = (int)((ref[c / 4] >> (8 * (c % 4))) & 0xFFu);
        const float unit =
            sv == 255u ? __uint_as_float(0x7FC00000u) : exp2f((float)((int)sv - rc + 1));
        uint32_t v[4];
        e2m1x8(*reinterpret_cast<const uint16_t*>(buf + G::v_half(8 * h + t, c, g)), v[0], v[1], v[2],
               v[3]);
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

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kThreads, Shape<D, NT>::kCtasPerSm)
    kv_attention(const KvAttentionArgs a) {
  using G = KvGroup<D>;
  using L = Shape<D, NT>;
  constexpr int CB = G::kBlocks, NW = (CB + 3) / 4;
  constexpr int kRows = L::kRows, kStages = L::kStages, kWarps = L::kWarps, kThreads = L::kThreads;
  constexpr bool kQInRegs = !L::kShared;
  constexpr int kU = L::kTogether;
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, tq = lane & 3;
  const KvView& cache = a.cache;
  const int heads = cache.kv_heads, group = a.q_heads / heads;
  float* merge = reinterpret_cast<float*>(smem + L::kMerge);
  float* m_sh = reinterpret_cast<float*>(smem + L::kStats);
  float* l_sh = m_sh + kWarps * kRows;
  float* factor_sh =
      reinterpret_cast<float*>(smem + L::kRowInfo) + (L::kShared ? 0 : warp) * 3 * kRows;
  int* lo_sh = reinterpret_cast<int*>(factor_sh + kRows);
  int* hi_sh = lo_sh + kRows;
  Part* parts_sh = reinterpret_cast<Part*>(smem + L::kParts);
  long long* scan = reinterpret_cast<long long*>(smem + L::kScan);
  int* scan2 = reinterpret_cast<int*>(smem + L::kScan2);
  long long* prefix = reinterpret_cast<long long*>(smem + L::kPrefix);
  int2* cached = reinterpret_cast<int2*>(prefix + a.batch.entries);
  uint8_t* ring = smem + L::kRing + warp * kStages * L::kStageBytes;
  uint8_t* k_scales = smem + L::kScales + warp * L::kScaleBytes;  // float [32 keys][CB]
  uint8_t* v_scales = k_scales + 32 * CB * 4;                    // f16x2 [16 pairs of keys][CB]
  const uint32_t bar = smem_u32(smem + L::kBars) + warp * kStages * 8;
  __shared__ int last_sh[2];

  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(bar + 8 * s, 1);
    mbar_init_fence();
  }
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();

  // ---- the division of the work
  Entry own{-1, 0, 0, 0};
  if ((int)threadIdx.x < a.batch.entries) own = load_entry(a, threadIdx.x);
  long long total = 0;
  int longest = 1;
  float items = 0.f;
  {
    long long steps_here = 0;
    for (int b = threadIdx.x; b < a.batch.entries; b += kThreads) {
      const Entry e = b < kThreads ? own : load_entry(a, b);
      if (b < kCached) cached[b] = make_int2(e.slot, e.len);
      const int steps = steps_of<kRows>(e, group, a.window), tiles = tiles_of<kRows>(e, group);
      steps_here += (long long)steps * tiles;
      items += (float)tiles;
      if (e.n > 0) longest = max(longest, steps);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      steps_here += __shfl_xor_sync(kAll, steps_here, off);
      items += __shfl_xor_sync(kAll, items, off);
    }
    longest = __reduce_max_sync(kAll, longest);
    if (lane == 0) {
      scan[warp] = steps_here;
      scan2[warp] = longest;
      scan2[kWarps + warp] = __float_as_int(items);
    }
    __syncthreads();
    items = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      total += scan[w];
      longest = max(longest, scan2[w]);
      items += __int_as_float(scan2[kWarps + w]);
    }
    total *= heads;
    items *= (float)heads;
  }
  const float warps = (float)(gridDim.x * kWarps);
  unsigned q_steps, align;
  if (!L::kShared && 2.f * items <= warps) {
    // Few items: q for which one pass does, whatever the lengths are (an item wastes less than a
    // piece).  Rather than that, whole items to a CTA, if that costs less than a join through memory
    // does, which is about three steps.
    const float loose = ceilf((float)total / (warps - items));
    const float aligned = (float)kWarps * items < warps
                              ? fmaxf(ceilf((float)total / (warps - (float)kWarps * items)),
                                      (float)((longest + kWarps - 1) / kWarps))
                              : 1e30f;
    align = aligned <= loose + ((float)longest > loose ? 3.f : 0.f) ? kWarps : 1;
    q_steps = (unsigned)fmaxf(1.f, fminf(align > 1 ? aligned : loose, 1e9f));
  } else {
    // Some lengths of a piece, each with the pieces in a row and with every item at the start of
    // a CTA, are rated in steps: the passes' longest pieces, two steps for what a pass begins and
    // ends with, three for a join through memory.
    const int fair = (int)fminf(ceilf((float)total / warps), 6e7f);
    __syncthreads();
    {
      const unsigned q = steps_choice<kWarps>(warp, fair, longest);
      float loose = 0.f, aligned = 0.f;  // units (exact where it matters, below 2^24)
      for (int b = lane; b < a.batch.entries; b += 32) {
        const Entry e = load_entry(a, b, cached);
        const unsigned pieces = ((unsigned)steps_of<kRows>(e, group, a.window) + q - 1) / q;
        const float tiles = (float)tiles_of<kRows>(e, group);
        loose += tiles * (float)pieces;
        aligned += tiles * (float)((pieces + kWarps - 1) / kWarps);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        loose += __shfl_xor_sync(kAll, loose, off);
        aligned += __shfl_xor_sync(kAll, aligned, off);
      }
      const float units = (float)heads * (lane == 0 ? loose * (1.f / kWarps) : aligned);
      const float passes = ceilf(units / (float)gridDim.x);
      const bool across = (float)longest > (float)q * (lane == 0 ? 1.f : (float)kWarps);
      const float cost =
          (passes <= 1.f ? (float)q : fmaxf((float)q, (float)fair + 0.75f * (float)q)) +
          2.f * passes + (across ? 3.f : 0.f);
      // joins across CTAs have room for so many
      const bool fits =
          (!across || units <= (float)(kKvMaxUnits / NT)) && (!L::kShared || lane == 1);
      if (lane < 2) scan2[2 * warp + lane] = fits ? (int)fminf(cost * 16.f, 1e9f) : 0x7FFFFFFF;
    }
    __syncthreads();
    const int rated = lane < 2 * kWarps ? scan2[lane] : 0x7FFFFFFF;
    const int cheapest = __reduce_min_sync(kAll, rated);
    const int choice = __ffs(__ballot_sync(kAll, rated == cheapest)) - 1;
    q_steps = steps_choice<kWarps>(choice >> 1, fair, longest);
    align = choice & 1 ? kWarps : 1;
  }
  const Divisor by_q(q_steps);
  const auto places_of = [&](const Entry& e, unsigned& pieces) {  // of one item
    pieces = by_q.of((unsigned)steps_of<kRows>(e, group, a.window) + q_steps - 1);
    return align > 1 ? (pieces + kWarps - 1) / kWarps * kWarps : pieces;
  };
  // Places of the entries before each entry.  A small batch is gone through by every warp for
  // itself whenever it looks for a place; else prefix[] holds them.
  const bool small = a.batch.entries <= 128 && (float)total + items * (float)kWarps < 2e9f;
  total = 0;
  if (small) {
    unsigned all = 0;
    for (int b = lane; b < a.batch.entries; b += 32) {
      const Entry e = load_entry(a, b, cached);
      unsigned pieces;
      all += tiles_of<kRows>(e, group) * heads * places_of(e, pieces);
    }
    total = __reduce_add_sync(kAll, all);
  } else {
    for (int base = 0; base < a.batch.entries; base += kThreads) {
      const int b = base + threadIdx.x;
      long long cost = 0;
      if (b < a.batch.entries) {
        const Entry e = b < kThreads ? own : load_entry(a, b);
        unsigned pieces;
        cost = (long long)tiles_of<kRows>(e, group) * heads * places_of(e, pieces);
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
    __syncthreads();
  }
  const bool no_joins = (unsigned)longest <= q_steps;

  const bool vec = (reinterpret_cast<uintptr_t>(a.q) & 15u) == 0 && a.q_token % 8 == 0 &&
                   a.q_head % 8 == 0;
  const uint32_t ring_at = smem_u32(ring);
  int stage = 0;
  uint32_t phase = 0;
  bool dead = false;  // a wait ran out
  for (int unit = blockIdx.x; (long long)unit * kWarps < total; unit += gridDim.x) {
    // ---- the warp's piece
    const long long slot = (long long)unit * kWarps + warp;
    Part part;
    part.pieces = 0;
    part.slot0 = 0;
    part.tile = part.head = part.first = part.n = 0;
    Entry entry{-1, 0, 0, 0};
    Span span{0, 0};
    int from = 0, steps = 0;  // the piece: steps [from, from + steps) of the tile
    if (slot < total) {
      // the entry that it belongs to, and its place among that entry's
      unsigned long long rest = 0;
      int lo = 0;
      unsigned pieces, places;
      if (small) {
        unsigned before = 0;
        for (int b0 = 0; b0 < a.batch.entries; b0 += 32) {
          const int b = b0 + lane;
          unsigned cost = 0, lane_pieces = 0, lane_places = 0;
          Entry e{-1, 0, 0, 0};
          if (b < a.batch.entries) {
            e = load_entry(a, b, cached);
            lane_places = places_of(e, lane_pieces);
            cost = tiles_of<kRows>(e, group) * heads * lane_places;
          }
          unsigned incl = cost;
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const unsigned t = __shfl_up_sync(kAll, incl, off);
            if (lane >= off) incl += t;
          }
          const unsigned hit = __ballot_sync(kAll, before + incl > (unsigned)slot);
          if (hit) {
            lo = __ffs(hit) - 1;
            rest = (unsigned)slot - before - __shfl_sync(kAll, incl - cost, lo);
            pieces = __shfl_sync(kAll, lane_pieces, lo);
            places = __shfl_sync(kAll, lane_places, lo);
            entry.slot = __shfl_sync(kAll, e.slot, lo);
            entry.len = __shfl_sync(kAll, e.len, lo);
            entry.first = __shfl_sync(kAll, e.first, lo);
            entry.n = __shfl_sync(kAll, e.n, lo);
            break;
          }
          before += __shfl_sync(kAll, incl, 31);
        }
      } else {
        int hi = a.batch.entries;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (prefix[mid] <= slot) lo = mid; else hi = mid;
        }
        rest = slot - prefix[lo];
        entry = load_entry(a, lo, cached);
        places = places_of(entry, pieces);
      }
      const int tiles = max(1, tiles_of<kRows>(entry, group));
      const unsigned item = rest >> 32 ? (unsigned)(rest / places) : Divisor(places).of((unsigned)rest);
      const unsigned piece = (unsigned)(rest - (unsigned long long)item * places);
      // (within bounds also if someone rewrites the lengths meanwhile)
      int turn = 0;
      part.head = item;
      if (item >= (unsigned)heads) {
        turn = min((int)(item / heads), tiles - 1);
        part.head = item - (item / heads) * heads;
      }
      part.tile = turn & 1 ? tiles - 1 - (turn >> 1) : turn >> 1;
      part.slot0 = slot - piece;
      part.first = entry.first;
      part.n = entry.n;
      span = tile_span<kRows>(entry, part.tile, group, a.window);
      if (piece < pieces) {
        part.pieces = pieces;
        from = piece * q_steps;
        steps = min((int)q_steps, (span.end + kStep - 1) / kStep - span.first - from);
        if (steps < 0 || dead) steps = 0;
      }
    }
    const int rows = entry.n * group - part.tile * kRows;  // of the tile's, those that are real

    // The i-th step's groups are looked up by lane i % 32, 32 steps at a time, and copied into
    // the stages in turn.
    const uint8_t *src0 = nullptr, *src1 = nullptr;
    uint32_t bytes0 = 0;
    int page0 = 0, page1 = 0;
    const auto look_up = [&](int i0) {
      const int pos = (span.first + from + i0 + lane) * kStep;
      if (i0 + lane >= steps) return;
      const int32_t* row = cache.table + (long long)entry.slot * cache.columns;
      page0 = row[pos >> cache.page_shift];
      page1 = cache.page_size < kStep && pos + 16 < span.end ? row[(pos + 16) >> cache.page_shift] : 0;
    };
    // (a page out of range: the flag, and NaN from the workspace in its place)
    const auto group_at = [&](int page, int pos) -> const uint8_t* {
      if (kv_page_there(cache, page)) return kv_group(cache, page, a.layer, part.head, pos, G::kBytes);
      atomicOr(cache.flag, WD_KV_FLAG_BAD_INDEX);
      return a.none;
    };
    const auto plan = [&](int i0) {
      const int pos = (span.first + from + i0 + lane) * kStep;
      src1 = nullptr;
      if (i0 + lane >= steps) return;
      src0 = group_at(page0, pos);
      bytes0 = G::kBytes;
      if (pos + 16 < span.end) {
        if (cache.page_size >= kStep)  // the step lies within a page, its groups side by side
          bytes0 = 2 * G::kBytes;
        else
          src1 = group_at(page1, pos + 16);
      }
    };
    const auto gone = [&](int key) {  // is the page of a key out of range?
      return key < span.end &&
             !kv_page_there(cache, cache.table[(long long)entry.slot * cache.columns +
                                               (key >> cache.page_shift)]);
    };
    look_up(0);

    // the queries, on their way while the first groups are asked for
    constexpr int kFetches = L::kShared ? (kRows * (D / 8) + kThreads - 1) / kThreads : CB;
    Words<4> query[kFetches];
#pragma unroll
    for (int i = 0; i < kFetches; ++i) {
      // shared: 8 channels of any row; else channels 32i + 8tq of row g, the lane's own fragment
      const int x = threadIdx.x + i * kThreads;
      const int row = L::kShared ? x / (D / 8) : g;
      const int ch = L::kShared ? x % (D / 8) * 8 : 32 * i + 8 * tq;
      const int flat = part.tile * kRows + row;
      const int token = entry.n > 1 ? flat / group : 0;
      query[i] = Words<4>{{0u, 0u, 0u, 0u}};
      if (row < kRows && row < rows && (L::kShared || part.pieces > 0))
        query[i] = load8(a, (entry.first + token) * a.q_token +
                                (part.head * group + flat - token * group) * a.q_head + ch, vec);
    }

    const auto issue = [&](int to_stage) {
      const uint32_t to = ring_at + to_stage * L::kStageBytes, full = bar + 8 * to_stage;
      mbar_arrive_expect_tx(full, bytes0 + (src1 ? G::kBytes : 0));
      bulk_g2s_nohint(to, src0, bytes0, full);
      if (src1) bulk_g2s_nohint(to + G::kBytes, src1, G::kBytes, full);
    };
    plan(0);
    if (lane < kStages && lane < steps) issue((stage + lane) % kStages);
    __syncwarp();

    // ---- the queries as fragments: channel 32c + 8t + 4j + 2i + {0,1} of row 8nt + g is
    // register i of product j in lane 4g + t
    uint4 qf[kQInRegs ? CB : 1];
    const uint8_t* q_sh = smem + L::kQ;
    if constexpr (L::kShared) {
      __syncthreads();  // the pass before has read its own
#pragma unroll
      for (int i = 0; i < kFetches; ++i) {
        const int x8 = threadIdx.x + i * kThreads;
        const int row = x8 / (D / 8), e8 = x8 % (D / 8);
        if (row >= kRows) break;  // (whole warps)
        float x[8];
        widen8(query[i], a.half, x);
        uint32_t bits = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) bits = max(bits, __float_as_uint(x[q]) & 0x7FFFFFFFu);
#pragma unroll
        for (int off = 1; off < D / 8; off <<= 1)
          bits = max(bits, __shfl_xor_sync(kAll, bits, off));
        const RowScale r = row_scale(bits);
        *reinterpret_cast<uint4*>(smem + L::kQ +
                                  (((row >> 3) * CB + (e8 >> 2)) * 32 + (row & 7) * 4 + (e8 & 3)) * 16) =
            row_fragment(x, r);
        if (e8 == 0) {
          const int pos = entry.len - entry.n + (entry.n > 1 ? (part.tile * kRows + row) / group : 0);
          const bool real = row < rows;  // no row: nothing to hide, never stored
          factor_sh[row] = pos < 0 ? 1.f : power_factor(r, a.row_scale);  // (sees nothing: no NaN)
          lo_sh[row] = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
          hi_sh[row] = real ? pos : span.end - 1;
        }
      }
      __syncthreads();
    } else {
      uint32_t bits = 0;
      float x[CB][8];
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        widen8(query[c], a.half, x[c]);
#pragma unroll
        for (int q = 0; q < 8; ++q) bits = max(bits, __float_as_uint(x[c][q]) & 0x7FFFFFFFu);
      }
      bits = max(bits, __shfl_xor_sync(kAll, bits, 1));
      bits = max(bits, __shfl_xor_sync(kAll, bits, 2));
      const RowScale r = row_scale(bits);
#pragma unroll
      for (int c = 0; c < CB; ++c) qf[c] = row_fragment(x[c], r);
      __syncwarp();
      if (tq == 0) {
        const int pos = entry.len - entry.n + (entry.n > 1 ? (part.tile * kRows + g) / group : 0);
        const bool real = g < rows;
        factor_sh[g] = pos < 0 ? 1.f : power_factor(r, a.row_scale);  // (sees nothing: no NaN)
        lo_sh[g] = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
        hi_sh[g] = real ? pos : span.end - 1;
      }
      __syncwarp();
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

    for (int i = 0; i < steps; ++i) {
      const bool landed = mbar_wait(bar + 8 * stage, phase);
      const int step_at = (span.first + from + i) * kStep;

      // ---- the scales of key step_at + lane, for the lanes whose products want them
      bool inside = step_at + lane < span.end;
      const uint8_t* scale_at = ring + stage * L::kStageBytes + (lane >> 4) * G::kBytes + (lane & 15) * CB;
      const Words<NW> kt = lds_scales<CB>(scale_at + G::kKScale);
      Words<NW> vt = lds_scales<CB>(scale_at + G::kVScale);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        float4 f;
        const uint32_t lo = e8m0x2(kt.v[w]);
        f.x = __uint_as_float(lo << 16) * a.key_scale;
        f.y = __uint_as_float(lo & 0xFFFF0000u) * a.key_scale;
        if constexpr (CB == 2) {
          *reinterpret_cast<float2*>(k_scales + lane * 8) = make_float2(f.x, f.y);
        } else {
          const uint32_t hi = e8m0x2(kt.v[w] >> 16);
          f.z = __uint_as_float(hi << 16) * a.key_scale;
          f.w = __uint_as_float(hi & 0xFFFF0000u) * a.key_scale;
          *reinterpret_cast<float4*>(k_scales + lane * 4 * CB + 16 * w) = f;
        }
      }
      // 2^(s - ref + 1) of V: the exponent field is s - ref + 16, here first four times that in
      // the byte it belongs in.  Keys that no row sees take the reference itself; their
      // probabilities are zero.
      const auto put_v_scales = [&]() {
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const uint32_t d = 4u * (inside ? vt.v[w] : ref[w]) - 4u * (ref[w] - 0x10101010u);
          const uint32_t other = __shfl_xor_sync(kAll, d, 1);
          const bool second = lane & 1;
          if constexpr (CB == 2) {
            const uint32_t both = second ? __byte_perm(other, d, 0x5410) << 0
                                         : __byte_perm(d, other, 0x5410) << 8;
            *reinterpret_cast<uint32_t*>(v_scales + (lane >> 1) * 8 + (lane & 1) * 4) =
                both & 0xFF00FF00u;
          } else {
            const uint32_t both = second ? __byte_perm(other, d, 0x7632) : __byte_perm(d, other, 0x5410);
            *reinterpret_cast<uint2*>(v_scales + (lane >> 1) * 4 * CB + 16 * w + (lane & 1) * 8) =
                make_uint2((both << 8) & 0xFF00FF00u, both & 0xFF00FF00u);
          }
        }
        __syncwarp();
      };
      bool odd = !landed;  // are all V scales within [ref - 15, ref]?
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const uint32_t v = CB == 2 ? vt.v[w] | (ref[w] & 0xFFFF0000u) : vt.v[w];
        const uint32_t t0 = ((ref[w] & 0x00FF00FFu) | 0x80008000u) - (v & 0x00FF00FFu);
        const uint32_t t1 = (((ref[w] >> 8) & 0x00FF00FFu) | 0x80008000u) - ((v >> 8) & 0x00FF00FFu);
        odd |= inside && ((t0 | t1) & 0x7FF07FF0u) != 0u;
      }
      put_v_scales();
      bool slow = false;

#pragma unroll
      for (int u0 = 0; u0 < 2; u0 += kU) {
        const int j0 = step_at + 16 * u0;
        if (u0 > 0 && j0 >= span.end) break;  // was not copied
        const uint8_t* buf = ring + stage * L::kStageBytes + u0 * G::kBytes;

        // ---- S^T = K Q^T
        float s[kU][NT][4];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          scores<D, NT>(buf + u * G::kBytes, k_scales + (u0 + u) * 16 * CB * 4, qf, q_sh, lane, s[u]);

        // ---- does anything change: a larger logit, a V scale out of range?
        const bool whole = j0 >= seen_lo && j0 + 16 * kU - 1 <= seen_hi;
        float top[NT][2];
        bool grow = odd;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float t = -INFINITY;
#pragma unroll
            for (int u = 0; u < kU; ++u)
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
            grow |= top[nt][e] > m[nt][e] + kSlack;
          }
        const auto hide = [&](int u) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u][nt][e] = -INFINITY;
        };
        if (kU == 1 && u0 > 0 && slow && gone(j0)) hide(0);
        if (__any_sync(kAll, grow)) {
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
          if (__any_sync(kAll, odd)) {
            bool bad = false;
            // what lies before the window of all rows (the first row's) takes part in nothing, and a key
            // that not every row sees must not push what the others see out of FP32
            const int key = step_at + lane;
            inside = inside && key >= lo_sh[0];
            // Scales that are all NaN may be those of a page that is not there: nobody sees its keys.
            uint32_t nan = CB == 2 ? vt.v[0] | 0xFFFF0000u : vt.v[0];
#pragma unroll
            for (int w = 1; w < NW; ++w) nan &= vt.v[w];
            bool hidden = false;
            if (__any_sync(kAll, nan == kAll)) {
              inside = inside && !gone(key);
#pragma unroll
              for (int u = 0; u < kU; ++u)
                if (gone(j0 + 16 * u)) hide(u);
              hidden = kU == 1 && gone(step_at + 16);  // (its turn comes)
            }
            const uint32_t limit = !inside ? 0u : key >= seen_lo && key <= seen_hi ? 254u : kSharedMost;
#pragma unroll
            for (int c = 0; c < CB; ++c) {
              const uint32_t sh = 8 * (c % 4), mine_c = (vt.v[c / 4] >> sh) & 0xFFu;
              const uint32_t old = (ref[c / 4] >> sh) & 0xFFu;
              const uint32_t most =
                  max(old, __reduce_max_sync(kAll, mine_c != 255u ? min(mine_c, limit) : 0u));
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
            slow = __any_sync(kAll, bad) || hidden;
            __syncwarp();
            put_v_scales();
            odd = false;
          }
        }

        // ---- P = 2^kBias exp2(x - m)
        uint32_t p[kU][2][NT];  // P^T fragments: tokens 16u + 8h + 2tq + {0, 1} of column g
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float z0 = m[nt][0] == -INFINITY ? 0.f : kBias - m[nt][0];
          const float z1 = m[nt][1] == -INFINITY ? 0.f : kBias - m[nt][1];
#pragma unroll
          for (int u = 0; u < kU; ++u)
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
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (!slow)
            values<D, NT>(buf + u * G::kBytes, v_scales + (u0 + u) * 8 * CB * 4, p[u], lane, o);
          else if (!gone(j0 + 16 * u))
            values_singly<D, NT>(buf + u * G::kBytes, p[u], ref, j0 + 16 * u, span.end, lo_sh, hi_sh,
                                 lane, o);
        }
      }
      if (dead) {
        // give up, but not before the copies in flight have landed (or as long again has passed)
        for (int j = 0; j < kStages && i + j < steps; ++j)
          mbar_wait(bar + 8 * ((stage + j) % kStages), stage + j < kStages ? phase : phase ^ 1u);
        break;
      }

      // ---- refill the stage
      __syncwarp();
      const int next = i + kStages;
      if ((next & 31) == 0) {
        look_up(next);
        plan(next);
      }
      if (lane == (next & 31) && next < steps) issue(stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1u;
      }
    }

    // ---- the piece's result
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(kAll, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(kAll, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(kAll, l[nt][e], 16);
      }
    const auto unit_of = [&](int c) {
      return exp2_int((int)((ref[c / 4] >> (8 * (c % 4))) & 0xFFu) - 128);
    };
    // Values beyond 2^23 (which raise the reference that far, whoever sees them) may be so large that their sum,
    // each up to 2^14 times, is more than FP32 holds where their mean is not: a row's sums and
    // outputs then stand on a maximum 2^64 times as large.
    bool large = false;
#pragma unroll
    for (int w = 0; w < NW; ++w) large |= __vcmpgeu4(ref[w], 0x01010101u * kSharedMost) != 0u;
    if (__builtin_expect(large, 0)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float most = 0.f;
#pragma unroll
          for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              most = fmaxf(most, fmaxf(fabsf(o[c][j][nt][e]), fabsf(o[c][j][nt][2 + e])) * unit_of(c));
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) most = fmaxf(most, __shfl_xor_sync(kAll, most, off));
          if (!(most > 0x1p100f)) continue;
          m[nt][e] += 64.f;
          l[nt][e] *= 0x1p-64f;
#pragma unroll
          for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              o[c][j][nt][e] *= 0x1p-64f;
              o[c][j][nt][2 + e] *= 0x1p-64f;
            }
        }
    }
    const auto output = [&](int c, int nt, int e) {  // channels 32c + 4g + {0..3} of row 8nt + 2tq + e
      const float unit = unit_of(c);
      return make_float4(o[c][0][nt][e] * unit, o[c][0][nt][2 + e] * unit, o[c][1][nt][e] * unit,
                         o[c][1][nt][2 + e] * unit);
    };
    if (part.pieces == 1) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int c = 0; c < CB; ++c)
            store_row<D, kRows>(a, part, 8 * nt + 2 * tq + e, 32 * c + 4 * g, output(c, nt, e),
                                m[nt][e], l[nt][e]);
    }
    if (no_joins) continue;

    // ---- join the pieces of an item that this CTA has
    if (lane == 0) parts_sh[warp] = part;
    if (g == 0)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m_sh[warp * kRows + 8 * nt + 2 * tq + e] = m[nt][e];
          l_sh[warp * kRows + 8 * nt + 2 * tq + e] = l[nt][e];
        }
    uint32_t leads = 0, follows = 0, partial = 0;  // warps: first of an item here, further ones, of items that go on elsewhere
#pragma unroll
    for (int round = 0; round < L::kRounds; ++round) {
      if (round > 0) __syncthreads();
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        const int cr = c - round * L::kRoundBlocks;
        if (cr < 0 || cr >= L::kRoundBlocks) continue;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            *reinterpret_cast<float4*>(
                merge + (warp * kRows + 8 * nt + 2 * tq + e) * L::kMergeRow + 32 * cr + 4 * g) =
                output(c, nt, e);
      }
      __syncthreads();
      if (round == 0) {
        long long slot0 = 0;
        int pieces = 0;
        if (lane < kWarps) {
          slot0 = parts_sh[lane].slot0;
          pieces = parts_sh[lane].pieces;
        }
        const long long slot0_before = __shfl_up_sync(kAll, slot0, 1);
        const int pieces_before = __shfl_up_sync(kAll, pieces, 1);
        const bool follow = lane > 0 && pieces > 1 && pieces_before > 1 && slot0 == slot0_before;
        const bool whole = slot0 >= (long long)unit * kWarps &&
                           slot0 + pieces <= (long long)(unit + 1) * kWarps;
        follows = __ballot_sync(kAll, follow);
        leads = __ballot_sync(kAll, pieces > 1 && !follow);
        partial = __ballot_sync(kAll, pieces > 1 && !follow && !whole);
      }
      constexpr int kQuads = 8 * L::kRoundBlocks;  // four channels each, of a row
      for (int i = threadIdx.x; i < __popc(leads) * kRows * kQuads; i += kThreads) {
        uint32_t rest = leads;
        for (int skip = i / (kRows * kQuads); skip > 0; --skip) rest &= rest - 1;
        const int w0 = __ffs(rest) - 1;
        const int w1 = w0 + __ffs(~(follows >> (w0 + 1)));
        const int row = i % (kRows * kQuads) / kQuads, ch = 4 * (i % kQuads);
        float top = -INFINITY, sum = 0.f;
        for (int w = w0; w < w1; ++w) top = fmaxf(top, m_sh[w * kRows + row]);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int w = w0; w < w1; ++w) {
          const float f = top == -INFINITY ? 0.f : exp2_fast(m_sh[w * kRows + row] - top);
          const float lw = l_sh[w * kRows + row];
          // a warp whose keys were all NaN has no maximum, but a NaN sum
          sum += lw != lw ? lw : lw * f;
          const float4 v =
              *reinterpret_cast<const float4*>(merge + (w * kRows + row) * L::kMergeRow + ch);
          y.x = fmaf(v.x, f, y.x);
          y.y = fmaf(v.y, f, y.y);
          y.z = fmaf(v.z, f, y.z);
          y.w = fmaf(v.w, f, y.w);
        }
        const Part p = parts_sh[w0];
        const int at_ch = 32 * round * L::kRoundBlocks + ch;
        if (!(partial >> w0 & 1u)) {
          store_row<D, kRows>(a, p, row, at_ch, y, top, sum);
        } else {
          float* to = part_at<D, NT>(a, p, unit);
          __stcg(reinterpret_cast<float4*>(to + row * D + at_ch), y);
          if (at_ch == 0) {
            __stcg(to + kRows * D + row, top);
            __stcg(to + kRows * D + kRows + row, sum);
          }
        }
      }
    }
    __syncthreads();
    // ---- the CTA that arrives last at an item joins its parts, in their order
    const int pending = __popc(partial);  // the first warps' item, the last warps', or both
    if (pending > 0) {
      const int waiting[2] = {__ffs(partial) - 1, 31 - __clz(partial)};
      if ((int)threadIdx.x < pending) {
        const Part p = parts_sh[threadIdx.x == 0 ? waiting[0] : waiting[1]];
        const int first_unit = (int)(p.slot0 / kWarps);
        const uint32_t others = (uint32_t)((p.slot0 + p.pieces - 1) / kWarps - first_unit);
        // releases what the CTA wrote before its barrier, and acquires what the others released
        uint32_t before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                     : "=r"(before)
                     : "l"(a.counters + first_unit)
                     : "memory");
        const bool last = before == others;
        if (last) a.counters[first_unit] = 0;
        last_sh[threadIdx.x] = last;
      }
      __syncthreads();
      for (int which = 0; which < pending; ++which) {
        if (!last_sh[which]) continue;
        const Part part = parts_sh[which == 0 ? waiting[0] : waiting[1]];
        const int first_unit = (int)(part.slot0 / kWarps);
        const int parts = (int)((part.slot0 + part.pieces - 1) / kWarps) - first_unit + 1;
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
                const float* from = part_at<D, NT>(a, part, first_unit + x0 + x);
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
      __syncthreads();
    }
  }
}

template <int D, int NT>
cudaError_t run(const KvAttentionArgs& a, cudaStream_t s) {
  using L = Shape<D, NT>;
  const int bytes = L::shared_bytes(a.batch.entries);
  const void* fn = reinterpret_cast<const void*>(kv_attention<D, NT>);
  cudaError_t e = ensure_dynamic_smem(fn, bytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_attention<D, NT>, kKvSms * L::kCtasPerSm, L::kThreads, bytes, s, a);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionArgs& args, cudaStream_t s) {
  KvAttentionArgs a = args;
  int exponent;
  const float fraction = frexpf(fminf(fmaxf(a.scale * 1.4426950408889634f, FLT_MIN), FLT_MAX), &exponent);
  a.key_scale = ldexpf(fraction, -kKeyShift);
  a.row_scale = ldexpf(1.f, exponent > 127 ? 127 : exponent);
  const int group = a.q_heads / a.cache.kv_heads;
  const long long rows = (long long)a.max_q * group;
  // More rows than one tile here holds, and so on average too (a chunk among many single tokens would
  // have those in tiles of 256 rows): the other kernel.  16 entries, 4000 to 8000 keys, 4 key
  // heads, head_dim 128: 40 rows 89 us against 105 here, 64 rows 82 against 106, 128 rows 84 against 207;
  // head_dim 64: 62 against 72, 60 against 73, 61 against 141.  32 rows take 52 us here, 81 there.
  // Up to 64 rows of few entries and heads stay, as their long sequences are cut finer here: 64 rows of one
  // head over 131,072 keys 62 us against 105, 40 rows of 4 heads over 4000 23 against 28 (but 64
  // rows over 100 keys 14 against 11); 32 heads of 100 to 200 keys 16 against 14, 128 heads 28 against 16.
  const long long items = (long long)a.batch.entries * a.cache.kv_heads;
  const bool many = rows > (items < 64 ? 64 : 32) &&
                    (long long)a.batch.tokens * group > 32ll * a.batch.entries;
  if (many && kv_attention_rows_supported(a)) return launch_kv_attention_rows(a, s);
  switch (a.cache.head_dim) {
    case 64: return rows <= 8 ? run<64, 1>(a, s) : rows <= 16 ? run<64, 2>(a, s) : run<64, 4>(a, s);
    case 128:
      return rows <= 8 ? run<128, 1>(a, s) : rows <= 16 ? run<128, 2>(a, s) : run<128, 4>(a, s);
    default: return rows <= 8 ? run<256, 1>(a, s) : run<256, 2>(a, s);
  }
}

}  // namespace wd
