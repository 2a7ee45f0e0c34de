// wd_kv_attention_rows.cu - attention over the 4-bit cache for many query rows to a key head: chunks of
// a prompt (declared in include/wd_kv.h; few rows take wd_kv_attention.cu, which converts the
// keys again for every 32 rows).
//
// A CTA has a tile of 256 query rows (heads that share the key head, and tokens) in two halves of
// 128 and goes over the keys 64 at a time.  S = Q K^T and O = P V are tcgen05 products with S,
// P and O in tensor memory; every key tile is turned into FP16 once for all rows.  The warps
// have roles, with shared-memory barriers between them:
//   0-7   softmax of the two halves, a thread to a row: S from tensor memory, P back as the left
//         operand of P V, in S's place, O rescaled in place where the reference has moved
//   8-13  conversion: two warps write K, four V, scales applied, into a ring of swizzled tiles
//   14    the products, S two tiles ahead, so that they run during the softmax
//   15    bulk copies of the groups into a ring
//
//   - K: where the scales of a tile are within 2^22 of each other, its blocks are scaled by
//     2^(s - R), exactly, and 2^(R - 127) goes into the rows' softmax factor.  Else each token has its
//     own r, the largest scale of its blocks that are not all zero, 2^(s - r) is exact down to
//     2^-23, and 2^(r - 127) multiplies the logit in FP32 (as 2^(r - 153), the rest in the row's factor).  Smaller blocks are 0 in the tile, and the
//     softmax adds their part of the logits in FP32 (a query may be zero where the large ones are).
//   - V: blocks are scaled by 2^(s - R), exactly down to 2^-22, with R at least the largest scale
//     met for the block of channels (16 times it where it was set, so that it is seldom
//     set again; keys that some of the rows do not see raise it to 2^23 at most).  What is smaller or
//     larger, or NaN, is 0 in the tile, and added to O in FP32 one by one.
//   - Queries, P and the lazy maximum as in wd_kv_attention.cu.
// An item (entry, tile of rows, key head) is cut into pieces along the keys where there are not
// enough items for the GPU; the CTA that finishes last joins them in their order.
//
// Measured (bfloat16, head_dim 128, 8 query heads to a key head).  2432 tokens after 30,336, 4 key
// heads: 1275 us, 986 TFLOP/s, 0.52 of the cuBLAS rate; the products alone would take 1300
// cycles a tile of 64 keys, the softmax takes about 2300 (64 exponentials a thread at a quarter of the
// rate, and instructions that two warps to a scheduler do not hide).  Chunks of 200 to
// 256 tokens in two sequences of 4100 to 6001, 4 key heads: 81 us, where wd_kv_attention.cu
// takes 233; the 48 tiles of a piece cost 58 us, the rest is the start (7 us), Q and the joins.
// Tried: m16n8k16 products over ldmatrix fragments (354 us); two warps for V (130 us); products
// issued without uniform registers (2432 tokens: 1651 us, then 1328); 160 registers for the softmax
// warps and 88 for the others by setmaxnreg, which leaves no spills (1392; with 128 each, 32 bytes
// of stores and about 130 of loads are spilled); the rare keys noted in a word that two of the
// conversion warps write (1306 to 1345, head_dim 64 1043 against 1005).
#include "wd_kv_attention.cuh"

namespace wd {
namespace {

constexpr int kRows = 256;  // of a tile
constexpr int kKeys = 64;  // of a tile
constexpr int kStages = 3;  // of converted tiles
constexpr int kRaws = 3;    // of tiles as they are stored
constexpr int kSoftmaxThreads = 256;
// the first warps of the other roles (the last warp loads)
constexpr int kKeyWarp = 8, kValueWarp = 10, kIssueWarp = 14, kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxEntries = 1024;  // of a batch: they are kept in shared memory
constexpr int kAlike = 30;  // octaves around 1 in which a tile's R may be part of a row's factor
// Logits whose reference is beyond this are rounded before the reference is taken off: in one fused step the
// rounding of the reference alone, 2^-24 of it, would be an exponent.
constexpr float kSteep = 16384.f;
constexpr int kRoom = 4;  // octaves that a V reference is set above the largest scale
constexpr uint32_t kTmemColumns = 512;

template <int D>
struct Rows {
  using G = KvGroup<D>;
  static constexpr int kRawBytes = 4 * G::kBytes;
  static constexpr int kTileBytes = kKeys * D * 2;    // K or V of a tile, FP16
  static constexpr int kHalfBytes = 128 * D * 2;      // Q of a half
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kHalfBytes;
  static constexpr int kV = kK + kStages * kTileBytes;
  static constexpr int kRaw = kV + kStages * kTileBytes;
  // float [stages][kKeys]: 2^(r - 127 - kKeyShift) of K, negative if there is more of the key than the tile
  // has, -inf if it is not there
  static constexpr int kCol = kRaw + kRaws * kRawBytes;
  static constexpr int kFactor = kCol + kStages * kKeys * 4;  // FP16 [kKeys][4]: of V
  // uint32 [stages][4]: V's references, whether there is more of it; K's 2^(R - 127 - kFactorShift), or 0
  static constexpr int kInfo = kFactor + kKeys * 8;
  static constexpr int kBars = kInfo + kStages * 16;
  // uint64, one after the other:
  static constexpr int kRawFull = 0, kRawFree = kRawFull + kRaws, kFull = kRawFree + kRaws,
                       kFree = kFull + kStages, kScore = kFree + kStages, kProb = kScore + 4,
                       kOut = kProb + 4, kQuery = kOut + 2, kJoinIn = kQuery + 2,
                       kJoinOut = kJoinIn + 1, kDrain = kJoinOut + 1, kBarriers = kDrain + 1;
  // int [4]: tensor memory, last, next to arrive at; groups of the raw tiles that are not there, a byte each
  static constexpr int kWords = kBars + 8 * kBarriers;
  static constexpr int kScan = (kWords + 31) / 16 * 16;  // int [16], float [16], int [16]
  static constexpr int kEntries = kScan + 192;           // Planned [entries]
  static constexpr int shared_bytes(int entries) { return kEntries + 32 * entries + 1024; }
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kRaw % 128 == 0, "alignment");
  static_assert(kCol % 16 == 0 && kInfo % 16 == 0 && kBars % 8 == 0, "alignment");
  static_assert(shared_bytes(kMaxEntries) <= 232448, "shared memory");
  // columns of tensor memory: O of the halves, and two S of each, whose place P takes
  static constexpr uint32_t kO = 0, kS = 2 * D;
  static_assert(kS + 4 * kKeys <= kTmemColumns, "tensor memory");
};

// n columns of the warp's 32 TMEM lanes, a lane to a thread.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
        "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
        "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
        "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
        "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]),
        "=r"(r[54]), "=r"(r[55]), "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]),
        "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]),
      "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
      "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
      "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]),
      "r"(addr)
      : "memory");
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t addr) {
  uint32_t r;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(addr)
      : "memory");
  return r;
}
__device__ __forceinline__ void tmem_st1(uint32_t addr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr), "r"(r) : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Descriptor of a 128-byte swizzled operand in shared memory: 8 rows of 128 bytes after one another,
// 1024 bytes to the next 8, `panel` bytes to the next 128 of the rows that run along the
// operand's M or N.
__device__ __forceinline__ uint64_t smem_operand(uint32_t addr, uint32_t panel) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(panel >> 4) << 16 |
         (uint64_t)(1024u >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// FP16 x FP16 -> FP32, M = 128; b_along_n: the right operand's rows run along N, not K.
__host__ __device__ constexpr uint32_t mma_kind(int n, bool b_along_n) {
  return 1u << 4 | (b_along_n ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_smem(uint32_t d, uint64_t a, uint64_t b, uint32_t kind,
                                         bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t kind,
                                         bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"((uint32_t)add)
      : "memory");
}
// One lane of a warp that runs together.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// `bar` gets an arrival when the products issued so far are done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

// Byte of 16-byte chunk `chunk` of a row of a tile of `rows` rows: panels of 128 bytes.
__device__ __forceinline__ int tile_at(int rows, int row, int chunk) {
  return (chunk >> 3) * rows * 128 + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
}

// FP16 2^-d (a subnormal from 15 on, exact), 0 from 24 on, where 0.5 x 2^-d, of E2M1, is no FP16 number; d >= 0.
__device__ __forceinline__ uint32_t half_power(int d) {
  return d < 15 ? (uint32_t)(15 - d) << 10 : d < 24 ? 1u << (24 - d) : 0u;
}

// Whether V that is 2^-d of the reference is in the tile: else it is added on its own.
__device__ __forceinline__ bool in_tile(int d) { return (unsigned)d <= 22u; }

// Whether a block of K that is 2^-d of its token's largest is in the tile (as half_power has it).
__device__ __forceinline__ bool key_in_tile(int d) { return d <= 23; }

// Where the keys of one head and layer of a sequence lie.
struct Keys {
  const int32_t* row;   // of the table
  const uint8_t* base;  // the head in page 0
  long long page_bytes;
  int page_shift, num_pages;
};
__device__ __forceinline__ Keys keys_of(const KvView& c, int slot, int layer, int head) {
  return Keys{c.table + (long long)slot * c.columns,
              c.pool + layer * c.layer_bytes + (long long)head * c.head_bytes, c.page_bytes,
              c.page_shift, c.num_pages};
}
// The group of a key whose page is there (within the pool whatever the table says by now).
template <int D>
__device__ __forceinline__ const uint8_t* group_of(const Keys& k, int key) {
  const int page = k.row[key >> k.page_shift];
  return k.base + (page >= 0 && page < k.num_pages ? page : 0) * k.page_bytes +
         ((key & ((1 << k.page_shift) - 1)) >> 4) * KvGroup<D>::kBytes;
}

// What of a key's sum with a query row is not in its tile, times 2^-kKeyShift.  grp: the key's group, of which it
// is token t; q: the tile of the row's half, in shared memory.
template <int D>
__device__ __forceinline__ float key_rest(const uint8_t* grp, int t, const uint8_t* q, int row) {
  using G = KvGroup<D>;
  int top = 0;
  float sum = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass)
#pragma unroll 1
    for (int c = 0; c < G::kBlocks; ++c) {
      const int s = grp[G::kKScale + t * G::kBlocks + c];
      if (pass == 1 && (s == 255 || key_in_tile(top - s))) continue;
      uint32_t any = 0;
      float part = 0.f;
#pragma unroll 1
      for (int t8 = 0; t8 < 4; ++t8) {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(grp + G::k_word(t, c, t8));
        any |= w & 0x77777777u;
        if (pass == 0) continue;
        uint32_t k[4];
        e2m1x8(w, k[0], k[1], k[2], k[3]);
        const uint4 x = *reinterpret_cast<const uint4*>(q + tile_at(128, row, 4 * c + t8));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&k[e]));
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&xs[e]));
          part = fmaf(a.y, b.y, fmaf(a.x, b.x, part));
        }
      }
      if (pass == 0 && (s == 255 || any != 0u)) top = max(top, s);
      if (pass == 1 && any != 0u) sum += part * exp2f((float)(s - 127 - kKeyShift));
    }
  return sum;
}

// Whether a tile has keys of which there is more, or that are not there.
__device__ __forceinline__ bool rare_tile(const float* col, int lane) {
  return __any_sync(kAll, signbit(col[lane]) || signbit(col[32 + lane]));
}
// The scores of such a tile times `col`, in place, key by key.
template <int D>
__device__ __noinline__ void rare_scores(const Keys k, uint32_t s_at, const float* col, int j0, int end,
                                         const uint8_t* q, int row) {
#pragma unroll 1
  for (int t = 0; t < kKeys && j0 + t < end; ++t) {
    const float by = col[t];
    float sum = -INFINITY;
    if (by != -INFINITY) {
      sum = __uint_as_float(tmem_ld1(s_at + t)) * fabsf(by);
      if (by < 0.f) sum += key_rest<D>(group_of<D>(k, j0 + t), (j0 + t) & 15, q, row);
    }
    tmem_st1(s_at + t, __float_as_uint(sum));
  }
  tmem_st_wait();
}
// The tile's logits, in place, less the reference `from`: -inf but for keys lo to hi of the tile.
__device__ __noinline__ void steep_scores(uint32_t s_at, const float* col, float factor, float from, int lo,
                                          int hi) {
#pragma unroll 1
  for (int t = 0; t < kKeys; ++t) {
    float v = __uint_as_float(tmem_ld1(s_at + t));
    if (col) v *= col[t];
    v = t < lo || t > hi ? -INFINITY : __fsub_rn(__fmul_rn(v, factor), from);
    tmem_st1(s_at + t, __float_as_uint(v));
  }
  tmem_st_wait();
}

// Two FP32 values in one register pair: one instruction for both.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ int byte_of(uint32_t w, int c) { return (int)(w >> (8 * c) & 0xFFu); }

// A piece as its warps see it.
struct Piece {
  Part part;
  int slot, len, key0, tiles, end, rows;
  int lo;                  // no row sees keys before it,
  int shared_lo, shared;   // and every row sees those from shared_lo up to `shared`
};

// An entry and its share of the work: each of its tiles of rows, for each key head, is cut into pieces;
// those of the entries before come first.
struct Planned {
  Entry entry;
  int row_tiles, seen;  // tiles of rows, and of keys that one of them sees at most
  int before, pieces;
};

// Not inlined: every role looks up its pieces, and with as much more code the roles' loops are
// fetched more slowly (57 items in 2 pieces: 83 us, inlined 89).
__device__ __noinline__ Piece find_piece(const Planned* plan, int entries, int heads, int group,
                                         int window, unsigned q, int unit) {
  int lo = 0, hi = entries;
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan[mid].before <= unit) lo = mid; else hi = mid;
  }
  const Planned& e = plan[lo];
  const unsigned rest = (unsigned)(unit - e.before), pieces = (unsigned)e.pieces;
  const unsigned item = rest / pieces, piece = rest - item * pieces;
  const int turn = (int)(item / heads);
  Piece p;
  p.part.slot0 = unit - piece;
  p.part.pieces = (int)pieces;
  p.part.head = (int)(item % heads);
  p.part.tile = turn & 1 ? e.row_tiles - 1 - (turn >> 1) : turn >> 1;
  p.part.first = e.entry.first;
  p.part.n = e.entry.n;
  const Span span = tile_span<kRows>(e.entry, p.part.tile, group, window);
  p.slot = e.entry.slot;
  p.len = e.entry.len;
  p.end = span.end;
  p.key0 = (int)min((long long)span.first * kStep / kKeys * kKeys + (long long)piece * q * kKeys,
                    (long long)(span.end + kKeys - 1) / kKeys * kKeys);
  p.tiles = max(0, min((int)q, (span.end - p.key0 + kKeys - 1) / kKeys));
  p.rows = min(kRows, e.entry.n * group - p.part.tile * kRows);
  const int pos0 = p.len - p.part.n + (p.part.n > 1 ? p.part.tile * kRows / group : 0);  // first row's
  p.lo = window > 0 ? max(0, pos0 - window + 1) : 0;
  p.shared_lo = window > 0 ? max(0, p.end - window) : 0;
  p.shared = pos0 + 1;
  return p;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_rows(const KvAttentionArgs a) {
  using G = KvGroup<D>;
  using L = Rows<D>;
  constexpr int CB = G::kBlocks;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((0u - smem_u32(smem_raw)) & 1023u);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const KvView& cache = a.cache;
  const int heads = cache.kv_heads, group = a.q_heads / heads;
  int* scan = reinterpret_cast<int*>(smem + L::kScan);
  float* scan_items = reinterpret_cast<float*>(smem + L::kScan + 64);
  int* scan_longest = reinterpret_cast<int*>(smem + L::kScan + 128);
  Planned* plan = reinterpret_cast<Planned*>(smem + L::kEntries);
  volatile int* words = reinterpret_cast<volatile int*>(smem + L::kWords);
  const uint32_t bars = smem_u32(smem + L::kBars);
  const auto bar = [&](int i) { return bars + 8 * i; };
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRaws; ++i) {
      mbar_init(bar(L::kRawFull + i), 1);
      mbar_init(bar(L::kRawFree + i), kIssueWarp - kKeyWarp);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(L::kFull + i), kIssueWarp - kKeyWarp);
      mbar_init(bar(L::kFree + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::kScore + 2 * i), 2);
      mbar_init(bar(L::kScore + 2 * i + 1), 2);
      mbar_init(bar(L::kProb + 2 * i), 4);
      mbar_init(bar(L::kProb + 2 * i + 1), 4);
      mbar_init(bar(L::kOut + i), 1);
      mbar_init(bar(L::kQuery + i), 128);
    }
    mbar_init(bar(L::kJoinIn), kSoftmaxThreads);
    mbar_init(bar(L::kJoinOut), 1);
    mbar_init(bar(L::kDrain), 1);
    mbar_init_fence();
    words[2] = blockIdx.x;
  }
  if (warp == kIssueWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(smem + L::kWords)),
                 "r"(kTmemColumns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tmem_fence_before();
  }
  grid_dependency_wait();  // nothing above reads what an earlier kernel may write
  grid_launch_dependents();

  // ---- the division of the work: pieces of q tiles of keys
  float items = 0.f;
  int longest = 1;
#pragma unroll 1
  for (int b = threadIdx.x; b < a.batch.entries; b += kThreads) {
    const Entry e = load_entry(a, b);
    const int tiles = tiles_of<kRows>(e, group);
    // (one more: a window's tiles start anywhere)
    const int seen = (steps_of<kRows>(e, group, a.window) + 2) / 2;
    plan[b].entry = e;
    plan[b].row_tiles = tiles;
    plan[b].seen = seen;
    items += (float)tiles;
    if (e.n > 0) longest = max(longest, seen);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) items += __shfl_xor_sync(kAll, items, off);
  longest = __reduce_max_sync(kAll, longest);
  if (lane == 0) {
    scan_items[warp] = items;
    scan_longest[warp] = longest;
  }
  __syncthreads();
  items = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    items += scan_items[w];
    longest = max(longest, scan_longest[w]);
  }
  items *= (float)heads;
  // Into how many pieces is the longest item cut?  Each lane rates a number: passes of the CTAs over
  // all pieces, each as long as its tiles and what a piece costs besides (about twelve tiles), and
  // the parts that an item's last CTA reads (about 2/3 of a tile each).  One piece needs no
  // parts; else there is room for kKvMaxRowUnits.  Measured: 64 items of up to 126 tiles 86 us in 2
  // pieces each, 97 in 4; 57 items of up to 94 tiles 83 us in 2 pieces, 95 in 5.
  unsigned q = longest;
  bool cut = false;
  if (items < 1.5f * (float)gridDim.x) {
    constexpr int kPieces[16] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 12, 16, 20, 26, 38, 76, 152};
    int pieces = 1;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((lane & 15) == i) pieces = kPieces[i];
    const unsigned tiles = (longest + pieces - 1) / pieces;
    int units = 0;
#pragma unroll 1
    for (int b = 0; b < a.batch.entries; ++b)
      units += plan[b].row_tiles * heads * (int)((plan[b].seen + tiles - 1) / tiles);
    float cost = (float)((units + gridDim.x - 1) / gridDim.x) * (float)(tiles + 12) +
                 (pieces > 1 ? 0.7f * (float)pieces + 2.f : 0.f);
    if (pieces > 1 && (units > kKvMaxRowUnits || tiles < 2)) cost = INFINITY;
    const uint32_t best = __reduce_min_sync(kAll, __float_as_uint(cost));
    const int winner = __ffs(__ballot_sync(kAll, __float_as_uint(cost) == best)) - 1;
    q = __shfl_sync(kAll, tiles, winner);
    cut = __shfl_sync(kAll, pieces, winner) > 1;
  }
  int total = 0;
#pragma unroll 1
  for (int base = 0; base < a.batch.entries; base += kThreads) {
    const int b = base + threadIdx.x;
    int cost = 0;
    if (b < a.batch.entries) {
      plan[b].pieces = cut ? (plan[b].seen + q - 1) / q : 1;
      cost = plan[b].row_tiles * heads * plan[b].pieces;
    }
    int incl = cost;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(kAll, incl, off);
      if (lane >= off) incl += t;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    int below = total, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) below += scan[w];
      all += scan[w];
    }
    if (b < a.batch.entries) plan[b].before = below + incl - cost;
    total += all;
  }
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = (uint32_t)words[0];

  const auto find = [&](int unit) {
    return find_piece(plan, a.batch.entries, heads, group, a.window, q, unit);
  };
  // A wait of all lanes of a warp; false, and the flag, where it ran out: the role then ends.
  const auto wait = [&](int i, uint32_t parity) {
    if (__all_sync(kAll, mbar_try_wait(bar(i), parity))) return true;
    const bool ok = __all_sync(kAll, mbar_wait(bar(i), parity));
    if (!ok && lane == 0) atomicOr(cache.flag, WD_KV_FLAG_TIMEOUT);
    return ok;
  };

  const auto load_role = [&]() {
    uint32_t count = 0;  // tiles so far
    bool ok = true;
#pragma unroll 1
    for (int unit = blockIdx.x; ok && unit < total; unit += gridDim.x) {
      const Piece p = find(unit);
#pragma unroll 1
      for (int i = 0; i < p.tiles; ++i, ++count) {
        const int r = count % kRaws;
        if (count >= kRaws && !wait(L::kRawFree + r, (count / kRaws - 1) & 1)) {
          ok = false;
          break;
        }
        const int pos = p.key0 + i * kKeys + 16 * lane;
        const bool asked = lane < 4 && pos < p.end;
        const int page = asked ? kv_page(cache, p.slot, pos >> cache.page_shift) : 0;
        const bool mine = asked && page >= 0;
        const uint32_t groups = __ballot_sync(kAll, mine);
        const uint32_t gone = __ballot_sync(kAll, asked && page < 0);
        if (lane == 0) {
          smem[L::kWords + 12 + r] = (uint8_t)gone;
          mbar_arrive_expect_tx(bar(L::kRawFull + r), __popc(groups) * G::kBytes);
        }
        __syncwarp();
        if (mine)
          bulk_g2s_nohint(smem_u32(smem + L::kRaw) + r * L::kRawBytes + lane * G::kBytes,
                          kv_group(cache, page, a.layer, p.part.head, pos, G::kBytes), G::kBytes,
                          bar(L::kRawFull + r));
      }
    }
    // nothing in flight at the end, whatever the others did
    for (uint32_t c = count < kRaws ? 0 : count - kRaws; c < count; ++c)
      wait(L::kRawFull + c % kRaws, (c / kRaws) & 1);
  };

  const auto convert_role = [&]() {
    const bool values = warp >= kValueWarp;
    const int own = warp - (values ? kValueWarp : kKeyWarp);  // which of the tile's keys
    uint32_t count = 0;
#pragma unroll 1
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
      const Piece p = find(unit);
      uint32_t ref = 0;  // V's references, a byte to a block
#pragma unroll 1
      for (int i = 0; i < p.tiles; ++i, ++count) {
        const int r = count % kRaws, st = count % kStages;
        if (!wait(L::kRawFull + r, (count / kRaws) & 1)) return;
        const uint8_t* raw = smem + L::kRaw + r * L::kRawBytes;
        const int left = p.end - (p.key0 + i * kKeys);  // keys of the tile
        const uint32_t gone = smem[L::kWords + 12 + r];  // groups that are not there
        // the scales of all keys, 32h + lane, of which every warp makes the same
        uint32_t sc[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 32 * h + lane;
          sc[h] = lds_scales<CB>(raw + (t >> 4) * G::kBytes +
                                 (values ? G::kVScale : G::kKScale) + (t & 15) * CB).v[0];
          // (nobody sees these: any number of the others' size)
          if (gone != 0u && (gone >> (t >> 4) & 1u)) sc[h] = values ? ref : 0x7F7F7F7Fu;
        }
        if (!values) {
          // scales that are alike in all of the tile become one factor of its logits
          int high = 0, low = 255;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (32 * h + lane >= left) continue;
#pragma unroll
            for (int c = 0; c < CB; ++c) {
              high = max(high, byte_of(sc[h], c));
              low = min(low, byte_of(sc[h], c));
            }
          }
          high = __reduce_max_sync(kAll, high);
          low = __reduce_min_sync(kAll, low);
          const bool alike = gone == 0u &&
              high - low <= 22 && high >= 127 - kAlike && high <= 127 + kAlike;
          const int t = 32 * own + lane;
          const uint32_t mine = own ? sc[1] : sc[0];
          const uint8_t* codes = raw + (t >> 4) * G::kBytes + (t & 15) * 16 * CB;
          int top = high;
          bool rest = false;  // the token has blocks that are not in the tile
          if (!alike) {
            uint32_t any[CB] = {};
            for (int j = 0; j < 4; ++j) {
              const Words<CB> w = lds<CB>(codes + j * 4 * CB);
#pragma unroll
              for (int c = 0; c < CB; ++c) any[c] |= w.v[c];
            }
            top = 0;
#pragma unroll
            for (int c = 0; c < CB; ++c) {
              const int s = byte_of(mine, c);
              if (s == 255 || (any[c] & 0x77777777u)) top = max(top, s);
            }
#pragma unroll
            for (int c = 0; c < CB; ++c)
              rest |= t < left && (any[c] & 0x77777777u) && !key_in_tile(top - byte_of(mine, c));
          }
          uint32_t f[CB];
#pragma unroll
          for (int c = 0; c < CB; ++c) f[c] = half_power(max(0, top - byte_of(mine, c))) * 0x10001u;
          if (count >= kStages && !wait(L::kFree + st, (count / kStages - 1) & 1)) return;
          uint8_t* to = smem + L::kK + st * L::kTileBytes;
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            const int c4 = ((t >> 1) & 3) ^ j;  // in this order the banks are taken once each
            const Words<CB> w = lds<CB>(codes + c4 * 4 * CB);
#pragma unroll
            for (int c = 0; c < CB; ++c) {
              uint4 v;
              e2m1x8(w.v[c], v.x, v.y, v.z, v.w);
              v = make_uint4(mul_half2(v.x, f[c]), mul_half2(v.y, f[c]), mul_half2(v.z, f[c]),
                             mul_half2(v.w, f[c]));
              *reinterpret_cast<uint4*>(to + tile_at(kKeys, t, 4 * c + c4)) = v;
            }
          }
          float col = t >= left ? 0.f : top == 255 ? __uint_as_float(0x7FC00000u)
                                                   : exp2f((float)(top - 127 - kKeyShift));
          if (rest) col = -col;
          if (gone != 0u && (gone >> (t >> 4) & 1u)) col = -INFINITY;
          reinterpret_cast<float*>(smem + L::kCol)[st * kKeys + t] = col;
          if (own == 0 && lane == 0)
            *reinterpret_cast<float*>(smem + L::kInfo + 16 * st + 8) =
                alike ? exp2f((float)(high - 127 - kFactorShift)) : 0.f;
        } else {
          // Mostly all scales are within 2^15 below the references.
          bool odd = false, other = false;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t d0 = ((ref & 0x00FF00FFu) | 0x80008000u) - (sc[h] & 0x00FF00FFu);
            const uint32_t d1 = ((ref >> 8 & 0x00FF00FFu) | 0x80008000u) - (sc[h] >> 8 & 0x00FF00FFu);
            odd |= 32 * h + lane < left && ((d0 | d1) & 0x7FF07FF0u) != 0u;
          }
          if (__any_sync(kAll, odd)) {
            // What no row sees takes part in nothing, and a key that not every row sees must not push what the
            // others see out of FP32: it raises the reference to kSharedMost at most.
            int most[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int t = 32 * h + lane, key = p.key0 + i * kKeys + t;
              most[h] = key < p.lo || t >= left ? -1
                        : key >= p.shared_lo && key < p.shared ? 254 : (int)kSharedMost - kRoom;
            }
#pragma unroll
            for (int c = 0; c < CB; ++c) {
              int s = 0;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int x = byte_of(sc[h], c);
                if (x != 255) s = max(s, min(x, most[h]));
              }
              s = __reduce_max_sync(kAll, s);
              if (s > byte_of(ref, c))
                ref = (ref & ~(0xFFu << (8 * c))) | (uint32_t)min(s + kRoom, 254) << (8 * c);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int c = 0; c < CB; ++c) {
                const int s = byte_of(sc[h], c);
                other |= most[h] >= 0 && (s == 255 || !in_tile(byte_of(ref, c) - s));
              }
            other = __any_sync(kAll, other);
          }
          // the factors of the warp's 16 keys, a lane to half of a key's
          uint8_t* factors = smem + L::kFactor + own * 16 * 8;
          {
            const int t = 16 * own + (lane & 15), c0 = lane >> 4 ? CB / 2 : 0;
            const uint32_t mine =
                __shfl_sync(kAll, own & 2 ? sc[1] : sc[0], t & 31) >> (8 * c0);
            uint32_t f = 0;
#pragma unroll
            for (int c = 0; c < CB / 2; ++c) {
              const int s = byte_of(mine, c), d = byte_of(ref, c0 + c) - s;
              if (t < left && s != 255 && in_tile(d)) f |= half_power(d) << (16 * c);
            }
            if constexpr (CB == 4)
              *reinterpret_cast<uint32_t*>(factors + 8 * (lane & 15) + 2 * c0) = f;
            else
              *reinterpret_cast<uint16_t*>(factors + 8 * (lane & 15) + 2 * c0) = (uint16_t)f;
          }
          __syncwarp();
          if (count >= kStages && !wait(L::kFree + st, (count / kStages - 1) & 1)) return;
          uint8_t* to = smem + L::kV + st * L::kTileBytes;
          const int g = lane >> 2, tq = lane & 3;
#pragma unroll 1
          for (int j = 0; j < 2; ++j) {  // eight keys each
            const int t = 8 * j + 2 * tq;
            const Words<CB> w = lds<CB>(raw + own * G::kBytes + G::kCodeBytes + j * 128 * CB +
                                        g * 16 * CB + tq * 4 * CB);
#pragma unroll
            for (int par = 0; par < 2; ++par) {
              const uint2 f = *reinterpret_cast<const uint2*>(factors + 8 * (t + par));
#pragma unroll
              for (int cp = 0; cp < CB / 2; ++cp) {
                const uint32_t ff = cp ? f.y : f.x;
                const uint32_t f0 = __byte_perm(ff, 0, 0x1010), f1 = __byte_perm(ff, 0, 0x3232);
                uint32_t v[4];
                e2m1x8(w.v[par * (CB / 2) + cp], v[0], v[1], v[2], v[3]);
                const int key = 16 * own + t + par, chunk = 8 * cp + (g >> 1), rest = (g & 1) * 8;
                *reinterpret_cast<uint2*>(to + tile_at(kKeys, key, chunk) + rest) =
                    make_uint2(mul_half2(v[0], f0), mul_half2(v[1], f0));
                *reinterpret_cast<uint2*>(to + tile_at(kKeys, key, chunk + 4) + rest) =
                    make_uint2(mul_half2(v[2], f1), mul_half2(v[3], f1));
              }
            }
          }
          if (own == 0 && lane == 0)
            *reinterpret_cast<uint2*>(smem + L::kInfo + 16 * st) =
                make_uint2(ref, other ? 1u : 0u);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(L::kFull + st));
          mbar_arrive(bar(L::kRawFree + r));
        }
      }
    }
  };

  // The warp runs this together, and what the products' operands are made of is known to be
  // the same in all lanes (a shuffle from one lane): they then come from uniform registers, without
  // which a product takes twice as long to issue as to run.
  const auto issue_role = [&]() {
    uint32_t count = 0, queries[2] = {0, 0}, probs[2] = {0, 0};
    const uint64_t q0 = smem_operand(smem_u32(smem + L::kQ), 0),
                   k0 = smem_operand(smem_u32(smem + L::kK), 0),
                   v0 = smem_operand(smem_u32(smem + L::kV), kKeys * 128);
    const uint32_t tm = __shfl_sync(kAll, tmem, 0);
    const auto s_at = [&](int x, uint32_t n) { return tm + L::kS + (2 * x + (n & 1)) * kKeys; };
    const auto score = [&](int x, uint32_t n, int st) {  // (16-byte units are added to descriptors)
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_smem(s_at(x, n),
                   q0 + (uint32_t)(x * L::kHalfBytes + (k >> 2) * 128 * 128 + (k & 3) * 32) / 16,
                   k0 + (uint32_t)(st * L::kTileBytes + (k >> 2) * kKeys * 128 + (k & 3) * 32) / 16,
                   mma_kind(kKeys, false), k > 0);
        mma_commit(bar(L::kScore + 2 * x + (n & 1)));
        mbar_arrive(bar(L::kScore + 2 * x + (n & 1)));  // (passes on what the conversion wrote)
      }
      __syncwarp();
    };
    const int end = __shfl_sync(kAll, total, 0);
#pragma unroll 1
    for (int unit = blockIdx.x; unit < end; unit += gridDim.x) {
      const Piece p = find(unit);
      const int tiles = __shfl_sync(kAll, p.tiles, 0);
      const int halves = __shfl_sync(kAll, p.rows, 0) > 128 ? 2 : 1;
      if (tiles == 0) continue;
      if (!wait(L::kFull + count % kStages, (count / kStages) & 1)) return;
#pragma unroll
      for (int x = 0; x < 2; ++x)
        if (x < halves) {
          if (!wait(L::kQuery + x, queries[x] & 1)) return;
          ++queries[x];
          tmem_fence_after();
          score(x, probs[x], count % kStages);
        }
      if (tiles > 1) {
        if (!wait(L::kFull + (count + 1) % kStages, ((count + 1) / kStages) & 1)) return;
        tmem_fence_after();
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (x < halves) score(x, probs[x] + 1, (count + 1) % kStages);
      }
#pragma unroll 1
      for (int i = 0; i < tiles; ++i, ++count) {
        const int st = count % kStages, next = (count + 2) % kStages;
        const bool more = i + 2 < tiles;
#pragma unroll
        for (int x = 0; x < 2; ++x)
          if (x < halves) {
            if (!wait(L::kProb + 2 * x + (probs[x] & 1), (probs[x] >> 1) & 1)) return;
            tmem_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kKeys / 16; ++k)
                mma_tmem(tm + L::kO + x * D, s_at(x, probs[x]) + 8 * k,
                         v0 + (uint32_t)(st * L::kTileBytes + k * 16 * 128) / 16,
                         mma_kind(D, true), true);
              mma_commit(bar(L::kOut + x));
              if (x == halves - 1) mma_commit(bar(L::kFree + st));
            }
            __syncwarp();
            if (more) {
              if (x == 0 && !wait(L::kFull + next, ((count + 2) / kStages) & 1)) return;
              tmem_fence_after();
              score(x, probs[x], next);  // into P's place, behind the product that reads it
            }
            ++probs[x];
          }
      }
    }
  };

  const auto softmax_role = [&]() {
    const int x = warp >> 2;                  // the half
    const int row = threadIdx.x;              // of the tile
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // the warp's lanes of tensor memory
    const uint32_t o_at = tmem + lanes + L::kO + x * D;
    const bool vec =
        ((reinterpret_cast<uintptr_t>(a.q) & 15) | (a.q_token & 7) | (a.q_head & 7)) == 0;
    uint32_t count = 0, mine = 0, joins = 0;  // tiles so far, of them those of this half
    uint32_t outs = 0;                        // products P V of this half that are known to be done
    const auto wait_outs = [&](uint32_t n) {
#pragma unroll 1
      for (; outs < n; ++outs)
        if (!wait(L::kOut + x, outs & 1)) return false;
      tmem_fence_after();
      return true;
    };
#pragma unroll 1
    for (int unit = blockIdx.x; unit < total; unit += gridDim.x) {
      const Piece p = find(unit);
      const bool real = row < p.rows;
      const int flat = p.part.tile * kRows + row;
      const int token = real ? flat / group : 0;
      const int head = p.part.head * group + flat - token * group;
      const long long at = (long long)(p.part.first + token) * a.q_heads + head;
      const bool active = x == 0 || p.rows > 128;
      const int pos = p.len - p.part.n + token;
      float m = -INFINITY, l = 0.f, factor = 0.f;
      uint32_t ref = 0;
      bool steep = false;  // a reference of one of the warp's rows is beyond kSteep
      if (active && p.tiles > 0) {
        // ---- the row's query
        const long long q_at = (p.part.first + token) * a.q_token + head * a.q_head;
        Words<4> w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 8; ++c) w[c] = Words<4>{{0u, 0u, 0u, 0u}};
        if (real && vec) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = load8(a, q_at + 8 * c, true);
        } else if (real) {
#pragma unroll
          for (int c = 0; c < D / 8; ++c) w[c] = load8(a, q_at + 8 * c, false);
        }
        uint32_t bits = 0;  // the largest magnitude: of 16 bits each it is the largest integer
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k) bits = __vmaxu2(bits, w[c].v[k] & 0x7FFF7FFFu);
        bits = max(bits & 0xFFFFu, bits >> 16);
        bits = a.half ? __float_as_uint(__half2float(__ushort_as_half((unsigned short)bits)))
                      : bits << 16;
        const RowScale scale = row_scale(bits);
        factor = pos < 0 ? 1.f : row_factor(scale, a.scale);  // (sees nothing: no NaN)
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          float v[8];
          widen8(w[c], a.half, v);
          *reinterpret_cast<uint4*>(smem + L::kQ + x * L::kHalfBytes + tile_at(128, row & 127, c)) =
              row_fragment(v, scale);
        }
        fence_async_smem();
        __syncwarp();
        uint32_t none[32] = {};
#pragma unroll
        for (int c = 0; c < CB; ++c) tmem_st32(o_at + 32 * c, none);
        tmem_st_wait();
        tmem_fence_before();
        mbar_arrive(bar(L::kQuery + x));
      }
      const int row_lo = real && a.window > 0 ? max(0, pos - a.window + 1) : 0;
      const int row_hi = real ? pos : 0x7FFFFFFF;  // no row: nothing to hide, never stored
      if (!active) {
        count += p.tiles;
      } else {
#pragma unroll 1
        for (int i = 0; i < p.tiles; ++i, ++count, ++mine) {
          const int st = count % kStages, j0 = p.key0 + i * kKeys;
          if (!wait(L::kScore + 2 * x + (mine & 1), (mine >> 1) & 1)) return;
          tmem_fence_after();
          if (i > 1) outs = max(outs, mine - 1);  // S came behind P V of two tiles before
          const uint32_t s_at = tmem + lanes + L::kS + (2 * x + (mine & 1)) * kKeys;
          uint32_t sr[64];
          tmem_ld64(s_at, sr);
          const uint4 info = *reinterpret_cast<const uint4*>(smem + L::kInfo + 16 * st);
          const bool whole = __all_sync(kAll, j0 >= row_lo && j0 + kKeys - 1 <= row_hi);
          const float* col = reinterpret_cast<const float*>(smem + L::kCol) + st * kKeys;
          float f = factor;
          if (info.z) {
            f *= __uint_as_float(info.z);
            if (f == 0.f) f = 1.2e-38f;  // (-inf stays -inf)
          } else {
            f = shifted_factor(f);
            if (rare_tile(col, lane)) {
              rare_scores<D>(keys_of(cache, p.slot, a.layer, p.part.head), s_at, col, j0, p.end,
                             smem + L::kQ + x * L::kHalfBytes, row & 127);
              tmem_ld64(s_at, sr);
            } else {
#pragma unroll
              for (int n = 0; n < kKeys; ++n)
                sr[n] = __float_as_uint(__uint_as_float(sr[n]) * col[n]);
            }
          }
          if (!whole) {
#pragma unroll
            for (int n = 0; n < kKeys; ++n)
              if (j0 + n < row_lo || j0 + n > row_hi) sr[n] = 0xFF800000u;
          }
          float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int n = 0; n < kKeys; n += 2)
            top4[n / 2 & 3] =
                max3(top4[n / 2 & 3], __uint_as_float(sr[n]), __uint_as_float(sr[n + 1]));
          const float top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]) * f;
          const bool moved = i > 0 && info.x != ref;
          if (__any_sync(kAll, top > m + kSlack) || moved) {
            const float t = top > m + kSlack ? top : m;
            const float keep = m == -INFINITY ? (t == m ? 1.f : 0.f) : exp2_fast(m - t);
            l = m == -INFINITY ? l : l * keep;  // (a sum of NaN is not forgotten)
            m = t;
            steep = __any_sync(kAll, fabsf(m) >= kSteep && m != -INFINITY);
            if (i > 0) {
              if (!wait_outs(mine)) return;
#pragma unroll 1
              for (int c = 0; c < CB; ++c) {
                const float down = keep * exp2f((float)(byte_of(ref, c) - byte_of(info.x, c)));
                uint32_t o[32];
                tmem_ld32(o_at + 32 * c, o);
#pragma unroll
                for (int n = 0; n < 32; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * down);
                tmem_st32(o_at + 32 * c, o);
              }
            }
          }
          ref = info.x;
          float z = m == -INFINITY ? 0.f : kBias - m;
          if (steep) {
            steep_scores(s_at, info.z || rare_tile(col, lane) ? nullptr : col, f, m == -INFINITY ? 0.f : m,
                         row_lo - j0, row_hi - j0);
            tmem_ld64(s_at, sr);
            f = 1.f;
            z = kBias;
          }
          uint64_t sums[2] = {0, 0};
          const uint64_t f2 = pair(__float_as_uint(f), __float_as_uint(f)),
                         z2 = pair(__float_as_uint(z), __float_as_uint(z));
          uint32_t pr[32];
#pragma unroll
          for (int n = 0; n < kKeys; n += 2) {
            const uint64_t e = fma2(pair(sr[n], sr[n + 1]), f2, z2);
            const float p0 = exp2_fast(__uint_as_float((uint32_t)e)),
                        p1 = exp2_fast(__uint_as_float((uint32_t)(e >> 32)));
            sums[n / 2 & 1] =
                add2(sums[n / 2 & 1], pair(__float_as_uint(p0), __float_as_uint(p1)));
            pr[n / 2] = pack_half2(p0, p1);
          }
          const uint64_t both = add2(sums[0], sums[1]);
          l += __uint_as_float((uint32_t)both) + __uint_as_float((uint32_t)(both >> 32));
          tmem_st32(s_at, pr);
          tmem_st_wait();
          if (info.y) {
            // ---- what of the tile's V is not in it
            if (!wait_outs(mine)) return;
            const Keys keys = keys_of(cache, p.slot, a.layer, p.part.head);
#pragma unroll 1
            for (int t = 0; t < kKeys && j0 + t < p.end; ++t) {
              if (col[t] == -INFINITY) continue;  // (not there)
              const int key = j0 + t;
              const uint8_t* grp = group_of<D>(keys, key);
              const uint32_t weights = tmem_ld1(s_at + t / 2);
              const __half2 two = *reinterpret_cast<const __half2*>(&weights);
              const float weight = t & 1 ? __high2float(two) : __low2float(two);
              const bool seen = key >= row_lo && key <= row_hi;
#pragma unroll 1
              for (int c = 0; c < CB; ++c) {
                const int s = grp[G::kVScale + (key & 15) * CB + c], d = byte_of(ref, c) - s;
                if (s != 255 && in_tile(d)) continue;
                const float by = !seen ? 0.f
                                 : s == 255 ? __uint_as_float(0x7FC00000u) : weight * exp2f((float)-d);
                uint32_t o[32];
                tmem_ld32(o_at + 32 * c, o);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  uint32_t v[4];
                  e2m1x8(*reinterpret_cast<const uint16_t*>(grp + G::v_half(key & 15, c, k)), v[0],
                         v[1], v[2], v[3]);
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const __half2 v2 = *reinterpret_cast<const __half2*>(&v[e >> 1]);
                    o[4 * k + e] =
                        __float_as_uint(fmaf(by, e & 1 ? __high2float(v2) : __low2float(v2),
                                             __uint_as_float(o[4 * k + e])));
                  }
                }
                tmem_st32(o_at + 32 * c, o);
                tmem_st_wait();
              }
            }
          }
          // (a barrier's wait tells a phase from the next one only: never two behind)
          if (i + 1 == p.tiles && !wait_outs(mine)) return;
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(L::kProb + 2 * x + (mine & 1)));
        }
        if (!wait_outs(mine)) return;
      }

      // ---- the piece's result: its own softmax, the maximum and the sum
      const float inv = l == 0.f ? 0.f : 1.f / l;
      constexpr long long kPartFloats = (long long)kRows * (D + 2);
      float* part = a.partial + unit * kPartFloats;
      const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0;
      const auto put = [&](int ch, const float (&y)[16]) {  // sixteen channels of the row
        uint16_t* to = static_cast<uint16_t*>(a.out) + at * D + ch;
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (a.half) {
            h[k] = pack_half2(y[2 * k], y[2 * k + 1]);
          } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
            h[k] = *reinterpret_cast<const uint32_t*>(&b);
          }
        }
        if (wide) {
          reinterpret_cast<uint4*>(to)[0] = make_uint4(h[0], h[1], h[2], h[3]);
          reinterpret_cast<uint4*>(to)[1] = make_uint4(h[4], h[5], h[6], h[7]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            to[2 * k] = (uint16_t)h[k];
            to[2 * k + 1] = (uint16_t)(h[k] >> 16);
          }
        }
      };
      if (active) {
#pragma unroll 1
        for (int ch = 0; ch < D; ch += 16) {
          uint32_t o[16] = {};
          if (p.tiles > 0) tmem_ld16(o_at + ch, o);
          const float unit_c = exp2f((float)(byte_of(ref, ch / 32) - 127));
          float y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __uint_as_float(o[e]) * inv * unit_c;
          if (real && p.part.pieces == 1) {
            put(ch, y);
          } else if (real) {  // four channels of all rows after one another
            float4* to = reinterpret_cast<float4*>(part) + ch / 4 * kRows + row;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              __stcg(to + e * kRows,
                     make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]));
          }
          __syncwarp();
        }
        tmem_fence_before();
        if (real) {
          if (p.part.pieces > 1) {
            __stcg(part + kRows * D + row, m);
            __stcg(part + kRows * (D + 1) + row, l);
          } else if (a.lse) {
            a.lse[at] = l == 0.f ? -INFINITY : (m - kBias) * 0.6931471805599453f + logf(l);
          }
        }
      }
      __syncwarp();
      if (p.part.pieces == 1) {
        if (threadIdx.x == 0) words[2] = unit + gridDim.x;
        continue;
      }
      mbar_arrive(bar(L::kJoinIn));
      if (warp == 0) {
        if (!wait(L::kJoinIn, joins & 1)) return;
        if (lane == 0) {
          uint32_t before;
          asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;"
                       : "=r"(before)
                       : "l"(a.counters + p.part.slot0)
                       : "memory");
          const bool last = before == p.part.pieces - 1u;
          if (last) a.counters[p.part.slot0] = 0;
          words[1] = last;
          words[2] = unit + gridDim.x;
          mbar_arrive(bar(L::kJoinOut));
        }
        __syncwarp();
      }
      if (!wait(L::kJoinOut, joins & 1)) return;
      ++joins;
      if (words[1] && real) {
        // every part is there: join them in their order
        const float* from = a.partial + p.part.slot0 * kPartFloats;
        const float* m_at = from + kRows * D + row;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 4
        for (int k = 0; k < p.part.pieces; ++k) top = fmaxf(top, __ldcg(m_at + k * kPartFloats));
#pragma unroll 4
        for (int k = 0; k < p.part.pieces; ++k) {
          const float lk = __ldcg(m_at + k * kPartFloats + kRows);
          const float f = top == -INFINITY ? 0.f : exp2_fast(__ldcg(m_at + k * kPartFloats) - top);
          sum += lk != lk ? lk : lk * f;  // a piece of nothing but NaN has no maximum
        }
        const float all = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
        for (int ch = 0; ch < D; ch += 16) {
          float y[16] = {};
#pragma unroll 1
          for (int k0 = 0; k0 < p.part.pieces; k0 += 4) {  // four parts' loads at a time
            float by[4];
            float4 v[4][4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const bool in = k0 + k < p.part.pieces;
              const float* pk = from + (in ? k0 + k : k0) * kPartFloats;
              const float lk = __ldcg(pk + kRows * (D + 1) + row);
              const float f =
                  top == -INFINITY ? 0.f : exp2_fast(__ldcg(pk + kRows * D + row) - top);
              by[k] = in ? (lk != lk ? lk : lk * f) * all : 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (in)
                  v[k][e] = __ldcg(reinterpret_cast<const float4*>(pk) + (ch / 4 + e) * kRows + row);
                else
                  v[k][e] = make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[4 * e] = fmaf(v[k][e].x, by[k], y[4 * e]);
                y[4 * e + 1] = fmaf(v[k][e].y, by[k], y[4 * e + 1]);
                y[4 * e + 2] = fmaf(v[k][e].z, by[k], y[4 * e + 2]);
                y[4 * e + 3] = fmaf(v[k][e].w, by[k], y[4 * e + 3]);
              }
          }
          put(ch, y);
        }
        if (a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (top - kBias) * 0.6931471805599453f + logf(sum);
      }
    }
  };

  if (warp < kKeyWarp) {
    softmax_role();
  } else if (warp < kIssueWarp) {
    convert_role();
  } else if (warp == kIssueWarp) {
    issue_role();
    __syncwarp();
    if (elect_one()) mma_commit(bar(L::kDrain));
    __syncwarp();
    mbar_wait(bar(L::kDrain), 0);  // nothing of it runs on
    __syncwarp();
  } else {
    load_role();
  }
  tmem_fence_before();
  __syncthreads();
  // Where a wait ran out, the pieces that were not got to arrive all the same: an item's counter is zero
  // again when its last piece has, and the calls behind this one find it so.
  if (cut && threadIdx.x == 0) {
#pragma unroll 1
    for (int unit = words[2]; unit < total; unit += gridDim.x) {
      const Piece p = find(unit);
      if (p.part.pieces > 1 && atomicAdd(a.counters + p.part.slot0, 1u) == p.part.pieces - 1u)
        a.counters[p.part.slot0] = 0;
    }
  }
  if (warp == kIssueWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kTmemColumns));
  }
}

template <int D>
cudaError_t run(const KvAttentionArgs& a, cudaStream_t s) {
  const int bytes = Rows<D>::shared_bytes(a.batch.entries);
  const void* fn = reinterpret_cast<const void*>(kv_attention_rows<D>);
  const cudaError_t e = ensure_dynamic_smem(fn, bytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_attention_rows<D>, kKvSms, kThreads, bytes, s, a);
}

}  // namespace

bool kv_attention_rows_supported(const KvAttentionArgs& a) {
  return a.cache.head_dim <= 128 && a.batch.entries <= kMaxEntries;
}

cudaError_t launch_kv_attention_rows(const KvAttentionArgs& a, cudaStream_t s) {
  return a.cache.head_dim == 64 ? run<64>(a, s) : run<128>(a, s);
}

}  // namespace wd
