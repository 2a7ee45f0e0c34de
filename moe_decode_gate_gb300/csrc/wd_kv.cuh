// wd_kv.cuh - what the kernels of the 4-bit cache share: the layout of a group
// of 16 tokens, the view of a cache that they get, and the launch interface
// between them and the C-ABI (wd_kv_capi.cu).  The layout itself is described
// in include/wd_kv.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/wd_kv.h"
#include "wd_launch.h"

namespace wd {

// The layout of a group for one head_dim.
template <int D>
struct KvGroup {
  static constexpr int kBlocks = D / 32;                          // scale blocks to a token
  static constexpr int kSlabBlocks = kBlocks < 4 ? kBlocks : 4;   // blocks to a slab
  static constexpr int kSlabs = kBlocks / kSlabBlocks;
  static constexpr int kSlabBytes = 16 * 16 * kSlabBlocks;        // codes of 16 tokens
  static constexpr int kCodeBytes = 8 * D;                        // K or V codes
  static constexpr int kKScale = 2 * kCodeBytes;                  // offset of the K scales
  static constexpr int kVScale = kKScale + 16 * kBlocks;
  static constexpr int kBytes = kVScale + 16 * kBlocks;

  // byte of channels 32*block + 8*t8 + {0..7} of token t: 4 bytes of K codes
  __host__ __device__ static constexpr int k_word(int t, int block, int t8) {
    return (block / kSlabBlocks) * kSlabBytes + t * 16 * kSlabBlocks + t8 * 4 * kSlabBlocks +
           (block % kSlabBlocks) * 4;
  }
  // byte of channels 32*block + 4*g + {0..3} of token t: 2 bytes of V codes
  __host__ __device__ static constexpr int v_half(int t, int block, int g) {
    return kCodeBytes + (block / kSlabBlocks) * kSlabBytes + (t / 8) * 128 * kSlabBlocks +
           g * 16 * kSlabBlocks + (t % 8 / 2) * 4 * kSlabBlocks + (t % 2) * 2 * kSlabBlocks +
           (block % kSlabBlocks) * 2;
  }
};

// A cache as the kernels see it.
struct KvView {
  uint8_t* pool;
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  uint32_t* flag;  // the workspace's error flag
  int num_pages, slots, columns, page_size, page_shift, layers, kv_heads, head_dim;
  long long page_bytes;   // all layers
  long long layer_bytes;  // one layer of a page
  int head_bytes;         // one head of one layer of a page
};

// The batch of new tokens: entry b is slot seqs[b] (null: b) and owns tokens
// [q_start[b], q_start[b + 1]) (null: token b).
struct KvBatch {
  const int32_t* seqs;
  const int32_t* q_start;
  int entries, tokens;
};

// Length of slot s as the kernels may use it: no more than its table holds.
__device__ __forceinline__ int kv_length(const KvView& v, int s) {
  const int n = v.lengths[s];
  const int most = v.columns << v.page_shift;
  if (n < 0 || n > most) {
    atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
    return n < 0 ? 0 : most;
  }
  return n;
}

// Slot of entry b, or -1 (and the flag) if it is out of range.
__device__ __forceinline__ int kv_slot(const KvView& v, const KvBatch& q, int b) {
  const int s = q.seqs ? q.seqs[b] : b;
  if ((unsigned)s < (unsigned)v.slots) return s;
  atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
  return -1;
}

// First token and number of tokens of entry b, within [0, tokens).
__device__ __forceinline__ void kv_tokens(const KvView& v, const KvBatch& q, int b, int& first,
                                          int& n) {
  if (!q.q_start) {
    first = b;
    n = b < q.tokens ? 1 : 0;
    return;
  }
  first = q.q_start[b];
  const long long end = q.q_start[b + 1];
  if (first < 0 || end < first || end > q.tokens) {
    atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
    first = 0;
    n = 0;
    return;
  }
  n = (int)end - first;
}

// Whether the pool has this page.
__device__ __forceinline__ bool kv_page_there(const KvView& v, int p) {
  return (unsigned)p < (unsigned)v.num_pages;
}

// The page in column j of slot s; -1 (and the flag) if the id is out of range.
__device__ __forceinline__ int kv_page(const KvView& v, int s, int j) {
  const int p = v.table[(long long)s * v.columns + j];
  if (kv_page_there(v, p)) return p;
  atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
  return -1;
}

// Address of the 16-token group that holds position `pos` of a head.
__device__ __forceinline__ uint8_t* kv_group(const KvView& v, int page, int layer, int head,
                                             int pos, int group_bytes) {
  return v.pool + page * v.page_bytes + layer * v.layer_bytes + (long long)head * v.head_bytes +
         ((pos & (v.page_size - 1)) >> 4) * group_bytes;
}

// Scratch inside a cache's workspace.  Attention: arrival counters and partial results of the
// units (what a CTA does in one pass) of items that several CTAs share: two to a unit of
// 8 rows, one to a unit of 256.  Pages: lists of page ids, chunk counts, staged table rows and
// per-slot owners.
constexpr int kKvSms = 152;           // what the attention's grid is made for
constexpr int kKvMaxUnits = 8 * kKvSms;  // units of 8 query rows that there is room for
constexpr int kKvMaxRowUnits = 2 * kKvSms;  // of 256 query rows
constexpr int kKvNoneBytes = 2 * KvGroup<256>::kBytes;
constexpr int kKvChunkPages = 4096;   // pages that one CTA counts in wd_kv_compact

struct KvScratch {
  uint32_t* counters;  // [kKvMaxUnits], zero between calls
  uint8_t* none;       // [kKvNoneBytes], 0xFF: the groups of a page that is not there
  float* partial;      // [2 * kKvMaxUnits][8][head_dim + 2] or [kKvMaxRowUnits][256][head_dim + 2]
  int32_t* list_a;     // [num_pages]
  int32_t* list_b;     // [num_pages]
  int32_t* list_c;     // [num_pages]
  int32_t* chunk;      // [chunks of num_pages + 8]
  int32_t* rows;       // [slots][columns]
  int32_t* plan;       // [5][slots]
  int32_t* owner;      // [slots]
  size_t bytes;        // all of it, the flag's 256 bytes included
};
// Launch as a programmatic dependent: the kernel may start while the one before it
// on the stream drains.  Each of them waits for the results of that one before its first
// read of memory.
template <typename... Params, typename... Args>
cudaError_t kv_launch(void (*kernel)(Params...), int grid, int block, int shared, cudaStream_t s,
                      const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = (size_t)shared;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

KvScratch kv_scratch(const wd_kv_cache& c);
KvView kv_view(const wd_kv_cache& c);

struct KvAppendArgs {
  KvView cache;
  KvBatch batch;
  int layer;
  const void *k, *v;
  long long k_token, k_head, v_token, v_head;  // strides in elements
  void *k_out, *v_out;
  wd_kv_dtype dtype;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t s);

struct KvAttentionArgs {
  KvView cache;
  KvBatch batch;
  int layer;
  const void* q;
  long long q_token, q_head;
  int q_heads;
  void* out;
  float* lse;
  float scale;
  float key_scale, row_scale;  // of launch_kv_attention's own: scale log2 e = key_scale 2^kKeyShift row_scale
  int window, max_q;
  bool half;  // FP16 (else BF16)
  uint32_t* counters;
  const uint8_t* none;
  float* partial;
};
cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t s);

cudaError_t launch_kv_reserve(const KvView& v, const KvScratch& w, const int32_t* seqs,
                              const int32_t* counts, int n, int32_t* ok, cudaStream_t s);
cudaError_t launch_kv_fork(const KvView& v, const KvScratch& w, const int32_t* src,
                           const int32_t* dst, int n, int32_t* ok, cudaStream_t s);
cudaError_t launch_kv_compact(const KvView& v, const KvScratch& w, int32_t* table_out,
                              int32_t* refs_out, int32_t* page_map, cudaStream_t s);

}  // namespace wd
