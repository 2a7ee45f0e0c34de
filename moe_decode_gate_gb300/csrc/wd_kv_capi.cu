// wd_kv_capi.cu - the C-ABI of the 4-bit cache (declared in include/wd_kv.h):
// argument checks on the host, the workspace's layout, and the launches.
// Nothing here allocates or synchronises except wd_kv_read_error_flag.
#include <string.h>

#include "wd_kv.cuh"

namespace wd {
namespace {

constexpr size_t kFlagBytes = 256;

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool dims_ok(int layers, int kv_heads, int head_dim, int page_size) {
  return layers >= 1 && layers <= 1024 && kv_heads >= 1 && kv_heads <= 256 &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) &&
         (page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128 ||
          page_size == 256);
}

int group_bytes(int head_dim) { return 16 * (head_dim + 2 * (head_dim / 32)); }

wd_status check_dims(const wd_kv_cache* c) {
  if (!c) return WD_ERR_INVALID_ARG;
  if (!dims_ok(c->layers, c->kv_heads, c->head_dim, c->page_size)) return WD_ERR_UNSUPPORTED_SHAPE;
  if (c->num_pages < 1 || c->num_pages > (1 << 24) || c->slots < 1 || c->slots > 65536 ||
      c->columns < 1 || c->columns > (1 << 20))
    return WD_ERR_UNSUPPORTED_SHAPE;
  return WD_OK;
}

wd_status check_cache(const wd_kv_cache* c) {
  const wd_status st = check_dims(c);
  if (st != WD_OK) return st;
  if (!c->pool || !c->table || !c->lengths || !c->refs || !c->workspace)
    return WD_ERR_INVALID_ARG;
  if (!aligned(c->pool, 16) || !aligned(c->table, 4) || !aligned(c->lengths, 4) ||
      !aligned(c->refs, 4) || !aligned(c->workspace, 256))
    return WD_ERR_INVALID_ARG;
  if (c->workspace_bytes < kv_scratch(*c).bytes) return WD_ERR_WORKSPACE_TOO_SMALL;
  return WD_OK;
}

wd_status check_batch(const wd_kv_cache* c, int layer, const int32_t* seqs, const int32_t* q_start,
                      int entries, int tokens) {
  if (layer < 0 || layer >= c->layers || entries < 0 || entries > WD_KV_MAX_ENTRIES || tokens < 0 ||
      tokens > WD_KV_MAX_TOKENS || !aligned(seqs, 4) || !aligned(q_start, 4))
    return WD_ERR_INVALID_ARG;
  if (!q_start && tokens > entries) return WD_ERR_INVALID_ARG;
  if (!seqs && entries > c->slots) return WD_ERR_INVALID_ARG;
  return WD_OK;
}

}  // namespace

KvScratch kv_scratch(const wd_kv_cache& c) {
  uint8_t* p = static_cast<uint8_t*>(c.workspace) + kFlagBytes;
  size_t used = kFlagBytes;
  const auto take = [&](size_t bytes) {
    uint8_t* at = p;
    p += round256(bytes);
    used += round256(bytes);
    return at;
  };
  KvScratch w;
  const size_t pages = c.num_pages, slots = c.slots;
  w.counters = reinterpret_cast<uint32_t*>(take(4 * (size_t)kKvMaxUnits));
  w.none = take(kKvNoneBytes);
  w.partial = reinterpret_cast<float*>(
      take(4 * ((size_t)c.head_dim + 2) *
           (c.head_dim <= 128 ? (size_t)kKvMaxRowUnits * 256 : 2 * (size_t)kKvMaxUnits * 8)));
  w.list_a = reinterpret_cast<int32_t*>(take(4 * pages));
  w.list_b = reinterpret_cast<int32_t*>(take(4 * pages));
  w.list_c = reinterpret_cast<int32_t*>(take(4 * pages));
  w.chunk = reinterpret_cast<int32_t*>(take(4 * ((pages + kKvChunkPages - 1) / kKvChunkPages + 8)));
  w.rows = reinterpret_cast<int32_t*>(take(4 * slots * c.columns));
  w.plan = reinterpret_cast<int32_t*>(take(4 * 5 * slots));
  w.owner = reinterpret_cast<int32_t*>(take(4 * slots));
  w.bytes = used;
  return w;
}

KvView kv_view(const wd_kv_cache& c) {
  KvView v;
  v.pool = static_cast<uint8_t*>(c.pool);
  v.table = c.table;
  v.lengths = c.lengths;
  v.refs = c.refs;
  v.flag = static_cast<uint32_t*>(c.workspace);
  v.num_pages = c.num_pages;
  v.slots = c.slots;
  v.columns = c.columns;
  v.page_size = c.page_size;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  v.layers = c.layers;
  v.kv_heads = c.kv_heads;
  v.head_dim = c.head_dim;
  v.head_bytes = c.page_size / 16 * group_bytes(c.head_dim);
  v.layer_bytes = (long long)c.kv_heads * v.head_bytes;
  v.page_bytes = c.layers * v.layer_bytes;
  return v;
}

}  // namespace wd

using namespace wd;

extern "C" {

size_t wd_kv_page_bytes(int layers, int kv_heads, int head_dim, int page_size) {
  if (!dims_ok(layers, kv_heads, head_dim, page_size)) return 0;
  return (size_t)layers * kv_heads * (page_size / 16) * group_bytes(head_dim);
}

size_t wd_kv_workspace_size(const wd_kv_cache* cache) {
  if (check_dims(cache) != WD_OK) return 0;
  return kv_scratch(*cache).bytes;
}

wd_status wd_kv_workspace_init(const wd_kv_cache* cache, wd_stream_t stream) {
  const wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // the flag's slot and the counters behind it
  cudaError_t e = cudaMemsetAsync(cache->workspace, 0, kFlagBytes + 4 * kKvMaxUnits, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(kv_scratch(*cache).none, 0xFF, kKvNoneBytes, s);
  return cuda_status(e);
}

wd_status wd_kv_read_error_flag(const wd_kv_cache* cache, wd_stream_t stream, int* flag) {
  const wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  if (!flag) return WD_ERR_INVALID_ARG;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, cache->workspace, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(cache->workspace, 0, sizeof(v), s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  // A call that gave up leaves its counters at zero; whatever the reason was, the next one starts from that.
  if (e == cudaSuccess && (v & WD_KV_FLAG_TIMEOUT))
    e = cudaMemsetAsync(kv_scratch(*cache).counters, 0, 4 * kKvMaxUnits, s);
  if (e != cudaSuccess) return cuda_status(e);
  *flag = (int)(v & (WD_KV_FLAG_BAD_INDEX | WD_KV_FLAG_TIMEOUT | WD_KV_FLAG_NO_PAGES));
  if (v & WD_KV_FLAG_TIMEOUT) return WD_ERR_PIPELINE_TIMEOUT;
  if (v & WD_KV_FLAG_NO_PAGES) return WD_ERR_OUT_OF_PAGES;
  return (v & WD_KV_FLAG_BAD_INDEX) ? WD_ERR_BAD_INDEX : WD_OK;
}

wd_status wd_kv_reserve(const wd_kv_cache* cache, const int32_t* seqs, const int32_t* counts,
                        int n, int32_t* ok, wd_stream_t stream) {
  const wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  if (n < 0 || n > cache->slots || (n > 0 && !counts) || !aligned(seqs, 4) || !aligned(counts, 4) ||
      !aligned(ok, 4))
    return WD_ERR_INVALID_ARG;
  if (n == 0) return WD_OK;
  return cuda_status(launch_kv_reserve(kv_view(*cache), kv_scratch(*cache), seqs, counts, n, ok,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

wd_status wd_kv_append(const wd_kv_cache* cache, int layer, const void* k, const void* v,
                       wd_kv_dtype dtype, int64_t k_stride_token, int64_t k_stride_head,
                       int64_t v_stride_token, int64_t v_stride_head, void* k_out, void* v_out,
                       const int32_t* seqs, const int32_t* q_start, int entries, int tokens,
                       wd_stream_t stream) {
  wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  st = check_batch(cache, layer, seqs, q_start, entries, tokens);
  if (st != WD_OK) return st;
  if (dtype != WD_KV_BF16 && dtype != WD_KV_FP16 && dtype != WD_KV_FP32) return WD_ERR_INVALID_ARG;
  const uintptr_t size = dtype == WD_KV_FP32 ? 4 : 2;
  if (tokens == 0 || entries == 0) return WD_OK;
  if (!k || !v || !k_out != !v_out) return WD_ERR_INVALID_ARG;
  if (!aligned(k, size) || !aligned(v, size) || !aligned(k_out, size) || !aligned(v_out, size))
    return WD_ERR_INVALID_ARG;
  KvAppendArgs a{};
  a.cache = kv_view(*cache);
  a.batch = KvBatch{seqs, q_start, entries, tokens};
  a.layer = layer;
  a.k = k;
  a.v = v;
  a.k_token = k_stride_token;
  a.k_head = k_stride_head;
  a.v_token = v_stride_token;
  a.v_head = v_stride_head;
  a.k_out = k_out;
  a.v_out = v_out;
  a.dtype = dtype;
  return cuda_status(launch_kv_append(a, reinterpret_cast<cudaStream_t>(stream)));
}

wd_status wd_kv_attention(const wd_kv_cache* cache, int layer, const void* q, wd_kv_dtype dtype,
                          int64_t q_stride_token, int64_t q_stride_head, int q_heads, void* out,
                          float* lse, const int32_t* seqs, const int32_t* q_start, int entries,
                          int tokens, int max_q, float scale, int window, wd_stream_t stream) {
  wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  st = check_batch(cache, layer, seqs, q_start, entries, tokens);
  if (st != WD_OK) return st;
  if ((dtype != WD_KV_BF16 && dtype != WD_KV_FP16) || q_heads < 1 || q_heads > 4096 ||
      q_heads % cache->kv_heads || max_q < 0 || window < 0)
    return WD_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !(scale < INFINITY)) return WD_ERR_INVALID_ARG;
  if ((long long)tokens * q_heads >= (1ll << 31)) return WD_ERR_UNSUPPORTED_SHAPE;
  if (tokens == 0 || entries == 0) return WD_OK;
  if (!q || !out || !aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4))
    return WD_ERR_INVALID_ARG;
  const KvScratch w = kv_scratch(*cache);
  KvAttentionArgs a{};
  a.cache = kv_view(*cache);
  a.batch = KvBatch{seqs, q_start, entries, tokens};
  a.layer = layer;
  a.q = q;
  a.q_token = q_stride_token;
  a.q_head = q_stride_head;
  a.q_heads = q_heads;
  a.out = out;
  a.lse = lse;
  a.scale = scale;
  a.window = window;
  a.max_q = q_start ? (max_q > 0 && max_q < tokens ? max_q : tokens) : 1;
  a.half = dtype == WD_KV_FP16;
  a.counters = w.counters;
  a.none = w.none;
  a.partial = w.partial;
  return cuda_status(launch_kv_attention(a, reinterpret_cast<cudaStream_t>(stream)));
}

wd_status wd_kv_fork(const wd_kv_cache* cache, const int32_t* src, const int32_t* dst, int n,
                     int32_t* ok, wd_stream_t stream) {
  const wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  if (n < 0 || n > cache->slots || (n > 0 && !dst) || !aligned(src, 4) || !aligned(dst, 4) ||
      !aligned(ok, 4))
    return WD_ERR_INVALID_ARG;
  if (n == 0) return WD_OK;
  return cuda_status(launch_kv_fork(kv_view(*cache), kv_scratch(*cache), src, dst, n, ok,
                                    reinterpret_cast<cudaStream_t>(stream)));
}

wd_status wd_kv_free(const wd_kv_cache* cache, const int32_t* seqs, int n, wd_stream_t stream) {
  return wd_kv_fork(cache, nullptr, seqs, n, nullptr, stream);
}

wd_status wd_kv_compact(const wd_kv_cache* cache, int32_t* table_out, int32_t* refs_out,
                        int32_t* page_map, wd_stream_t stream) {
  const wd_status st = check_cache(cache);
  if (st != WD_OK) return st;
  if (!table_out != !refs_out || !aligned(table_out, 4) || !aligned(refs_out, 4) ||
      !aligned(page_map, 4))
    return WD_ERR_INVALID_ARG;
  const KvView v = kv_view(*cache);
  return cuda_status(launch_kv_compact(v, kv_scratch(*cache), table_out ? table_out : v.table,
                                       refs_out ? refs_out : v.refs, page_map,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
