// wd_kv_pages.cu - handing out, forking, freeing and compacting the pages of
// the 4-bit cache (declared in include/wd_kv.h).
//
// A page is free when refs[page] == 0; there is no free list to keep in order,
// and the lowest free pages go first, so results do not depend on the timing of
// anything.  Each operation is a plan (who gets which page: scans over refs and
// over the requests) and the work that it describes (table rows, counts, and the
// pages' bytes, which are what it costs: a page of 48 layers is over a megabyte).
// Counts change by integer atomics, whose order does not show.
//
// Calls whose plan is short run as one kernel: every CTA makes the whole plan for
// itself, copies its share of the pages, and the last one to finish writes the
// bookkeeping, which nobody reads any more.  Where the plan is long it is made once,
// and the operation takes three kernels.  (Measured, GB300: four beams, 48 layers 10.0
// us in three kernels, 8.3 in one; 4096 small pages compacted 10.0 and 5.4.)
#include "wd_device.cuh"
#include "wd_kv.cuh"

namespace wd {
namespace {

constexpr int kPlan = 1024;  // threads of the planning CTA
constexpr int kCopy = 256;   // threads that copy a piece of a page
// What is done in one kernel: the pool's scan takes one look of kPlan threads, the tables one CTA.
constexpr int kOnePages = 16 * kPlan;
constexpr int kOneCells = 1 << 16;

// Exclusive scan of one int per thread of a kPlan-thread CTA; `total` is the sum.
__device__ __forceinline__ int block_scan(int v, int& total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int t = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += t;
  }
  __syncthreads();  // the sums of the scan before have been read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    const int mine = warp_sums[lane];
    int s = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int t = __shfl_up_sync(0xFFFFFFFFu, s, off);
      if (lane >= off) s += t;
    }
    warp_sums[lane] = s - mine;
    if (lane == 31) warp_sums[32] = s;
  }
  __syncthreads();
  total = warp_sums[32];
  return warp_sums[warp] + incl - v;
}

// Calls take(rank, page) for the lowest free pages, rank 0 first, until
// `wanted` are found or the pool ends; returns how many there are of them.
// All threads of the CTA.
template <typename F>
__device__ __forceinline__ int find_free(const KvView& v, int wanted, int* warp_sums, F take) {
  constexpr int kEach = 16;
  const bool vec = (reinterpret_cast<uintptr_t>(v.refs) & 15u) == 0;
  int found = 0;
  for (int base = 0; base < v.num_pages && found < wanted; base += kPlan * kEach) {
    const int at = base + threadIdx.x * kEach;
    uint32_t free_bits = 0;
    if (vec && at + kEach <= v.num_pages) {
#pragma unroll
      for (int k = 0; k < kEach; k += 4) {
        const int4 r = *reinterpret_cast<const int4*>(v.refs + at + k);
        free_bits |= (r.x == 0 ? 1u : 0u) << k | (r.y == 0 ? 2u : 0u) << k |
                     (r.z == 0 ? 4u : 0u) << k | (r.w == 0 ? 8u : 0u) << k;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (at + k < v.num_pages && v.refs[at + k] == 0) free_bits |= 1u << k;
    }
    int total;
    int rank = found + block_scan(__popc(free_bits), total, warp_sums);
    while (free_bits) {
      const int k = __ffs(free_bits) - 1;
      free_bits &= free_bits - 1;
      if (rank < wanted) take(rank, at + k);
      ++rank;
    }
    found += total;
  }
  return min(found, wanted);
}

// Marks, for each slot that the call names, the first request that names it.
__device__ __forceinline__ void mark_owners(const KvView& v, const int32_t* slots_of, int n,
                                            int32_t* owner) {
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int s = slots_of ? slots_of[i] : i;
    if ((unsigned)s < (unsigned)v.slots) __stcg(owner + s, 0x7FFFFFFF);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int s = slots_of ? slots_of[i] : i;
    if ((unsigned)s < (unsigned)v.slots) atomicMin(owner + s, i);
  }
  __syncthreads();
}

// ------------------------------------------------------------- reserve ---

__global__ void __launch_bounds__(kPlan)
    kv_reserve(const KvView v, const KvScratch w, const int32_t* seqs, const int32_t* counts,
               int n, int32_t* ok) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ int warp_sums[33];
  __shared__ int wanted_sh;
  int32_t* begin = w.plan;              // pages that the requests before i ask for
  int32_t* need = w.plan + v.slots;     // pages of request i, -1: refused
  mark_owners(v, seqs, n, w.owner);
  int before = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    int pages = -1;
    if (i < n) {
      const int s = seqs ? seqs[i] : i;
      const int add = counts[i];
      if ((unsigned)s < (unsigned)v.slots && add >= 0 && __ldcg(w.owner + s) == i) {
        const long long len = kv_length(v, s);
        const long long most = (long long)v.columns << v.page_shift;
        if (len + add <= most)
          pages = (int)(((len + add + v.page_size - 1) >> v.page_shift) -
                        ((len + v.page_size - 1) >> v.page_shift));
      } else {
        atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      }
    }
    int total;
    const int excl = block_scan(pages > 0 ? pages : 0, total, warp_sums);
    if (i < n) {
      begin[i] = before + excl;
      need[i] = pages;
    }
    // A call may ask for more than an int counts: kPlan requests of 2^20 pages are 2^30, and from there on
    // none is served any more.
    before = total > (1 << 30) - before ? 1 << 30 : before + total;
  }
  if (threadIdx.x == 0) wanted_sh = before;
  __syncthreads();
  const int wanted = wanted_sh;
  // the pages, in rank order: list_a[rank]
  const int found = find_free(v, wanted, warp_sums,
                              [&](int rank, int page) { __stcg(w.list_a + rank, page); });
  __syncthreads();
  for (int i = threadIdx.x >> 5; i < n; i += kPlan / 32) {  // a warp to a request
    const int lane = threadIdx.x & 31;
    const int s = seqs ? seqs[i] : i;
    const int pages = need[i];
    const bool served = pages == 0 || (pages > 0 && begin[i] <= found - pages);
    if (served) {
      const int len = kv_length(v, s);
      const int have = (len + v.page_size - 1) >> v.page_shift;
      for (int k = lane; k < pages; k += 32) {
        const int page = __ldcg(w.list_a + begin[i] + k);
        v.table[(long long)s * v.columns + have + k] = page;
        v.refs[page] = 1;
      }
      __syncwarp();
      if (lane == 0) v.lengths[s] = len + counts[i];
    } else if (lane == 0) {
      atomicOr(v.flag, pages > 0 ? WD_KV_FLAG_NO_PAGES : WD_KV_FLAG_BAD_INDEX);
    }
    if (ok && lane == 0) ok[i] = served ? 1 : 0;
  }
}

// ---------------------------------------------------------------- fork ---

// The plan of a fork, per request: what becomes of the slot.
struct ForkPlan {
  int32_t* whole;  // pages shared with the source, -1: the slot stays as it is
  int32_t* page;   // the new last page, -1: none
  int32_t* from;   // the page that it is a copy of
  int32_t* old;    // pages that the slot held
  int32_t* length; // its new length
};
__device__ __host__ __forceinline__ ForkPlan fork_plan(const KvScratch& w, int slots) {
  const long long n = slots;
  return ForkPlan{w.plan, w.plan + n, w.plan + 2 * n, w.plan + 3 * n, w.plan + 4 * n};
}

__global__ void __launch_bounds__(kPlan)
    kv_fork_plan(const KvView v, const KvScratch w, const int32_t* src, const int32_t* dst, int n,
                 int32_t* ok) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ int warp_sums[33];
  const ForkPlan p = fork_plan(w, v.slots);
  mark_owners(v, dst, n, w.owner);
  int before = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    bool copy = false;
    if (i < n) {
      const int d = dst[i], s = src ? src[i] : -1;
      int whole = -1, from = -1, old = 0, len = 0;
      if ((unsigned)d < (unsigned)v.slots && s >= -1 && s < v.slots && __ldcg(w.owner + d) == i) {
        old = (kv_length(v, d) + v.page_size - 1) >> v.page_shift;
        len = s < 0 ? 0 : kv_length(v, s);
        if (s == d) {
          whole = -2;  // stays, but not refused
        } else {
          whole = len >> v.page_shift;
          copy = (len & (v.page_size - 1)) != 0;
          if (copy) from = kv_page(v, s, whole);
          if (copy && from < 0) {  // refused: there is nothing to copy
            copy = false;
            whole = -1;
          }
        }
      } else {
        atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      }
      p.whole[i] = whole;
      p.from[i] = from;
      p.old[i] = old;
      p.length[i] = len;
    }
    int total;
    const int rank = before + block_scan(copy ? 1 : 0, total, warp_sums);
    if (i < n) p.page[i] = copy ? rank : -1;
    before += total;
  }
  const int found = find_free(v, before, warp_sums,
                              [&](int rank, int page) { __stcg(w.list_a + rank, page); });
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int rank = p.page[i];
    if (rank >= 0) {
      const bool have = rank < found;
      p.page[i] = have ? __ldcg(w.list_a + rank) : -1;
      if (!have) {
        p.whole[i] = -1;
        p.from[i] = -1;
        atomicOr(v.flag, WD_KV_FLAG_NO_PAGES);
      }
    }
    if (ok) ok[i] = p.whole[i] != -1 ? 1 : 0;
  }
}

// Bytes that kCopy threads copy at a time, each with eight 16-byte loads in flight.  (With
// streaming loads and stores and 32 CTAs to an SM: a compaction that moves 411 MB 124.7 us, 97 % of
// the copy bandwidth; four loads, 8 CTAs and the caches' own ways took 141.)
constexpr int kLoads = 8;
constexpr int kPiece = kLoads * kCopy * 16;

// Up to kPiece bytes (a multiple of 16) from src to dst by kCopy threads, this one `me` of them.
__device__ __forceinline__ void copy_piece(uint8_t* dst, const uint8_t* src, int bytes, int me) {
  const uint4* in = reinterpret_cast<const uint4*>(src);
  uint4* out = reinterpret_cast<uint4*>(dst);
  const int n = bytes >> 4;
  uint4 x[kLoads];
#pragma unroll
  for (int q = 0; q < kLoads; ++q)
    if (me + q * kCopy < n) x[q] = __ldcs(in + me + q * kCopy);
#pragma unroll
  for (int q = 0; q < kLoads; ++q)
    if (me + q * kCopy < n) __stcs(out + me + q * kCopy, x[q]);
}

// The t-th piece of a page, page after page: the pages' pieces are dealt out to teams of kCopy
// threads over the whole grid.  page_of(k) gives the k-th copy's source and destination, -1 for none.
template <typename F>
__device__ __forceinline__ void copy_pages(const KvView& v, int count, F page_of) {
  const int pieces = (int)((v.page_bytes + kPiece - 1) / kPiece);
  const int teams = gridDim.x * (blockDim.x / kCopy);
  // (neighbouring teams to different CTAs, so that few pieces occupy many SMs)
  const int team = threadIdx.x / kCopy * gridDim.x + blockIdx.x;
  for (long long t = team; t < (long long)count * pieces; t += teams) {
    const int2 pair = page_of((int)(t / pieces));
    if (pair.y < 0) continue;
    const long long off = t % pieces * kPiece;
    copy_piece(v.pool + pair.y * v.page_bytes + off, v.pool + pair.x * v.page_bytes + off,
               (int)min((long long)kPiece, v.page_bytes - off), threadIdx.x % kCopy);
  }
}

// True in all threads of the CTA of the grid that gets here last, with what the others wrote visible.
__device__ __forceinline__ bool last_cta(uint32_t* counter) {
  __shared__ int last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) {
    last = atomicAdd(counter, 1u) == gridDim.x - 1;
    if (last) *counter = 0;
    __threadfence();
  }
  __syncthreads();
  return last != 0;
}

// Stage the new table rows (the table itself is still being read), change the
// counts, and copy the partly filled pages.
__global__ void __launch_bounds__(kCopy) kv_fork_work(const KvView v, const KvScratch w,
                                                      const int32_t* src, const int32_t* dst,
                                                      int n) {
  grid_dependency_wait();
  grid_launch_dependents();
  const ForkPlan p = fork_plan(w, v.slots);
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int whole = p.whole[i];
    if (whole < 0) continue;
    const int d = dst[i], s = src ? src[i] : -1, page = p.page[i], old = p.old[i];
    const int most = max(old, whole + 1);
    for (int j = threadIdx.x; j < v.columns && j < most; j += kCopy) {
      int next = -1;
      if (j < whole) {
        next = v.table[(long long)s * v.columns + j];
        if ((unsigned)next < (unsigned)v.num_pages)
          atomicAdd(v.refs + next, 1);
        else
          atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      } else if (j == whole && page >= 0) {
        next = page;
        atomicAdd(v.refs + next, 1);
      }
      if (j < old) {
        const int gone = v.table[(long long)d * v.columns + j];
        if ((unsigned)gone < (unsigned)v.num_pages)
          atomicSub(v.refs + gone, 1);
        else
          atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      }
      w.rows[(long long)i * v.columns + j] = next;
    }
  }
  copy_pages(v, n, [&](int i) {
    return p.whole[i] < 0 ? make_int2(-1, -1) : make_int2(p.from[i], p.page[i]);
  });
}

// The rows and lengths, now that nothing reads the old ones any more.
__global__ void __launch_bounds__(kCopy) kv_fork_rows(const KvView v, const KvScratch w,
                                                      const int32_t* dst, int n) {
  grid_dependency_wait();
  grid_launch_dependents();
  const ForkPlan p = fork_plan(w, v.slots);
  for (int i = blockIdx.x; i < n; i += gridDim.x) {
    const int whole = p.whole[i];
    if (whole < 0) continue;
    const int d = dst[i];
    const int most = min(v.columns, max(p.old[i], whole + 1));
    for (int j = threadIdx.x; j < most; j += kCopy)
      v.table[(long long)d * v.columns + j] = w.rows[(long long)i * v.columns + j];
    if (threadIdx.x == 0) v.lengths[d] = p.length[i];
  }
}

// The whole operation for up to kOneRequests requests, a pool of up to kOnePages pages and rows of up to
// kOneCells cells in all.
constexpr int kOneRequests = 256;

__global__ void __launch_bounds__(kPlan)
    kv_fork_one(const KvView v, const KvScratch w, const int32_t* src, const int32_t* dst, int n,
                int32_t* ok) {
  __shared__ int warp_sums[33], dst_sh[kOneRequests], src_sh[kOneRequests], whole_sh[kOneRequests],
      from_sh[kOneRequests], page_sh[kOneRequests], found_sh[kOneRequests];
  grid_dependency_wait();
  grid_launch_dependents();
  const int i = threadIdx.x;
  int d = -1, s = -1;
  if (i < n) {
    d = dst[i];
    s = src ? src[i] : -1;
    dst_sh[i] = d;
    src_sh[i] = s;
  }
  __syncthreads();
  bool copy = false;
  int whole = -1, from = -1, old = 0, len = 0;
  if (i < n) {
    bool good = (unsigned)d < (unsigned)v.slots && s >= -1 && s < v.slots;
    for (int k = 0; k < i; ++k) good &= dst_sh[k] != d;
    if (good) {
      old = (kv_length(v, d) + v.page_size - 1) >> v.page_shift;
      len = s < 0 ? 0 : kv_length(v, s);
      if (s == d) {
        whole = -2;  // stays, but not refused
      } else {
        whole = len >> v.page_shift;
        copy = (len & (v.page_size - 1)) != 0;
        if (copy) from = kv_page(v, s, whole);
        if (copy && from < 0) {  // refused: there is nothing to copy
          copy = false;
          whole = -1;
        }
      }
    } else {
      atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
    }
  }
  int wanted;
  const int rank = block_scan(copy ? 1 : 0, wanted, warp_sums);
  const int found = find_free(v, wanted, warp_sums, [&](int r, int page) { found_sh[r] = page; });
  __syncthreads();
  int page = -1;
  if (copy) {
    if (rank < found) {
      page = found_sh[rank];
    } else {
      whole = -1;
      atomicOr(v.flag, WD_KV_FLAG_NO_PAGES);
    }
  }
  if (i < n) {
    whole_sh[i] = whole;
    from_sh[i] = from;
    page_sh[i] = page;
  }
  __syncthreads();
  copy_pages(v, n, [&](int k) { return make_int2(from_sh[k], page_sh[k]); });
  if (!last_cta(w.counters)) return;
  // the rows, staged first: a slot may be source and destination
  __shared__ int old_sh[kOneRequests];
  if (i < n) old_sh[i] = old;
  __syncthreads();
  const int lane = i & 31;
  for (int k = i >> 5; k < n; k += kPlan / 32) {
    const int wh = whole_sh[k];
    if (wh < 0) continue;
    const int most = min(v.columns, max(old_sh[k], wh + 1));
    for (int j = lane; j < most; j += 32) {
      int next = -1;
      if (j < wh) {
        next = v.table[(long long)src_sh[k] * v.columns + j];
        if ((unsigned)next < (unsigned)v.num_pages)
          atomicAdd(v.refs + next, 1);
        else
          atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      } else if (j == wh && page_sh[k] >= 0) {
        next = page_sh[k];
        atomicAdd(v.refs + next, 1);
      }
      if (j < old_sh[k]) {
        const int gone = v.table[(long long)dst_sh[k] * v.columns + j];
        if ((unsigned)gone < (unsigned)v.num_pages)
          atomicSub(v.refs + gone, 1);
        else
          atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      }
      w.rows[(long long)k * v.columns + j] = next;
    }
  }
  __syncthreads();
  for (int k = i >> 5; k < n; k += kPlan / 32) {
    const int wh = whole_sh[k];
    if (wh < 0) continue;
    const int most = min(v.columns, max(old_sh[k], wh + 1));
    for (int j = lane; j < most; j += 32)
      v.table[(long long)dst_sh[k] * v.columns + j] = w.rows[(long long)k * v.columns + j];
  }
  if (i < n) {
    if (whole >= 0) v.lengths[d] = len;
    if (ok) ok[i] = whole != -1 ? 1 : 0;
  }
}

// ------------------------------------------------------------- compact ---

// Live pages of each chunk of kKvChunkPages pages.
__global__ void __launch_bounds__(kPlan) kv_compact_count(const KvView v, const KvScratch w) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ int sums[32];
  const int base = blockIdx.x * kKvChunkPages;
  int live = 0;
#pragma unroll
  for (int k = 0; k < kKvChunkPages / kPlan; ++k) {
    const int at = base + k * kPlan + threadIdx.x;
    if (at < v.num_pages && v.refs[at] > 0) ++live;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) live += __shfl_xor_sync(0xFFFFFFFFu, live, off);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = live;
  __syncthreads();
  if (threadIdx.x == 0) {
    int t = 0;
    for (int k = 0; k < 32; ++k) t += sums[k];
    w.chunk[blockIdx.x] = t;
  }
}

// list_a: where each page goes, -1 for a free one, -2 - k for the k-th mover;
// list_b: the movers; list_c: the holes that they move to.  chunk[chunks] =
// live pages, chunk[chunks + 1] = movers.
__global__ void __launch_bounds__(kPlan)
    kv_compact_plan(const KvView v, const KvScratch w, int chunks) {
  grid_dependency_wait();
  grid_launch_dependents();
  __shared__ int warp_sums[33];
  int live_total = 0, live_before = 0, live_to_split = 0, total;
  for (int base = 0; base < chunks; base += kPlan) {
    const int k = base + threadIdx.x;
    const int c = k < chunks ? w.chunk[k] : 0;
    block_scan(c, total, warp_sums);
    live_total += total;
    block_scan(k < (int)blockIdx.x ? c : 0, total, warp_sums);
    live_before += total;
  }
  const int split = live_total / kKvChunkPages;  // the chunk that page live_total is in
  for (int base = 0; base < split; base += kPlan) {
    const int k = base + threadIdx.x;
    block_scan(k < split ? w.chunk[k] : 0, total, warp_sums);
    live_to_split += total;
  }
  int in_split = 0;
  for (int at = split * kKvChunkPages + threadIdx.x; at < live_total; at += kPlan)
    in_split += v.refs[at] > 0 ? 1 : 0;
  block_scan(in_split, total, warp_sums);
  const int below = live_to_split + total;  // live pages below live_total
  constexpr int kEach = kKvChunkPages / kPlan;
  const int at = blockIdx.x * kKvChunkPages + threadIdx.x * kEach;
  bool live[kEach];
  int mine = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    live[k] = at + k < v.num_pages && v.refs[at + k] > 0;
    mine += live[k] ? 1 : 0;
  }
  int rank = live_before + block_scan(mine, total, warp_sums);  // live pages before `at`
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int page = at + k;
    if (page < v.num_pages) {
      int to = -1;
      if (live[k]) {
        to = page;
        if (page >= live_total) {
          w.list_b[rank - below] = page;
          to = -2 - (rank - below);
        }
      } else if (page < live_total) {
        w.list_c[page - rank] = page;
      }
      w.list_a[page] = to;
    }
    rank += live[k] ? 1 : 0;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    w.chunk[chunks] = live_total;
    w.chunk[chunks + 1] = live_total - below;
  }
}

// Move the pages and rewrite the bookkeeping.  Movers lie at or above the live
// count and holes below it, so no page is read after it was written.
__global__ void __launch_bounds__(kCopy)
    kv_compact_work(const KvView v, const KvScratch w, int chunks, int32_t* table_out,
                    int32_t* refs_out, int32_t* page_map) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int movers = w.chunk[chunks + 1];
  const long long threads = (long long)gridDim.x * kCopy;
  const long long me = (long long)blockIdx.x * kCopy + threadIdx.x;
  for (long long e = me; e < (long long)v.slots * v.columns; e += threads) {
    const int page = v.table[e];
    int to = -1;
    if (page >= 0) {
      if (page < v.num_pages) {
        to = w.list_a[page];
        if (to <= -2) to = w.list_c[-2 - to];
      } else {
        atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      }
    }
    table_out[e] = to;
  }
  for (long long page = me; page < v.num_pages; page += threads) {
    const int to = w.list_a[page];
    if (to == page) {
      if (refs_out != v.refs) refs_out[page] = v.refs[page];
    } else if (to <= -2) {  // a mover: its count goes with it
      const int hole = w.list_c[-2 - to];
      refs_out[hole] = v.refs[page];
      refs_out[page] = 0;
    } else if (page >= w.chunk[chunks]) {  // free, and no mover's place
      refs_out[page] = 0;
    }
    if (page_map) page_map[page] = to <= -2 ? w.list_c[-2 - to] : to;
  }
  copy_pages(v, movers, [&](int k) { return make_int2(w.list_b[k], w.list_c[k]); });
}

// The whole operation for a pool of up to kOnePages pages and tables of up to kOneCells cells.
// kEach: pages to a thread of the plan.
template <int kEach>
__global__ void __launch_bounds__(kPlan)
    kv_compact_one(const KvView v, uint32_t* counter, int32_t* table_out, int32_t* refs_out,
                   int32_t* page_map) {
  constexpr int kPages = kEach * kPlan;
  constexpr uint16_t kNowhere = 0xFFFF;
  extern __shared__ __align__(16) uint16_t lists[];
  __shared__ int warp_sums[33];
  uint16_t* mover = lists;              // [kPages / 2]
  uint16_t* hole = lists + kPages / 2;  // [kPages / 2]
  uint16_t* to = lists + kPages;        // [kPages] where a page goes, kNowhere for a free one
  grid_dependency_wait();
  grid_launch_dependents();
  const int at = threadIdx.x * kEach;
  uint32_t live = 0;
  if ((reinterpret_cast<uintptr_t>(v.refs) & 15u) == 0 && at + kEach <= v.num_pages) {
#pragma unroll
    for (int k = 0; k < kEach; k += 4) {
      const int4 r = *reinterpret_cast<const int4*>(v.refs + at + k);
      live |= ((r.x > 0 ? 1u : 0u) | (r.y > 0 ? 2u : 0u) | (r.z > 0 ? 4u : 0u) | (r.w > 0 ? 8u : 0u)) << k;
    }
  } else {
    for (int k = 0; k < kEach; ++k)
      if (at + k < v.num_pages && v.refs[at + k] > 0) live |= 1u << k;
  }
  int total, below;
  int rank = block_scan(__popc(live), total, warp_sums);  // live pages before `at`
  const int under = min(max(total - at, 0), kEach);       // of the thread's pages, those below `total`
  block_scan(__popc(live & ((1u << under) - 1u)), below, warp_sums);
  uint32_t goes[kEach / 2];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int page = at + k;
    const bool is_live = live >> k & 1u;
    const uint32_t stays = is_live ? (uint32_t)page : kNowhere;
    goes[k / 2] = k & 1 ? goes[k / 2] | stays << 16 : stays;
    if (is_live) {
      if (page >= total) mover[rank - below] = (uint16_t)page;
      ++rank;
    } else if (page < total) {
      hole[page - rank] = (uint16_t)page;
    }
  }
#pragma unroll
  for (int k = 0; k < kEach / 4; ++k)
    reinterpret_cast<uint2*>(to + at)[k] = make_uint2(goes[2 * k], goes[2 * k + 1]);
  __syncthreads();
  const int movers = total - below;
  for (int k = threadIdx.x; k < movers; k += kPlan) to[mover[k]] = hole[k];
  __syncthreads();
  // Bookkeeping of its own is written by all CTAs, each its share; the cache's own by the
  // last one to finish, when nobody reads it any more.
  const bool apart = table_out != v.table && refs_out != v.refs;
  const int first = apart ? blockIdx.x * kPlan + threadIdx.x : threadIdx.x;
  const int step = apart ? gridDim.x * kPlan : kPlan;
  const auto write_tables = [&]() {
    for (int e = first; e < v.slots * v.columns; e += step) {
      const int page = v.table[e];
      if (page >= v.num_pages) atomicOr(v.flag, WD_KV_FLAG_BAD_INDEX);
      const int now = (unsigned)page < (unsigned)v.num_pages ? to[page] : kNowhere;
      table_out[e] = now == kNowhere ? -1 : now;
    }
  };
  const auto map_page = [&](int page) {
    if (page_map) page_map[page] = to[page] == kNowhere ? -1 : to[page];
  };
  if (apart) {
    write_tables();
    for (int page = first; page < v.num_pages; page += step) {
      map_page(page);
      if (to[page] != kNowhere) refs_out[to[page]] = v.refs[page];
      if (page >= total) refs_out[page] = 0;
    }
  }
  copy_pages(v, movers, [&](int k) { return make_int2(mover[k], hole[k]); });
  if (apart || !last_cta(counter)) return;
  write_tables();
  int count[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int page = k * kPlan + threadIdx.x;
    if (page >= v.num_pages) break;
    count[k] = v.refs[page];
    map_page(page);
  }
  __syncthreads();  // refs_out may be refs
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int page = k * kPlan + threadIdx.x;
    if (page >= v.num_pages) break;
    if (to[page] != kNowhere) refs_out[to[page]] = count[k];
    if (page >= total) refs_out[page] = 0;
  }
}

constexpr int kWorkCtas = kKvSms * 32;

// Whether up to `copies` page copies are few enough for the one-kernel forms.  Their CTAs are large, and
// copy less well than the many small ones of the other form: 97 MB take 38.0 us against 33.7.
bool few_bytes(const KvView& v, long long copies) { return copies * v.page_bytes <= (64ll << 20); }
// CTAs of kPlan threads for them.
int copying_ctas(const KvView& v, int copies) {
  const long long pieces = (v.page_bytes + kPiece - 1) / kPiece * copies;
  return (int)(pieces < 1 ? 1 : pieces < kKvSms ? pieces : kKvSms);
}

template <int kEach>
cudaError_t compact_one(const KvView& v, const KvScratch& w, int32_t* table_out, int32_t* refs_out,
                        int32_t* page_map, cudaStream_t s) {
  constexpr int kBytes = 2 * 2 * kEach * kPlan;
  const cudaError_t e =
      ensure_dynamic_smem(reinterpret_cast<const void*>(kv_compact_one<kEach>), kBytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kv_compact_one<kEach>, copying_ctas(v, v.num_pages / 2), kPlan, kBytes, s, v,
                   w.counters, table_out, refs_out, page_map);
}

}  // namespace

cudaError_t launch_kv_reserve(const KvView& v, const KvScratch& w, const int32_t* seqs,
                              const int32_t* counts, int n, int32_t* ok, cudaStream_t s) {
  return launch_dependent(kv_reserve, 1, kPlan, 0, s, v, w, seqs, counts, n, ok);
}

cudaError_t launch_kv_fork(const KvView& v, const KvScratch& w, const int32_t* src,
                           const int32_t* dst, int n, int32_t* ok, cudaStream_t s) {
  if (n <= kOneRequests && v.num_pages <= kOnePages && (long long)n * v.columns <= kOneCells &&
      few_bytes(v, n))
    return launch_dependent(kv_fork_one, copying_ctas(v, n), kPlan, 0, s, v, w, src, dst, n, ok);
  cudaError_t e = launch_dependent(kv_fork_plan, 1, kPlan, 0, s, v, w, src, dst, n, ok);
  if (e == cudaSuccess) e = launch_dependent(kv_fork_work, kWorkCtas, kCopy, 0, s, v, w, src, dst, n);
  if (e == cudaSuccess) e = launch_dependent(kv_fork_rows, n < 1024 ? n : 1024, kCopy, 0, s, v, w, dst, n);
  return e;
}

cudaError_t launch_kv_compact(const KvView& v, const KvScratch& w, int32_t* table_out,
                              int32_t* refs_out, int32_t* page_map, cudaStream_t s) {
  if (v.num_pages <= kOnePages && (long long)v.slots * v.columns <= kOneCells &&
      few_bytes(v, v.num_pages / 2))
    return v.num_pages <= 4 * kPlan ? compact_one<4>(v, w, table_out, refs_out, page_map, s)
                                    : compact_one<16>(v, w, table_out, refs_out, page_map, s);
  const int chunks = (v.num_pages + kKvChunkPages - 1) / kKvChunkPages;
  cudaError_t e = launch_dependent(kv_compact_count, chunks, kPlan, 0, s, v, w);
  if (e == cudaSuccess) e = launch_dependent(kv_compact_plan, chunks, kPlan, 0, s, v, w, chunks);
  if (e == cudaSuccess)
    e = launch_dependent(kv_compact_work, kWorkCtas, kCopy, 0, s, v, w, chunks, table_out, refs_out,
                  page_map);
  return e;
}

}  // namespace wd
