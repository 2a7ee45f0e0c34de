// wd_kv_attention.cu - attention over the 4-bit cache (declared in include/wd_kv.h).
//
// One CTA per (token, query head): each warp walks every fourth key, lane l
// holding channels l, l + 32, ... of the query and of its running output, with
// a running maximum and sum; the warps meet in shared memory at the end.
#include "wd_kv.cuh"

namespace wd {
namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const uint32_t m = code & 7u;
  const float a = m < 2u ? 0.5f * (float)m
                         : __uint_as_float(((126u + (m >> 1)) << 23) | ((m & 1u) << 22));
  return (code & 8u) ? -a : a;
}
__device__ __forceinline__ float scale_value(uint32_t s) {
  return __uint_as_float(s == 0u ? 0x00400000u : (s == 255u ? 0x7FC00000u : s << 23));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) kv_attention(const KvAttentionArgs a) {
  using G = KvGroup<D>;
  constexpr int C = D / 32;
  __shared__ float out_sh[kWarps][D], m_sh[kWarps], l_sh[kWarps];
  const KvView& c = a.cache;
  const int token = blockIdx.x / a.q_heads, qh = blockIdx.x % a.q_heads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int head = qh / (a.q_heads / c.kv_heads);
  int b = token;
  if (a.batch.q_start) {
    int lo = 0, hi = a.batch.entries;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.batch.q_start[mid] <= token) lo = mid + 1; else hi = mid;
    }
    b = lo - 1;
  }
  if (b < 0 || b >= a.batch.entries) return;
  int first, n;
  kv_tokens(c, a.batch, b, first, n);
  if (token >= first + n) return;
  const int s = kv_slot(c, a.batch, b);
  const int len = s < 0 ? 0 : kv_length(c, s);
  const int pos = len - n + token - first;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  float q[C], o[C];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const long long at = token * a.q_token + qh * a.q_head + 32 * k + lane;
    q[k] = a.half ? __half2float(static_cast<const __half*>(a.q)[at])
                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at]);
    o[k] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = lo + warp; j <= pos; j += kWarps) {
    const int page = kv_page(c, s, j >> c.page_shift);
    const uint8_t* g = kv_group(c, page, a.layer, head, j, G::kBytes);
    const int t = j & 15;
    float x = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const uint32_t w = g[G::k_word(t, k, lane >> 3) + ((lane & 7) >> 1)];
      x += q[k] * e2m1_value(w >> (4 * (lane & 1))) * scale_value(g[G::kKScale + t * C + k]);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    x *= a.scale;
    const float top = fmaxf(m, x);
    const float keep = __expf(m - top), p = __expf(x - top);
    l = l * keep + p;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const uint32_t w = g[G::v_half(t, k, lane >> 2) + ((lane & 3) >> 1)];
      o[k] = o[k] * keep + p * e2m1_value(w >> (4 * (lane & 1))) *
                               scale_value(g[G::kVScale + t * C + k]);
    }
    m = top;
  }
#pragma unroll
  for (int k = 0; k < C; ++k) out_sh[warp][32 * k + lane] = o[k];
  if (lane == 0) {
    m_sh[warp] = m;
    l_sh[warp] = l;
  }
  __syncthreads();
  float top = m_sh[0];
  for (int w = 1; w < kWarps; ++w) top = fmaxf(top, m_sh[w]);
  if (top == -INFINITY) top = 0.f;
  float sum = 0.f;
  for (int w = 0; w < kWarps; ++w) sum += l_sh[w] * __expf(m_sh[w] - top);
  for (int ch = threadIdx.x; ch < D; ch += kWarps * 32) {
    float y = 0.f;
    for (int w = 0; w < kWarps; ++w) y += out_sh[w][ch] * __expf(m_sh[w] - top);
    y = sum == 0.f ? 0.f : y / sum;
    const long long at = ((long long)token * a.q_heads + qh) * D + ch;
    if (a.half)
      static_cast<__half*>(a.out)[at] = __float2half_rn(y);
    else
      static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(long long)token * a.q_heads + qh] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_kv_attention(const KvAttentionArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)a.batch.tokens * a.q_heads;
  switch (a.cache.head_dim) {
    case 64: kv_attention<64><<<grid, kWarps * 32, 0, s>>>(a); break;
    case 128: kv_attention<128><<<grid, kWarps * 32, 0, s>>>(a); break;
    default: kv_attention<256><<<grid, kWarps * 32, 0, s>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace wd
