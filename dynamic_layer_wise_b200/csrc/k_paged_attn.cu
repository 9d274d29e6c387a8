// Attention of packed query rows over the paged K/V cache of their sequence.
#include "common.cuh"
#include "paged.h"

namespace dcu {
namespace {

// One warp per (row, head): out = sum_j p_j V_j / sum_j p_j with a running max,
// a key at a time, the head dim spread over the lanes.
template <class T>
__global__ void __launch_bounds__(128) k_paged_attn_rowhead(const PagedAttnArgs a) {
  pdl_enter();
  const dcu_pages &pg = a.pages;
  const int lane = threadIdx.x & 31;
  const int hd = pg.head_dim, G = a.n_heads / pg.n_kv_heads;
  const int rows = min(max(a.row_start[a.B], 0), a.max_rows);
  const long long items = (long long)rows * a.n_heads;
  const T *Q = static_cast<const T *>(a.q), *K = static_cast<const T *>(pg.k), *V = static_cast<const T *>(pg.v);
  for (long long it = blockIdx.x * 4ll + (threadIdx.x >> 5); it < items; it += gridDim.x * 4ll) {
    const int r = (int)(it / a.n_heads), h = (int)(it - (long long)r * a.n_heads);
    int lo = 0, hi = a.B - 1;  // the first sequence whose end is above r
    while (lo < hi) {
      const int m = (lo + hi) >> 1;
      if (a.row_start[m + 1] > r) hi = m;
      else lo = m + 1;
    }
    const int n = max(a.kv_len[lo], 0);
    float q[8], o[8], m_run = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int d = lane + 32 * e;
      q[e] = d < hd ? to_f(Q[((size_t)r * a.n_heads + h) * hd + d]) : 0.f;
      o[e] = 0.f;
    }
    for (int key = 0; key < n; ++key) {
      const int pi = key / pg.page_size;
      const int page = pi < a.max_pages ? a.table[(size_t)lo * a.max_pages + pi] : -1;
      if (page < 0 || page >= pg.n_pages) {
        if (lane == 0 && a.status) atomicOr(a.status, DCU_ST_BAD_PAGE);
        if (pi >= a.max_pages) break;
        continue;
      }
      const int64_t at = (int64_t)page * pg.page_stride + (int64_t)(key - pi * pg.page_size) * pg.slot_stride +
                         (int64_t)(h / G) * pg.head_stride;
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < hd) s = fmaf(q[e], to_f(K[at + lane + 32 * e]), s);
      s = warp_sum(s) * a.scale_log2;
      const float m_new = fmaxf(m_run, s);
      const float f = m_run == -INFINITY ? 0.f : exp2f(m_run - m_new), p = exp2f(s - m_new);
      m_run = m_new;
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (lane + 32 * e < hd) o[e] = fmaf(p, to_f(V[at + lane + 32 * e]), o[e] * f);
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < hd)
        static_cast<T *>(a.out)[((size_t)r * a.n_heads + h) * hd + lane + 32 * e] = from_f<T>(o[e] * inv);
  }
}

}  // namespace

int64_t paged_attention_workspace(const dcu_pages &) { return 16; }

cudaError_t launch_paged_attention(const PagedAttnArgs &a, void *, cudaStream_t s) {
  const long long items = (long long)a.max_rows * a.n_heads;
  const int grid = (int)(items / 4 + 1 < 148 * 16 ? items / 4 + 1 : 148 * 16);
  if (a.pages.dtype == DCU_BF16) launch_pdl(k_paged_attn_rowhead<bf16>, dim3(grid), dim3(128), 0, s, a);
  else launch_pdl(k_paged_attn_rowhead<float>, dim3(grid), dim3(128), 0, s, a);
  return cudaGetLastError();
}

}  // namespace dcu
