// Host-side launchers of the paged K/V cache kernels (internal).  Arguments
// have been checked by the entry points in paged.cu.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dcu.h"

namespace dcu {

constexpr int kPagedMaxB = 65536;  // every CTA of the planning prologues scans the B counts

// ---- plans and the K/V write (k_paged.cu)
cudaError_t launch_page_table(const int32_t *lens, int B, int page_size, int max_pages, int n_pages,
                              const int32_t *pool, int n_pool, const int32_t *first, int32_t *table, int32_t *held,
                              int32_t *next, int32_t *status, cudaStream_t s);
cudaError_t launch_slot_map(const int32_t *table, int B, int max_pages, int page_size, int n_pages,
                            const int32_t *count, const int32_t *pos, int pos_stride, const int32_t *first,
                            int max_rows, int32_t *row_start, int32_t *row_pos, int32_t *slot, int32_t *status,
                            cudaStream_t s);
cudaError_t launch_paged_write(const float *qkv, int max_rows, const int32_t *n_rows, const int32_t *row_pos,
                               const int32_t *slot, const float2 *rope, int max_pos, int n_heads,
                               const dcu_pages &pages, void *q, int32_t *status, cudaStream_t s);

// ---- attention (k_paged_attn.cu)
struct PagedAttnArgs {
  const void *q;
  void *out;
  const int32_t *row_start, *kv_len, *table;
  dcu_pages pages;
  int32_t B, max_rows, max_pages, n_heads;
  int32_t page_shift;  // log2(page_size), -1 when it is no power of two
  float scale_log2;    // scale * log2(e)
  bool whole;          // no item is cut: fewer items than CTAs, and short ones (whole_items)
  int32_t *status;
};
int64_t paged_attention_workspace(const dcu_pages &pages);
cudaError_t launch_paged_attention(const PagedAttnArgs &a, void *workspace, cudaStream_t s);

}  // namespace dcu
