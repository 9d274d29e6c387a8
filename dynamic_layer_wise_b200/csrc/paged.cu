// C entry points of the paged K/V cache: argument checks, then one launcher
// call each.  No allocation, no synchronisation, no state between calls.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "kernels.h"
#include "paged.h"

using namespace dcu;

namespace {

int pg_fail(int code, const char *msg) noexcept {
  try {
    set_global_error(msg);
  } catch (...) {
  }
  return code;
}

int pg_cuda(cudaError_t e, const char *call) noexcept {
  if (e == cudaSuccess) return DCU_OK;
  cudaGetLastError();  // reported here: not left for the next call
  try {
    set_global_error((std::string(call) + ": " + cudaGetErrorString(e)).c_str());
  } catch (...) {
  }
  return DCU_ECUDA;
}

bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

struct Span {
  const void *p;  // NULL: not given
  int64_t bytes;
};
// Whether an output overlaps an input or another output: the kernels' threads read and write in no order.
bool clash(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span *o = outs.begin(); o != outs.end(); ++o) {
    if (!o->p || !o->bytes) continue;
    for (const Span *x = outs.begin(); x != o; ++x)
      if (x->p && x->bytes && overlap(o->p, o->bytes, x->p, x->bytes)) return true;
    for (const Span &x : ins)
      if (x.p && x.bytes && overlap(o->p, o->bytes, x.p, x.bytes)) return true;
  }
  return false;
}

bool mis(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

const char *bad_pages(const dcu_pages *p) {
  if (!p || !p->k || !p->v) return "pages: null pointer";
  if (p->dtype != DCU_F32 && p->dtype != DCU_BF16) return "pages: dtype must be DCU_F32 or DCU_BF16";
  if (p->n_pages <= 0 || p->page_size <= 0 || (int64_t)p->n_pages * p->page_size >= (1ll << 31))
    return "pages: n_pages and page_size must be positive with n_pages * page_size < 2^31";
  if (p->n_kv_heads <= 0 || p->head_dim <= 0 || p->head_dim % 16 || p->head_dim > 256)
    return "pages: n_kv_heads must be positive and head_dim a multiple of 16 up to 256";
  const int64_t v = p->dtype == DCU_BF16 ? 8 : 4;
  if (mis(p->k, 16) || mis(p->v, 16)) return "pages: k and v must be 16-byte aligned";
  if (p->page_stride < 0 || p->slot_stride < 0 || p->head_stride < 0 || p->page_stride % v || p->slot_stride % v ||
      p->head_stride % v)
    return "pages: strides must be non-negative multiples of 16 bytes";
  return nullptr;
}

}  // namespace

extern "C" {

int dcu_page_table(const int32_t *lens, int32_t B, int32_t page_size, int32_t max_pages, int32_t n_pages,
                   const int32_t *pool, int32_t n_pool, const int32_t *first, int32_t *table, int32_t *held,
                   int32_t *next, int32_t *status, dcu_stream_t stream) {
  if (!lens || !table || !held || !next || B <= 0 || B > kPagedMaxB || page_size <= 0 || max_pages <= 0 ||
      max_pages > (1 << 27) || n_pages <= 0 || n_pool < 0 || (int64_t)n_pages * page_size >= (1ll << 31) || next == first)
    return pg_fail(DCU_EINVAL, "dcu_page_table: bad argument");
  if (!pool && n_pool != n_pages && n_pool != 0)
    return pg_fail(DCU_EINVAL, "dcu_page_table: without a pool, n_pool must be n_pages");
  if (clash({{table, 4ll * B * max_pages}, {held, 4ll * B}, {next, 4}, {status, 4}},
            {{lens, 4ll * B}, {pool, 4ll * n_pool}, {first, 4}}))
    return pg_fail(DCU_EINVAL, "dcu_page_table: an output overlaps another array");
  return pg_cuda(launch_page_table(lens, B, page_size, max_pages, n_pages, pool, n_pool, first, table, held, next,
                                   status, (cudaStream_t)stream),
                 "dcu_page_table");
}

int dcu_slot_map(const int32_t *table, int32_t B, int32_t max_pages, int32_t page_size, int32_t n_pages,
                 const int32_t *count, const int32_t *pos, int32_t pos_stride, const int32_t *first,
                 int32_t max_rows, int32_t *row_start, int32_t *row_pos, int32_t *slot, int32_t *status,
                 dcu_stream_t stream) {
  if (!table || !count || !row_start || B <= 0 || B > kPagedMaxB || max_pages <= 0 || page_size <= 0 ||
      n_pages <= 0 || (int64_t)n_pages * page_size >= (1ll << 31) || max_rows < 0 ||
      (max_rows > 0 && (!row_pos || !slot)) || (pos && (pos_stride <= 0 || first)))
    return pg_fail(DCU_EINVAL, "dcu_slot_map: bad argument");
  if (clash({{row_start, 4ll * (B + 1)}, {row_pos, 4ll * max_rows}, {slot, 4ll * max_rows}, {status, 4}},
            {{table, 4ll * B * max_pages}, {count, 4ll * B}, {pos, 4ll * B * pos_stride}, {first, 4ll * B}}))
    return pg_fail(DCU_EINVAL, "dcu_slot_map: an output overlaps another array");
  return pg_cuda(launch_slot_map(table, B, max_pages, page_size, n_pages, count, pos, pos_stride, first, max_rows,
                                 row_start, row_pos, slot, status, (cudaStream_t)stream),
                 "dcu_slot_map");
}

int dcu_rope_table(float *tab, int32_t max_pos, int32_t head_dim, float theta, dcu_stream_t stream) {
  if (!tab || mis(tab, 8) || max_pos <= 0 || head_dim <= 0 || head_dim % 2 || !(theta > 0.f) || std::isinf(theta))
    return pg_fail(DCU_EINVAL, "dcu_rope_table: bad argument");
  return pg_cuda(launch_rope_table(reinterpret_cast<float2 *>(tab), max_pos, head_dim, theta, (cudaStream_t)stream),
                 "dcu_rope_table");
}

int dcu_paged_write(const float *qkv, int32_t max_rows, const int32_t *n_rows, const int32_t *row_pos,
                    const int32_t *slot, const float *rope, int32_t max_pos, int32_t n_heads,
                    const dcu_pages *pages, void *q, int32_t *status, dcu_stream_t stream) {
  if (const char *m = bad_pages(pages)) return pg_fail(DCU_EINVAL, m);
  if (max_rows < 0 || n_heads <= 0 || (max_rows > 0 && (!qkv || !slot || !q || (rope && !row_pos))) ||
      (rope && max_pos <= 0))
    return pg_fail(DCU_EINVAL, "dcu_paged_write: bad argument");
  if (mis(qkv, 16) || mis(rope, 16) || mis(q, 16))
    return pg_fail(DCU_EINVAL, "dcu_paged_write: qkv, rope and q must be 16-byte aligned");
  if ((int64_t)n_heads + 2ll * pages->n_kv_heads > (1ll << 19))  // (32 items a head, 512 a block, 65535 slices)
    return pg_fail(DCU_EINVAL, "dcu_paged_write: too many heads");
  if ((pages->n_pages > 1 && !pages->page_stride) || (pages->page_size > 1 && !pages->slot_stride) ||
      (pages->n_kv_heads > 1 && !pages->head_stride))
    return pg_fail(DCU_EINVAL, "dcu_paged_write: pages with a zero stride cannot be written");
  if (max_rows == 0) return DCU_OK;
  if (pages->k == pages->v) return pg_fail(DCU_EINVAL, "dcu_paged_write: K and V share their pages");
  const int64_t es = pages->dtype == DCU_BF16 ? 2 : 4, rh = (int64_t)max_rows * pages->head_dim;
  if (overlap(q, rh * n_heads * es, qkv, rh * (n_heads + 2ll * pages->n_kv_heads) * 4))
    return pg_fail(DCU_EINVAL, "dcu_paged_write: q overlaps qkv");
  if (clash({{q, rh * n_heads * es}, {status, 4}},
            {{n_rows, 4}, {row_pos, 4ll * max_rows}, {slot, 4ll * max_rows}, {rope, rope ? 4ll * max_pos * pages->head_dim : 0}}))
    return pg_fail(DCU_EINVAL, "dcu_paged_write: q overlaps another array");
  return pg_cuda(launch_paged_write(qkv, max_rows, n_rows, row_pos, slot, reinterpret_cast<const float2 *>(rope),
                                    max_pos, n_heads, *pages, q, status, (cudaStream_t)stream),
                 "dcu_paged_write");
}

int dcu_paged_attention_workspace(const dcu_pages *pages, int64_t *bytes) {
  if (const char *m = bad_pages(pages)) return pg_fail(DCU_EINVAL, m);
  if (!bytes) return pg_fail(DCU_EINVAL, "dcu_paged_attention_workspace: bytes is NULL");
  *bytes = paged_attention_workspace(*pages);
  return DCU_OK;
}

int dcu_paged_attention(const void *q, int32_t max_rows, const int32_t *row_start, int32_t B, const int32_t *kv_len,
                        const int32_t *table, int32_t max_pages, int32_t n_heads, const dcu_pages *pages, float scale,
                        void *out, void *workspace, int64_t workspace_bytes, int32_t *status, dcu_stream_t stream) {
  if (const char *m = bad_pages(pages)) return pg_fail(DCU_EINVAL, m);
  if (!row_start || !kv_len || !table || B <= 0 || B > kPagedMaxB || max_pages <= 0 || max_rows < 0 ||
      n_heads <= 0 || n_heads % pages->n_kv_heads || n_heads > (1 << 20) || !std::isfinite(scale * 1.4426950408889634f) ||
      (max_rows > 0 && (!q || !out)))
    return pg_fail(DCU_EINVAL, "dcu_paged_attention: bad argument");
  if (mis(q, 16) || mis(out, 16) || mis(workspace, 16))
    return pg_fail(DCU_EINVAL, "dcu_paged_attention: q, out and workspace must be 16-byte aligned");
  if (max_rows == 0) return DCU_OK;
  if ((int64_t)max_rows * (n_heads / pages->n_kv_heads) >= (1ll << 30))  // queries of a kv head are counted in 32 bits
    return pg_fail(DCU_EINVAL, "dcu_paged_attention: too many rows x heads of a group");
  const int64_t qb = (int64_t)max_rows * n_heads * pages->head_dim * (pages->dtype == DCU_BF16 ? 2 : 4);
  if (overlap(q, qb, out, qb)) return pg_fail(DCU_EINVAL, "dcu_paged_attention: out may not overlap q");
  if (!workspace || workspace_bytes < paged_attention_workspace(*pages))
    return pg_fail(DCU_EINVAL, "dcu_paged_attention: workspace smaller than dcu_paged_attention_workspace");
  if (clash({{out, qb}, {workspace, paged_attention_workspace(*pages)}, {status, 4}},
            {{q, qb}, {row_start, 4ll * (B + 1)}, {kv_len, 4ll * B}, {table, 4ll * B * max_pages}}))
    return pg_fail(DCU_EINVAL, "dcu_paged_attention: out or the workspace overlaps another array");
  PagedAttnArgs a;
  a.q = q;
  a.out = out;
  a.row_start = row_start;
  a.kv_len = kv_len;
  a.table = table;
  a.pages = *pages;
  a.B = B;
  a.max_rows = max_rows;
  a.max_pages = max_pages;
  a.n_heads = n_heads;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (pages->page_size == 1 << i) a.page_shift = i;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.whole = false;
  a.status = status;
  return pg_cuda(launch_paged_attention(a, workspace, (cudaStream_t)stream), "dcu_paged_attention");
}

}  // extern "C"
