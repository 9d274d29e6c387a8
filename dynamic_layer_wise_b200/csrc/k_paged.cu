// Plans of a paged K/V cache (block table, slot map) and the RoPE + K/V write
// of the recomputed rows into their slots.
#include "common.cuh"
#include "paged.h"

namespace dcu {
namespace {

__device__ __forceinline__ void flag(int32_t *status, int bit) {
  if (status) atomicOr(status, bit);
}

// Exclusive prefix sum of one int64 per thread in thread order (as
// block_exclusive_scan, but wide: page and row totals may pass 2^31).
__device__ __forceinline__ long long scan64(long long v, long long *red, long long *total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[w] = x;
  __syncthreads();
  long long base = 0, t = 0;
  for (int i = 0; i < nw; ++i) {
    if (i == w) base = t;
    t += red[i];
  }
  __syncthreads();
  *total = t;
  return base + x - v;
}

// ------------------------------------------------------------------ block table
// need_b = ceil(max(len_b, 0) / P), 0 when it exceeds the table row; E_b = its
// inclusive prefix sum.  Request b is served iff first + E_b <= n_pool, and E
// never decreases, so the served requests are a prefix and page j of request b
// is pool[first + E_b - need_b + j]: every table entry is independent of the
// others.  CTA (x, y) writes columns [y C, y C + C) of rows [x R, x R + R) and
// sums the needs of the rows before its own for itself (a few KB from L2)
// instead of waiting for another CTA.
// Measured: 4 requests 2.6 us (a launch), 2000 ragged ones of up to 1024 pages
// (8 MB of table, 3.7 MB of pool) 7.4 us, 1.6 TB/s: short of memory's rate (1.8
// us) by the chain launch - lengths - sums - pool entry - store, and by the rounds
// of a CTA's rows (four here), each of which waits for its pool entries.
__device__ __forceinline__ long long pages_needed(int len, int page_size, int max_pages) {
  if (len <= 0) return 0;
  const unsigned n = ((unsigned)len + (unsigned)page_size - 1u) / (unsigned)page_size;
  return n > (unsigned)max_pages ? 0 : n;
}

constexpr int kTabThreads = 256;
constexpr int kTabCols = 4096;
constexpr int kTabBatch = 4;

__global__ void __launch_bounds__(kTabThreads)
    k_page_table(const int32_t *__restrict__ lens, int B, int page_size, int max_pages, int n_pages,
                 const int32_t *__restrict__ pool, int n_pool, const int32_t *__restrict__ first_p, int rows_per_cta,
                 int32_t *__restrict__ table, int32_t *__restrict__ held, int32_t *__restrict__ next,
                 int32_t *status) {
  pdl_enter();
  __shared__ long long red[32];
  __shared__ int s_src[kTabThreads], s_held[kTabThreads];
  const int b0 = blockIdx.x * rows_per_cta, nr = min(rows_per_cta, B - b0);
  const int c0 = blockIdx.y * kTabCols, c1 = min(max_pages, c0 + kTabCols);
  const int first = first_p ? *first_p : 0;
  const bool ok = first >= 0 && first <= n_pool;
  const long long avail = ok ? (long long)n_pool - first : 0;
  long long before = 0;
  for (int b = threadIdx.x; b < b0; b += kTabThreads) before += pages_needed(lens[b], page_size, max_pages);
  long long base;
  scan64(before, red, &base);
  const int i = threadIdx.x, b = b0 + i;
  const int len = i < nr ? lens[b] : 0;
  const long long need = pages_needed(len, page_size, max_pages);
  long long tot;
  const long long end = base + scan64(need, red, &tot) + need;
  if (i < nr) {
    const bool fits = end <= avail;
    s_held[i] = fits ? (int)need : 0;
    s_src[i] = fits ? first + (int)(end - need) : 0;
    if (blockIdx.y == 0) {
      held[b] = fits ? (int)need : 0;
      if (!fits && need > 0) flag(status, DCU_ST_NO_PAGE);
      if (len > 0 && need == 0) flag(status, DCU_ST_NO_PAGE);
      // the last served request writes next (row 0 when none is)
      const long long after = b + 1 < B ? end + pages_needed(lens[b + 1], page_size, max_pages) : avail + 1;
      if (fits && after > avail) *next = first + (int)end;
      if (b == 0 && !fits) *next = first;
    }
  }
  __syncthreads();
  // columns dealt out to the threads, kTabBatch pool loads of a thread in flight
  const int nc = c1 - c0;
  for (int r = 0; r < nr; ++r) {
    int32_t *row = table + (size_t)(b0 + r) * max_pages + c0;
    const int h = s_held[r] - c0, src = s_src[r] + c0;
    for (int c = threadIdx.x; c < nc; c += kTabThreads * kTabBatch) {
      int pg[kTabBatch];
#pragma unroll
      for (int e = 0; e < kTabBatch; ++e) {
        const int k = c + e * kTabThreads;
        pg[e] = k < h ? (pool ? pool[src + k] : src + k) : -1;
      }
#pragma unroll
      for (int e = 0; e < kTabBatch; ++e) {
        const int k = c + e * kTabThreads;
        if (k >= nc) break;
        if (k < h && (pg[e] < 0 || pg[e] >= n_pages)) {
          pg[e] = -1;
          flag(status, DCU_ST_BAD_PAGE);
        }
        row[k] = pg[e];
      }
    }
  }
}

// ------------------------------------------------------------------ slot map
// Row t of the packed rows belongs to the sequence b with S_b <= t < S_{b+1}
// (S: prefix sums of the counts).  A CTA owns kMapRows consecutive rows, so the
// work is even however ragged the counts are; it scans the counts in chunks of
// kMapChunk into shared memory and finds each row's sequence by bisection.
// CTA 0 scans them all and writes row_start.  Measured: 65 rows 2.6 us, the rows
// of 500 ragged requests 4.0 us: launches and dependent loads (counts, position,
// table entry); the bytes would take 0.1 us.
constexpr int kMapThreads = 256;
constexpr int kMapPer = 4;
constexpr int kMapChunk = kMapThreads * kMapPer;
constexpr int kMapRows = 512;

__global__ void __launch_bounds__(kMapThreads)
    k_slot_map(const int32_t *__restrict__ table, int B, int max_pages, int page_size, int n_pages,
               const int32_t *__restrict__ count, const int32_t *__restrict__ pos, int pos_stride,
               const int32_t *__restrict__ first, int max_rows, int32_t *__restrict__ row_start,
               int32_t *__restrict__ row_pos, int32_t *__restrict__ slot, int32_t *status) {
  pdl_enter();
  __shared__ long long red[32];
  __shared__ long long s_end[kMapChunk];  // inclusive prefix sums of the chunk's counts
  const long long t0 = (long long)blockIdx.x * kMapRows, t1 = min((long long)max_rows, t0 + kMapRows);
  long long base = 0;
  for (int c0 = 0; c0 < B; c0 += kMapChunk) {
    int n[kMapPer];
    long long mine = 0;
#pragma unroll
    for (int e = 0; e < kMapPer; ++e) {
      const int b = c0 + threadIdx.x * kMapPer + e;
      int k = b < B ? max(count[b], 0) : 0;
      if (pos && k > pos_stride) {
        k = pos_stride;
        flag(status, DCU_ST_BAD_ROW);
      }
      n[e] = k;
      mine += k;
    }
    long long total;
    long long run = base + scan64(mine, red, &total);
#pragma unroll
    for (int e = 0; e < kMapPer; ++e) {
      const int b = c0 + threadIdx.x * kMapPer + e;
      if (blockIdx.x == 0 && b < B) row_start[b] = (int)min(run, (long long)max_rows);
      run += n[e];
      s_end[threadIdx.x * kMapPer + e] = run;
      if (blockIdx.x == 0 && b == B - 1) {
        row_start[B] = (int)min(run, (long long)max_rows);
        if (run > max_rows) flag(status, DCU_ST_BAD_ROW);
      }
    }
    __syncthreads();
    const long long lo = max(t0, base), hi = min(t1, base + total);
    for (long long t = lo + threadIdx.x; t < hi; t += kMapThreads) {
      int a = 0, z = kMapChunk - 1;  // the first sequence whose end is above t
      while (a < z) {
        const int m = (a + z) >> 1;
        if (s_end[m] > t) z = m;
        else a = m + 1;
      }
      const int b = c0 + a;
      const int j = (int)(t - (a ? s_end[a - 1] : base));
      long long p;
      if (pos) {
        const int32_t *pr = pos + (size_t)b * pos_stride + j;
        p = pr[0];
        if (j > 0 && pr[-1] >= p) flag(status, DCU_ST_BAD_ROW);
      } else {
        p = (first ? (long long)first[b] : 0) + j;
      }
      int sl = -1;
      if (p >= 0 && p <= 0x7fffffffll) {
        const int pi = (int)((unsigned)p / (unsigned)page_size);
        if (pi < max_pages) {
          const int pg = table[(size_t)b * max_pages + pi];
          if (pg >= 0 && pg < n_pages) sl = pg * page_size + ((int)p - pi * page_size);
        }
      }
      if (sl < 0) flag(status, DCU_ST_BAD_PAGE);
      row_pos[t] = (int)max(-1ll, min(p, 0x7fffffffll));
      slot[t] = sl;
    }
    base += total;
    if (blockIdx.x != 0 && base >= t1) break;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ RoPE + K/V write
// A work item is elements j .. j + 3 of both halves of a head (4 pairs of q or k;
// of v merely 8 elements): 32 bytes read, two vectors written, and a warp's loads
// and stores are whole lines.  (Items of 8 pairs, whose lanes read every other 16
// bytes, measured before: 1.03 to 1.09 times as long in bf16, 1.1 to 1.17 in
// float32, 1.4 for 512 rows in L2.)
__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
}
__device__ __forceinline__ void store4(bf16 *p, const float (&v)[4]) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(v[0], v[1]), y = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// grid (rows, slices of a row): each thread has one item of one row, and its 32
// bytes are on the way before the row's slot and position and the row count are
// known: rows not in use are read for nothing (the count awaited first, measured: 65
// rows 2.25 in place of 2.13 us, 512 rows of which 51 are used 1.72 in place of 2.07,
// thousands of rows the same either way).  A row is
// streamed once and written once, so memory bounds it: 6148 rows of 28 + 2 x 4
// heads of 128 take 29.0 us, 6.0 TB/s (a plain copy: 6.46); 65 rows of 96 heads
// 2.1 to 2.6 us, a launch.  q, K and V are rounded once, from the fp32 rotation.
constexpr int kWriteMax = 512;  // most threads of a CTA

template <class T>
__global__ void __launch_bounds__(kWriteMax)
    k_paged_write(const float *__restrict__ qkv, int max_rows, const int32_t *__restrict__ n_rows,
                  const int32_t *__restrict__ row_pos, const int32_t *__restrict__ slot,
                  const float2 *__restrict__ rope, int max_pos, int H, const dcu_pages pg, T *__restrict__ q,
                  int32_t *status) {
  pdl_enter();
  const int hd = pg.head_dim, KV = pg.n_kv_heads, half = hd / 2;
  const int per = half / 4, items = (H + 2 * KV) * per;
  const int t = blockIdx.x, u = blockIdx.y * blockDim.x + threadIdx.x;
  if (u >= items) return;
  const int head = u / per, j = (u - head * per) * 4;
  const bool is_v = head >= H + KV;
  const float *x = qkv + (size_t)t * (size_t)(H + 2 * KV) * hd + (size_t)head * hd + j;
  float a[4], b[4];
  load4(x, a);
  load4(x + half, b);
  const int sl = slot[t], p = rope ? row_pos[t] : 0, used = n_rows ? *n_rows : max_rows;
  if (t >= used) return;
  const unsigned n_slots = (unsigned)pg.n_pages * (unsigned)pg.page_size;  // below 2^31
  const bool good = !rope || (p >= 0 && p < max_pos);
  if (u == 0) {
    const int bits = (!good || (t == 0 && used > max_rows) ? DCU_ST_BAD_ROW : 0) |
                     ((unsigned)sl + 1u > n_slots ? DCU_ST_BAD_PAGE : 0);  // (-1 is no slot, and no fault)
    if (bits) flag(status, bits);
  }
  T *dst;
  if (head < H) {
    dst = q + ((size_t)t * H + head) * hd + j;
  } else {
    if (!good || (unsigned)sl >= n_slots) return;
    const int page = (int)((unsigned)sl / (unsigned)pg.page_size);
    dst = static_cast<T *>(is_v ? pg.v : pg.k) + (int64_t)page * pg.page_stride +
          (int64_t)(sl - page * pg.page_size) * pg.slot_stride + (int64_t)(head - H - (is_v ? KV : 0)) * pg.head_stride + j;
  }
  if (rope && !is_v) {
    const float4 *cs = reinterpret_cast<const float4 *>(rope + (size_t)(good ? p : 0) * half + j);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float4 c = __ldg(cs + e / 2);
      const float a0 = a[e] * c.x - b[e] * c.y, b0 = b[e] * c.x + a[e] * c.y;
      const float a1 = a[e + 1] * c.z - b[e + 1] * c.w, b1 = b[e + 1] * c.z + a[e + 1] * c.w;
      a[e] = good ? a0 : 0.f;
      b[e] = good ? b0 : 0.f;
      a[e + 1] = good ? a1 : 0.f;
      b[e + 1] = good ? b1 : 0.f;
    }
  }
  store4(dst, a);
  store4(dst + half, b);
}

}  // namespace

cudaError_t launch_page_table(const int32_t *lens, int B, int page_size, int max_pages, int n_pages,
                              const int32_t *pool, int n_pool, const int32_t *first, int32_t *table, int32_t *held,
                              int32_t *next, int32_t *status, cudaStream_t s) {
  // rows per CTA: at most 4 CTAs of row groups per SM, at most one thread per row
  int per = (B + 148 * 4 - 1) / (148 * 4);
  if (per > kTabThreads) per = kTabThreads;
  const dim3 grid((B + per - 1) / per, (max_pages + kTabCols - 1) / kTabCols);
  return launch_pdl(k_page_table, grid, dim3(kTabThreads), 0, s, lens, B, page_size, max_pages, n_pages, pool, n_pool,
                    first, per, table, held, next, status);
}

cudaError_t launch_slot_map(const int32_t *table, int B, int max_pages, int page_size, int n_pages,
                            const int32_t *count, const int32_t *pos, int pos_stride, const int32_t *first,
                            int max_rows, int32_t *row_start, int32_t *row_pos, int32_t *slot, int32_t *status,
                            cudaStream_t s) {
  const int grid = max_rows > 0 ? (int)(((long long)max_rows + kMapRows - 1) / kMapRows) : 1;
  return launch_pdl(k_slot_map, dim3(grid), dim3(kMapThreads), 0, s, table, B, max_pages, page_size, n_pages, count,
                    pos, pos_stride, first, max_rows, row_start, row_pos, slot, status);
}

cudaError_t launch_paged_write(const float *qkv, int max_rows, const int32_t *n_rows, const int32_t *row_pos,
                               const int32_t *slot, const float2 *rope, int max_pos, int n_heads,
                               const dcu_pages &pages, void *q, int32_t *status, cudaStream_t s) {
  // a row's items in as few slices as fit a CTA, in equal parts
  const int items = (n_heads + 2 * pages.n_kv_heads) * (pages.head_dim / 8);
  const int slices = (items + kWriteMax - 1) / kWriteMax;
  const int threads = ((items + slices - 1) / slices + 31) / 32 * 32;
  const dim3 grid(max_rows, slices);
  if (pages.dtype == DCU_BF16)
    return launch_pdl(k_paged_write<bf16>, grid, dim3(threads), 0, s, qkv, max_rows, n_rows, row_pos, slot, rope,
                      max_pos, n_heads, pages, (bf16 *)q, status);
  return launch_pdl(k_paged_write<float>, grid, dim3(threads), 0, s, qkv, max_rows, n_rows, row_pos, slot, rope,
                      max_pos, n_heads, pages, (float *)q, status);
}

}  // namespace dcu
