// The line of work of the paged attention kernels: every (sequence, kv head,
// query tile) is an item of ceil(keys / KB) units, units are numbered in item
// order, and each CTA takes an equal range of them.  Lengths and rows are only
// on the device, so each CTA derives the cut itself.
#pragma once
#include "common.cuh"
#include "gemm_tc.h"
#include "paged.h"

namespace dcu {

constexpr int kMaxRanges = 148;  // most CTAs (work ranges) of a launch

// A share of an item that a range boundary cuts: what the merge needs.
struct Share {
  int32_t last;   // last range that holds a share of the item begun in this range; -1: none is cut here
  int32_t row0;   // first packed row of the sequence
  int32_t q0;     // first query (pair index in the sequence and kv head) of the tile
  int32_t nq;     // queries of the tile
  int32_t kvh;
  int32_t slot;   // the share of this range: 0 its first segment, 1 its last one
};

namespace {

// key / page_size: a shift for the usual powers of two
__device__ __forceinline__ unsigned div_page(const PagedAttnArgs &a, unsigned key) {
  return a.page_shift >= 0 ? key >> a.page_shift : key / (unsigned)a.pages.page_size;
}

// The items of sequence b.
struct Seq {
  int row0, nq, tiles, tq, nk, nblk;  // first row, queries per kv head, tiles, queries per tile, keys, blocks per item
  __device__ __forceinline__ long long units(int KV) const { return (long long)KV * tiles * nblk; }
};
// FLAG: sets the status bits of the sequence, once a CTA (find_range's first look at it).
template <int R, int KB, bool FLAG = false>
__device__ __forceinline__ Seq seq_of(const PagedAttnArgs &a, int b) {
  Seq s;
  const int r0 = a.row_start[b], r1 = a.row_start[b + 1];
  const int lo = min(max(r0, 0), a.max_rows), hi = min(max(r1, 0), a.max_rows);
  const int rows = max(hi - lo, 0);
  s.row0 = lo;
  s.nq = rows * (a.n_heads / a.pages.n_kv_heads);
  s.tiles = (s.nq + R - 1) / R;
  s.tq = s.tiles ? ((s.nq + s.tiles - 1) / s.tiles + 7) / 8 * 8 : 0;
  const long long cap = (long long)a.max_pages * a.pages.page_size;
  const int n = max(a.kv_len[b], 0);
  if (FLAG) {
    const int bits = (r0 < 0 || r1 < r0 || r1 > a.max_rows ? DCU_ST_BAD_ROW : 0) | (n > cap && rows ? DCU_ST_BAD_PAGE : 0);
    if (bits && a.status) atomicOr(a.status, bits);
  }
  s.nk = (int)min((long long)n, cap);
  s.nblk = max(1, (int)(((long long)s.nk + KB - 1) / KB));  // an empty sequence still gets its zeros
  return s;
}

// A place in the line of units: block blk of (b, kv head, tile).
struct Place {
  int b, kvh, tile, blk;
  Seq s;
};
// The next sequence with rows.  Those without are passed one by one, about 80 ns each: one row of 8 heads x 64 over 500
// keys takes 7.7 us alone, 44 us with 500 sequences without rows behind it.
template <int R, int KB>
__device__ __forceinline__ void next_seq(const PagedAttnArgs &a, Place &p) {
  while (++p.b < a.B) {
    p.s = seq_of<R, KB>(a, p.b);
    if (p.s.tiles) break;
  }
}
template <int R, int KB>
__device__ __forceinline__ void advance(const PagedAttnArgs &a, Place &p, int n) {
  p.blk += n;
  while (p.b < a.B && p.blk >= p.s.nblk) {
    p.blk -= p.s.nblk;
    if (++p.tile == p.s.tiles) {
      p.tile = 0;
      if (++p.kvh == a.pages.n_kv_heads) {
        p.kvh = 0;
        next_seq<R, KB>(a, p);
      }
    }
  }
}


// The range [u0, u1) of a CTA.  Either the line is cut evenly (range i of the
// launch holds q + 1 units when i < rem, else q), or, where the items are few,
// every item is cut by itself into equal parts: then no CTA works on two items,
// and an item has fewer shares.
struct Range {
  long long u0, u1, q;
  int rem, last;  // last -1: the even cut; else the last range of the only item, whose units count from 0
  bool any;
  // the range that holds unit u, the last one of an item that the range has a part of
  __device__ __forceinline__ int of(long long u) const {
    if (last >= 0) return last;
    const long long wide = rem * (q + 1);
    return u < wide ? (int)(u / (q + 1)) : rem + (int)((u - wide) / q);
  }
};

__device__ __forceinline__ long long div_ll(long long a, int b) {
  return a < (1ll << 32) ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Cuts `total` units for the CTA; kept out of line of the place search so that
// one sequence (B == 1) needs neither the scan nor a barrier.
__device__ __forceinline__ void cut_even(Range &rg, long long total, int ranges) {
  const int bid = (int)blockIdx.x;
  rg.last = -1;
  rg.any = bid < ranges;
  rg.q = ranges ? div_ll(total, ranges) : 0;
  rg.rem = (int)(total - rg.q * ranges);
  rg.u0 = bid * rg.q + min(bid, rg.rem);
  rg.u1 = rg.u0 + rg.q + (bid < rg.rem ? 1 : 0);
}
// Item, kv head, tile and block of unit `off` of sequence p.s.
__device__ __forceinline__ void locate(Place &p, long long off) {
  const long long item = div_ll(off, p.s.nblk);
  p.blk = (int)(off - item * p.s.nblk);
  p.kvh = (int)div_ll(item, p.s.tiles);
  p.tile = (int)(item - (long long)p.kvh * p.s.tiles);
}

// part `part` of `parts` of item `item` of sequence p.s
__device__ __forceinline__ void cut_item(Range &rg, Place &p, int item, int part, int parts, int first_range) {
  rg.u0 = div_ll((long long)part * p.s.nblk, parts);
  rg.u1 = div_ll((long long)(part + 1) * p.s.nblk, parts);
  rg.last = first_range + parts - 1;
  p.blk = (int)rg.u0;
  p.kvh = item / p.s.tiles;
  p.tile = item - p.kvh * p.s.tiles;
}

// All W warps of the CTA: its range and its first place, in shared memory (each
// thread's own copies of what the search holds would cost the kernels registers).
// A launch uses the whole grid unless that leaves a range less than `least` units
// of an item that is cut: as many ranges as there are items, or as many as have
// `least` units, whichever is more.  The cut is by items where that makes the
// longest range at most `turn` units longer than the even cut does: what a
// CTA's change of items costs.
template <int R, int KB, int W>
__device__ __forceinline__ void find_range(const PagedAttnArgs &a, Place *place, Range *range, long long *scan,
                                           int least, int turn) {
  const int KV = a.pages.n_kv_heads;
  Range rg;
  if (a.B == 1) {
    Place p;
    p.b = 0;
    p.s = seq_of<R, KB, true>(a, 0);
    const long long total = p.s.units(KV);
    const long long items = (long long)KV * p.s.tiles;
    const int ranges = (int)min((long long)gridDim.x, max(items, div_ll(total + least - 1, least)));
    cut_even(rg, total, ranges);
    if (total > 0 && items <= ranges) {
      const int f = a.whole ? 1 : ranges / (int)items;
      if (a.whole || (p.s.nblk + f - 1) / f <= (int)rg.q + (rg.rem ? 1 : 0) + turn) {
        const int item = (int)blockIdx.x / f;
        rg.any = item < items;
        if (rg.any) cut_item(rg, p, item, (int)blockIdx.x - item * f, f, item * f);
      }
    }
    if (rg.any && rg.last < 0) locate(p, rg.u0);
    if (threadIdx.x == 0) {
      *place = p;
      *range = rg;
    }
    __syncthreads();
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.B + 32 * W - 1) / (32 * W);
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  long long mine = 0, items = 0;
  Place p;  // with one sequence per thread (B <= 32 W) its items are kept
  p.b = b0;
  for (int b = b0; b < b1; ++b) {
    p.s = seq_of<R, KB, true>(a, b);
    mine += p.s.units(KV);
    items += (long long)KV * p.s.tiles;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
  if (lane == 31) {
    scan[warp] = x;
    scan[W + warp] = items;
  }
  __syncthreads();
  long long base = 0, total = 0;
  items = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i == warp) base = total;
    total += scan[i];
    items += scan[W + i];
  }
  const int ranges = (int)min((long long)gridDim.x, max(items, div_ll(total + least - 1, least)));
  if (items > 0 && items <= (int)gridDim.x) {
    // parts of at most cut[c] units: the first c that gives no more parts than there are CTAs.  The counts (at most
    // items + total / cut, below 300) are added up packed, 16 bits for each c.
    constexpr int NC = 4;
    __shared__ unsigned long long s_cnt[W];
    const int even = a.whole ? 1 << 30 : (int)div_ll(total + ranges - 1, ranges);
    const int cut[NC] = {even, even + turn / 4, even + turn / 2, even + turn};
    unsigned long long n = 0;
    for (int b = b0; b < b1; ++b) {
      const Seq s = per == 1 ? p.s : seq_of<R, KB>(a, b);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        n += (unsigned long long)(KV * s.tiles * (((unsigned)s.nblk + cut[c] - 1u) / (unsigned)cut[c])) << (16 * c);
    }
    unsigned long long upto = n, before = 0, all4 = 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) s_cnt[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (i == warp) before = all4;
      all4 += s_cnt[i];
    }
    before += upto - n;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int all = (int)(all4 >> (16 * c) & 0xffffu), mine_r = (int)(n >> (16 * c) & 0xffffu);
      if (all > (int)gridDim.x) continue;
      int at_r = (int)(before >> (16 * c) & 0xffffu);
      const int bid = (int)blockIdx.x;
      if (bid >= at_r && bid < at_r + mine_r) {  // exactly one thread, or none
        int f = 0;
        for (p.b = b0; p.b < b1; ++p.b) {
          if (per > 1) p.s = seq_of<R, KB>(a, p.b);
          f = (p.s.nblk + cut[c] - 1) / cut[c];
          if (bid < at_r + KV * p.s.tiles * f) break;
          at_r += KV * p.s.tiles * f;
        }
        const int item = (bid - at_r) / f;
        cut_item(rg, p, item, bid - at_r - item * f, f, at_r + item * f);
        rg.any = true;
        *place = p;
        *range = rg;
      }
      if (tid == 0 && bid >= all) {
        rg.any = false;
        *range = rg;
      }
      __syncthreads();
      return;
    }
  }
  cut_even(rg, total, ranges);
  long long at = base + x - mine;
  if (rg.any && rg.u0 >= at && rg.u0 < at + mine) {  // exactly one thread
    if (per > 1)
      for (p.b = b0; p.b < b1; ++p.b) {
        p.s = seq_of<R, KB>(a, p.b);
        if (rg.u0 < at + p.s.units(KV)) break;
        at += p.s.units(KV);
      }
    locate(p, rg.u0 - at);
    *place = p;
  }
  if (tid == 0) *range = rg;
  __syncthreads();
}

// The (row, head) pairs of a tile: query r is row r0 + (h0 + r) / G, head h0 + r
// modulo G of the group.
struct Pairs {
  int row0, h0, G;
  float inv;
  __device__ __forceinline__ Pairs(const Seq &s, int q0, int G_) : G(G_), inv(1.f / (float)G_) {
    row0 = s.row0 + q0 / G;
    h0 = q0 % G;
  }
  // element offset of query r (< 256) of kv head kvh in [rows][H][hd]; exact: h0 + r is far below 2^21, where the
  // fp32 product's error stays below the distance 0.5 / G to the next integer
  __device__ __forceinline__ size_t at(int r, int kvh, int H, int hd) const {
    const int i = h0 + r;
    const int d = G == 1 ? i : (int)(((float)i + 0.5f) * inv);
    return ((size_t)(row0 + d) * H + kvh * G + (i - d * G)) * hd;
  }
};

// Place of dim d of query q in a share of kr queries: groups of 4 dims, so the
// threads that write a share (one query each) store whole lines.
__device__ __forceinline__ size_t share_at(size_t share, int kr, int dp, int q, int d) {
  return ((share * (dp / 4) + d / 4) * kr + q) * 4 + (d & 3);
}
__device__ __forceinline__ void load_query16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void load_query_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

}  // namespace

// The shares of a launch in the workspace: two per range at most, kr queries each.
struct ShareBuf {
  float *o;      // [ranges][2][dp / 4][kr][4]
  float2 *ml;    // [ranges][2][kr] (max in log2 units, sum)
  Share *desc;   // [ranges]
  ShareBuf(void *ws, int kr, int dp)
      : o(static_cast<float *>(ws)), ml(reinterpret_cast<float2 *>(o + (size_t)kMaxRanges * 2 * kr * dp)),
        desc(reinterpret_cast<Share *>(ml + (size_t)kMaxRanges * 2 * kr)) {}
  static constexpr int64_t bytes(int kr, int dp) {
    return (int64_t)kMaxRanges * 2 * kr * (dp * 4 + 8) + (int64_t)kMaxRanges * sizeof(Share);
  }
};

// Tensor maps of a layer's pages: box of kb slots, dims (d, head, slot, page)
// when head_first, else (d, slot, head, page).
struct PageMaps {
  CUtensorMap k, v;
  int box, head_first;
};
// k_paged_attn.cu
bool page_maps(const dcu_pages &p, int kb, PageMaps *m);
cudaError_t paged_grid(int *grid);  // one range per SM
// Whether no item of a call is to be cut, which spares the merge: at most `most` units of kb keys an item, by what the
// table holds, and not more tiles of r queries than CTAs, by the rows and sequences.  Measured with 4 units (narrow
// kernel: 4 blocks a warp), cut / whole, us in a graph: 65 rows of 32 heads x 512 keys 14.3 / 11.8, one row x 256 keys
// 9.5 / 6.8, 33 float32 rows of 4 heads x 256 keys 11.1 / 9.6 (2.2 us less from Python in each case); with 8 units 65
// rows x 1024 keys 15.2 / 15.8, one row x 1024 keys 10.9 / 12.8.
inline bool whole_items(const PagedAttnArgs &a, int r, int kb, int most, int grid) {
  const long long q = (long long)a.max_rows * (a.n_heads / a.pages.n_kv_heads);
  return (long long)a.max_pages * a.pages.page_size <= (long long)kb * most &&
         ((q + r - 1) / r + a.B - 1) * a.pages.n_kv_heads <= grid;
}
cudaError_t launch_paged_merge(const PagedAttnArgs &a, int kr, int grid, const ShareBuf &sb, cudaStream_t s);

// k_paged_attn_tc.cu: bf16, boxes of 8 .. 64 slots of one page
constexpr int kTcQueries = 128;  // queries of a tile
int tc_box_keys(const dcu_pages &p);  // slots of a box (page_size % 8 == 0)
cudaError_t launch_paged_attention_tc(const PagedAttnArgs &a, const PageMaps &m, void *ws, cudaStream_t s);

}  // namespace dcu
