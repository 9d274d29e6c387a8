// Attention of packed query rows over the paged K/V cache of their sequence:
// out[r][h] = sum_j w_j V_j, w = softmax_j(scale q . K_j) over the keys j of
// the row's sequence, read through its block table.  This file: few queries a
// sequence (one tile of 8), float32, and pages or scales that the tcgen05 kernel
// of k_paged_attn_tc.cu does not take; and the merge that both share (not launched
// where no item is cut).
//
// Work.  A query is a (row, query head) pair; an item is (sequence, kv head,
// tile of at most R queries), so a tile reads its keys once for the whole GQA
// group of its rows.  The keys of an item are cut into blocks of KB.  All
// blocks of all items, in item order, form one line of units that is cut into
// equal ranges, one per CTA (one CTA per SM): every SM reads the same number of
// keys whatever the lengths are, a long sequence is split over many SMs and
// short ones share an SM.  (Few items are cut one by one into equal parts: then
// no CTA changes items.)  Lengths and rows are only on the device, so each CTA
// derives the cut itself from the prefix sum of the sequences' unit counts.
//
// Inside a CTA the units go round-robin to its warps.  Each warp streams its
// own blocks through a private ring of shared memory and keeps its own running
// maximum, sum and O = P V, all fp32; nothing but the end of an item synchronises
// the warps.  Where a page holds whole blocks and the strides nest, a block comes
// as TMA tiles (its rows past the length are cleared, a bad page is not loaded);
// else key by key with 16-byte cp.async, zero-filled past the length and for bad
// pages.  Either way nothing outside the sequence gets into a product.
// The ring runs across item ends, so loads keep flowing while a finished item
// is merged.  Where a CTA's range cuts an item, its share (O, max, sum) goes to
// the workspace and k_paged_merge joins the shares in range order.
//
// bf16 blocks run on mma.sync m16n8k16 with the operands swapped (S^T = K Q^T,
// O^T += V^T P^T): the 16-wide M holds keys or head dims, the 8-wide N holds
// queries, so a single token with 7 or 8 heads in a group fills the tile.  P is
// split into a high and a low bf16 part, two products instead of one: the
// weights keep 16 bits at a cost that the memory-bound loop hides.  float32
// blocks run on the CUDA cores in fp32.
//
// What bounds it: reading the pages.  One row a sequence, 28/4 heads of 128:
// 64 ragged sequences (1.06 GB) 186 us, 5.7 TB/s; one of 131072 keys (268 MB)
// 52.2 us, 5.1 TB/s.  The rings hold 192 KB an SM, 28 MB on the GPU; loaded key by
// key with cp.async, 64 x 8192 keys took 289 us instead of 197.  Short calls are a
// chain of latencies (lengths, table, keys, blocks, joins): 33 float32 rows over
// 256 keys of 4 heads 9.7 us.  float32, one row over 32 x 8192 keys: 5.5 TB/s with
// 16/16 heads of 128, 5.1 with 28/4, 4.1 with head dim 256 (room for 4 warps only); a
// group of 16 heads has two tiles, which each read the keys (2.0 TB/s of them).  Over
// one sequence of 8192 keys 16/16 heads take 3.7 TB/s, and many rows compute 11 to 21
// TFLOP/s in tiles of 8 queries.
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace dcu {
namespace {

// One kernel variant: head dims up to DP (shorter ones zero-padded in shared memory).
template <int DP, bool F32, int NT>
struct Cfg {
  static constexpr int kKB = F32 ? 8 : 16;                       // keys of a block
  static constexpr int kW = DP == 256 ? 4 : F32 ? 12 : 8;  // warps
  static constexpr int kR = 8 * NT;                              // queries of a tile: NT groups of 8
  static constexpr int kEs = F32 ? 4 : 2;                        // element size
  static constexpr int kRow = DP * kEs;                          // bytes of a key row
  static constexpr int kStage = 2 * kKB * kRow;                  // K and V of a block
  static constexpr int kNst = DP == 256 ? 3 : F32 ? (DP == 64 ? 4 : 2) : (DP == 64 ? 5 : 3);  // ring stages of a warp
  static constexpr int kQPitch = kRow + 16;                      // padded query row
  static constexpr int kRing = kW * kNst * kStage;
  static constexpr int kQ = kR * kQPitch;
  static constexpr int kRed = (kW / 2) * DP * 8 * 4;             // merge buffer: half the warps, 8 queries
  static constexpr int kP = F32 ? kW * 64 * 4 : 0;               // float32: P of a block, per warp
  static constexpr int kSmem = kRing + kQ + kRed + kP + 1024;  // + alignment of the ring
  static constexpr int kThreads = 32 * kW;
  static_assert(kSmem + 2800 <= 227 * 1024, "dynamic and static shared memory of an SM");
  static constexpr int kND = F32 ? (DP > 128 ? DP / 128 : 1) : 0;  // float32: 4-dim chunks of O per lane and query
  static constexpr int kAcc = F32 ? 8 * kND : DP / 16;           // float4s of O per lane and query group
};

__device__ __forceinline__ uint32_t su32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cpa16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cpa_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cpa_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// transpose of an 8 x 8 tile of 16-bit values held one row pair per lane
__device__ __forceinline__ uint32_t movm(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// 2^x; results below 2^-126 become 0 (they round away in every sum here)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16-byte chunk c of key row r in a block's K or V: boxes of KB rows x 128
// bytes with the 128-byte swizzle (the layout that a TMA tile load writes).
template <int KB>
__device__ __forceinline__ uint32_t kv_off(int r, int c) {
  return (uint32_t)((c >> 3) * (KB * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// A block to be loaded: its page (TMA: one page; cp.async: the page of the
// lane's key), the slot offset of its first key, kv head and valid keys.
struct Req {
  int pg, blk, kvh, nk;
};

template <int DP, bool F32, int NT, bool TMA>
__global__ void __launch_bounds__(Cfg<DP, F32, NT>::kThreads, 1)
    k_paged_attn(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, int head_first, float *__restrict__ part_o, float2 *__restrict__ part_ml,
                 Share *__restrict__ shares) {
  using C = Cfg<DP, F32, NT>;
  constexpr int KB = C::kKB, W = C::kW, R = C::kR, NST = C::kNst;
  constexpr int CPR = C::kRow / 16;  // 16-byte chunks of a key row
  constexpr uint32_t FULL = (1u << KB) - 1u;
  pdl_enter();
  extern __shared__ uint8_t sm_raw[];
  __shared__ long long s_scan[2 * W];
  __shared__ Place s_place;
  __shared__ Range s_range;
  __shared__ uint32_t s_mask[W][NST];
  __shared__ float2 s_ml[W][R];
  __shared__ float2 s_fin[R];  // joined (max, sum) of a query
  __shared__ __align__(8) uint64_t s_bar[W][NST];
  __shared__ int s_abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int hd = a.pages.head_dim, KV = a.pages.n_kv_heads, G = a.n_heads / KV;
  if (TMA) fence_proxy_async_global();  // the pages may have been written by the kernel just waited for
  if (TMA && tid == 0) {
    for (int i = 0; i < W * NST; ++i) mbar_init(su32(&s_bar[0][0]) + 8u * i, 1);
    fence_barrier_init();
    s_abort = 0;
  }

  // ---- this CTA's range of the units and its first place
  // at least a block per warp; a change of items costs about four of each (measured with one and four: one row x 8192
  // keys x 32 heads 31.5 and 29.7 us, x 40 heads 36.6 and 35.1; nothing slower)
  find_range<R, KB, W>(a, &s_place, &s_range, s_scan, W, 4 * W);
  Place seg = s_place;  // start of the current segment (the part of an item inside the range)
  const Range rg = s_range;
  if (!rg.any) {
    if (tid == 0) shares[blockIdx.x].last = -1;
    return;
  }
  const long long u0 = rg.u0, u1 = rg.u1;

  uint8_t *sm = sm_raw + ((1024u - (su32(sm_raw) & 1023u)) & 1023u);
  const uint32_t sm32 = su32(sm);
  const uint32_t ring = sm32 + (uint32_t)(warp * NST * C::kStage);
  const uint32_t bars = su32(&s_bar[warp][0]);
  uint8_t *q_sm = sm + C::kRing;
  float *red = reinterpret_cast<float *>(sm + C::kRing + C::kQ);  // [W / 2][DP][8]
  [[maybe_unused]] float *p_sm = reinterpret_cast<float *>(sm + C::kRing + C::kQ + C::kRed) + warp * 64;

  // ---- the warp's loader: blocks u0 + warp, + W, ...
  Place ld = seg;
  advance<R, KB>(a, ld, warp);
  long long ld_u = u0 + warp;
  const unsigned psz = (unsigned)a.pages.page_size;
  // the next block of this warp: starts the look-up of its page(s), which `issue` uses later
  auto request = [&]() {
    Req r{-1, 0, 0, 0};
    if (ld_u < u1) {
      r.blk = ld.blk;
      r.kvh = ld.kvh;
      r.nk = ld.s.nk;
      const int key = ld.blk * KB + (TMA ? 0 : lane);
      if (key < r.nk && (TMA || lane < KB))
        r.pg = a.table[(size_t)ld.b * a.max_pages + div_page(a, (unsigned)key)];
      ld_u += W;
      if (ld_u < u1) advance<R, KB>(a, ld, W);
    }
    return r;
  };
  auto issue = [&](const Req &r, int st) {
    const uint32_t dst = ring + (uint32_t)(st * C::kStage);
    const int key0 = r.blk * KB;
    if constexpr (TMA) {
      const int nv = min(KB, r.nk - key0);  // <= 0: nothing to load
      const bool ok = nv > 0 && r.pg >= 0 && r.pg < a.pages.n_pages;
      if (lane == 0) {
        s_mask[warp][st] = ok ? FULL >> (KB - nv) : 0u;
        const uint32_t bar = bars + 8u * st;
        mbar_expect_tx(bar, ok ? (uint32_t)C::kStage : 0u);
        if (ok) {
          const int y = key0 - (int)(div_page(a, (unsigned)key0) * psz);
#pragma unroll
          for (int i = 0; i < CPR / 8; ++i) {
            const int x = i * (128 / C::kEs), c1 = head_first ? r.kvh : y, c2 = head_first ? y : r.kvh;
            tma_load_4d(dst + (uint32_t)(i * KB * 128), &kmap, x, c1, c2, r.pg, bar);
            tma_load_4d(dst + (uint32_t)(KB * C::kRow + i * KB * 128), &vmap, x, c1, c2, r.pg, bar);
          }
        } else if (nv > 0 && a.status) {
          atomicOr(a.status, DCU_ST_BAD_PAGE);
        }
      }
    } else {
      const int key = key0 + lane;
      const bool in = lane < KB && key < r.nk;
      const bool ok = in && r.pg >= 0 && r.pg < a.pages.n_pages;
      if (in && !ok && a.status) atomicOr(a.status, DCU_ST_BAD_PAGE);
      long long off = 0;
      if (ok)
        off = (long long)r.pg * a.pages.page_stride +
              (long long)((unsigned)key - div_page(a, (unsigned)key) * psz) * a.pages.slot_stride +
              (long long)r.kvh * a.pages.head_stride;
      const uint32_t mask = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) s_mask[warp][st] = mask;
      const char *kb = static_cast<const char *>(a.pages.k), *vb = static_cast<const char *>(a.pages.v);
#pragma unroll
      for (int i = 0; i < KB * CPR / 32; ++i) {
        const int rr = (i * 32 + lane) / CPR, c = (i * 32 + lane) % CPR;
        const long long o = __shfl_sync(0xffffffffu, off, rr);
        const bool v = ((mask >> rr) & 1u) && c * (16 / C::kEs) < hd;
        const long long byte = v ? o * C::kEs + c * 16 : 0;
        const uint32_t d = dst + kv_off<KB>(rr, c);
        cpa16(d, kb + byte, v);
        cpa16(d + (uint32_t)(KB * C::kRow), vb + byte, v);
      }
      cpa_commit();
    }
  };
  int left = (int)max(0ll, (u1 - u0 - warp + W - 1) / W);  // blocks of this warp not yet asked for
  Req nxt{};
  {
    Req first[NST - 1];
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) first[i] = request();
    nxt = request();
#pragma unroll
    for (int i = 0; i < NST - 1; ++i) {
      if (i < left) issue(first[i], i);
      else if (!TMA) cpa_commit();
    }
    left -= NST - 1;
  }
  int st_load = NST - 1, st_use = 0;
  uint32_t parity = 0;
  [[maybe_unused]] bool alive = true;
  [[maybe_unused]] int undone = 0;  // blocks issued but not waited for

  // ---- segments
  long long u = u0 + warp;  // the warp's next unit
  for (long long s0 = u0; s0 < u1;) {
    const Seq &sq = seg.s;
    const long long s1 = min(u1, s0 + (sq.nblk - seg.blk));
    const int q0 = seg.tile * sq.tq, nq = min(sq.tq, sq.nq - q0);
    const int ngrp = NT == 1 ? 1 : (nq + 7) >> 3;
    const Pairs pairs(sq, q0, G);
    // queries of the tile -> shared memory (zeros past nq and past head_dim)
    for (int i = tid; i < ngrp * 8 * CPR; i += C::kThreads) {
      const int r = i / CPR, c = i - r * CPR;
      const bool in = r < nq && c * (16 / C::kEs) < hd;
      const char *src = static_cast<const char *>(a.q) +
                        (pairs.at(in ? r : 0, seg.kvh, a.n_heads, hd) * C::kEs + (in ? c * 16 : 0));
      uint8_t *dst = q_sm + r * C::kQPitch + c * 16;
      if constexpr (TMA)
        load_query16(su32(dst), src, in);
      else  // (waiting for an asynchronous copy here would drain the ring's)
        *reinterpret_cast<uint4 *>(dst) = in ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
    }
    if constexpr (TMA) load_query_wait();
    __syncthreads();
    // B fragments of a single query group stay in registers: dims 32 kk + 8 i of the 8 queries
    [[maybe_unused]] uint32_t qf[F32 || NT > 1 ? 1 : DP / 32][4];
    if constexpr (!F32 && NT == 1) {
#pragma unroll
      for (int kk = 0; kk < DP / 32; ++kk)
        ldsm4(su32(q_sm) + (uint32_t)((lane & 7) * C::kQPitch + (4 * kk + (lane >> 3)) * 16), qf[kk]);
    }

    float m_run[NT][2], l_run[NT][2];
    float o[NT][C::kAcc][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m_run[n][0] = m_run[n][1] = -INFINITY;
      l_run[n][0] = l_run[n][1] = 0.f;
#pragma unroll
      for (auto &x : o[n]) x[0] = x[1] = x[2] = x[3] = 0.f;
    }

    for (; u < s1; u += W) {
      if constexpr (TMA) {
        if (alive) {
          alive = __all_sync(0xffffffffu, wait_bounded(bars + 8u * st_use, parity, &s_abort, a.status));
          if (!alive) undone = min(NST - 1, left + NST - 1);
        }
        if (!alive) continue;  // the wait gave up (DCU_ST_TIMEOUT): nothing more is loaded or read
      } else {
        cpa_wait<NST - 2>();
        __syncwarp();
      }
      if (left > 0) {  // the stage read in the last pass
        issue(nxt, st_load);
        nxt = request();
      } else if (!TMA) {
        cpa_commit();
      }
      --left;
      st_load = st_load + 1 == NST ? 0 : st_load + 1;
      const uint32_t kt = ring + (uint32_t)(st_use * C::kStage), vt = kt + (uint32_t)(KB * C::kRow);
      const uint32_t mask = s_mask[warp][st_use];
      if (++st_use == NST) {
        st_use = 0;
        parity ^= 1u;
      }
      if (mask == 0u) {
        __syncwarp();
        continue;
      }
      if (TMA && mask != FULL) {
        // past the sequence's end the page holds anything: P is 0 there, V must be
        const int nv = __popc(mask);
        for (int i = lane; i < (KB - nv) * CPR; i += 32)
          *reinterpret_cast<uint4 *>(sm + (vt - sm32) + kv_off<KB>(nv + i / CPR, i % CPR)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // before the stage's next TMA load
        __syncwarp();
      }
      if constexpr (!F32) {
        float s[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
        // S^T[key][query]: A = K (16 keys x 16 dims), B = Q^T
        [[maybe_unused]] float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kk = 0; kk < DP / 32; ++kk) {
          uint32_t ka[2][4];
#pragma unroll
          for (int h2 = 0; h2 < 2; ++h2)
            ldsm4(kt + kv_off<KB>((lane & 7) + ((lane >> 3) & 1) * 8, 4 * kk + 2 * h2 + (lane >> 4)), ka[h2]);
          if constexpr (NT == 1) {  // two chains of products
            mma16816(s[0], ka[0], qf[kk][0], qf[kk][1]);
            mma16816(s2, ka[1], qf[kk][2], qf[kk][3]);
          } else {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (n < ngrp) {
                uint32_t qa[4];
                ldsm4(su32(q_sm) + (uint32_t)((n * 8 + (lane & 7)) * C::kQPitch + (4 * kk + (lane >> 3)) * 16), qa);
                mma16816(s[n], ka[0], qa[0], qa[1]);
                mma16816(s[n], ka[1], qa[2], qa[3]);
              }
            }
          }
        }
        if constexpr (NT == 1) {
#pragma unroll
          for (int e = 0; e < 4; ++e) s[0][e] += s2[e];
        }
        uint32_t ph[NT][2], pl[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n < ngrp) {
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = s[n][e] * a.scale_log2;
            if (mask != FULL) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (!((mask >> (g + (e >> 1) * 8)) & 1u)) x[e] = -INFINITY;
            }
            float mx[2] = {fmaxf(x[0], x[2]), fmaxf(x[1], x[3])};
#pragma unroll
            for (int of = 4; of < 32; of <<= 1) {
              mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], of));
              mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], of));
            }
            // The maximum moves only when a block exceeds it by more than 8 (log2 units), so P stays below 2^8 and
            // most blocks rescale nothing; O, the sum and P share it, so the result is the same.
            const bool grow = mx[0] > m_run[n][0] + 8.f || mx[1] > m_run[n][1] + 8.f;
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float m2 = fmaxf(m_run[n][c], mx[c]);
                const float f = m_run[n][c] == -INFINITY ? 0.f : ex2(m_run[n][c] - m2);
                m_run[n][c] = m2;
                l_run[n][c] *= f;
#pragma unroll
                for (int i = 0; i < DP / 16; ++i) {
                  o[n][i][c] *= f;
                  o[n][i][c + 2] *= f;
                }
              }
            }
            float p[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float m = m_run[n][e & 1];
              p[e] = ex2(x[e] - (m == -INFINITY ? 0.f : m));
              lo[e] = p[e] - __bfloat162float(__float2bfloat16_rn(p[e]));
            }
            l_run[n][0] += p[0] + p[2];
            l_run[n][1] += p[1] + p[3];
            ph[n][0] = movm(pack2(p[0], p[1]));
            ph[n][1] = movm(pack2(p[2], p[3]));
            pl[n][0] = movm(pack2(lo[0], lo[1]));
            pl[n][1] = movm(pack2(lo[2], lo[3]));
          }
        }
        // O^T[dim][query] += V^T P^T: A = V^T (16 dims x 16 keys)
#pragma unroll
        for (int i = 0; i < DP / 16; ++i) {
          uint32_t va[4];
          ldsm4t(vt + kv_off<KB>((lane & 7) + (lane >> 4) * 8, 2 * i + ((lane >> 3) & 1)), va);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (n < ngrp) {
              mma16816(o[n][i], va, ph[n][0], ph[n][1]);
              mma16816(o[n][i], va, pl[n][0], pl[n][1]);
            }
          }
        }
      } else {
        // lane = (keys 2 (lane / 8) and + 1, every 8th 16-byte chunk of the row), all 8 queries: a query chunk read from
        // shared memory serves two keys (reading the queries again for every key would bound the loop), and the 8 lanes
        // of a key read 8 bank groups
        const uint8_t *kr = sm + (kt - sm32);
        const int t8 = lane & 7, ka = (lane >> 3) * 2;
        float s[2][8];
#pragma unroll
        for (int r = 0; r < 8; ++r) s[0][r] = s[1][r] = 0.f;
#pragma unroll 2
        for (int i = 0; i < CPR / 8; ++i) {
          const int c = 8 * i + t8;
          const float4 k0 = *reinterpret_cast<const float4 *>(kr + kv_off<KB>(ka, c));
          const float4 k1 = *reinterpret_cast<const float4 *>(kr + kv_off<KB>(ka + 1, c));
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float4 qv = *reinterpret_cast<const float4 *>(q_sm + r * C::kQPitch + c * 16);
            s[0][r] = fmaf(qv.x, k0.x, fmaf(qv.y, k0.y, fmaf(qv.z, k0.z, fmaf(qv.w, k0.w, s[0][r]))));
            s[1][r] = fmaf(qv.x, k1.x, fmaf(qv.y, k1.y, fmaf(qv.z, k1.z, fmaf(qv.w, k1.w, s[1][r]))));
          }
        }
        // sums over the 8 lanes, each step keeping half of the values: bit 2 of the lane takes its key, bits 1 and 0 the
        // queries, which ends with key g = lane / 4 and queries 2 t, 2 t + 1
        float x[2];
        {
          float h4[8], h2[4];
          const bool b2 = lane & 4, b1 = lane & 2, b0 = lane & 1;
#pragma unroll
          for (int r = 0; r < 8; ++r)
            h4[r] = (b2 ? s[1][r] : s[0][r]) + __shfl_xor_sync(0xffffffffu, b2 ? s[0][r] : s[1][r], 4);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            h2[r] = (b1 ? h4[4 + r] : h4[r]) + __shfl_xor_sync(0xffffffffu, b1 ? h4[r] : h4[4 + r], 2);
          const bool v = (mask >> g) & 1u;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float sv = (b0 ? h2[2 + c] : h2[c]) + __shfl_xor_sync(0xffffffffu, b0 ? h2[c] : h2[2 + c], 1);
            x[c] = v ? sv * a.scale_log2 : -INFINITY;
          }
        }
        float mx[2] = {x[0], x[1]};
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], of));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], of));
        }
        const bool grow = mx[0] > m_run[0][0] + 8.f || mx[1] > m_run[0][1] + 8.f;
        if (__any_sync(0xffffffffu, grow)) {
          float f[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float m2 = fmaxf(m_run[0][c], mx[c]);
            f[c] = m_run[0][c] == -INFINITY ? 0.f : exp2f(m_run[0][c] - m2);
            m_run[0][c] = m2;
            l_run[0][c] *= f[c];
          }
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float fr = __shfl_sync(0xffffffffu, f[r & 1], r >> 1);
#pragma unroll
            for (int i = 0; i < C::kND; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[0][r * C::kND + i][e] *= fr;
          }
        }
        float p[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          p[c] = exp2f(x[c] - (m_run[0][c] == -INFINITY ? 0.f : m_run[0][c]));
          l_run[0][c] += p[c];
        }
        __syncwarp();
        *reinterpret_cast<float2 *>(p_sm + g * 8 + 2 * t) = make_float2(p[0], p[1]);
        __syncwarp();
        // O: the lane's chunk(s) of the head dim; DP == 64: half a warp takes every other key
        constexpr int ND = C::kND, KS = DP == 64 ? 2 : 1;
        const uint8_t *vr = sm + (vt - sm32);
#pragma unroll
        for (int k2 = 0; k2 < KB / KS; ++k2) {
          const int key = KS == 2 ? 2 * k2 + (lane >> 4) : k2;
          const float4 pa = *reinterpret_cast<const float4 *>(p_sm + key * 8);
          const float4 pb = *reinterpret_cast<const float4 *>(p_sm + key * 8 + 4);
          const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
          for (int i = 0; i < ND; ++i) {
            const int c = (KS == 2 ? (lane & 15) : lane) + 32 * i;
            const float4 vv = *reinterpret_cast<const float4 *>(vr + kv_off<KB>(key, c));
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              float(&od)[4] = o[0][r * ND + i];
              od[0] = fmaf(pr[r], vv.x, od[0]);
              od[1] = fmaf(pr[r], vv.y, od[1]);
              od[2] = fmaf(pr[r], vv.z, od[2]);
              od[3] = fmaf(pr[r], vv.w, od[3]);
            }
          }
        }
      }
      __syncwarp();  // all lanes are done with the stage
    }

    // ---- the segment's end: join the warps
    const bool starts = seg.blk == 0, ends = s1 - s0 == sq.nblk - seg.blk;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float l = l_run[n][c];
#pragma unroll
        for (int of = 4; of < 32; of <<= 1) l += __shfl_xor_sync(0xffffffffu, l, of);
        l_run[n][c] = l;
        if (g == 0) s_ml[warp][n * 8 + 2 * t + c] = make_float2(m_run[n][c], l);
      }
    __syncthreads();
    if (tid < ngrp * 8) {
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w2 = 0; w2 < W; ++w2) M = fmaxf(M, s_ml[w2][tid].x);
#pragma unroll
      for (int w2 = 0; w2 < W; ++w2) {
        const float2 ml = s_ml[w2][tid];
        L += ml.x == -INFINITY ? ml.y : ml.y * exp2f(ml.x - M);  // (a sum without a maximum: 0, or NaN)
      }
      s_fin[tid] = make_float2(M, L);
    }
    const int slot = s0 == u0 ? 0 : 1;  // the range's first segment, or its last one
    const size_t share = (size_t)blockIdx.x * 2 + slot;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n < ngrp) {
        // factor of this warp's share of queries 8 n + 2 t, + 1
        float f[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float M = -INFINITY;
#pragma unroll
          for (int w2 = 0; w2 < W; ++w2) M = fmaxf(M, s_ml[w2][n * 8 + 2 * t + c].x);
          f[c] = m_run[n][c] == -INFINITY ? 0.f : exp2f(m_run[n][c] - M);
        }
        if constexpr (!F32) {
#pragma unroll
          for (int i = 0; i < DP / 16; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][i][e] *= f[e & 1];
        } else {
          constexpr int ND = C::kND;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const float fr = __shfl_sync(0xffffffffu, f[r & 1], r >> 1);
#pragma unroll
            for (int i = 0; i < ND; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float x = o[0][r * ND + i][e] * fr;
                if (DP == 64) x += __shfl_xor_sync(0xffffffffu, x, 16);
                o[0][r * ND + i][e] = x;
              }
          }
        }
        // the upper half of the warps hands its shares to the lower half, whose W / 2 sums stay in the buffer
#pragma unroll
        for (int half = 1; half >= 0; --half) {
          if ((warp >= W / 2) == (half == 1)) {
            float *bw = red + (size_t)(warp % (W / 2)) * DP * 8;  // [dim][8 queries], float32: [8 queries][dim]
            if constexpr (!F32) {
#pragma unroll
              for (int i = 0; i < DP / 16; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float2 *d = reinterpret_cast<float2 *>(bw + (i * 16 + g + 8 * e) * 8 + 2 * t);
                  float2 v = make_float2(o[n][i][2 * e], o[n][i][2 * e + 1]);
                  if (half == 0) {
                    const float2 w2 = *d;
                    v.x += w2.x;
                    v.y += w2.y;
                  }
                  *d = v;
                }
            } else {
              constexpr int ND = C::kND;
              if (DP != 64 || lane < 16) {
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                  if (r >= nq) break;
#pragma unroll
                  for (int i = 0; i < ND; ++i) {
                    float4 *d = reinterpret_cast<float4 *>(bw + r * DP + (lane + 32 * i) * 4);
                    const float(&x)[4] = o[0][r * ND + i];
                    float4 v = make_float4(x[0], x[1], x[2], x[3]);
                    if (half == 0) {
                      const float4 w2 = *d;
                      v.x += w2.x;
                      v.y += w2.y;
                      v.z += w2.z;
                      v.w += w2.w;
                    }
                    *d = v;
                  }
                }
              }
            }
          }
          __syncthreads();
        }
        // sum of the W / 2 buffers: whole items are normalised and stored, cut ones go to the workspace
        for (int i = tid; i < DP * 8 / 2; i += C::kThreads) {
          const int qr = F32 ? i / (DP / 2) : i & 7, d = (F32 ? i % (DP / 2) : i >> 3) * 2;
          if (n * 8 + qr >= nq || d >= hd) continue;
          float x0 = 0.f, x1 = 0.f;
#pragma unroll
          for (int w2 = 0; w2 < W / 2; ++w2) {
            const float *x = red + (size_t)w2 * DP * 8 + (F32 ? qr * DP + d : d * 8 + qr);
            x0 += x[0];
            x1 += x[F32 ? 1 : 8];
          }
          const float M = s_fin[n * 8 + qr].x, L = s_fin[n * 8 + qr].y;
          if (starts && ends) {
            const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
            const size_t at = pairs.at(n * 8 + qr, seg.kvh, a.n_heads, hd) + d;
            if constexpr (F32)
              *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(x0 * inv, x1 * inv);
            else
              *reinterpret_cast<uint32_t *>(static_cast<bf16 *>(a.out) + at) = pack2(x0 * inv, x1 * inv);
          } else {
            *reinterpret_cast<float2 *>(part_o + share_at(share, R, DP, n * 8 + qr, d)) = make_float2(x0, x1);
            if (d == 0) part_ml[share * R + n * 8 + qr] = make_float2(M, L);
          }
        }
        if (n + 1 < NT) __syncthreads();
      }
    }
    if (s1 == u1 && tid == 0) {
      Share sh;
      sh.last = -1;
      if (starts && !ends) {
        sh.last = rg.of(s0 + sq.nblk - 1);
        sh.row0 = sq.row0;
        sh.q0 = q0;
        sh.nq = nq;
        sh.kvh = seg.kvh;
        sh.slot = slot;
      }
      shares[blockIdx.x] = sh;
    }
    advance<R, KB>(a, seg, (int)(s1 - s0));
    s0 = s1;
    __syncthreads();  // the next segment reuses the query tile, the sums and the buffer
  }
  if constexpr (TMA) {
    for (int i = 0; i < undone; ++i) {  // after a timeout: no copy may land once the CTA has left
      wait_drain(bars + 8u * st_use, parity);
      if (++st_use == NST) {
        st_use = 0;
        parity ^= 1u;
      }
    }
  } else {
    cpa_wait<0>();
  }
}

// Joins the shares of the items that range boundaries cut: for a query,
// out = sum_i w_i O_i, w_i = 2^(m_i - M) / sum_j 2^(m_j - M) l_j, over its
// shares i.  An item that begins in range r has its first share there (slot 1,
// or 0 when it is that range's only segment) and the others in slot 0 of the
// following ranges.  A piece of work is 8 neighbouring queries x a quarter of
// the head dim; lane = (query, group of 4 dims), so a warp's loads are whole
// 128-byte lines of a share.  The pieces of all items form one line, dealt out
// to the warps of the launch; when there are fewer than CTAs (a single token
// over a long cache: few queries, many shares), a CTA takes a piece and its
// warps split the shares.  Every sum has a fixed order.
constexpr int kMergeThreads = 256;

template <int DP, class T>
__global__ void __launch_bounds__(kMergeThreads)
    k_paged_merge(const __grid_constant__ PagedAttnArgs a, int R, int ranges, const float *__restrict__ part_o,
                  const float2 *__restrict__ part_ml, const Share *__restrict__ shares) {
  constexpr int W = kMergeThreads / 32, NI = DP / 64;  // groups of 4 dims per lane
  constexpr int kBatch = 8 / NI;                       // shares whose loads are in flight together
  pdl_enter();
  __shared__ int s_end[kMaxRanges];
  __shared__ Share s_share[kMaxRanges];
  __shared__ int s_red[32];
  __shared__ float4 s_part[W][NI][32];
  __shared__ float2 s_pml[W][8];
  static_assert(kMaxRanges <= kMergeThreads, "one thread per range");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int mine = 0;
  if (tid < ranges) {
    const Share sh = shares[tid];
    s_share[tid] = sh;
    if (sh.last >= 0) mine = 4 * ((sh.nq + 7) / 8);
  }
  int total;
  const int pre = block_exclusive_scan(mine, s_red, &total);
  if (tid < ranges) s_end[tid] = pre + mine;
  __syncthreads();
  const int G = a.n_heads / a.pages.n_kv_heads, hd = a.pages.head_dim;
  const bool whole = total <= (int)gridDim.x;  // a CTA per piece
  const int step = whole ? gridDim.x : gridDim.x * W;
  for (int i = whole ? blockIdx.x : blockIdx.x * W + warp; i < total; i += step) {
    int r = 0, z = ranges - 1;  // the first range whose end is above i
    while (r < z) {
      const int m = (r + z) >> 1;
      if (s_end[m] > i) z = m;
      else r = m + 1;
    }
    const Share sh = s_share[r];
    const int piece = i - (s_end[r] - 4 * ((sh.nq + 7) / 8));
    const int qr = (piece >> 2) * 8 + (lane & 7);
    const int d0 = (piece & 3) * (DP / 4) + (lane >> 3) * 4;  // the lane's dims: d0 + 16 n .. + 3
    const bool in = qr < sh.nq;
    float M = -INFINITY, L = 0.f, acc[NI][4];
#pragma unroll
    for (int n = 0; n < NI; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    const int di = whole ? W : 1;
    for (int j0 = whole ? r + warp : r; j0 <= sh.last; j0 += kBatch * di) {
      float2 ml[kBatch];
      float4 v[kBatch][NI];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int j = j0 + k * di;
        const size_t share = (size_t)j * 2 + (j == r ? sh.slot : 0);
        ml[k] = make_float2(-INFINITY, 0.f);
        if (j <= sh.last && in) {
          ml[k] = part_ml[share * R + qr];
#pragma unroll
          for (int n = 0; n < NI; ++n)
            v[k][n] = *reinterpret_cast<const float4 *>(part_o + share_at(share, R, DP, qr, d0 + 16 * n));
        }
      }
      float m2 = M;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) m2 = fmaxf(m2, ml[k].x);
      const float f = M == -INFINITY ? 0.f : exp2f(M - m2);
      M = m2;
      L *= f;
#pragma unroll
      for (int n = 0; n < NI; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[n][e] *= f;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (j0 + k * di > sh.last || !in) break;
        const float w = ml[k].x == -INFINITY ? 0.f : exp2f(ml[k].x - M);
        L += ml[k].x == -INFINITY ? 0.f : w * ml[k].y;
#pragma unroll
        for (int n = 0; n < NI; ++n) {
          acc[n][0] += w * v[k][n].x;
          acc[n][1] += w * v[k][n].y;
          acc[n][2] += w * v[k][n].z;
          acc[n][3] += w * v[k][n].w;
        }
      }
    }
    if (whole) {  // join the warps, in order
#pragma unroll
      for (int n = 0; n < NI; ++n) s_part[warp][n][lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
      if (lane < 8) s_pml[warp][lane] = make_float2(M, L);
      __syncthreads();
      if (warp == 0) {
        M = -INFINITY;
#pragma unroll
        for (int k = 0; k < W; ++k) M = fmaxf(M, s_pml[k][lane & 7].x);
        L = 0.f;
#pragma unroll
        for (int n = 0; n < NI; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) {
          const float2 ml = s_pml[k][lane & 7];
          const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
          L += ml.x == -INFINITY ? 0.f : w * ml.y;
#pragma unroll
          for (int n = 0; n < NI; ++n) {
            const float4 x = s_part[k][n][lane];
            acc[n][0] += w * x.x;
            acc[n][1] += w * x.y;
            acc[n][2] += w * x.z;
            acc[n][3] += w * x.w;
          }
        }
      }
      __syncthreads();
      if (warp != 0) continue;
    }
    if (!in) continue;
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
    const int pq = sh.q0 + qr, row = sh.row0 + pq / G, h = sh.kvh * G + pq % G;
    T *dst = static_cast<T *>(a.out) + ((size_t)row * a.n_heads + h) * hd + d0;
#pragma unroll
    for (int n = 0; n < NI; ++n) {
      if (d0 + 16 * n >= hd) continue;
      if constexpr (sizeof(T) == 2)
        *reinterpret_cast<uint2 *>(dst + 16 * n) =
            make_uint2(pack2(acc[n][0] * inv, acc[n][1] * inv), pack2(acc[n][2] * inv, acc[n][3] * inv));
      else
        *reinterpret_cast<float4 *>(dst + 16 * n) =
            make_float4(acc[n][0] * inv, acc[n][1] * inv, acc[n][2] * inv, acc[n][3] * inv);
    }
  }
}

template <int DP, bool F32, int NT, bool TMA>
cudaError_t launch_variant(const PagedAttnArgs &a, const PageMaps &m, void *ws, cudaStream_t s) {
  using C = Cfg<DP, F32, NT>;
  static std::atomic<uint64_t> attr{0};
  if (cudaError_t e = ensure_smem_limit(k_paged_attn<DP, F32, NT, TMA>, C::kSmem, attr)) return e;
  int grid = 0;
  if (cudaError_t e = paged_grid(&grid)) return e;
  const ShareBuf sb(ws, C::kR, DP);
  PagedAttnArgs b = a;
  b.whole = whole_items(a, C::kR, C::kKB, 4 * C::kW, grid);
  if (cudaError_t e = launch_pdl(k_paged_attn<DP, F32, NT, TMA>, dim3(grid), dim3(C::kThreads), C::kSmem, s, b, m.k,
                                 m.v, m.head_first, sb.o, sb.ml, sb.desc))
    return e;
  return b.whole ? cudaSuccess : launch_paged_merge(a, C::kR, grid, sb, s);
}

template <int DP, bool F32, int NT>
cudaError_t launch(const PagedAttnArgs &a, void *ws, cudaStream_t s) {
  PageMaps m = {};
  if (page_maps(a.pages, Cfg<DP, F32, NT>::kKB, &m)) return launch_variant<DP, F32, NT, true>(a, m, ws, s);
  return launch_variant<DP, F32, NT, false>(a, m, ws, s);
}

}  // namespace

// Tensor maps (head dim, then slot and head by stride, page) with boxes of 128
// bytes x kb slots.  false, and the kernel loads key by key with cp.async,
// where a block of kb keys could cross a page or the strides do not nest (each
// a multiple of the one below and past its extent, as a tensor map wants).
bool page_maps(const dcu_pages &p, int kb, PageMaps *m) {
  if (p.page_size % kb) return false;
  const bool f32 = p.dtype == DCU_F32;
  const uint64_t es = f32 ? 4 : 2, row = (uint64_t)p.head_dim * es;
  uint64_t slot = (uint64_t)p.slot_stride * es, head = (uint64_t)p.head_stride * es;
  if (p.n_kv_heads == 1) head = slot;  // the stride of a single head does not matter
  const bool hf = head <= slot;
  const uint64_t s0 = hf ? head : slot, s1 = hf ? slot : head;
  const uint64_t n0 = hf ? (uint64_t)p.n_kv_heads : (uint64_t)p.page_size;
  const uint64_t n1 = hf ? (uint64_t)p.page_size : (uint64_t)p.n_kv_heads;
  const uint64_t s2 = p.n_pages == 1 ? s1 * n1 : (uint64_t)p.page_stride * es;
  if (s0 < row || s1 < s0 * n0 || s1 % s0 || s2 < s1 * n1 || s2 % s1 || s2 >= (1ull << 40)) return false;
  const uint64_t dims[4] = {(uint64_t)p.head_dim, n0, n1, (uint64_t)p.n_pages};
  const uint64_t st[3] = {s0, s1, s2};
  const uint32_t box[4] = {(uint32_t)(128 / es), hf ? 1u : (uint32_t)kb, hf ? (uint32_t)kb : 1u, 1u};
  m->box = kb;
  m->head_first = hf;
  return encode_tmap_4d(&m->k, f32, p.k, dims, st, box) && encode_tmap_4d(&m->v, f32, p.v, dims, st, box);
}

cudaError_t paged_grid(int *grid) {
  int dev = 0, sms = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) return e;
  *grid = sms < kMaxRanges ? sms : kMaxRanges;
  return cudaSuccess;
}

cudaError_t launch_paged_merge(const PagedAttnArgs &a, int kr, int grid, const ShareBuf &sb, cudaStream_t s) {
  const int hd = a.pages.head_dim;
  // two CTAs per SM
  auto go = [&](auto kern) {
    return launch_pdl(kern, dim3(2 * grid), dim3(kMergeThreads), 0, s, a, kr, grid, sb.o, sb.ml, sb.desc);
  };
  if (a.pages.dtype == DCU_F32)
    return hd <= 64 ? go(k_paged_merge<64, float>) : hd <= 128 ? go(k_paged_merge<128, float>)
                                                               : go(k_paged_merge<256, float>);
  return hd <= 64 ? go(k_paged_merge<64, bf16>) : hd <= 128 ? go(k_paged_merge<128, bf16>)
                                                            : go(k_paged_merge<256, bf16>);
}

int64_t paged_attention_workspace(const dcu_pages &p) {
  const int dp = p.head_dim <= 64 ? 64 : p.head_dim <= 128 ? 128 : 256;
  if (p.dtype == DCU_F32) return ShareBuf::bytes(8, dp);
  return ShareBuf::bytes(kTcQueries, dp);
}

cudaError_t launch_paged_attention(const PagedAttnArgs &a, void *ws, cudaStream_t s) {
  const int hd = a.pages.head_dim;
  if (a.pages.dtype == DCU_F32)
    return hd <= 64 ? launch<64, true, 1>(a, ws, s)
                    : hd <= 128 ? launch<128, true, 1>(a, ws, s) : launch<256, true, 1>(a, ws, s);
  // Queries per sequence and kv head, on average (max_rows bounds the rows).  Up to 8 fill one mma.sync group; above,
  // the tcgen05 kernel where it applies.  Measured, this kernel / that one, us a call: 1 x 1024 keys, 32 heads x 128:
  // 1 query 10.9 / 13.3, 9 queries 12.7 / 13.5; 1 x 8192 keys: 8 queries 30.0 / 34.2, 12 queries 44.4 / 34.5; 64 x
  // 2000 keys, 28/4 heads: 7 queries 53 / 58, 14 queries 91 / 59; 128 x 100 keys, 8 heads x 64: 8 queries 30.5 / 37.9,
  // 12 queries 50.5 / 38.4.  These are of equal rows a sequence.  The rule sees a mean only, and one kernel takes all: 64
  // tokens over 200 to 2000 keys and a prompt of 400 rows, 32 heads x 128, take 400 us together, 261 and 21 apart.
  if ((long long)a.max_rows * (a.n_heads / a.pages.n_kv_heads) <= 8ll * a.B)
    return hd <= 64 ? launch<64, false, 1>(a, ws, s)
                    : hd <= 128 ? launch<128, false, 1>(a, ws, s) : launch<256, false, 1>(a, ws, s);
  PageMaps m = {};
  if (a.scale_log2 > 0.f && a.pages.page_size % 8 == 0 && page_maps(a.pages, tc_box_keys(a.pages), &m))
    return launch_paged_attention_tc(a, m, ws, s);
  return hd <= 64 ? launch_variant<64, false, 4, false>(a, m, ws, s)
                  : hd <= 128 ? launch_variant<128, false, 4, false>(a, m, ws, s)
                              : launch_variant<256, false, 2, false>(a, m, ws, s);
}

}  // namespace dcu
