// Paged attention of many query rows per sequence on the 5th-gen tensor cores
// (bf16, head_dim up to 128).  Same line of work, shares and merge as
// k_paged_attn.cu, with items of up to 256 queries (two MMA tiles of 128, one
// TMEM lane per query) and units of 128 keys:
//
//   warp 0     TMA producer: the pages of a chunk of 128 keys, boxes of
//              box_keys slots x 64 dims (128-byte swizzle), K and V rings of
//              two stages; a box past the sequence's end or on a bad page is
//              read at a page coordinate outside the tensor, i.e. as zeros
//   warps 1, 2 MMA issuers of tile A and of tile B (one thread each): S_t =
//              Q_t K^T (M = 128 queries, N = 128 keys) and O_t += P_t V (P_t in
//              tensor memory, V MN-major)
//   warps 4-11 and 12-19  softmax of tile A and of tile B: thread = (query, half
//              of the sub-chunk's keys)
//
// A chunk is worked in two sub-chunks of 64 keys, each with a TMEM score buffer
// of its own per tile, so S of the next sub-chunk is there when the softmax
// gets to it and only the softmax is on the critical path; the two tiles share
// every K and V stage.  An item of at most 128 queries gives both tiles the
// same queries and every other chunk, each with its own maximum, sum and O, and
// the two are joined at its end.
// TMEM: two score buffers of 64 columns for A, two for B, O_A and O_B of 128
// columns; P (bf16 pairs) overwrites scores that the same thread has read.
// P is rounded to bf16 once, as in the dense attention of a step: a second
// product for the low part would cost half as much again on the pipe that
// bounds this kernel.
//
// Every mbarrier wait is bounded; on expiry the CTA sets DCU_ST_TIMEOUT, drains
// its copies and MMAs in flight, frees TMEM and exits.
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace dcu {
namespace {

constexpr int kKC = 128;              // keys of a unit
constexpr int kSub = 64;              // keys of a sub-chunk
constexpr int kStages = 2;            // K and V ring depth
constexpr int kSoftWarps = 8;         // per tile
constexpr int kSoft0 = 4;             // first softmax warp
constexpr int kWarps = kSoft0 + 2 * kSoftWarps;
constexpr int kThreads = 32 * kWarps;

template <int DP>
struct TcCfg {
  static constexpr uint32_t kTile = 128u * DP * 2u;  // a Q tile, or K or V of a chunk: DP / 64 blocks of 16 KB
  static constexpr uint32_t kSmem = (2 + 2 * kStages) * kTile + 1024u;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kO = 256;                // O_t at column 256 + 128 t
};

__device__ __forceinline__ uint32_t tile_off(int r, int c) {  // 16-byte chunk c of row r
  return (uint32_t)(c >> 3) * 16384u + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
__device__ __forceinline__ float ex2a(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t packb(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

// true in one lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attn_tc(const __grid_constant__ PagedAttnArgs a, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, int head_first, int box, float *__restrict__ part_o,
                    float2 *__restrict__ part_ml, Share *__restrict__ shares) {
  using C = TcCfg<DP>;
  constexpr int R = kTcQueries, OC = DP / 2;  // O columns of a half
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t bars[4 * kStages + 16];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ long long s_scan[kWarps];
  __shared__ Place s_place;
  __shared__ float s_mx[2][2][2][128];  // [sub-chunk parity][tile][half] maximum of the half's keys
  __shared__ float s_l[2][2][128];      // [tile][half] share of the row sum
  __shared__ float s_m[2][128];         // [tile] final row maximum
  __shared__ uint32_t s_bad[4];         // [chunk % 4] boxes of the chunk on bad pages
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = (smem_u32(sm_raw) + 1023u) & ~1023u;
  uint8_t *sm = sm_raw + (sbase - smem_u32(sm_raw));
  const uint32_t q_s = sbase, k_s = sbase + 2 * C::kTile, v_s = k_s + kStages * C::kTile;
  const uint32_t bar0 = smem_u32(bars);
  auto K_FULL = [&](uint32_t s) { return bar0 + 8u * s; };
  auto K_EMPTY = [&](uint32_t s) { return bar0 + 8u * (kStages + s); };
  auto V_FULL = [&](uint32_t s) { return bar0 + 8u * (2 * kStages + s); };
  auto V_EMPTY = [&](uint32_t s) { return bar0 + 8u * (3 * kStages + s); };
  auto S_FULL = [&](int t, uint32_t b) { return bar0 + 8u * (4 * kStages + 2 * t + b); };
  auto P_FULL = [&](int t, uint32_t b) { return bar0 + 8u * (4 * kStages + 4 + 2 * t + b); };
  auto PV_DONE = [&](int t) { return bar0 + 8u * (4 * kStages + 8 + t); };
  auto DRAIN = [&](int t) { return bar0 + 8u * (4 * kStages + 10 + t); };
  const uint32_t Q_FULL = bar0 + 8u * (4 * kStages + 12), O_FINAL = Q_FULL + 8u;
  // tile A's softmax warps, per segment of two tiles whose last chunk ends inside a page: V's rows there are cleared.
  // (Tile B may be a chunk ahead or behind, so P_FULL of tile A would not do: a parity wait is only sound within one
  // phase.)
  const uint32_t V_CLEAR = Q_FULL + 16u, A_BEGUN = Q_FULL + 24u;  // A_BEGUN: tile A has its first scores of a segment

  if (tid == 0) {
    // a stage is empty, and a segment final, once both tiles say so (a tile that has the chunk to itself, twice)
    for (uint32_t s = 0; s < kStages; ++s) {
      mbar_init(K_FULL(s), 1);
      mbar_init(K_EMPTY(s), 2);
      mbar_init(V_FULL(s), 1);
      mbar_init(V_EMPTY(s), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(DRAIN(t), 1);
      for (uint32_t b = 0; b < 2; ++b) {
        mbar_init(S_FULL(t, b), 2);  // the scores (commit), and the issuer itself (it has seen the chunk's K_FULL)
        mbar_init(P_FULL(t, b), kSoftWarps);
      }
      mbar_init(PV_DONE(t), 1);
    }
    mbar_init(Q_FULL, 2 * kSoftWarps);
    mbar_init(O_FINAL, 2);
    mbar_init(V_CLEAR, kSoftWarps);
    mbar_init(A_BEGUN, kSoftWarps);
    abort_flag = 0;
    fence_barrier_init();
    prefetch_tmap(&kmap);
    prefetch_tmap(&vmap);
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  pdl_enter();
  fence_proxy_async_global();  // the pages may have been written by the kernel just waited for
  tc_fence_before();
  Place seg;
  const Range rg = find_range<R, kKC, kWarps>(a, seg, &s_place, s_scan, 1);  // (a barrier inside)
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int *abort_v = &abort_flag;
  const int KV = a.pages.n_kv_heads, G = a.n_heads / KV, hd = a.pages.head_dim;

  if (!rg.any) {
    if (tid == 0) shares[blockIdx.x].last = -1;
  } else if (warp == 0) {
    // ---- TMA producer
    Place &ld = seg;
    const int nb = kKC / box;                     // boxes of a chunk (of each 64-dim half)
    const int my = lane % nb, half = lane / nb;   // the lane's box: lanes 0 .. nb * DP / 64 - 1 issue
    const bool mine = half < DP / 64;
    auto look = [&]() {
      const int key = ld.blk * kKC + my * box;
      return mine && key < ld.s.nk ? a.table[(size_t)ld.b * a.max_pages + div_page(a, (unsigned)key)] : -1;
    };
    int pg = look();
    uint32_t issued = 0;
    bool ok = true;
    for (long long u = rg.u0; u < rg.u1 && ok; ++u) {
      const uint32_t st = issued % kStages, ph = ((issued / kStages) & 1u) ^ 1u;
      const int key = ld.blk * kKC + my * box, kvh = ld.kvh;
      const bool in = mine && key < ld.s.nk, good = in && pg >= 0 && pg < a.pages.n_pages;
      if (in && !good && half == 0 && a.status) atomicOr(a.status, DCU_ST_BAD_PAGE);
      const uint32_t bad = __ballot_sync(0xffffffffu, in && !good) & ((1u << nb) - 1u);  // lanes of half 0
      const int w = good ? pg : a.pages.n_pages;  // outside the tensor: zeros
      const int y = good ? key - (int)(div_page(a, (unsigned)key) * (unsigned)a.pages.page_size) : 0;
      const int c1 = head_first ? kvh : y, c2 = head_first ? y : kvh;
      const uint32_t dst = (uint32_t)half * 16384u + (uint32_t)(my * box) * 128u;
      if (u + 1 < rg.u1) {
        advance<R, kKC>(a, ld, 1);
        pg = look();
      }
      for (int v = 0; v < 2 && ok; ++v) {
        ok = __all_sync(0xffffffffu, wait_bounded(v ? V_EMPTY(st) : K_EMPTY(st), ph, abort_v, a.status));
        if (!ok) break;
        const uint32_t bar = v ? V_FULL(st) : K_FULL(st);
        if (lane == 0) {
          // read by the softmax once it has S of the chunk; by then tile A and B are past the entry's last use
          if (!v) s_bad[issued & 3u] = bad;
          mbar_expect_tx(bar, C::kTile);
        }
        __syncwarp();
        if (mine) tma_box((v ? v_s : k_s) + st * C::kTile + dst, v ? &vmap : &kmap, half * 64, c1, c2, w, bar);
        if (v) ++issued;
      }
    }
    if (!ok) {  // wait, bounded, for the copies still in flight
      for (uint32_t s = 0; s < kStages; ++s) {
        const uint32_t nk = issued > s ? (issued - 1 - s) / kStages : 0;  // last full phase of the stage
        if (issued > s) {
          wait_drain(K_FULL(s), nk & 1u);
          wait_drain(V_FULL(s), nk & 1u);
        }
      }
      const uint32_t s = issued % kStages;  // a K load whose V was not issued (ends at once if there was none)
      wait_drain(K_FULL(s), (issued / kStages) & 1u);
    }
  } else if (warp == 1 || warp == 2) {
    // ---- MMA issuer of tile t: the warp runs as one, an elected lane issues
    const int t = warp - 1;
    const uint32_t id_s = idesc_bf16(128, kSub), id_o = idesc_bf16_bmn(128, DP);
    const uint32_t s_tm = tmem + 128u * t, o_tm = tmem + C::kO + 128u * t;
    const uint64_t qd = sw128_desc(q_s), kd0 = sw128_desc(k_s), vd0 = sw128_mn_desc(v_s, 16384u);
    constexpr uint64_t kStep = C::kTile >> 4;  // descriptor distance of two stages (and of the Q tiles)
    bool ok = true, any = false;
    uint32_t g = 0, nseg = 0;      // chunks of the CTA, segments
    uint32_t u = 0, clears = 0;    // sub-chunks of this tile, V_CLEAR phases
    auto wait = [&](uint32_t bar, uint32_t par) {
      ok = ok && __all_sync(0xffffffffu, wait_bounded(bar, par & 1u, abort_v, a.status));
      return ok;
    };
    // scores of sub-chunk h of the chunk in stage st, into buffer h
    auto issue_s = [&](uint32_t st, uint32_t h, bool alone) {
      const uint64_t kd = kd0 + st * kStep + h * (uint64_t)(kSub * 128 >> 4), qq = alone ? qd : qd + t * kStep;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const uint64_t off = (uint64_t)((kk >> 2) * (16384 >> 4) + 2 * (kk & 3));
          tc_mma(s_tm + h * 64u, qq + off, kd + off, id_s, kk > 0 ? 1u : 0u);
        }
        tc_commit(S_FULL(t, h));
        mbar_arrive(S_FULL(t, h));
        if (h) {
          tc_commit(K_EMPTY(st));
          if (alone) tc_commit(K_EMPTY(st));
        }
      }
      __syncwarp();
      any = true;
    };
    for (long long s0 = rg.u0; s0 < rg.u1 && ok; ++nseg) {
      const long long s1 = min(rg.u1, s0 + (seg.s.nblk - seg.blk));
      const int n = (int)(s1 - s0);
      const bool alone = min(seg.s.tq, seg.s.nq - seg.tile * seg.s.tq) <= 128;
      const int j0 = alone ? t : 0, dj = alone ? 2 : 1;  // this tile's chunks: j0, j0 + dj, ...
      // every segment in turn, also one without a chunk of this tile: a wait may be at most one phase behind
      if (!wait(Q_FULL, nseg)) break;
      if (j0 < n) {
        const uint32_t st = (g + j0) % kStages;
        if (!wait(K_FULL(st), (g + j0) / kStages)) break;
        // tile B starts half a sub-chunk late, so that the two tiles' exponentials take turns
        if (!alone && t == 1 && n > 2 && !wait(A_BEGUN, nseg)) break;
        tc_fence_after();
        issue_s(st, 0, alone);
        issue_s(st, 1, alone);
      }
      for (int j = j0; j < n && ok; j += dj) {
        const uint32_t gj = g + (uint32_t)j, st = gj % kStages, gn = gj + (uint32_t)dj, sn = gn % kStages;
        const bool last = j + dj >= n;
        for (uint32_t h = 0; h < 2; ++h, ++u) {
          if (!wait(P_FULL(t, h), u >> 1)) break;
          if (h == 0) {
            if (!wait(V_FULL(st), gj / kStages)) break;
            // the rows of V past the end of an item's last chunk are cleared by the softmax warps of tile A, or of the
            // one tile that takes the chunk, before their P_FULL (tile B: V_CLEAR)
            if (!alone && t == 1 && seg.s.nk - (seg.blk + j) * kKC < kKC && !wait(V_CLEAR, clears++)) break;
          }
          tc_fence_after();
          const uint64_t vd = vd0 + st * kStep + h * (uint64_t)(kSub * 128 >> 4);
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk)
              tc_mma_ts(o_tm, s_tm + h * 64u + (uint32_t)((kk >> 1) * 32 + 16 + (kk & 1) * 8),
                        vd + (uint64_t)(kk * (2048 >> 4)), id_o, (j > j0 || h > 0 || kk > 0) ? 1u : 0u);
            tc_commit(PV_DONE(t));
            if (h) {
              tc_commit(V_EMPTY(st));
              if (alone) tc_commit(V_EMPTY(st));
            }
          }
          __syncwarp();
          // the buffer's next scores overwrite P: after P V has read it
          if ((!last && h == 0 && !wait(K_FULL(sn), gn / kStages)) || !wait(PV_DONE(t), u)) break;
          if (!last) {
            tc_fence_after();
            issue_s(sn, h, alone);
          }
        }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(O_FINAL);
      __syncwarp();
      g += (uint32_t)n;
      advance<R, kKC>(a, seg, n);
      s0 = s1;
    }
    if (!ok && any) {
      if (elect_one()) tc_commit(DRAIN(t));
      __syncwarp();
      wait_drain(DRAIN(t), 0);
    }
  } else if (warp >= kSoft0) {
    // ---- softmax
    const int t = (warp - kSoft0) / kSoftWarps, pt = ((warp - kSoft0) % kSoftWarps) / 4, q4 = warp & 3;
    const int qi = q4 * 32 + lane;                       // query of the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t s_tm = tmem + 128u * t + lane_off, o_tm = tmem + C::kO + 128u * t + lane_off + (uint32_t)(pt * OC);
    const int st_id = tid - 32 * kSoft0;
    const float sc = a.scale_log2;
    auto pair_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + t * 4 + q4) : "memory"); };
    uint32_t u = 0, g = 0, nseg = 0;  // sub-chunks of this tile, chunks of the CTA, segments
    bool alive = true;
    constexpr int kPart = kSub / 2;   // keys of a thread in a sub-chunk
    for (long long s0 = rg.u0; s0 < rg.u1; ++nseg) {
      const Seq &sq = seg.s;
      const long long s1 = min(rg.u1, s0 + (sq.nblk - seg.blk));
      const int n = (int)(s1 - s0);
      const int q0 = seg.tile * sq.tq, nq = min(sq.tq, sq.nq - q0);
      const bool alone = nq <= 128;
      const Pairs pairs(sq, q0, G);
      const int j0 = alone ? t : 0, dj = alone ? 2 : 1;  // this tile's chunks: j0, j0 + dj, ...
      // queries -> shared memory (zero rows past nq, zero dims past head_dim); the last segment's MMAs have read
      // theirs (O_FINAL)
      {
        const int rows = nq > 128 ? 256 : 128;
        for (int i = st_id; i < rows * (DP / 8); i += 64 * kSoftWarps) {
          const int r = i / (DP / 8), c = i - r * (DP / 8);
          const bool in = r < nq && c * 8 < hd;
          load_query16(q_s + (uint32_t)(r >> 7) * C::kTile + tile_off(r & 127, c),
                       static_cast<const bf16 *>(a.q) + pairs.at(in ? r : 0, seg.kvh, a.n_heads, hd) + (in ? c * 8 : 0),
                       in);
        }
        load_query_wait();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(Q_FULL);
      }
      float m_run = -INFINITY, l_run = 0.f;
      const int ns = j0 < n ? 2 * ((n - j0 + dj - 1) / dj) : 0;  // this tile's sub-chunks
      const bool used = (alone ? 0 : t * 128) + q4 * 32 < nq;     // this warp has queries
      for (int i = 0; i < ns; ++i, ++u) {
        const int j = j0 + (i >> 1) * dj, key0 = (seg.blk + j) * kKC + (i & 1) * kSub;
        const uint32_t hb = (uint32_t)(i & 1), s_buf = s_tm + hb * 64u;
        if (alive) alive = __all_sync(0xffffffffu, wait_bounded(S_FULL(t, hb), (u >> 1) & 1u, abort_v, a.status));
        const int nv = sq.nk - key0 - pt * kPart;  // valid keys of this thread
        const uint32_t gj = g + (uint32_t)j;
        if (t == 0 && i == 0 && lane == 0) mbar_arrive(A_BEGUN);
        if (used) {
        uint32_t sr[kPart];  // raw scores: the scale (> 0) commutes with the maximum and enters the exponent
        float mc = -INFINITY;
        if (alive) {
          tc_fence_after();
          tmem_ld32_issue(s_buf + (uint32_t)(pt * kPart), sr);
          tmem_wait_ld_tie32(sr);
          const uint32_t bad = s_bad[gj & 3u];
          if (nv < kPart || bad) {
            uint32_t valid = nv >= kPart ? ~0u : nv <= 0 ? 0u : (1u << nv) - 1u;
            const int k0 = (i & 1) * kSub + pt * kPart;  // this thread's keys in the chunk: one box, or two of 16
            if ((bad >> (k0 / box)) & 1u) valid &= box >= kPart ? 0u : ~0u << box;
            if (box < kPart && ((bad >> (k0 / box + 1)) & 1u)) valid &= (1u << box) - 1u;
#pragma unroll
            for (int c = 0; c < kPart; ++c)
              if (!((valid >> c) & 1u)) sr[c] = 0xff800000u;  // -inf
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < kPart; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
          mc = sc * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        s_mx[u & 1][t][pt][qi] = mc;
        pair_sync();
        mc = fmaxf(mc, s_mx[u & 1][t][1 - pt][qi]);
        if (!alive) continue;
        // The maximum moves only when a sub-chunk exceeds it by more than 8 (log2 units): P stays below 2^8, most
        // sub-chunks rescale nothing, and P, the sum and O share it.
        const bool grow = mc > m_run + 8.f;
        const float m_new = grow ? mc : m_run;
        const float alpha = grow ? (m_run == -INFINITY ? 0.f : ex2a(m_run - m_new)) : 1.f;
        if (i > 0 && __any_sync(0xffffffffu, grow)) {
          // P V of the sub-chunk before must be in O.  The wait is within a phase: P V of the one before that was
          // complete before S_FULL, and this one's cannot be before its P_FULL.
          alive = __all_sync(0xffffffffu, wait_bounded(PV_DONE(t), (u - 1) & 1u, abort_v, a.status));
          if (!alive) continue;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < OC / 16; ++c) {
            float ov[16];
            tmem_ld16(o_tm + (uint32_t)(c * 16), ov);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] *= alpha;
            tmem_st16(o_tm + (uint32_t)(c * 16), ov);
          }
        }
        m_run = m_new;
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kPart / 2; ++c) {
          const float p0 = ex2a(fmaf(__uint_as_float(sr[2 * c]), sc, -m_use));
          const float p1 = ex2a(fmaf(__uint_as_float(sr[2 * c + 1]), sc, -m_use));
          ps[c & 3] += p0 + p1;
          sr[c] = packb(p0, p1);
        }
        // P: 16 columns over the upper half of this thread's own scores
        tmem_st16u(s_buf + (uint32_t)(pt * kPart + 16), sr);
        l_run = l_run * alpha + ((ps[0] + ps[1]) + (ps[2] + ps[3]));
        }
        if (hb == 0 && (alone || t == 0) && sq.nk - key0 < kKC) {
          // past the sequence's end its page holds anything: P is 0 there, V must be.  Boxes wholly past it came as
          // zeros; the rows are cleared after the copy and before P_FULL lets P V start.
          alive = __all_sync(0xffffffffu, wait_bounded(V_FULL(gj % kStages), (gj / kStages) & 1u, abort_v, a.status));
          if (!alive) continue;
          const int r0 = max(sq.nk - key0, 0), r1 = min(kKC, (r0 + box - 1) / box * box);
          for (int w = st_id & (32 * kSoftWarps - 1); w < (r1 - r0) * (DP / 8); w += 32 * kSoftWarps)
            *reinterpret_cast<uint4 *>(sm + (v_s - sbase) + (gj % kStages) * C::kTile +
                                       tile_off(r0 + w / (DP / 8), w % (DP / 8))) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (!alone && lane == 0) mbar_arrive(V_CLEAR);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(P_FULL(t, hb));
      }
      // ---- the segment's end
      if (alive) alive = __all_sync(0xffffffffu, wait_bounded(O_FINAL, nseg & 1u, abort_v, a.status));
      s_l[t][pt][qi] = l_run;
      if (pt == 0) s_m[t][qi] = m_run;
      const bool starts = seg.blk == 0, ends = n == sq.nblk - seg.blk;
      const int slot = s0 == rg.u0 ? 0 : 1;
      const size_t share = (size_t)blockIdx.x * 2 + slot;
      // O columns of this thread, and its query: tiles of their own, half a row per thread; alone, the four threads of
      // a row take a quarter each of both O's (fa, fb: their weights)
      int q, c0, nc;
      float m, l, fa = 1.f, fb = 0.f;
      if (alone) {
        asm volatile("bar.sync %0, 128;" ::"r"(9 + q4) : "memory");
        const float ma = s_m[0][qi], mb = s_m[1][qi];
        m = fmaxf(ma, mb);
        fa = ma == -INFINITY ? 0.f : ex2a(ma - m);
        fb = mb == -INFINITY ? 0.f : ex2a(mb - m);
        l = (s_l[0][0][qi] + s_l[0][1][qi]) * fa + (s_l[1][0][qi] + s_l[1][1][qi]) * fb;
        q = qi;
        nc = DP / 4;
        c0 = (2 * pt + t) * nc;
      } else {
        pair_sync();
        m = m_run;
        l = s_l[t][0][qi] + s_l[t][1][qi];
        q = t * 128 + qi;
        nc = DP / 2;
        c0 = pt * nc;
      }
      if (alive) {
        tc_fence_after();
        bf16 *dst = static_cast<bf16 *>(a.out) + pairs.at(q < nq ? q : 0, seg.kvh, a.n_heads, hd);
        float *po = part_o + share_at(share, R, DP, q, 0);
        const float inv = starts && ends ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
        const uint32_t oa = tmem + C::kO + (alone ? 0u : 128u * t) + lane_off;
#pragma unroll 1
        for (int c = c0; c < c0 + nc; c += 16) {
          float ov[16];
          tmem_ld16(oa + (uint32_t)c, ov);
          if (alone) {
            float ob[16];
            if (n > 1) tmem_ld16(oa + 128u + (uint32_t)c, ob);
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] = n > 1 ? ov[e] * fa + ob[e] * fb : ov[e];
          }
          if (q < nq && c < hd) {
#pragma unroll
            for (int e = 0; e < 16; ++e) ov[e] *= inv;
            if (starts && ends) {
              uint4 *d = reinterpret_cast<uint4 *>(dst + c);
#pragma unroll
              for (int e = 0; e < 2; ++e)
                d[e] = make_uint4(packb(ov[8 * e], ov[8 * e + 1]), packb(ov[8 * e + 2], ov[8 * e + 3]),
                                  packb(ov[8 * e + 4], ov[8 * e + 5]), packb(ov[8 * e + 6], ov[8 * e + 7]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *reinterpret_cast<float4 *>(po + (c / 4 + e) * (R * 4)) =
                    make_float4(ov[4 * e], ov[4 * e + 1], ov[4 * e + 2], ov[4 * e + 3]);
            }
          }
        }
        if (q < nq && c0 == 0 && !(starts && ends)) part_ml[share * R + q] = make_float2(m, l);
        tc_fence_before();
      }
      if (s1 == rg.u1 && st_id == 0) {
        Share sh;
        sh.last = starts && !ends && alive ? rg.of(s0 + sq.nblk - 1) : -1;
        sh.row0 = sq.row0;
        sh.q0 = q0;
        sh.nq = nq;
        sh.kvh = seg.kvh;
        sh.slot = slot;
        shares[blockIdx.x] = sh;
      }
      g += (uint32_t)n;
      advance<R, kKC>(a, seg, n);
      s0 = s1;
    }
  }
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int DP>
cudaError_t launch_dp(const PagedAttnArgs &a, const PageMaps &m, void *ws, cudaStream_t s) {
  using C = TcCfg<DP>;
  static std::atomic<uint64_t> attr{0};
  if (cudaError_t e = ensure_smem_limit(k_paged_attn_tc<DP>, (int)C::kSmem, attr)) return e;
  int grid = 0;
  if (cudaError_t e = paged_grid(&grid)) return e;
  const ShareBuf sb(ws, kTcQueries, DP);
  if (cudaError_t e = launch_pdl(k_paged_attn_tc<DP>, dim3(grid), dim3(kThreads), C::kSmem, s, a, m.k, m.v,
                                 m.head_first, m.box, sb.o, sb.ml, sb.desc))
    return e;
  return launch_paged_merge(a, kTcQueries, grid, sb, s);
}

}  // namespace

int tc_box_keys(const dcu_pages &p) {
  int box = 16;
  while (box < 128 && p.page_size % (2 * box) == 0) box *= 2;
  return box;
}

cudaError_t launch_paged_attention_tc(const PagedAttnArgs &a, const PageMaps &m, void *ws, cudaStream_t s) {
  return a.pages.head_dim <= 64 ? launch_dp<64>(a, m, ws, s) : launch_dp<128>(a, m, ws, s);
}

}  // namespace dcu
