// Paged attention of many query rows per sequence on the 5th-gen tensor cores
// (bf16).  Same line of work, shares and merge as k_paged_attn.cu, with items of
// up to 128 queries (one TMEM lane each) and units of 128 keys, worked in
// sub-chunks of 64:
//
//   warps 0, 3  TMA producers of K and of V: the pages of a sub-chunk, boxes of
//               `box` slots x 64 dims (128-byte swizzle), into a ring each; a box
//               past the sequence's end or on a bad page is read at a page
//               coordinate outside the tensor, i.e. as zeros.  The warp looks 32
//               boxes up at a time, one thread issues them
//   warps 1, 2  MMA issuers (one thread each): S_u = Q K_u^T (M = 128
//               queries, N = 64 keys) into one of five score buffers in tensor
//               memory, and O += P_u V_u (P_u in tensor memory, V MN-major); one
//               warp for both spent 0.9 us a sub-chunk on waits and issues
//   warps 4-19  softmax, four sets of four warps: set u % 4 takes sub-chunk u, a
//               thread is a query and has all 64 keys
//
// The only thing that goes from one sub-chunk to the next is the running maximum
// (O, P and the sums share it): a set waits for its predecessor's maximum, not
// for its exponentials, so four sub-chunks are in the softmax at a time, two more
// in the MMAs, and neither's latency is on the critical path.  (Two tiles of 128
// queries taking turns on two buffers each, measured before: 1.3 us per 128
// queries x 128 keys, bound by the chain softmax - P V - S of each tile.)
//
// What bounds a sub-chunk (4736 rows x 8192 keys x 4 heads, head dim 128: 72 to 78
// us with the GPU's clock, 1.02 to 1.10 PFLOP/s): the five score buffers.  From
// the issue of S to the end of P V takes about 4300 cycles - 750 until S is seen,
// 600 for the maximum, 450 until it is handed on, 1700 for the exponentials (whose
// units four warps of a scheduler share), 750 for P V - and a fifth of that is the
// 870 cycles of a sub-chunk, of which the products are 512.  Six buffers have no room beside Q in
// tensor memory, and Q in shared memory makes S bound by its bytes there (384
// cycles instead of 256); three sets that keep their 64 scores in registers took
// 1.2 times as long, ring stages of two sub-chunks 1.04 times, and the next item's
// queries loaded under the last one's epilogue (for registers) 1.05 times.
// Shorter calls are bound by what surrounds the loop: 161 rows x 8192 keys of 32
// heads take 47 us, of which 32 are the loop (64 sub-chunks), 9.5 the way to the
// first P V (search 1.6, Q 2, first keys 2.5, first softmax 3), 5 the merge.
//
// TMEM: five score buffers of 64 columns, Q, O of head_dim columns (head_dim
// above 128: four buffers, Q in shared memory); P (bf16 pairs) overwrites the
// second half of its scores, which are in registers by then.  P is rounded to bf16 once, as in the dense attention of a step: a second
// product for the low part would cost half as much again on the tensor pipe.
//
// Every mbarrier wait is bounded; on expiry the CTA sets DCU_ST_TIMEOUT, drains
// its copies and MMAs in flight, frees TMEM and exits.  A parity wait is only
// sound for a phase that is the current or the last one of its barrier; where
// that is not plain from the order of the waits, a comment says why it holds.
#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace dcu {
namespace {

constexpr int kKC = 128;              // keys of a unit
constexpr int kSub = 64;              // keys of a sub-chunk
// Units that a change of items costs (O out, Q in, the pipeline refilled: 5 us, a unit takes 1 us).  Measured with 4, 8
// and 12: 60 heads x 100 rows x 8192 keys 63, 56 and 56 us, 50 heads of 64 dims 39, 39 and 43.
constexpr int kTurn = 8;
constexpr uint32_t kSets = 4;         // softmax sets
constexpr int kSoft0 = 4;             // first softmax warp
constexpr int kWarps = kSoft0 + 4 * kSets;
constexpr int kThreads = 32 * kWarps;

template <int DP>
struct TcCfg {
  // Q: in tensor memory (bf16 pairs), or, where that leaves too few score buffers, in shared memory: DP / 64 blocks of
  // 128 rows x 128 bytes
  static constexpr bool kQTmem = DP <= 128;
  static constexpr uint32_t kQ = kQTmem ? 0u : 128u * DP * 2u;
  static constexpr uint32_t kTile = 64u * DP * 2u;   // K or V of a sub-chunk: DP / 64 blocks of 64 rows x 128 bytes
  // ring depths (sub-chunks) and score buffers: what shared memory (227 KB) and tensor memory (512 columns) hold
  static constexpr uint32_t kKStages = DP == 256 ? 2 : 6, kVStages = DP == 256 ? 2 : 7, kBufs = DP == 256 ? 4 : 5;
  static constexpr uint32_t kSmem = kQ + (kKStages + kVStages) * kTile + 1024u;
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kQCol = 64 * kBufs;      // columns of Q and of O
  static constexpr uint32_t kO = kQCol + (kQTmem ? 64 : 0);
  static_assert(kO + DP <= kTmemCols, "tensor memory");
};

template <int ROWS>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {  // 16-byte chunk c of row r of a tile of ROWS rows
  return (uint32_t)(c >> 3) * (uint32_t)(ROWS * 128) + (uint32_t)r * 128u + ((uint32_t)((c & 7) ^ (r & 7)) << 4);
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

__device__ __forceinline__ void mask32(uint32_t (&r)[32], uint32_t valid) {
#pragma unroll
  for (int c = 0; c < 32; ++c)
    if (!((valid >> c) & 1u)) r[c] = 0xff800000u;  // -inf
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
  constexpr int R = kTcQueries;
  constexpr uint32_t kKStages = C::kKStages, kVStages = C::kVStages, kBufs = C::kBufs;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t bars[2 * (kKStages + kVStages) + 3 * kBufs + 4 + 4 * kSets];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ long long s_scan[2 * kWarps];
  __shared__ Place s_place;
  __shared__ Range s_range;
  __shared__ float s_max[kSets][128];   // [set] running maximum after the set's sub-chunk
  __shared__ float2 s_ml[kSets][128];   // [set] (maximum, sum) at the end of a segment
  __shared__ uint32_t s_bad[16];        // [sub-chunk % 16] its boxes on bad pages
  __shared__ int2 s_box[2][32];         // [K, V][box of the producer's batch] slot, page
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = (smem_u32(sm_raw) + 1023u) & ~1023u;
  uint8_t *sm = sm_raw + (sbase - smem_u32(sm_raw));
  const uint32_t q_s = sbase, k_s = sbase + C::kQ, v_s = k_s + kKStages * C::kTile;
  const uint32_t bar0 = smem_u32(bars);
  auto K_FULL = [&](uint32_t s) { return bar0 + 8u * s; };
  auto K_EMPTY = [&](uint32_t s) { return bar0 + 8u * (kKStages + s); };
  auto V_FULL = [&](uint32_t s) { return bar0 + 8u * (2 * kKStages + s); };
  auto V_EMPTY = [&](uint32_t s) { return bar0 + 8u * (2 * kKStages + kVStages + s); };
  const uint32_t bar1 = bar0 + 8u * (2 * (kKStages + kVStages));
  auto S_FULL = [&](uint32_t b) { return bar1 + 8u * b; };                   // scores of buffer b are there
  auto P_FULL = [&](uint32_t b) { return bar1 + 8u * (kBufs + b); };         // its P is there
  auto PV_DONE = [&](uint32_t b) { return bar1 + 8u * (2 * kBufs + b); };    // its P V is in O
  const uint32_t Q_FULL = bar1 + 8u * (3 * kBufs), O_FINAL = Q_FULL + 8u, DRAIN = Q_FULL + 16u;  // DRAIN: two
  auto MAX = [&](uint32_t set, int q4) { return Q_FULL + 32u + 8u * (set * 4u + (uint32_t)q4); };  // s_max[set] of 32 rows

  if (tid == 0) {
    for (uint32_t i = 0; i < 2 * (kKStages + kVStages); ++i) mbar_init(bar0 + 8u * i, 1);
    for (uint32_t b = 0; b < kBufs; ++b) {
      mbar_init(S_FULL(b), 2);  // the scores (commit), and the issuer itself (it has seen K_FULL, and so s_bad)
      mbar_init(P_FULL(b), 4);
      mbar_init(PV_DONE(b), 1);
    }
    for (uint32_t i = 0; i < 4 * kSets; ++i) mbar_init(MAX(0, 0) + 8u * i, 1);
    mbar_init(Q_FULL, 4 * kSets);
    mbar_init(O_FINAL, 1);
    mbar_init(DRAIN, 1);
    mbar_init(DRAIN + 8u, 1);
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
  // (a barrier inside; two units at least: measured with 1, 2, 4 and 8, 65 rows of 28/4 heads x 1024 keys take 16.8, 15.7,
  // 16.6 and 18.6 us, 65 rows of 32 heads x 256 keys 13.1, 11.7, 11.8 and 11.7, of 8 heads x 2048 keys 13.6, 14.3, 15.6, 19.0)
  find_range<R, kKC, kWarps>(a, &s_place, &s_range, s_scan, 2, kTurn);
  Place seg = s_place;
  const int units = s_range.any ? (int)(s_range.u1 - s_range.u0) : 0;
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  volatile int *abort_v = &abort_flag;
  const int KV = a.pages.n_kv_heads, G = a.n_heads / KV, hd = a.pages.head_dim;

  if (!units) {
    if (tid == 0) shares[blockIdx.x].last = -1;
  } else if (warp == 0 || warp == 3) {
    // ---- TMA producers
    const bool is_v = warp == 3;
    const uint32_t stages = is_v ? kVStages : kKStages, ring = is_v ? v_s : k_s;
    const uint32_t full0 = is_v ? V_FULL(0) : K_FULL(0), empty0 = is_v ? V_EMPTY(0) : K_EMPTY(0);
    const CUtensorMap *map = is_v ? &vmap : &kmap;
    // A batch is 32 boxes: each lane looks its box up (one batch ahead) and leaves its place in shared memory, then one
    // thread issues.  (Each sub-chunk looked up and issued by the whole warp, measured before: 1130 cycles a sub-chunk,
    // more than anything else in the kernel took.)
    const int nb = kSub / box, per = 32 / nb;  // boxes of a sub-chunk (of each 64-dim block), sub-chunks of a batch
    int2 *const places = s_box[is_v];
    uint32_t st = 0, par = 1, u = 0;  // stage, its EMPTY parity, sub-chunk
    bool ok = true;
    for (int left = units; left > 0 && ok;) {
      const int ns = 2 * min(left, seg.s.nblk - seg.blk), kvh = seg.kvh;
      // first key of the lane's box in the batch of sub-chunk h of the segment, and its page (-1: none)
      auto key_of = [&](int h) { return (unsigned)(seg.blk * kKC) + (unsigned)h * kSub + (unsigned)(lane * box); };
      auto look = [&](int h) {
        const unsigned key = key_of(h);
        return h < ns && key < (unsigned)seg.s.nk ? a.table[(size_t)seg.b * a.max_pages + div_page(a, key)] : -1;
      };
      int pg = look(0);
      for (int h0 = 0; h0 < ns && ok; h0 += per) {
        const unsigned key = key_of(h0);
        const bool in = key < (unsigned)seg.s.nk, good = in && pg >= 0 && pg < a.pages.n_pages;
        const uint32_t bad = __ballot_sync(0xffffffffu, in && !good);
        // outside the tensor: zeros
        places[lane] = make_int2(good ? (int)(key - div_page(a, key) * (unsigned)a.pages.page_size) : 0,
                                 good ? pg : a.pages.n_pages);
        __syncwarp();
        pg = look(h0 + per);
        const int n = min(per, ns - h0);
        int done = 0;  // sub-chunks issued
        if (elect_one()) {
          for (; done < n; ++done) {
            if (!wait_bounded(empty0 + 8u * st, par, abort_v, a.status)) break;
            if (!is_v) {
              const uint32_t mine = (bad >> (done * nb)) & ((1u << nb) - 1u);
              s_bad[(u + (uint32_t)done) & 15u] = mine;  // read by the softmax with the scores, long before it is reused
              if (mine && a.status) atomicOr(a.status, DCU_ST_BAD_PAGE);
            }
            const uint32_t bar = full0 + 8u * st, to = ring + st * C::kTile;
            mbar_expect_tx(bar, C::kTile);
            for (int x = 0; x < nb; ++x) {
              const int2 at = places[done * nb + x];
#pragma unroll
              for (int blk = 0; blk < DP / 64; ++blk)
                tma_box(to + (uint32_t)(blk * kSub * 128) + (uint32_t)(x * box) * 128u, map, blk * 64,
                        head_first ? kvh : at.x, head_first ? at.x : kvh, at.y, bar);
            }
            if (++st == stages) {
              st = 0;
              par ^= 1u;
            }
          }
        }
        // the issuing thread need not be the same one each time
        done = (int)__reduce_max_sync(0xffffffffu, (unsigned)done);
        ok = done == n;
        u += (uint32_t)done;
        st = u % stages;
        par = ((u / stages) & 1u) ^ 1u;
        __syncwarp();
      }
      advance<R, kKC>(a, seg, ns / 2);
      left -= ns / 2;
    }
    if (!ok)  // wait, bounded, for the copies still in flight: the last phase of every stage
      for (uint32_t s = 0; s < stages; ++s)
        if (u > s) wait_drain(full0 + 8u * s, ((u - 1 - s) / stages) & 1u);
  } else if (warp <= 2) {
    // ---- MMA issuers: one thread waits and issues
    if (elect_one()) {
      const bool pv = warp == 2;
      const uint32_t id_s = idesc_bf16(128, kSub), id_o = idesc_bf16_bmn(128, DP);
      [[maybe_unused]] const uint64_t qd = sw128_desc(q_s);
      const uint64_t kd0 = sw128_desc(k_s), vd0 = sw128_mn_desc(v_s, kSub * 128u);
      constexpr uint64_t kStep = C::kTile >> 4;  // descriptor distance of two stages
      bool ok = true, any = false;
      uint32_t nseg = 0;                                        // segments
      uint32_t st = 0, st_par = 0, b = 0, b_par = 0;            // stage and buffer of the sub-chunk, their FULL parities
      const uint32_t stages = pv ? kVStages : kKStages;
      auto step = [&]() {
        if (++st == stages) {
          st = 0;
          st_par ^= 1u;
        }
        if (++b == kBufs) {
          b = 0;
          b_par ^= 1u;
        }
      };
      auto wait = [&](uint32_t bar, uint32_t par) {
        ok = wait_bounded(bar, par & 1u, abort_v, a.status);
        return ok;
      };
      for (int left = units; left > 0 && ok; ++nseg) {
        const int ns = 2 * min(left, seg.s.nblk - seg.blk);
        if (!pv) {
          if (!wait(Q_FULL, nseg)) break;
          for (int i = 0; i < ns; ++i, step()) {
            // the buffer's last P V has read its P (the first time there is none, and that parity has passed)
            if (!wait(K_FULL(st), st_par) || !wait(PV_DONE(b), b_par ^ 1u)) break;
            tc_fence_after();
            const uint64_t kd = kd0 + st * kStep;
#pragma unroll
            for (int kk = 0; kk < DP / 16; ++kk) {
              const uint64_t kdk = kd + (uint64_t)((kk >> 2) * (kSub * 128 >> 4) + 2 * (kk & 3));
              if constexpr (C::kQTmem)
                tc_mma_ts(tmem + b * 64u, tmem + C::kQCol + (uint32_t)(kk * 8), kdk, id_s, kk > 0 ? 1u : 0u);
              else
                tc_mma(tmem + b * 64u, qd + (uint64_t)((kk >> 2) * (16384 >> 4) + 2 * (kk & 3)), kdk, id_s,
                       kk > 0 ? 1u : 0u);
            }
            tc_commit(S_FULL(b));
            mbar_arrive(S_FULL(b));
            tc_commit(K_EMPTY(st));
            any = true;
          }
        } else {
          for (int i = 0; i < ns; ++i, step()) {
            if (!wait(V_FULL(st), st_par) || !wait(P_FULL(b), b_par)) break;
            tc_fence_after();
            const uint64_t vd = vd0 + st * kStep;
#pragma unroll
            for (int kk = 0; kk < kSub / 16; ++kk)
              tc_mma_ts(tmem + C::kO, tmem + b * 64u + 32u + (uint32_t)(kk * 8), vd + (uint64_t)(kk * (2048 >> 4)), id_o,
                        (i > 0 || kk > 0) ? 1u : 0u);
            tc_commit(PV_DONE(b));
            tc_commit(V_EMPTY(st));
            if (i == ns - 1) tc_commit(O_FINAL);
            any = true;
          }
        }
        if (!ok) break;
        advance<R, kKC>(a, seg, ns / 2);
        left -= ns / 2;
      }
      if (!ok && any) {
        const uint32_t drain = DRAIN + (pv ? 8u : 0u);
        tc_commit(drain);
        wait_drain(drain, 0);
      }
    }
  } else if (warp >= kSoft0) {
    // ---- softmax
    const uint32_t set = (uint32_t)(warp - kSoft0) / 4u;
    const int q4 = warp & 3, qi = q4 * 32 + lane;        // query of the tile = TMEM lane
    const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
    const uint32_t o_tm = tmem + C::kO + lane_off;
    const int st_id = tid - 32 * kSoft0;
    const float sc = a.scale_log2;
    uint32_t g = 0, nseg = 0;  // chunks of the CTA before the segment, segments
    bool alive = true;
    for (int at = 0; at < units; ++nseg) {
      const Seq &sq = seg.s;
      const int n = min(units - at, sq.nblk - seg.blk), ns = 2 * n;
      const int q0 = seg.tile * sq.tq, nq = min(sq.tq, sq.nq - q0);
      const Pairs pairs(sq, q0, G);
      // queries (zero rows past nq, zero dims past head_dim) -> tensor memory, 32 dims of a row per thread, or shared
      // memory; the last segment's MMAs have read theirs (O_FINAL)
      const bf16 *qg = static_cast<const bf16 *>(a.q);
      if constexpr (C::kQTmem) {
        if (set < DP / 32) {
          uint32_t qv[16];
          const bf16 *src = qg + pairs.at(qi < nq ? qi : 0, seg.kvh, a.n_heads, hd);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int d = (int)set * 32 + c * 8;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (qi < nq && d < hd) v = *reinterpret_cast<const uint4 *>(src + d);
            qv[4 * c] = v.x;
            qv[4 * c + 1] = v.y;
            qv[4 * c + 2] = v.z;
            qv[4 * c + 3] = v.w;
          }
          tmem_st16u(tmem + C::kQCol + set * 16u + lane_off, qv);
          tmem_wait_st();
        }
        tc_fence_before();
      } else {
        for (int i = st_id; i < 128 * (DP / 8); i += 128 * (int)kSets) {
          const int r = i / (DP / 8), c = i - r * (DP / 8);
          const bool in = r < nq && c * 8 < hd;
          load_query16(q_s + tile_off<128>(r, c), qg + pairs.at(in ? r : 0, seg.kvh, a.n_heads, hd) + (in ? c * 8 : 0), in);
        }
        load_query_wait();
        fence_proxy_async_smem();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(Q_FULL);
      const bool used = q4 * 32 < nq;             // this warp has queries
      float m_own = -INFINITY, l_run = 0.f;       // the maximum of this set's last sub-chunk, its share of the sum
      for (int i = (int)((set - 2 * g) & 3u); i < ns; i += (int)kSets) {
        const uint32_t u = 2 * g + (uint32_t)i, b = u % kBufs, s_tm = tmem + b * 64u + lane_off;
        const int left = sq.nk - seg.blk * kKC - i * kSub;  // keys of the sequence from the sub-chunk's first on
        // (a buffer's phase before this one is long over: the set that had it has handed its maximum down to this one)
        if (alive) alive = __all_sync(0xffffffffu, wait_bounded(S_FULL(b), (u / kBufs) & 1u, abort_v, a.status));
        if (!alive) continue;  // nothing is handed on any more: every wait now fails
        if (i > 0 && !used) {
          alive = __all_sync(0xffffffffu, wait_bounded(MAX((set + 3u) & 3u, q4), ((u - 1) >> 2) & 1u, abort_v, a.status));
          if (!alive) continue;
        }
        if (used) {
          tc_fence_after();
          // Raw scores: the scale (> 0) commutes with the maximum and enters the exponent.  The first 32 keys are read
          // again for the exponentials rather than kept, which holds the thread within its registers.
          uint32_t lo = ~0u, hi = ~0u;  // valid keys
          const uint32_t bad = s_bad[u & 15u];
          const bool cut = left < kSub || bad;
          if (cut) {
            unsigned long long v = left >= kSub ? ~0ull : left <= 0 ? 0ull : (1ull << left) - 1ull;
            for (int x = 0; x < kSub; x += box)
              if ((bad >> (x / box)) & 1u) v &= ~((box >= kSub ? ~0ull : (1ull << box) - 1ull) << x);
            lo = (uint32_t)v;
            hi = (uint32_t)(v >> 32);
          }
          uint32_t sr[32];
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            tmem_ld32_issue(s_tm + (uint32_t)(hf * 32), sr);
            tmem_wait_ld_tie32(sr);
            if (cut) mask32(sr, hf ? hi : lo);
#pragma unroll
            for (int c = 0; c < 32; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
          }
          const float mc = sc * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // The predecessor's maximum (its last phase is long over: this set has waited for it, or a segment has ended).
          float m_old = -INFINITY;
          if (i > 0) {
            const uint32_t ps = (set + 3u) & 3u;
            alive = __all_sync(0xffffffffu, wait_bounded(MAX(ps, q4), ((u - 1) >> 2) & 1u, abort_v, a.status));
            if (!alive) continue;
            m_old = s_max[ps][qi];
          }
          // The maximum moves only when a sub-chunk exceeds it by more than 8 (log2 units): P stays below 2^8, most
          // sub-chunks rescale nothing, and P, the sums and O share it.
          const bool grow = mc > m_old + 8.f;
          const float m_new = grow ? mc : m_old;
          s_max[set][qi] = m_new;
          __syncwarp();
          if (lane == 0) mbar_arrive(MAX(set, q4));
          if (i > 0 && __any_sync(0xffffffffu, grow)) {
            // O takes the new maximum between P V of the last sub-chunk (waited for; the one before on that barrier was
            // waited for by the issuer of this buffer's S) and of this one (after its P_FULL)
            alive = __all_sync(0xffffffffu, wait_bounded(PV_DONE((u - 1) % kBufs), ((u - 1) / kBufs) & 1u, abort_v, a.status));
            if (!alive) continue;
            tc_fence_after();
            const float alpha = grow ? (m_old == -INFINITY ? 0.f : ex2a(m_old - m_new)) : 1.f;
#pragma unroll 1
            for (int c = 0; c < DP / 16; ++c) {
              float ov[16];
              tmem_ld16(o_tm + (uint32_t)(c * 16), ov);
#pragma unroll
              for (int e = 0; e < 16; ++e) ov[e] *= alpha;
              tmem_st16(o_tm + (uint32_t)(c * 16), ov);
            }
          }
          if (m_new != m_own) {
            l_run *= m_own == -INFINITY ? 0.f : ex2a(m_own - m_new);
            m_own = m_new;
          }
          const float m_use = m_new == -INFINITY ? 0.f : m_new;
          float ps[4] = {0.f, 0.f, 0.f, 0.f};
          // P: keys 32 .. 63 first (columns 48 .. 63 of the buffer), then keys 0 .. 31 (columns 32 .. 47)
#pragma unroll
          for (int hf = 1; hf >= 0; --hf) {
            if (hf == 0) {
              tmem_ld32_issue(s_tm, sr);
              tmem_wait_ld_tie32(sr);
              if (cut) mask32(sr, lo);
            }
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float p0 = ex2a(fmaf(__uint_as_float(sr[2 * c]), sc, -m_use));
              const float p1 = ex2a(fmaf(__uint_as_float(sr[2 * c + 1]), sc, -m_use));
              ps[c & 3] += p0 + p1;
              sr[c] = packb(p0, p1);
            }
            tmem_st16u(s_tm + (uint32_t)(hf ? 48 : 32), sr);
          }
          l_run += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        } else if (lane == 0) {
          mbar_arrive(MAX(set, q4));  // (the phases count sub-chunks in every segment)
        }
        if (left < kSub) {
          // Past the sequence's end its page holds anything: P is 0 there, V must be.  Boxes wholly past it came as
          // zeros; the rest of the last box is cleared after the copy and before P_FULL lets P V start.  (The stage held
          // sub-chunk u - kVStages; the issuer of this buffer's S has waited for P V of sub-chunk u - kBufs.)
          const uint32_t st = u % kVStages, before = u - kVStages;
          if (kVStages < kBufs && u >= kVStages) {
            alive = __all_sync(0xffffffffu, wait_bounded(PV_DONE(before % kBufs), (before / kBufs) & 1u, abort_v, a.status));
            if (!alive) continue;
          }
          alive = __all_sync(0xffffffffu, wait_bounded(V_FULL(st), (u / kVStages) & 1u, abort_v, a.status));
          if (!alive) continue;
          const int r0 = max(left, 0), r1 = (r0 + box - 1) / box * box;
          for (int w = qi; w < (r1 - r0) * (DP / 8); w += 128)
            *reinterpret_cast<uint4 *>(sm + (v_s - sbase) + st * C::kTile +
                                       tile_off<kSub>(r0 + w / (DP / 8), w % (DP / 8))) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(P_FULL(b));
      }
      // ---- the segment's end: the sets' sums, and a quarter of O's columns for each
      if (alive) alive = __all_sync(0xffffffffu, wait_bounded(O_FINAL, nseg & 1u, abort_v, a.status));
      s_ml[set][qi] = make_float2(m_own, l_run);
      asm volatile("bar.sync %0, 128;" ::"r"(1 + q4) : "memory");
      const bool starts = seg.blk == 0, ends = n == sq.nblk - seg.blk;
      const int slot = at ? 1 : 0;
      if (alive && used) {
        tc_fence_after();
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (uint32_t s = 0; s < kSets; ++s) m = fmaxf(m, s_ml[s][qi].x);  // the maximum never falls: the last sub-chunk's
#pragma unroll
        for (uint32_t s = 0; s < kSets; ++s) {
          const float2 ml = s_ml[s][qi];
          l += ml.x == -INFINITY ? ml.y : ml.y * ex2a(ml.x - m);
        }
        const size_t share = (size_t)blockIdx.x * 2 + slot;
        bf16 *dst = static_cast<bf16 *>(a.out) + pairs.at(qi < nq ? qi : 0, seg.kvh, a.n_heads, hd);
        float *po = part_o + share_at(share, R, DP, qi, 0);
        const float inv = starts && ends ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
#pragma unroll
        for (int c = (int)set * (DP / 4); c < (int)set * (DP / 4) + DP / 4; c += 16) {
          float ov[16];
          tmem_ld16(o_tm + (uint32_t)c, ov);
          if (qi < nq && c < hd) {
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
        if (set == 0 && qi < nq && !(starts && ends)) part_ml[share * R + qi] = make_float2(m, l);
        tc_fence_before();
      }
      if (at + n == units && st_id == 0) {
        Share sh;
        sh.last = starts && !ends && alive ? s_range.of(s_range.u0 + at + sq.nblk - 1) : -1;
        sh.row0 = sq.row0;
        sh.q0 = q0;
        sh.nq = nq;
        sh.kvh = seg.kvh;
        sh.slot = slot;
        shares[blockIdx.x] = sh;
      }
      g += (uint32_t)n;
      advance<R, kKC>(a, seg, n);
      at += n;
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
  PagedAttnArgs b = a;
  b.whole = whole_items(a, kTcQueries, kKC, 4, grid);
  if (cudaError_t e = launch_pdl(k_paged_attn_tc<DP>, dim3(grid), dim3(kThreads), C::kSmem, s, b, m.k, m.v,
                                 m.head_first, m.box, sb.o, sb.ml, sb.desc))
    return e;
  return b.whole ? cudaSuccess : launch_paged_merge(a, kTcQueries, grid, sb, s);
}

}  // namespace

int tc_box_keys(const dcu_pages &p) {
  int box = 8;  // the rows of a swizzle atom
  while (box < kSub && p.page_size % (2 * box) == 0) box *= 2;
  return box;
}

cudaError_t launch_paged_attention_tc(const PagedAttnArgs &a, const PageMaps &m, void *ws, cudaStream_t s) {
  return a.pages.head_dim <= 64 ? launch_dp<64>(a, m, ws, s)
                                : a.pages.head_dim <= 128 ? launch_dp<128>(a, m, ws, s) : launch_dp<256>(a, m, ws, s);
}

}  // namespace dcu
