// paged_long.cuh -- attention of many new tokens per sequence over a paged
// cache (the work list, the mask and the merge are in paged.cuh).
//
// The pipeline of the training forward (fwd.cuh) over the paged work list:
// one CTA per SM, an item is up to 256 rows of one head group, two Q tiles of
// 128 rows that two softmax warpgroups process while the tensor core works on
// the other tile:
//   S_t = Q_t K^T   tcgen05.mma from 128B-swizzled shared memory, fp32 in TMEM
//   P_t = 2^(S_t - m)   one thread per row, P written over S_t as 16 bits
//   O_t += P_t V    tcgen05.mma, A = P_t from TMEM
// Rows of a tile are (token, head of the group), the heads fastest: one TMA
// box of the [T][Hq][d] queries gives them in that order, so heads that share
// their keys share the tile.  The producer warp gathers a 128-key tile from
// its pages, one box per page, head and 64 columns.  Boxes without any needed
// key are fetched from outside the tensor, which fills with zeros and reads
// nothing; the rest of a partly needed box may hold no numbers, so before V is
// used on a tile that the item's key range cuts, a helper warp clears the rows
// outside the range (0 times no number is no number).  Scores of such keys are
// replaced, not added to, by the mask.
//
// Bound by the exponentials and the tensor core (a 128 x 128 tile takes 1024
// cycles of the 16 special-function lanes and 512 of the tensor core).
#pragma once

#include "fwd.cuh"
#include "paged.cuh"

namespace spa {

template <int D>
struct PagedLongCfg : FwdCfg<D> {
  static constexpr int ROWS = 256, TK = 128;
  using F = FwdCfg<D>;
  static constexpr uint32_t OFF_PLAN = F::OFF_BAR + 256;
  static constexpr uint32_t USED = OFF_PLAN + 512;
  static constexpr uint32_t SMEM_BYTES = USED + 1024 > 116u * 1024 ? USED + 1024 : 116u * 1024;
  static_assert(SMEM_BYTES <= kMaxSmemPerBlock, "shared memory");
};

struct PagedLongBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[2], v_full[2], kv_empty[2];
  uint64_t v_fixed[2];  // the helper warp has cleared the rows outside the key range
  uint64_t s_full[2], p_full[2], o_done[2], o_free[2];
  uint64_t turn[2];
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(PagedLongBars) <= 256, "barrier space");

// One piece of an item as the two Q tiles see it.
struct PagedTiles {
  int rows[2];     // rows of the tile that exist
  int64_t pos[2];  // position of the tile's first and last token
  int64_t last[2];
  int a[2], b[2];  // its key tiles within the piece
  bool act[2];
  int u0, u1;
};

template <int TK>
__device__ __forceinline__ PagedTiles paged_tiles(const PagedParams& p, const PagedWalk<TK>& w) {
  PagedTiles U;
  const PagedItem& it = w.it;
  const int per = 128 / p.group;  // tokens per Q tile
  U.u0 = w.t0;
  U.u1 = w.t1 - 1;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int tok = max(0, min(per, it.tokens - t * per));
    U.rows[t] = tok * p.group;
    U.pos[t] = it.pos0 + t * per;
    U.last[t] = U.pos[t] + tok - 1;
    const int64_t jlo = max64(0, U.pos[t] - p.hi[it.hg] + 1), jhi = min64(U.last[t] - p.lo[it.hg], it.kv - 1);
    U.act[t] = tok > 0 && jhi >= jlo;
    U.a[t] = U.act[t] ? max((int)(jlo / TK), w.t0) : 0;
    U.b[t] = U.act[t] ? min((int)(jhi / TK), w.t1 - 1) : -1;
    U.act[t] = U.act[t] && U.a[t] <= U.b[t];
  }
  return U;
}

// The item's key range cuts tile `t`: some of its rows are not to be used.
template <int TK>
__device__ __forceinline__ bool paged_cut(const PagedItem& it, int t) {
  return (int64_t)t * TK < it.jlo || (int64_t)t * TK + TK - 1 > it.jhi;
}

template <class E, int D, bool TURN>
__global__ void __launch_bounds__(384, 1)
    spa_paged_long_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using C = PagedLongCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  if (!smem_fits(smem_raw, smem, C::USED)) return;
  PagedLongBars* bars = reinterpret_cast<PagedLongBars*>(smem + C::OFF_BAR);
  PagedPlanSmem& plan = *reinterpret_cast<PagedPlanSmem*>(smem + C::OFF_PLAN);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t sQ = ptx::smem_u32(smem + C::OFF_Q);
  const uint32_t sK = ptx::smem_u32(smem + C::OFF_K);
  const uint32_t sV = ptx::smem_u32(smem + C::OFF_V);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars->q_full[i], 1);
      ptx::mbar_init(&bars->q_empty[i], 1);
      ptx::mbar_init(&bars->k_full[i], 1);
      ptx::mbar_init(&bars->v_full[i], 1);
      ptx::mbar_init(&bars->v_fixed[i], 1);
      ptx::mbar_init(&bars->kv_empty[i], 3);  // one release per MMA issuer, one of the helper's
      ptx::mbar_init(&bars->s_full[i], 1);
      ptx::mbar_init(&bars->p_full[i], 128);
      ptx::mbar_init(&bars->o_done[i], 1);
      ptx::mbar_init(&bars->o_free[i], 128);
      ptx::mbar_init(&bars->turn[i], 128);
      ptx::mbar_init(&bars->drain[i], 1);
    }
    bars->abort = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(&bars->tmem_base, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  if (warp == 8 && lane == 0) {
    ptx::prefetch_tmap(&tm_q);
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  ptx::tc_fence_before();
  paged_plan<C::TK, C::NTHREADS>(p, plan);
  ptx::tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;
  PagedWalk<C::TK> w(p, plan.run);

  if (warp >= 8) {
    ptx::regs_dec<C::CONTROL_REGS>();
    if (warp == 11) {
      // ---------------------------------------------------------- helper: clears unused V rows
      // It follows every tile, cut or not, and releases the stage like an MMA
      // issuer, so that the waits on v_full keep step with its phases.
      int g = 0;
      bool ok = true;
      while (ok && w.next()) {
        const PagedItem& it = w.it;
        for (int t = w.t0; ok && t < w.t1; ++t, ++g) {
          const int s = g % C::NS;
          ok = __all_sync(0xffffffffu, bar_wait(&bars->v_full[s], (g / C::NS) & 1, abort_flag));
          if (!ok) break;
          if (!paged_cut<C::TK>(it, t)) {
            if (lane == 0) ptx::mbar_arrive(&bars->kv_empty[s]);
            continue;
          }
          const int64_t j0 = (int64_t)t * C::TK;
          const int first = (int)min64(max64(it.jlo - j0, 0), C::TK);    // rows [0, first) and
          const int end = (int)min64(max64(it.jhi + 1 - j0, 0), C::TK);  // [end, TK) are not used
          const int n = first + (C::TK - end);
          for (int e = lane; e < n * 8; e += 32) {
            const int r = e / 8 < first ? e / 8 : end + e / 8 - first;
#pragma unroll
            for (int c = 0; c < C::DB; ++c)
              ptx::st_shared_v4(sV + s * C::KV_BYTES + c * (C::BK * 128) + r * 128 + (e % 8) * 16, 0u, 0u, 0u, 0u);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            ptx::mbar_arrive(&bars->v_fixed[s]);
            ptx::mbar_arrive(&bars->kv_empty[s]);
          }
        }
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
      const int box_shift = min(p.page_shift, 7), boxes = C::TK >> box_shift;
      PagedPages pages;
      int nq[2] = {0, 0};
      int g = 0;
      bool ok = true;
      while (ok && w.next()) {
        const PagedItem& it = w.it;
        const PagedTiles U = paged_tiles(p, w);
        const int hk = it.hg / p.kv_div;
        if (lane == 0 && p.kv_len[it.b] > it.kv) atomicExch(&g_spa_status, kStatusInval);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || !U.act[t]) continue;
          ok = __all_sync(0xffffffffu, bar_wait(&bars->q_empty[t], (nq[t] & 1) ^ 1, abort_flag));
          if (!ok) continue;
          ++nq[t];
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&bars->q_full[t], C::Q_BYTES);
            for (int c = 0; c < C::DB; ++c)
              ptx::tma_load_4d(smem + C::OFF_Q + t * C::Q_BYTES + c * (C::BQ * 128), &tm_q, &bars->q_full[t], c * 64,
                               0, it.hg, it.row0 + t * (128 / p.group));
          }
        }
        for (int t = w.t0; ok && t < w.t1; ++t, ++g) {
          const int s = g % C::NS;
          const int box_i = lane % boxes, cb = lane / boxes;  // box, 64-column block
          const int64_t box0 = (int64_t)t * boxes;
          const int id = pages.get(p, it, box0, box_shift, boxes, box_i, t == w.t0);
          ok = __all_sync(0xffffffffu, bar_wait(&bars->kv_empty[s], ((g / C::NS) & 1) ^ 1, abort_flag));
          if (!ok) break;
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(&bars->k_full[s], C::KV_BYTES);
            ptx::mbar_arrive_expect_tx(&bars->v_full[s], C::KV_BYTES);
          }
          __syncwarp();
          if (cb < C::DB) {
            const int64_t j = (box0 + box_i) << box_shift;
            const int c1 = (int)(j & ((1 << p.page_shift) - 1)), c2 = id < 0 ? -1 : id * p.Hk + hk;
            const uint32_t at = s * C::KV_BYTES + cb * (C::BK * 128) + (box_i << box_shift) * 128;
            ptx::tma_load_3d(smem + C::OFF_K + at, &tm_k, &bars->k_full[s], cb * 64, c1, c2);
            ptx::tma_load_3d(smem + C::OFF_V + at, &tm_v, &bars->v_full[s], cb * 64, c1, c2);
          }
          __syncwarp();
        }
      }
      // Exit path: every load this warp issued has landed before the CTA ends.
      if (lane == 0) {
        for (int t = 0; t < 2; ++t)
          if (nq[t] > 0) bar_drain(&bars->q_full[t], (nq[t] - 1) & 1);
        for (int s = 0; s < C::NS; ++s) {
          const int used = (g + C::NS - 1 - s) / C::NS;
          if (used > 0) {
            bar_drain(&bars->k_full[s], (used - 1) & 1);
            bar_drain(&bars->v_full[s], (used - 1) & 1);
          }
        }
      }
    } else {
      // ---------------------------------------------------------- MMA issuers
      // warp 9 issues every MMA of Q tile 0, warp 10 those of Q tile 1 (fwd.cuh)
      const int t = warp - 9;
      if (lane == 0) {
        constexpr uint32_t idesc_s = ptx::idesc_16_f32(E::kMmaFormat, 128, C::BK, false, false);
        constexpr uint32_t idesc_o = ptx::idesc_16_f32(E::kMmaFormat, 128, D, false, true);
        const uint64_t dq = ptx::sdesc_sw128(sQ + t * C::Q_BYTES, 0, 1024);
        const uint64_t dk0 = ptx::sdesc_sw128(sK, 0, 1024), dk1 = ptx::sdesc_sw128(sK + C::KV_BYTES, 0, 1024);
        const uint64_t dv0 = ptx::sdesc_sw128(sV, C::BK * 128, 1024);
        const uint64_t dv1 = ptx::sdesc_sw128(sV + C::KV_BYTES, C::BK * 128, 1024);
        const uint32_t tS = tmem + C::tm_s(t), tO = tmem + C::tm_o(t);
        uint64_t* s_full = &bars->s_full[t];
        uint64_t* p_full = &bars->p_full[t];
        int cq = 0, cp = 0, co = 0, g = 0;
        uint32_t fixed = 0;  // bit s: parity of the next v_fixed[s] phase
        bool ok = true;
        auto issue_s = [&](int slot) {
          const uint64_t db = slot ? dk1 : dk0;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::mma_bf16(tS, ptx::sdesc_advance(dq, (kk / 4) * (C::BQ * 128) + (kk % 4) * 32),
                          ptx::sdesc_advance(db, (kk / 4) * (C::BK * 128) + (kk % 4) * 32), idesc_s, kk > 0);
          ptx::mma_commit(s_full);
        };
        auto issue_pv = [&](int slot, bool first) {
          const uint64_t db = slot ? dv1 : dv0;
          ptx::mma_bf16_ts(tO, tS, db, idesc_o, !first);
#pragma unroll
          for (int kk = 1; kk < C::BK / 16; ++kk)
            ptx::mma_bf16_ts(tO, tS + kk * 8, ptx::sdesc_advance(db, kk * (16 * 128)), idesc_o, 1);
        };
        while (ok && w.next()) {
          const PagedTiles U = paged_tiles(p, w);
          if (U.u1 < U.u0) continue;
          const bool act_t = t ? U.act[1] : U.act[0];
          const int a_t = t ? U.a[1] : U.a[0];
          const int b_t = t ? U.b[1] : U.b[0];
          auto act = [&](int it) { return act_t && it >= a_t && it <= b_t; };
          const int g0 = g;
          auto slot = [&](int it) { return (g0 + it - U.u0) % C::NS; };
          auto ring_par = [&](int it) { return (uint32_t)(((g0 + it - U.u0) / C::NS) & 1); };
          if (act_t) ok = bar_wait(&bars->q_full[t], (cq++) & 1, abort_flag);
          bool first = true;
          ok = ok && bar_wait(&bars->k_full[slot(U.u0)], ring_par(U.u0), abort_flag);
          if (!ok) break;
          ptx::tc_fence_after();
          if (act(U.u0)) {
            issue_s(slot(U.u0));
            if (U.u0 == b_t) ptx::mma_commit(&bars->q_empty[t]);
          }
          for (int it = U.u0; ok && it <= U.u1; ++it) {
            const int s = slot(it);
            ok = bar_wait(&bars->v_full[s], ring_par(it), abort_flag);
            if (ok && paged_cut<C::TK>(w.it, it)) {
              ok = bar_wait(&bars->v_fixed[s], (fixed >> s) & 1, abort_flag);
              fixed ^= 1u << s;
            }
            if (!ok) break;
            if (act(it)) {
              // O_t += P_t V, then release the stage (this tile's reads of it are issued)
              ok = bar_wait(p_full, (cp++) & 1, abort_flag);
              if (ok && first) ok = bar_wait(&bars->o_free[t], ((co++) & 1) ^ 1, abort_flag);
              if (!ok) break;
              ptx::tc_fence_after();
              issue_pv(s, first);
              first = false;
              if (it == b_t) ptx::mma_commit(&bars->o_done[t]);
              ptx::mma_commit(&bars->kv_empty[s]);
            } else {
              ptx::mbar_arrive(&bars->kv_empty[s]);  // this tile does not use the stage
            }
            if (it + 1 <= U.u1) {
              ok = bar_wait(&bars->k_full[slot(it + 1)], ring_par(it + 1), abort_flag);
              if (!ok) break;
              ptx::tc_fence_after();
              if (act(it + 1)) {
                issue_s(slot(it + 1));
                if (it + 1 == b_t) ptx::mma_commit(&bars->q_empty[t]);
              }
            }
          }
          g = g0 + (U.u1 - U.u0 + 1);
        }
        // Exit path: every MMA this thread issued has completed.
        ptx::mma_commit(&bars->drain[t]);
        bar_drain(&bars->drain[t], 0);
      }
    }
    __syncwarp();
  } else {
    ptx::regs_inc<C::SOFTMAX_REGS>();
    // ------------------------------------------------------------ softmax warpgroups
    const int t = warp / 4;               // Q tile of this warpgroup
    const int r = threadIdx.x - 128 * t;  // row within the tile = TMEM lane
    const uint32_t lane_base = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t tS = tmem + lane_base + C::tm_s(t);
    const uint32_t tO = tmem + lane_base + C::tm_o(t);
    const float c2 = p.scale_log2;
    int cs = 0, cd = 0, job = -1, followers = 0;
    int turns = 0;  // waits on this warpgroup's turn barrier so far
    bool ok = true;
    while (ok && w.next()) {
      const PagedItem& it = w.it;
      const PagedTiles U = paged_tiles(p, w);
      const int32_t lo = p.lo[it.hg], hi = p.hi[it.hg];
      auto actv = [&](int tt, int kt) {
        return tt ? (U.act[1] && kt >= U.a[1] && kt <= U.b[1]) : (U.act[0] && kt >= U.a[0] && kt <= U.b[0]);
      };
      const bool act_t = t ? U.act[1] : U.act[0];
      const int a_t = t ? U.a[1] : U.a[0];
      const int b_t = t ? U.b[1] : U.b[0];
      const int rows_t = t ? U.rows[1] : U.rows[0];
      const int64_t pos_first = t ? U.pos[1] : U.pos[0], pos_last = t ? U.last[1] : U.last[0];
      const int64_t pos = pos_first + r / p.group;
      const bool live = r < rows_t;
      if (!w.whole && w.begins) {
        job = w.item;
        followers = (int)((it.cost - w.len + plan.run.run - 1) / plan.run.run);
      }
      const int64_t orow = paged_row(p, it, live ? t * 128 + r : 0);
      float* slot = paged_slot(p, blockIdx.x, w.begins, C::ROWS, D);
      float* slot_ml = slot + C::ROWS * D + t * 128 + r;
      if (!act_t) {
        // no key of this piece is attended to by this tile's rows
        if (live && w.whole) {
          uint16_t* dst = p.o + orow * D;
          for (int c = 0; c < D; c += 8) ptx::st_global_v4(dst + c, 0u, 0u, 0u, 0u);
          p.lse[orow] = -INFINITY;
        } else if (live) {
          slot_ml[0] = -INFINITY;
          slot_ml[C::ROWS] = 0.f;
        }
        continue;
      }
      // Running max (base-2 units) and sum.  Rows that do not exist start as if
      // they had seen a key, so that their warp can take the fast path.
      float m_ref = live ? -INFINITY : 0.f, l = 0.f;
      for (int kt = a_t; kt <= b_t; ++kt) {
        int prev;
        if (t == 1 && actv(0, kt)) prev = 0;
        else if (actv(1, kt - 1)) prev = 1;
        else if (actv(0, kt - 1)) prev = 0;
        else prev = -1;  // a piece's first step waits for no turn
        int nxt = -1;
        if (t == 0 && actv(1, kt)) nxt = 1;
        else if (actv(0, kt + 1)) nxt = 0;
        else if (actv(1, kt + 1)) nxt = 1;  // and a piece's last step passes none
        const bool pass_turn = nxt == 1 - t;
        const int64_t j0 = (int64_t)kt * C::BK;
        const bool interior = pos_first - (j0 + C::BK - 1) >= lo && pos_last - j0 < hi && j0 + C::BK <= it.kv;
        // otherwise this row's permitted keys are the columns clo .. clo + span
        int clo = 0;
        uint32_t span = 127;
        if (!interior) {
          const int64_t c_first = max64(pos - hi + 1 - j0, 0);
          const int64_t c_last = min64(min64(pos - lo - j0, it.kv - 1 - j0), 127);
          if (!live || c_last < c_first) {
            clo = 128;
            span = 0;
          } else {
            clo = (int)c_first;
            span = (uint32_t)(c_last - c_first);
          }
        }
        const bool fast = __all_sync(0xffffffffu, m_ref != -INFINITY);
        ok = __all_sync(0xffffffffu, bar_wait(&bars->s_full[t], (cs++) & 1, abort_flag));
        if (!ok) break;
        if (TURN && prev == 1 - t)
          ok = __all_sync(0xffffffffu, bar_wait(&bars->turn[t], (turns++) & 1, abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
        auto hand_turn = [&]() {
          if (TURN && pass_turn) ptx::mbar_arrive(&bars->turn[1 - t]);
        };
        // Fast path, for every tile after a row's first: exponentiate against
        // the current reference while tracking this tile's max; only if some
        // row's max rose past the reference by more than 2^8 is the tile done
        // again by the two-pass path (S is still intact then).
        bool done = false;
        if (fast) {
          const float2 c2v = make_float2(c2, c2);
          const float2 mnv = make_float2(-m_ref, -m_ref);
          float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
          float mx0 = -INFINITY, mx1 = -INFINITY;
          uint32_t pk[2][32];
          uint32_t sr[2][32];
          ptx::tmem_ld32(tS, sr[0]);
          ptx::tmem_wait_ld();
          ptx::reg_fence(sr[0]);
#define SPA_PAGED_FAST_CHUNKS(INTERIOR)                                                            \
  _Pragma("unroll") for (int q = 0; q < 4; ++q) {                                                  \
    if (q < 3) ptx::tmem_ld32(tS + (q + 1) * 32, sr[(q + 1) & 1]); /* next chunk in flight */      \
    const uint32_t* cur = sr[q & 1];                                                               \
    const int cb = q * 32 - clo;                                                                   \
    _Pragma("unroll") for (int e = 0; e < 32; e += 4) {                                            \
      float s0 = __uint_as_float(cur[e]), s1 = __uint_as_float(cur[e + 1]);                        \
      float s2 = __uint_as_float(cur[e + 2]), s3 = __uint_as_float(cur[e + 3]);                    \
      if (!(INTERIOR)) {                                                                           \
        s0 = (uint32_t)(cb + e) <= span ? s0 : -INFINITY;                                          \
        s1 = (uint32_t)(cb + e + 1) <= span ? s1 : -INFINITY;                                      \
        s2 = (uint32_t)(cb + e + 2) <= span ? s2 : -INFINITY;                                      \
        s3 = (uint32_t)(cb + e + 3) <= span ? s3 : -INFINITY;                                      \
      }                                                                                            \
      mx0 = ptx::fmax3(mx0, s0, s1);                                                               \
      mx1 = ptx::fmax3(mx1, s2, s3);                                                               \
      const float2 x01 = __ffma2_rn(make_float2(s0, s1), c2v, mnv);                                \
      const float2 x23 = __ffma2_rn(make_float2(s2, s3), c2v, mnv);                                \
      const float2 p01 = make_float2(ptx::exp2_approx(x01.x), ptx::exp2_approx(x01.y));            \
      const float2 p23 = make_float2(ptx::exp2_approx(x23.x), ptx::exp2_approx(x23.y));            \
      sa = __fadd2_rn(sa, p01);                                                                    \
      sb = __fadd2_rn(sb, p23);                                                                    \
      pk[q / 2][(q % 2) * 16 + e / 2] = E::pack(p01.x, p01.y);                                     \
      pk[q / 2][(q % 2) * 16 + e / 2 + 1] = E::pack(p23.x, p23.y);                                 \
    }                                                                                              \
    if (q < 3) {                                                                                   \
      ptx::tmem_wait_ld();                                                                         \
      ptx::reg_fence(sr[(q + 1) & 1]);                                                             \
    }                                                                                              \
  }
          if (interior) {
            SPA_PAGED_FAST_CHUNKS(true)
          } else {
            SPA_PAGED_FAST_CHUNKS(false)
          }
#undef SPA_PAGED_FAST_CHUNKS
          const bool over = live && fmaxf(mx0, mx1) * c2 > m_ref + 8.f;
          if (!__any_sync(0xffffffffu, over)) {
            hand_turn();
            ptx::tmem_st32(tS, pk[0]);
            ptx::tmem_st32(tS + 32, pk[1]);
            l += (sa.x + sa.y) + (sb.x + sb.y);
            done = true;
          }
        }
        if (!done) {
          // pass 1: row max of the raw scores (scale > 0 commutes with max)
          float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t sr[32];
            ptx::tmem_ld32(tS + q * 32, sr);
            ptx::tmem_wait_ld();
            ptx::reg_fence(sr);
            const int cb = q * 32 - clo;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              mx0 = fmaxf(mx0, (uint32_t)(cb + e) <= span ? __uint_as_float(sr[e]) : -INFINITY);
              mx1 = fmaxf(mx1, (uint32_t)(cb + e + 1) <= span ? __uint_as_float(sr[e + 1]) : -INFINITY);
            }
          }
          const float m_new = fmaxf(m_ref, fmaxf(mx0, mx1) * c2);
          const bool need = m_new > m_ref + 8.f;  // also true for a row's first finite max
          const bool need_o = need && (m_ref != -INFINITY);
          float alpha = 1.f;
          if (need) {
            alpha = ptx::exp2_approx(m_ref - m_new);  // 0 while the row had seen nothing
            l *= alpha;
            m_ref = m_new;
          }
          if (__any_sync(0xffffffffu, need_o)) {
            // O_t is stable: the PV of the previous key tile completed before S_t did
            const float a = need_o ? alpha : 1.f;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              ptx::tmem_ld32(tO + c, o);
              ptx::tmem_wait_ld();
              ptx::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
              ptx::tmem_st32(tO + c, o);
            }
          }
          // pass 2: p = exp2(s * scale_log2 - m), pairs over the first half of
          // S_t (chunk q of P covers columns [16q, 16q + 16), already read)
          const float mneg = (m_ref == -INFINITY) ? 0.f : -m_ref;
          float sm0 = 0.f, sm1 = 0.f;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            uint32_t sr[32], pk[16];
            ptx::tmem_ld32(tS + q * 32, sr);
            ptx::tmem_wait_ld();
            ptx::reg_fence(sr);
            const int cb = q * 32 - clo;
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0 = fmaf(__uint_as_float(sr[e]), c2, mneg), x1 = fmaf(__uint_as_float(sr[e + 1]), c2, mneg);
              x0 = (uint32_t)(cb + e) <= span ? x0 : -INFINITY;
              x1 = (uint32_t)(cb + e + 1) <= span ? x1 : -INFINITY;
              const float p0 = ptx::exp2_approx(x0), p1 = ptx::exp2_approx(x1);
              sm0 += p0;
              sm1 += p1;
              pk[e / 2] = E::pack(p0, p1);
            }
            ptx::tmem_st16(tS + q * 16, pk);
          }
          l += sm0 + sm1;
          hand_turn();
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bars->p_full[t]);
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      ok = __all_sync(0xffffffffu, bar_wait(&bars->o_done[t], (cd++) & 1, abort_flag));
      if (!ok) break;
      ptx::tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        ptx::tmem_ld32(tO + c, o);
        ptx::tmem_wait_ld();
        ptx::reg_fence(o);
        if (live && w.whole) {
          store_row32<E>(p.o + orow * D + c, o, inv);
        } else if (live) {
          float* dst = slot + (int64_t)(t * 128 + r) * D + c;
#pragma unroll
          for (int e = 0; e < 32; e += 8) ptx::st_global_v8(dst + e, o + e);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bars->o_free[t]);
      if (live && w.whole) {
        p.lse[orow] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
      } else if (live) {
        slot_ml[0] = m_ref;
        slot_ml[C::ROWS] = l;
      }
    }
    if (threadIdx.x == 0) paged_describe(p, ok ? job : -1, followers);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace spa
