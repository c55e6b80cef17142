// paged_long.cuh -- attention of many new tokens per sequence over a paged
// cache (the work list and the mask are in paged.cuh).
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
// Bound by the chain of one Q tile's step, S -> P -> O -> next S: 770 cycles to
// fetch the scores and find their max, 1440 for the exponentials (1024 of the
// special-function lanes), 1350 for the two products (2 x 512 of the tensor
// core, and the signals between them), against which the other tile's step is
// set.  4096 tokens of 32 heads over 16384 positions of one key/value head:
// 1215 TFLOP/s, 74 % of the measured bf16 rate (8 key/value heads, in a loop
// under the power cap: 970 to 1040).  Tried and slower there: 64-key
// tiles with S ahead of the softmax (the issuing thread's own instructions
// then take longer than the products: 970), a polynomial for part of the
// exponentials (more instructions than it saves lanes: 1130 at a quarter), the
// max beside the exponentials (spills: 1160).
#pragma once

#include "paged.cuh"

namespace spa {

// K and V have rings of their own: a K stage is free as soon as both tiles'
// S are done, a V stage after both tiles' O products, so that each is asked
// for about two steps before it is used (one ring for both, released after the
// O products, took 10 % longer over 16384 positions).
template <int D>
struct PagedLongCfg {
  static constexpr int ROWS = 256, TK = 128;
  static constexpr int BQ = 128, BK = TK, DB = D / 64;
  static constexpr int NK = D == 128 ? 3 : 4, NV = D == 128 ? 2 : 4;
  static constexpr uint32_t Q_BYTES = BQ * D * 2, KV_BYTES = BK * D * 2;
  static constexpr uint32_t OFF_Q = 0;
  static constexpr uint32_t OFF_K = OFF_Q + 2 * Q_BYTES;
  static constexpr uint32_t OFF_V = OFF_K + NK * KV_BYTES;
  static constexpr uint32_t OFF_BAR = OFF_V + NV * KV_BYTES;
  static constexpr uint32_t USED = OFF_BAR + 384;
  // at least 116 KB, so that one CTA (and its 512 TMEM columns) owns an SM
  static constexpr uint32_t SMEM_BYTES = USED + 1024 > 116u * 1024 ? USED + 1024 : 116u * 1024;
  static_assert(SMEM_BYTES <= kMaxSmemPerBlock, "shared memory");
  static constexpr int NTHREADS = 384;
  // register split (fwd.cuh): 168 per thread at launch
  static constexpr uint32_t LAUNCH_REGS = 168, SOFTMAX_REGS = 200, CONTROL_REGS = 104;
  static_assert(2 * SOFTMAX_REGS + CONTROL_REGS <= 3 * LAUNCH_REGS, "register split over budget");
  static constexpr uint32_t TMEM_COLS = 512;
  // tile t: S (and P over its first half) at t*256, O at t*256 + 128
  __host__ __device__ static constexpr uint32_t tm_s(int t) { return (uint32_t)(t * 256); }
  __host__ __device__ static constexpr uint32_t tm_o(int t) { return (uint32_t)t * 256u + 128u; }
};

struct PagedLongBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[4], k_empty[4];
  uint64_t v_full[4], v_empty[4];
  uint64_t v_fixed[4];   // the helper warp has cleared the rows outside the key range
  uint64_t s_full[2];
  uint64_t p_full[2][2];  // [tile][half of the keys]
  uint64_t o_done[2], o_free[2];
  uint64_t turn[2];       // turn[t]: softmax warpgroup t may form its exponentials
  uint64_t done[2][2];    // done[t][piece % 2]: warpgroup t is past its last turn of the piece
  uint64_t meet[2];       // warpgroup t's threads
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort;
  int last[2];            // warpgroup t's partial was its item's last to arrive
};
static_assert(sizeof(PagedLongBars) <= 384, "barrier space");

// A stage of a ring of N and the parity of its current phase.
template <int N>
struct RingSlot {
  int s = 0;
  uint32_t par = 0;
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      par ^= 1;
    }
  }
};

// One Q tile's part in a piece: its existing rows and its key tiles.
struct PagedTile {
  int rows;
  int a, b;  // b < a: no key of this piece is attended to
  int first_pos, last_pos;
  __device__ __forceinline__ bool has(int kt) const { return kt >= a && kt <= b; }
  __device__ __forceinline__ bool active() const { return b >= a; }
};

template <int TK>
__device__ __forceinline__ PagedTile paged_tile(const PagedParams& p, const PagedWalk<TK>& w, int t) {
  const PagedItem& it = w.it;
  const int per = 128 / p.group;  // tokens per Q tile
  const int tok = max(0, min(per, it.tokens - t * per));
  PagedTile U;
  U.rows = tok * p.group;
  U.first_pos = it.pos0 + t * per;
  U.last_pos = U.first_pos + tok - 1;
  const int64_t jlo = max64(0, (int64_t)U.first_pos - p.hi[it.hg] + 1);
  const int64_t jhi = min64((int64_t)U.last_pos - p.lo[it.hg], it.kv - 1);
  U.a = 1;
  U.b = 0;
  if (tok > 0 && jhi >= jlo) {
    U.a = max((int)(jlo / TK), w.t0);
    U.b = min((int)(jhi / TK), w.t1 - 1);
  }
  return U;
}

// The item's key range cuts tile `t`: some of its rows are not to be used.
template <int TK>
__device__ __forceinline__ bool paged_cut(const PagedItem& it, int t) {
  return t * TK < it.jlo || t * TK > it.jhi - (TK - 1);
}

// Scores of 32 columns that lie outside [lo, hi] (counted from the first of
// them) become -inf.
__device__ __forceinline__ void paged_mask32(uint32_t (&s)[32], int lo, int hi) {
  const uint32_t from = lo > 31 ? 0u : 0xffffffffu << max(lo, 0);
  const uint32_t to = hi < 0 ? 0u : 0xffffffffu >> (31 - min(hi, 31));
  const uint32_t keep = from & to;
#pragma unroll
  for (int e = 0; e < 32; ++e) s[e] = (keep >> e) & 1 ? s[e] : 0xff800000u;
}

// p = 2^(s c2 + mneg) of 32 scores as 16-bit pairs; adds them up in fp32.
// P is rounded once, as in the training forward.  That adds to o about the error
// of its own rounding: against fp64, o is off by 2.3e-3 of its norm in bf16 where
// rounding o alone gives 1.65e-3, and by 2.0e-4 against 1.5e-4 in fp16.  The
// second term that the kernel for few rows carries would cost half the products
// again here, where the products bound the step.
template <class E>
__device__ __forceinline__ void paged_exp32(const uint32_t (&s)[32], float2 c2v, float2 mnv, float2& sa, float2& sb,
                                            uint32_t (&pk)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), c2v, mnv);
    const float2 y = make_float2(ptx::exp2_approx(x.x), ptx::exp2_approx(x.y));
    if (e & 1) sb = __fadd2_rn(sb, y);
    else sa = __fadd2_rn(sa, y);
    pk[e] = E::pack(y.x, y.y);
  }
}

// One thread joins row r of an item from its pieces' partials, in their order
// (paged_join_row's sums over the layout of this kernel's partials).
template <class E, int D, int ROWS>
__device__ __forceinline__ void paged_join_thread(const PagedParams& p, int head, int pieces, int r, int64_t row) {
  float mx = -INFINITY;
  for (int i = 0; i < pieces; ++i) mx = ptx::fmax_nan(mx, paged_slot(p, head, i, ROWS, D)[ROWS * D + r]);
  float sum = 0.f, out[D];
#pragma unroll
  for (int e = 0; e < D; ++e) out[e] = 0.f;
  for (int i = 0; i < pieces; ++i) {
    const float* slot = paged_slot(p, head, i, ROWS, D);
    const float m = slot[ROWS * D + r];
    if (m == -INFINITY) continue;  // the row attends to nothing in this piece
    const float f = ptx::exp2_approx(m - mx);
    sum = fmaf(slot[ROWS * D + ROWS + r], f, sum);
#pragma unroll
    for (int e = 0; e < D; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(slot + (e / 8) * (8 * ROWS) + r * 8 + e % 8);
      out[e] = fmaf(f, v.x, out[e]);
      out[e + 1] = fmaf(f, v.y, out[e + 1]);
      out[e + 2] = fmaf(f, v.z, out[e + 2]);
      out[e + 3] = fmaf(f, v.w, out[e + 3]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* dst = p.o + row * D;
#pragma unroll
  for (int c = 0; c < D; c += 32) {
    uint32_t g[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) g[e] = __float_as_uint(out[c + e]);
    store_row32<E>(dst + c, g, inv);
  }
  p.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
}

template <class E, int D>
__global__ void __launch_bounds__(384, 1)
    spa_paged_long_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedParams p) {
  using C = PagedLongCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  if (!smem_fits(smem_raw, smem, C::USED)) return;
  PagedLongBars* bars = reinterpret_cast<PagedLongBars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t sQ = ptx::smem_u32(smem + C::OFF_Q);
  const uint32_t sK = ptx::smem_u32(smem + C::OFF_K);
  const uint32_t sV = ptx::smem_u32(smem + C::OFF_V);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars->q_full[i], 1);
      ptx::mbar_init(&bars->q_empty[i], 1);
      ptx::mbar_init(&bars->s_full[i], 1);
      ptx::mbar_init(&bars->p_full[i][0], 128);
      ptx::mbar_init(&bars->p_full[i][1], 128);
      ptx::mbar_init(&bars->o_done[i], 1);
      ptx::mbar_init(&bars->o_free[i], 128);
      ptx::mbar_init(&bars->turn[i], 128);
      ptx::mbar_init(&bars->done[i][0], 128);
      ptx::mbar_init(&bars->done[i][1], 128);
      ptx::mbar_init(&bars->meet[i], 128);
      ptx::mbar_init(&bars->drain[i], 1);
    }
    for (int i = 0; i < C::NK; ++i) {
      ptx::mbar_init(&bars->k_full[i], 1);
      ptx::mbar_init(&bars->k_empty[i], 2);  // one release per MMA issuer
    }
    for (int i = 0; i < C::NV; ++i) {
      ptx::mbar_init(&bars->v_full[i], 1);
      ptx::mbar_init(&bars->v_fixed[i], 1);
      ptx::mbar_init(&bars->v_empty[i], 3);  // one release per MMA issuer, one of the helper's
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
  __syncthreads();
  ptx::tc_fence_after();
  // The lengths are asked for while the plan is made (they are inputs, written
  // before it began), so that the walk finds them near.
  if ((int)threadIdx.x <= p.B) ptx::prefetch_l1(p.cu_q + threadIdx.x), ptx::prefetch_l1(p.kv_len + min((int)threadIdx.x, p.B - 1));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort;
  PagedWalk<C::TK> w(p, PagedRun(p));

  if (warp >= 8) {
    ptx::regs_dec<C::CONTROL_REGS>();
    if (warp == 11) {
      // ---------------------------------------------------------- helper: clears unused V rows
      // It follows every tile, cut or not, and releases the stage like an MMA
      // issuer, so that the waits on v_full keep step with its phases.
      RingSlot<C::NV> v;
      bool ok = true;
      while (ok && w.next()) {
        const PagedItem& it = w.it;
        for (int t = w.t0; t < w.t1; ++t, v.next()) {
          ok = __all_sync(0xffffffffu, bar_wait(&bars->v_full[v.s], v.par, abort_flag));
          if (!ok) break;
          const bool cut = paged_cut<C::TK>(it, t);
          if (cut) {
            const int j0 = t * C::TK;
            const int first = min(max(it.jlo - j0, 0), C::TK);    // rows [0, first) and
            const int end = min(max(it.jhi + 1 - j0, 0), C::TK);  // [end, TK) are not used
            const int n = first + (C::TK - end);
            for (int e = lane; e < n * 8; e += 32) {
              const int r = e / 8 < first ? e / 8 : end + e / 8 - first;
#pragma unroll
              for (int c = 0; c < C::DB; ++c)
                ptx::st_shared_v4(sV + v.s * C::KV_BYTES + c * (C::BK * 128) + r * 128 + (e % 8) * 16, 0u, 0u, 0u, 0u);
            }
            ptx::fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            if (cut) ptx::mbar_arrive(&bars->v_fixed[v.s]);
            ptx::mbar_arrive(&bars->v_empty[v.s]);
          }
        }
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- TMA producer
      // Asks for K of a tile one step ahead of V of the tile before.
      const int box_shift = min(p.page_shift, 7), boxes = C::TK >> box_shift;
      const int box_i = lane % boxes, cb = lane / boxes;  // box, 64-column block
      PagedPages pages;
      RingSlot<C::NK> k;
      RingSlot<C::NV> v;
      int nq[2] = {0, 0}, nk = 0, nv = 0;
      bool ok = true;
      while (ok && w.next()) {
        const PagedItem& it = w.it;
        const int hk = it.hg / p.kv_div;
        if (lane == 0 && p.kv_len[it.b] > it.kv) report_status(kStatusInval);
        // one 128-key tile of K or V into a stage, a box per page and 64 columns
        auto fetch = [&](const CUtensorMap* map, uint32_t at, uint64_t* bar, int t, int id) {
          if (lane == 0) ptx::mbar_arrive_expect_tx(bar, C::KV_BYTES);
          __syncwarp();
          if (cb < C::DB) {
            const int j = (t * boxes + box_i) << box_shift;
            ptx::tma_load_3d(smem + at + cb * (C::BK * 128) + (box_i << box_shift) * 128, map, bar, cb * 64,
                             j & ((1 << p.page_shift) - 1), id < 0 ? -1 : id * p.Hk + hk);
          }
          __syncwarp();
        };
        int id_v = -1;
        for (int t = w.t0; t <= w.t1; ++t) {
          int id = -1;
          if (t < w.t1) {
            id = pages.get(p, it, (int64_t)t * boxes, box_shift, boxes, box_i, t == w.t0);
            ok = __all_sync(0xffffffffu, bar_wait(&bars->k_empty[k.s], k.par ^ 1, abort_flag));
            if (!ok) break;
            fetch(&tm_k, C::OFF_K + k.s * C::KV_BYTES, &bars->k_full[k.s], t, id);
            k.next();
            ++nk;
            if (t == w.t0) {
              // Q after the first K: its buffers are free only when the piece
              // before has done its last S
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                if (!ok || !paged_tile(p, w, x).active()) continue;
                ok = __all_sync(0xffffffffu, bar_wait(&bars->q_empty[x], (nq[x] & 1) ^ 1, abort_flag));
                if (!ok) continue;
                ++nq[x];
                if (lane == 0) {
                  ptx::mbar_arrive_expect_tx(&bars->q_full[x], C::Q_BYTES);
                  for (int c = 0; c < C::DB; ++c)
                    ptx::tma_load_4d(smem + C::OFF_Q + x * C::Q_BYTES + c * (C::BQ * 128), &tm_q, &bars->q_full[x],
                                     c * 64, 0, it.hg, it.row0 + x * (128 / p.group));
                }
              }
              if (!ok) break;
            }
          }
          if (t > w.t0) {
            ok = __all_sync(0xffffffffu, bar_wait(&bars->v_empty[v.s], v.par ^ 1, abort_flag));
            if (!ok) break;
            fetch(&tm_v, C::OFF_V + v.s * C::KV_BYTES, &bars->v_full[v.s], t - 1, id_v);
            v.next();
            ++nv;
          }
          id_v = id;
        }
      }
      // (here, where nothing waits for its loads)
      if (blockIdx.x == 0 && lane == 0) report_missing_rows(p.cu_q, p.B, p.T);
      // Exit path: every load this warp issued has landed before the CTA ends.
      if (lane == 0) {
        for (int t = 0; t < 2; ++t)
          if (nq[t] > 0) bar_drain(&bars->q_full[t], (nq[t] - 1) & 1);
        for (int s = 0; s < C::NK; ++s) {
          const int used = (nk + C::NK - 1 - s) / C::NK;
          if (used > 0) bar_drain(&bars->k_full[s], (used - 1) & 1);
        }
        for (int s = 0; s < C::NV; ++s) {
          const int used = (nv + C::NV - 1 - s) / C::NV;
          if (used > 0) bar_drain(&bars->v_full[s], (used - 1) & 1);
        }
      }
    } else {
      // ---------------------------------------------------------- MMA issuers
      // warp 9 issues every MMA of Q tile 0, warp 10 those of Q tile 1; both
      // walk the piece's whole key range, so they agree on the rings
      const int t = warp - 9;
      if (lane == 0) {
        constexpr uint32_t idesc_s = ptx::idesc_16_f32(E::kMmaFormat, 128, C::BK, false, false);
        constexpr uint32_t idesc_o = ptx::idesc_16_f32(E::kMmaFormat, 128, D, false, true);
        const uint64_t dq = ptx::sdesc_sw128(sQ + t * C::Q_BYTES, 0, 1024);
        const uint64_t dk = ptx::sdesc_sw128(sK, 0, 1024), dv = ptx::sdesc_sw128(sV, C::BK * 128, 1024);
        const uint32_t tO = tmem + C::tm_o(t);
        const uint32_t tS = tmem + C::tm_s(t);
        uint64_t* s_full = &bars->s_full[t];
        RingSlot<C::NK> k;
        RingSlot<C::NV> v;
        int cq = 0, co = 0;
        uint32_t cp = 0;     // parity of the next P
        uint32_t fixed = 0;  // bit s: parity of the next v_fixed[s] phase
        bool ok = true;
        auto wait_k = [&]() { ok = ok && bar_wait(&bars->k_full[k.s], k.par, abort_flag); };
        auto wait_v = [&](int kt) {
          ok = ok && bar_wait(&bars->v_full[v.s], v.par, abort_flag);
          if (ok && paged_cut<C::TK>(w.it, kt)) {
            ok = bar_wait(&bars->v_fixed[v.s], (fixed >> v.s) & 1, abort_flag);
            fixed ^= 1u << v.s;
          }
        };
        auto issue_s = [&]() {
          const uint64_t db = ptx::sdesc_advance(dk, k.s * C::KV_BYTES);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::mma_bf16(tS, ptx::sdesc_advance(dq, (kk / 4) * (C::BQ * 128) + (kk % 4) * 32),
                          ptx::sdesc_advance(db, (kk / 4) * (C::BK * 128) + (kk % 4) * 32), idesc_s, kk > 0);
          ptx::mma_commit(s_full);
          ptx::mma_commit(&bars->k_empty[k.s]);
          k.next();
        };
        auto skip = [&](int kt) {  // a key tile that this Q tile does not use
          wait_k();
          if (ok) ptx::mbar_arrive(&bars->k_empty[k.s]);
          k.next();
          wait_v(kt);
          if (ok) ptx::mbar_arrive(&bars->v_empty[v.s]);
          v.next();
        };
        while (ok && w.next()) {
          if (w.t1 <= w.t0) continue;
          const PagedTile U = paged_tile(p, w, t);
          const int a = U.active() ? U.a : w.t1, b = U.active() ? U.b : w.t1 - 1;
          for (int kt = w.t0; ok && kt < a; ++kt) skip(kt);
          if (U.active()) {
            ok = ok && bar_wait(&bars->q_full[t], (cq++) & 1, abort_flag);
            wait_k();
            if (!ok) break;
            ptx::tc_fence_after();
            issue_s();
            if (a == b) ptx::mma_commit(&bars->q_empty[t]);
            for (int kt = a; kt <= b; ++kt) {
              // Everything else that the next products need is waited for before
              // P, so that they follow one another without a pause.
              if (kt < b) wait_k();
              wait_v(kt);
              if (kt == a) ok = ok && bar_wait(&bars->o_free[t], ((co++) & 1) ^ 1, abort_flag);
              const uint64_t db = ptx::sdesc_advance(dv, v.s * C::KV_BYTES);
              // O_t += P_t V, each half of the keys as soon as its P is there
              ok = ok && bar_wait(&bars->p_full[t][0], cp, abort_flag);
              if (!ok) break;
              ptx::tc_fence_after();
              ptx::mma_bf16_ts(tO, tS, db, idesc_o, kt != a);
#pragma unroll
              for (int kk = 1; kk < C::BK / 32; ++kk)
                ptx::mma_bf16_ts(tO, tS + kk * 8, ptx::sdesc_advance(db, kk * (16 * 128)), idesc_o, 1);
              ok = bar_wait(&bars->p_full[t][1], cp, abort_flag);
              if (!ok) break;
              ptx::tc_fence_after();
#pragma unroll
              for (int kk = C::BK / 32; kk < C::BK / 16; ++kk)
                ptx::mma_bf16_ts(tO, tS + kk * 8, ptx::sdesc_advance(db, kk * (16 * 128)), idesc_o, 1);
              cp ^= 1;
              if (kt < b) {
                issue_s();
                if (kt + 1 == b) ptx::mma_commit(&bars->q_empty[t]);
              } else {
                ptx::mma_commit(&bars->o_done[t]);
              }
              ptx::mma_commit(&bars->v_empty[v.s]);
              v.next();
            }
          }
          for (int kt = b + 1; ok && kt < w.t1; ++kt) skip(kt);
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
    const uint32_t tS = tmem + lane_base + C::tm_s(t), tO = tmem + lane_base + C::tm_o(t);
    const float c2 = p.scale_log2;
    int cs = 0, cd = 0, met = 0;
    // The two warpgroups take turns at the exponentials, so that one's overlap
    // the tensor core's work for the other (left to themselves they run side by
    // side, share the special-function lanes and then wait for the tensor core
    // together).  Order: (kt, tile 0), (kt, tile 1), (kt + 1, tile 0) ..; at every
    // change of owner the finishing warpgroup arrives on the other's turn
    // barrier.  Turns are passed and taken within a piece; a piece is begun when
    // the other warpgroup is past its last turn of the piece before, so that no
    // pass can run ahead of its take.
    int turns = 0;  // waits on this warpgroup's turn barrier so far
    int n = 0;      // pieces so far
    bool ok = true;
    for (; ok && w.next(); ++n) {
      if (n > 0)
        ok = __all_sync(0xffffffffu, bar_wait(&bars->done[1 - t][(n - 1) & 1], ((n - 1) >> 1) & 1, abort_flag));
      if (!ok) break;
      const PagedItem& it = w.it;
      const PagedTile U = paged_tile(p, w, t), V = paged_tile(p, w, 1 - t);  // this tile, the other
      const bool live = r < U.rows;
      // this row's place in a partial: 8 columns of all rows after one another,
      // so that 32 rows' 32-byte vectors lie side by side
      const int head = w.whole ? 0 : w.head();
      float* slot = paged_slot(p, head, blockIdx.x - head, C::ROWS, D) + (t * 128 + r) * 8;
      float* slot_ml = paged_slot(p, head, blockIdx.x - head, C::ROWS, D) + C::ROWS * D + t * 128 + r;
      const int64_t row = paged_row(p, it, live ? t * 128 + r : 0);
      // leaves the item's partial; whoever leaves the last joins them all
      auto leave = [&]() {
        __threadfence();
        ptx::mbar_arrive(&bars->meet[t]);
        ok = __all_sync(0xffffffffu, bar_wait(&bars->meet[t], (met++) & 1, abort_flag));
        if (ok && r == 0) bars->last[t] = atomicAdd(&p.arrived[2 * head + t], 1) == w.pieces() - 1;
        ptx::mbar_arrive(&bars->meet[t]);
        ok = __all_sync(0xffffffffu, ok && bar_wait(&bars->meet[t], (met++) & 1, abort_flag));
        if (!ok || !*(volatile int*)&bars->last[t]) return;
        __threadfence();
        if (live) paged_join_thread<E, D, C::ROWS>(p, head, w.pieces(), t * 128 + r, row);
      };
      if (!U.active()) {
        // no key of this piece is attended to by this tile's rows
        ptx::mbar_arrive(&bars->done[t][n & 1]);
        if (live && w.whole) {
          uint16_t* dst = p.o + row * D;
          for (int c = 0; c < D; c += 8) ptx::st_global_v4(dst + c, 0u, 0u, 0u, 0u);
          p.lse[row] = -INFINITY;
        } else if (live) {
          slot_ml[0] = -INFINITY;
          slot_ml[C::ROWS] = 0.f;
        }
        if (!w.whole) leave();
        continue;
      }
      // this row's permitted keys [row_lo, row_hi]; key tiles starting in
      // [in_lo, in_hi] are permitted to every row of the tile
      int row_lo, row_hi, in_lo, in_hi;
      {
        const int64_t lo = p.lo[it.hg], hi = p.hi[it.hg], pos = (int64_t)U.first_pos + r / p.group;
        row_lo = (int)max64(pos - hi + 1, 0);
        row_hi = live ? clamp_i32(min64(pos - lo, it.kv - 1)) : -1;
        in_lo = (int)max64(U.last_pos - hi + 1, 0);
        in_hi = clamp_i32(min64(U.first_pos - lo, it.kv - 1) - (C::BK - 1));
      }
      // Running max (base-2 units) and sum.  Rows that do not exist start as if
      // they had seen a key, so that their warp can take the fast path.
      float m_ref = live ? -INFINITY : 0.f, l = 0.f;
      for (int kt = U.a; kt <= U.b; ++kt) {
        const int other = kt + t;  // the next step's key tile if the other tile owns it
        const bool take_turn = V.has(other - 1), pass_turn = V.has(other);
        const int j0 = kt * C::BK;
        ok = __all_sync(0xffffffffu, bar_wait(&bars->s_full[t], (cs++) & 1, abort_flag));
        if (!ok) break;
        ptx::tc_fence_after();
        uint32_t s[4][32];  // the row's scores
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::tmem_ld32(tS + q * 32, s[q]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::reg_fence(s[q]);
        if (j0 < in_lo || j0 > in_hi) {
          // the columns of this row's permitted keys: [row_lo - j0, row_hi - j0]
#pragma unroll
          for (int q = 0; q < 4; ++q) paged_mask32(s[q], row_lo - j0 - 32 * q, row_hi - j0 - 32 * q);
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; e += 2)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            m4[q] = ptx::fmax3_nan(m4[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
        const float mx = ptx::fmax_nan(ptx::fmax3_nan(m4[0], m4[1], m4[2]), m4[3]) * c2;
        // The reference moves when a row sees its first key, and afterwards only
        // when the row's max rises past it by more than 2^8 (P stays below 2^8),
        // so that O is rescaled rarely.  A row that has seen no key uses 0.
        const bool moves = live && mx > m_ref + 8.f;  // also from -inf
        if (mx != mx) l = mx;  // a score that is no number: nor are o and lse
        if (__any_sync(0xffffffffu, moves)) {
          float alpha = 1.f;
          if (moves) {
            alpha = ptx::exp2_approx(m_ref - mx);  // 0 while the row had seen nothing
            m_ref = mx;
            l *= alpha;
          }
          if (kt > U.a) {
            // O_t is stable: the product before this tile completed before S_t did
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              ptx::tmem_ld16(tO + c, o);
              ptx::tmem_wait_ld();
              ptx::reg_fence(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              ptx::tmem_st16(tO + c, o);
            }
          }
        }
        if (take_turn) ok = __all_sync(0xffffffffu, bar_wait(&bars->turn[t], (turns++) & 1, abort_flag));
        if (!ok) break;
        // P over the first half of S, 16-bit pairs
        const float mneg = m_ref == -INFINITY ? 0.f : -m_ref;
        const float2 c2v = make_float2(c2, c2), mnv = make_float2(mneg, mneg);
        float2 sa = make_float2(0.f, 0.f), sb = make_float2(0.f, 0.f);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pk[16];
          if (q == 3 && pass_turn) ptx::mbar_arrive(&bars->turn[1 - t]);  // the other may start up
          paged_exp32<E>(s[q], c2v, mnv, sa, sb, pk);
          if (q == 2) {  // the first half has been stored meanwhile
            ptx::tmem_wait_st();
            ptx::tc_fence_before();
            ptx::mbar_arrive(&bars->p_full[t][0]);
          }
          ptx::tmem_st16(tS + q * 16, pk);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bars->p_full[t][1]);
        l += (sa.x + sa.y) + (sb.x + sb.y);
      }
      if (!ok) break;
      ptx::mbar_arrive(&bars->done[t][n & 1]);
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
          store_row32<E>(p.o + row * D + c, o, inv);
        } else if (live) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) ptx::st_global_v8(slot + (c + e) * C::ROWS, o + e);
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bars->o_free[t]);
      if (live && w.whole) {
        p.lse[row] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.69314718055994531f;
      } else if (live) {
        slot_ml[0] = l == l ? m_ref : l;  // (no number stays seen)
        slot_ml[C::ROWS] = l;
      }
      if (!w.whole) leave();
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

}  // namespace spa
