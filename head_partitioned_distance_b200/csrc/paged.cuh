// paged.cuh -- attention of new tokens over a paged cache, each head over its
// own band of causal distances: the work list shared by its kernels, the
// kernel for few rows per sequence (single tokens above all), and the joining
// of items whose keys were divided.  The kernel for many rows: paged_long.cuh.
//
// Row r of sequence b stands at position p = kv_len[b] - n_b + r and attends
// to the keys j < kv_len[b] with lo_h <= p - j < hi_h ("Making Every Head
// Count", Figure 1 caption, the bands; softmax over the permitted set: "Story
// of Attention -- Part 4", section 1).
//
// Work list.  An item is (sequence, head group, row block); a head group is
// `group` query heads that share a key/value head and, when group > 1, one
// band, so that each key is fetched once for all of them.  All items laid end
// to end, each as long as its key tiles plus what beginning and ending a piece
// costs, form one line that is cut into equal runs, one per CTA: sequences of
// any mixture of lengths load every SM alike, and a long sequence with few
// rows is spread over many SMs.  A plan kernel finds the cuts from the lengths
// on the device, so the host needs none of them and a captured call follows
// them.  An item that a cut divides leaves one partial (fp32 o, running max
// and sum) per piece; whoever leaves the last joins them all, in their order,
// so the result does not depend on which was last.
#pragma once

#include "common.cuh"
#include "elem.cuh"

namespace spa {

struct PagedParams {
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
  const uint16_t* q;  // [T][Hq][d]
  uint16_t* o;        // [T][Hq][d]
  float* lse;         // [T][Hq]
  int4* plan;         // PagedCut of every CTA and of the end; null: CTA i has item i
  int32_t* arrived;   // pieces that have left their partial, by the CTA that began the item (x 2 row halves)
  float* part;        // two partial slots per CTA
  int64_t pages;
  int B, T, Hq, max_q;
  int group;          // query heads per item
  int ng;             // head groups: Hq / group
  int kv_div;         // head groups per key/value head
  int Hk;
  int nblk;           // row blocks per (sequence, head group)
  int blk_tokens;     // tokens per row block
  int width, page_shift;
  int ctas;           // runs the line is cut into, at most
  int piece_cost;     // cost of a piece besides its key tiles, in key tiles
  int split_cost;     // what it costs that an item is divided, in key tiles
  int min_run;        // length of a run, at least
  int max_split;      // pieces of an item, about
  float scale_log2;
  int32_t lo[kMaxHeads];  // per head group
  int32_t hi[kMaxHeads];
};

struct PagedItem {
  int b, hg;
  int row0;      // first token row
  int tokens;    // token rows; 0: nothing to do
  int pos0;      // position of the first
  int jlo, jhi;  // keys that some row attends to (jhi < jlo: none)
  int kv;        // keys the sequence has (and the page table can name)
  int t0;        // first key tile
  int cost;      // key tiles; an item without keys counts one, one without rows none
  int next;      // without rows: how far on the next item is that may have some
};

// Positions and lengths are 32-bit; sums of them with band limits need more.
__device__ __forceinline__ int clamp_i32(int64_t v) { return (int)max64(min64(v, 2147483647LL), -2147483648LL); }

template <int TK>
__device__ __forceinline__ PagedItem paged_item(const PagedParams& p, int b, int hg, int blk) {
  PagedItem it;
  it.b = b;
  it.hg = hg;
  const int c0 = p.cu_q[b], n_all = p.cu_q[b + 1] - c0;
  const int len = p.kv_len[b];
  const int n = (c0 < 0 || c0 >= p.T) ? 0 : min(min(n_all, p.max_q), p.T - c0);
  const int first = blk * p.blk_tokens;
  it.row0 = c0 + first;
  it.tokens = max(0, min(p.blk_tokens, n - first));
  const int64_t pos0 = (int64_t)len - n_all + first;
  it.pos0 = clamp_i32(pos0);
  it.kv = (int)min64(max(len, 0), (int64_t)p.width << p.page_shift);
  it.jlo = (int)max64(0, pos0 - p.hi[hg] + 1);
  it.jhi = clamp_i32(min64(pos0 + it.tokens - 1 - p.lo[hg], it.kv - 1));
  const bool any = it.tokens > 0 && it.jhi >= it.jlo;
  it.t0 = any ? it.jlo / TK : 0;
  it.cost = it.tokens == 0 ? 0 : any ? it.jhi / TK - it.t0 + 1 : 1;
  // A head group's row blocks behind an empty one are empty too, and a sequence
  // without rows has none at all.  (Taken one by one, at 0.17 us each, they
  // could cost more than the attention: a prompt of 8192 tokens gives every
  // sequence of its batch 128 blocks per head group, and with 15 single tokens
  // took 3.1 ms instead of 0.5; and over tens of thousands of sequences one
  // role's steps could have outlasted another's wait.)
  it.next = (n > 0 ? p.nblk : (p.ng - hg) * p.nblk) - blk;
  return it;
}

template <int TK>
__device__ __forceinline__ PagedItem paged_item_at(const PagedParams& p, int item) {
  const int blk = item % p.nblk, rest = item / p.nblk;
  return paged_item<TK>(p, rest / p.ng, rest % p.ng, blk);
}

// Where a CTA's run begins: key tile `off` of an item (0: the item is whole
// from there on).  off > 0: CTA `head` began the item, which has `pieces`.
struct PagedCut {
  int item, off, head, pieces;
};

constexpr int kPagedPlanThreads = 512;
constexpr int kPagedMaxCtas = 296;

// One CTA.  Cuts the line into ctas runs and clears the arrival counts.  Every
// thread sums a share of the items; after a scan it knows where its share lies
// in the line and places the cuts that fall into it.  First at the nearest
// ends of items: where the longest run is then no longer than an even run and
// what dividing items costs, no item is divided.
template <int TK>
__global__ void __launch_bounds__(kPagedPlanThreads) spa_paged_plan_kernel(const __grid_constant__ PagedParams p) {
  constexpr int kWarps = kPagedPlanThreads / 32;
  __shared__ long long s_sum[kWarps];
  __shared__ int s_most[kWarps], s_end[kWarps];
  __shared__ int s_item[kPagedMaxCtas + 1], s_off[kPagedMaxCtas + 1];
  __shared__ long long s_at[kPagedMaxCtas + 1];  // where the cuts at ends of items lie
  // the kernel that follows may be launched: it waits for this one to end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int items = p.B * p.ng * p.nblk;
  const int per = (items + kPagedPlanThreads - 1) / kPagedPlanThreads;
  const int i0 = min((int)threadIdx.x * per, items), i1 = min(i0 + per, items);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  int step;  // from the item last asked for to the next that may have rows
  auto length = [&](int i) {
    const PagedItem it = paged_item_at<TK>(p, i);
    step = it.cost ? 1 : it.next;
    return it.cost ? it.cost + p.piece_cost : 0;
  };
  for (int c = threadIdx.x; c < 2 * p.ctas; c += kPagedPlanThreads) p.arrived[c] = 0;
  long long mine = 0;
  int most = 0, only = 0, end = 0;  // end: behind the last item with rows
  for (int i = i0; i < i1; i += step) {
    only = length(i);
    mine += only;
    most = max(most, only);
    end = only ? i + 1 : end;
  }
  long long incl = mine;
#pragma unroll
  for (int m = 1; m < 32; m *= 2) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += v;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  end = __reduce_max_sync(0xffffffffu, end);
  if (lane == 31) s_sum[warp] = incl;
  if (lane == 0) s_most[warp] = most, s_end[warp] = end;
  __syncthreads();
  long long before = incl - mine, total = 0;
  most = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
    most = max(most, s_most[w]);
    end = max(end, s_end[w]);
  }
  long long run = total < 2147483647LL - p.ctas ? (long long)(((uint32_t)total + p.ctas - 1) / (uint32_t)p.ctas)
                                                : (total + p.ctas - 1) / p.ctas;
  run = max(run, (long long)((most + p.max_split - 1) / p.max_split));
  run = max(run, (long long)p.min_run);
  // the first cut at or behind the share's beginning
  const int c0 = before + run < 2147483647LL ? (int)(((uint32_t)before + (uint32_t)run - 1) / (uint32_t)run)
                                             : (int)((before + run - 1) / run);
  auto place_cuts = [&](bool divide) {
    int c = c0;
    long long at = run * c, x = before;
    for (int i = i0; i < i1 && at < before + mine; i += step) {
      const int len = per == 1 ? only : length(i);
      for (; at < x + len && c <= p.ctas; at += run, ++c) {
        // a piece of no or one key tile is not worth its beginning: the cut
        // moves to the item's start or end
        const int off = (int)(at - x) - p.piece_cost;
        const bool start = divide ? off < 2 : 2 * (at - x) < len;
        const bool end = !start && (!divide || len - p.piece_cost - off < 2);
        s_item[c] = end ? i + 1 : i;
        s_off[c] = start || end ? 0 : off;
        s_at[c] = end ? x + len : x;
      }
      x += len;
    }
  };
  for (int c = threadIdx.x; c <= p.ctas; c += kPagedPlanThreads)
    if (run * c >= total) {
      s_item[c] = end;  // what has no rows behind that is nobody's
      s_off[c] = 0;
      s_at[c] = total;
    }
  place_cuts(false);
  __syncthreads();
  if (__syncthreads_or((int)threadIdx.x < p.ctas &&
                       s_at[threadIdx.x + 1] - s_at[threadIdx.x] > run + p.split_cost))
    place_cuts(true);
  __syncthreads();
  if ((int)threadIdx.x <= p.ctas) {
    // the cuts within the same item, by bisection: (item, off > 0) never falls
    const int c = threadIdx.x, item = s_item[c], off = s_off[c];
    int first = c, last = c;
    if (off > 0) {
      int a = -1;  // the last cut before them
      for (int hi = c; hi - a > 1;) {
        const int m = (a + hi) / 2;
        if (s_item[m] == item && s_off[m] > 0) hi = m;
        else a = m;
      }
      first = a + 1;
      int b = p.ctas + 1;  // the first cut behind them
      for (int lo = c; b - lo > 1;) {
        const int m = (lo + b) / 2;
        if (s_item[m] == item && s_off[m] > 0) lo = m;
        else b = m;
      }
      last = b - 1;
    }
    p.plan[c] = make_int4(item, off, first - 1, last - first + 2);
  }
}

// This CTA's run: from its cut to the next.
struct PagedRun {
  PagedCut from, to;
  __device__ __forceinline__ explicit PagedRun(const PagedParams& p) {
    if (!p.plan) {  // one whole item per CTA
      from = {(int)blockIdx.x, 0, 0, 0};
      to = {(int)blockIdx.x + 1, 0, 0, 0};
      return;
    }
    const int4 a = p.plan[blockIdx.x], b = p.plan[blockIdx.x + 1];
    from = {a.x, a.y, a.z, a.w};
    to = {b.x, b.y, b.z, b.w};
  }
};

// The pieces of a CTA's run, in order: key tiles [t0, t1) of one item each.
template <int TK>
struct PagedWalk {
  const PagedParams& p;
  const PagedRun run;
  int item;
  PagedItem it;
  int t0, t1;   // key tiles of this piece (none for an item without keys)
  bool whole;   // the piece is the whole item
  bool begins;  // it holds the item's first key tile
  __device__ __forceinline__ PagedWalk(const PagedParams& pp, const PagedRun& r) : p(pp), run(r), item(r.from.item - 1) {}
  __device__ __forceinline__ bool next() {
    do {
      ++item;
      if (item > run.to.item || (item == run.to.item && run.to.off == 0)) return false;
      it = paged_item_at<TK>(p, item);
      if (it.cost == 0) item += it.next - 1;
    } while (it.cost == 0);
    const int off = item == run.from.item ? run.from.off : 0;
    const int end = item == run.to.item ? run.to.off : it.cost;
    begins = off == 0;
    whole = begins && end == it.cost;
    t0 = it.t0 + off;
    t1 = it.jhi < it.jlo ? t0 : it.t0 + end;
    return true;
  }
  // of a piece that is not the whole item: who began the item, its pieces
  __device__ __forceinline__ int head() const { return begins ? (int)blockIdx.x : run.from.head; }
  __device__ __forceinline__ int pieces() const { return begins ? run.to.pieces : run.from.pieces; }
};

// Partial of `rows` rows: o [rows][d], then the maxima (base 2) and the sums.
__host__ __device__ constexpr int64_t paged_slot_floats(int rows, int d) { return (int64_t)rows * (d + 2); }

// A CTA's partials: the piece that begins an item goes to slot 2c + 1, one that
// goes on with an item begun by an earlier CTA to slot 2c.  Piece i of an item
// that CTA `head` began:
__device__ __forceinline__ float* paged_slot(const PagedParams& p, int head, int i, int rows, int d) {
  return p.part + (i ? 2 * ((int64_t)head + i) : 2 * (int64_t)head + 1) * paged_slot_floats(rows, d);
}

// Token row and head of row r of an item.
__device__ __forceinline__ int64_t paged_row(const PagedParams& p, const PagedItem& it, int r) {
  return ((int64_t)it.row0 + r / p.group) * p.Hq + it.hg * p.group + r % p.group;
}

// ------------------------------------------------------------------ few rows
// Items of at most 16 rows (new tokens x heads of the group).  Bound by the
// bytes of the keys and values: each CTA streams 64-key tiles of K and V into
// a shared-memory ring by TMA, page by page, and four warps share a tile, 16
// keys each, with their own running max and sum; both products are m16n8k16
// warp matrix instructions (the rows padded to 16: they take 28 % of the time
// the bytes take, and single rows need no tcgen05 tile of 128).  P stays in
// registers, which its accumulator layout lets serve as the A operand.  The
// four warps' results meet at the end of a piece.  Measured: 16 sequences of up
// to 32768 positions, 32 heads on 8 key/value heads, 1.66 GB in 252-260 us, 6.4
// to 6.6 TB/s; 8 sequences with 32 bands of 1024, 105 MB in 23 us, most of which
// is the latency of the first pages and of the end.
template <int D>
struct PagedShortCfg {
  static constexpr int TK = 64, ROWS = 16, WARPS = 4, NTHREADS = 160, CTAS_PER_SM = 2;
  static constexpr int NS = D == 128 ? 3 : 6;  // 96 KB of tiles in flight per CTA
  static constexpr uint32_t KV_BYTES = TK * D * 2, STAGE_BYTES = 2 * KV_BYTES;
  static constexpr uint32_t OFF_RED = NS * STAGE_BYTES;          // [WARPS][4 rows][D] fp32
  static constexpr uint32_t OFF_ML = OFF_RED + WARPS * 4 * D * 4;  // [2][WARPS][ROWS] fp32
  static constexpr uint32_t OFF_BAR = OFF_ML + 2 * WARPS * ROWS * 4;
  static constexpr uint32_t USED = OFF_BAR + 256;
  static constexpr uint32_t SMEM_BYTES = USED + 1024;  // alignment slack
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "shared memory of an SM");
};

struct PagedShortBars {
  uint64_t full[6], empty[6];
  int abort;
  int last;  // this CTA's piece was its item's last to arrive
};

template <class E>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (E::kIsBf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Page numbers of one item's key tiles, 32 boxes of `BOX` keys ahead in the
// producer warp's registers (lane i holds box base + i), so that the page
// table's latency is paid once per 32 boxes.  Boxes that hold no key any row
// attends to give -1 and are never looked up; so do page numbers out of range,
// which also raise the status word.  A load at page -1 lies outside the tensor
// and fills with zeros.
struct PagedPages {
  int64_t base = 0;
  int id = -1;
  // page of box `box + which`; the tile has the boxes [box, box + n), n <= 32
  __device__ __forceinline__ int get(const PagedParams& p, const PagedItem& it, int64_t box, int box_shift, int n,
                                     int which, bool fresh) {
    const int lane = threadIdx.x % 32;
    if (fresh || box < base || box + n > base + 32) {
      base = box;
      const int64_t j = (box + lane) << box_shift;
      id = -1;
      if (j <= it.jhi && j + (1 << box_shift) > it.jlo) {
        id = p.page_table[(int64_t)it.b * p.width + (j >> p.page_shift)];
        if (id < 0 || id >= p.pages) {
          id = -1;
          report_status(kStatusInval);
        }
      }
    }
    return __shfl_sync(0xffffffffu, id, (int)(box - base) + which);
  }
};

// One warp joins row r of an item from its pieces' partials, in their order:
//   o = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  lse = M + log2 of it.
template <class E, int D, int ROWS>
__device__ __forceinline__ void paged_join_row(const PagedParams& p, int head, int pieces, int r, int64_t row) {
  constexpr int CW = D / 32;
  const int lane = threadIdx.x % 32;
  float mx = -INFINITY;
  for (int i = lane; i < pieces; i += 32) mx = ptx::fmax_nan(mx, paged_slot(p, head, i, ROWS, D)[ROWS * D + r]);
#pragma unroll
  for (int k = 16; k > 0; k /= 2) mx = ptx::fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  float sum = 0.f, out[CW] = {};
  for (int i0 = 0; i0 < pieces; i0 += 32) {
    const int i = i0 + lane;
    float f = 0.f, li = 0.f;
    if (i < pieces) {
      const float* ml = paged_slot(p, head, i, ROWS, D) + ROWS * D + r;
      f = ml[0] == -INFINITY ? 0.f : ptx::exp2_approx(ml[0] - mx);
      li = ml[ROWS] * f;
    }
#pragma unroll 4
    for (int k = 0; k < min(32, pieces - i0); ++k) {
      const float fk = __shfl_sync(0xffffffffu, f, k);
      sum += __shfl_sync(0xffffffffu, li, k);
      const float* src = paged_slot(p, head, i0 + k, ROWS, D) + r * D + lane * CW;
      float v[CW];
      if constexpr (CW == 4) {
        const float4 u = *reinterpret_cast<const float4*>(src);
        v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
      } else {
        const float2 u = *reinterpret_cast<const float2*>(src);
        v[0] = u.x; v[1] = u.y;
      }
      // a piece in which the row attends to nothing counts for nothing
#pragma unroll
      for (int e = 0; e < CW; ++e) out[e] = fk == 0.f ? out[e] : fmaf(fk, v[e], out[e]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D) + lane * (CW / 2);
#pragma unroll
  for (int e = 0; e < CW / 2; ++e) dst[e] = E::pack(out[2 * e] * inv, out[2 * e + 1] * inv);
  if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
}

template <class E, int D>
__global__ void __launch_bounds__(160, 2)
    spa_paged_short_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ PagedParams p) {
  using C = PagedShortCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align1024(smem_raw);
  if (!smem_fits(smem_raw, smem, C::USED)) return;
  PagedShortBars* bars = reinterpret_cast<PagedShortBars*>(smem + C::OFF_BAR);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      ptx::mbar_init(&bars->full[s], 1);
      ptx::mbar_init(&bars->empty[s], C::WARPS);
    }
    bars->abort = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tm_k);
    ptx::prefetch_tmap(&tm_v);
  }
  __syncthreads();
  // The lengths are asked for while the plan is made (they are inputs, written
  // before it began), so that the walk finds them near.
  if ((int)threadIdx.x <= p.B) ptx::prefetch_l1(p.cu_q + threadIdx.x), ptx::prefetch_l1(p.kv_len + min((int)threadIdx.x, p.B - 1));
  asm volatile("griddepcontrol.wait;" ::: "memory");  // for the plan
  volatile int* abort_flag = &bars->abort;
  PagedWalk<C::TK> w(p, PagedRun(p));

  if (warp == C::WARPS) {
    // ------------------------------------------------------------ TMA producer
    const int box_shift = min(p.page_shift, 6), boxes = C::TK >> box_shift;
    const int n_op = boxes * 2 * (D / 64);  // copies per tile: boxes x (K, V) x 64-column blocks
    PagedPages pages;
    int g = 0;
    bool ok = true;
    while (ok && w.next()) {
      if (lane == 0 && p.kv_len[w.it.b] > w.it.kv) report_status(kStatusInval);
      const int hk = w.it.hg / p.kv_div;
      for (int t = w.t0; t < w.t1; ++t, ++g) {
        const int s = g % C::NS;
        const int box_i = lane % boxes, op = lane / boxes;  // op: (K or V) x column block
        const int64_t box0 = (int64_t)t * boxes;
        const int id0 = pages.get(p, w.it, box0, box_shift, boxes, box_i, t == w.t0);
        ok = __all_sync(0xffffffffu, bar_wait(&bars->empty[s], ((g / C::NS) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars->full[s], C::STAGE_BYTES);
        __syncwarp();
        if (lane < n_op) {
          const bool is_v = op >= D / 64;
          const int cb = op % (D / 64);
          const int64_t j = (box0 + box_i) << box_shift;
          ptx::tma_load_3d(smem + s * C::STAGE_BYTES + (is_v ? C::KV_BYTES : 0) + cb * (C::TK * 128) +
                               (box_i << box_shift) * 128,
                           is_v ? &tm_v : &tm_k, &bars->full[s], cb * 64, (int)(j & ((1 << p.page_shift) - 1)),
                           id0 < 0 ? -1 : id0 * p.Hk + hk);
        }
        __syncwarp();
      }
    }
    // (here, where nothing waits for its loads)
    if (blockIdx.x == 0 && lane == 0) report_missing_rows(p.cu_q, p.B, p.T);
    // every copy issued has landed before the CTA ends
    if (lane == 0)
      for (int s = 0; s < C::NS; ++s) {
        const int used = (g + C::NS - 1 - s) / C::NS;  // times this warp armed stage s
        if (used > 0) bar_drain(&bars->full[s], (used - 1) & 1);
      }
    return;
  }

  // ------------------------------------------------------------ four warps, 16 keys of a tile each
  const uint32_t s_base = ptx::smem_u32(smem);
  float* s_red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* s_m = reinterpret_cast<float*>(smem + C::OFF_ML);
  float* s_l = s_m + C::WARPS * C::ROWS;
  const int quad = lane / 4, qc = lane % 4;
  int g = 0;
  // A warp whose wait runs out of time computes no further tile, but walks on
  // through the pieces, so that the named barriers keep their four warps.
  bool ok = true;
  while (w.next()) {
    const PagedItem& it = w.it;
    const int rows = it.tokens * p.group;
    // this lane's two rows: their queries as A operands, their permitted keys
    uint32_t qf[D / 16][4];
    int a_lo[2], a_hi[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int r = quad + 8 * x;
      const bool live = r < rows;
      const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + paged_row(p, it, live ? r : 0) * D);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        qf[kk][x] = live ? src[kk * 8 + qc] : 0u;
        qf[kk][x + 2] = live ? src[kk * 8 + 4 + qc] : 0u;
      }
      const int64_t pos = (int64_t)it.pos0 + r / p.group;
      a_lo[x] = live ? (int)max64(0, pos - p.hi[it.hg] + 1) : 0;
      a_hi[x] = live ? clamp_i32(min64(pos - p.lo[it.hg], it.kv - 1)) : -1;
    }
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    float acc[D / 8][4];
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;

    for (int t = w.t0; ok && t < w.t1; ++t, ++g) {
      const int s = g % C::NS;
      ok = __all_sync(0xffffffffu, bar_wait(&bars->full[s], (g / C::NS) & 1, abort_flag));
      if (!ok) break;
      const int j0 = t * C::TK + warp * 16;  // at most 2^31 - 16: the last key stands below 2^31
      if (j0 <= it.jhi && j0 >= it.jlo - 15) {
        const uint32_t k_base = s_base + s * C::STAGE_BYTES, v_base = k_base + C::KV_BYTES;
        // S = Q K^T: two 8-key column tiles
        float sc[2][4] = {};
        {
          const int mat = lane / 8, key = warp * 16 + lane % 8 + (mat >= 2 ? 8 : 0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const int chunk = kk * 2 + (mat & 1);
            uint32_t kf[4];
            ldmatrix_x4(kf, k_base + (chunk / 8) * (C::TK * 128) + ptx::sw128_offset(key, chunk % 8));
            mma_16816<E>(sc[0], qf[kk], kf[0], kf[1]);
            mma_16816<E>(sc[1], qf[kk], kf[2], kf[3]);
          }
        }
        // masked scores become -inf; base-2 units
        // (P in two 16-bit terms, the second the rounding error of the first: one
        // term alone would add as much error to o as its own rounding, and the
        // bytes leave time for the second product)
        uint32_t pa[4], pb[4];
        float alpha[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int c_lo = a_lo[x] - j0, c_hi = a_hi[x] - j0;
          float v[4], mx = -INFINITY;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = (e / 2) * 8 + 2 * qc + (e & 1);
            v[e] = c >= c_lo && c <= c_hi ? sc[e / 2][2 * x + (e & 1)] * p.scale_log2 : -INFINITY;
            mx = ptx::fmax_nan(mx, v[e]);
          }
          mx = ptx::fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = ptx::fmax_nan(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float m_new = ptx::fmax_nan(m[x], mx);
          const float ref = m_new == -INFINITY ? 0.f : m_new;
          alpha[x] = ptx::exp2_approx(m[x] - ref);
          m[x] = m_new;
          float pe[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) pe[e] = ptx::exp2_approx(v[e] - ref);
          l[x] = fmaf(l[x], alpha[x], (pe[0] + pe[1]) + (pe[2] + pe[3]));
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            pa[x + 2 * e] = E::pack(pe[2 * e], pe[2 * e + 1]);
            const float2 first = E::unpack(pa[x + 2 * e]);
            pb[x + 2 * e] = E::pack(pe[2 * e] - first.x, pe[2 * e + 1] - first.y);
          }
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int n = 0; n < D / 8; ++n) {
            acc[n][0] *= alpha[0];
            acc[n][1] *= alpha[0];
            acc[n][2] *= alpha[1];
            acc[n][3] *= alpha[1];
          }
        }
        // O += P V.  Values of keys that no row attends to are cleared: what
        // stands there may be no number, and 0 times that is none either.
        {
          uint32_t keep[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int j = j0 + 8 * x + 2 * qc;
            keep[x] = (j >= it.jlo && j <= it.jhi ? 0xffffu : 0u) |
                      (j + 1 >= it.jlo && j < it.jhi ? 0xffff0000u : 0u);
          }
          const int mat = lane / 8, key = warp * 16 + lane % 8 + (mat & 1) * 8;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            const int chunk = n * 2 + mat / 2;
            uint32_t vf[4];
            ldmatrix_x4_trans(vf, v_base + (chunk / 8) * (C::TK * 128) + ptx::sw128_offset(key, chunk % 8));
            mma_16816<E>(acc[2 * n], pa, vf[0] & keep[0], vf[1] & keep[1]);
            mma_16816<E>(acc[2 * n + 1], pa, vf[2] & keep[0], vf[3] & keep[1]);
            mma_16816<E>(acc[2 * n], pb, vf[0] & keep[0], vf[1] & keep[1]);
            mma_16816<E>(acc[2 * n + 1], pb, vf[2] & keep[0], vf[3] & keep[1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&bars->empty[s]);
    }

    // ---------------------------------------------------------- the four warps' results meet
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
      l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
      if (qc == 0) {
        s_m[warp * C::ROWS + quad + 8 * x] = m[x];
        s_l[warp * C::ROWS + quad + 8 * x] = l[x];
      }
    }
    ptx::named_bar_sync(1, C::WARPS * 32);
    float f[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float mx = s_m[quad + 8 * x];
#pragma unroll
      for (int y = 1; y < C::WARPS; ++y) mx = ptx::fmax_nan(mx, s_m[y * C::ROWS + quad + 8 * x]);
      f[x] = m[x] == -INFINITY ? 0.f : ptx::exp2_approx(m[x] - mx);
    }
    const int head = w.whole ? 0 : w.head(), piece = blockIdx.x - head;
    float* slot = paged_slot(p, head, piece, C::ROWS, D);
    for (int r0 = 0; r0 < rows; r0 += 4) {
      const int x = r0 / 8;  // these four rows are the lanes' first or second
      if (quad - r0 % 8 >= 0 && quad - r0 % 8 < 4) {
        float* dst = s_red + (warp * 4 + quad - r0 % 8) * D + 2 * qc;
        const float fx = x ? f[1] : f[0];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
          *reinterpret_cast<float2*>(dst + n * 8) =
              make_float2((x ? acc[n][2] : acc[n][0]) * fx, (x ? acc[n][3] : acc[n][1]) * fx);
      }
      ptx::named_bar_sync(1, C::WARPS * 32);
      const int r = r0 + warp;  // one row per warp now, D / 32 columns per lane
      if (r < rows) {
        constexpr int CW = D / 32;
        float mx = s_m[r], sum = 0.f, out[CW] = {};
#pragma unroll
        for (int y = 1; y < C::WARPS; ++y) mx = ptx::fmax_nan(mx, s_m[y * C::ROWS + r]);
#pragma unroll
        for (int y = 0; y < C::WARPS; ++y) {
          const float my = s_m[y * C::ROWS + r];
          sum += my == -INFINITY ? 0.f : s_l[y * C::ROWS + r] * ptx::exp2_approx(my - mx);
#pragma unroll
          for (int e = 0; e < CW; ++e) out[e] += s_red[(y * 4 + warp) * D + lane * CW + e];
        }
        if (w.whole) {
          const int64_t row = paged_row(p, it, r);
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D) + lane * (CW / 2);
#pragma unroll
          for (int e = 0; e < CW / 2; ++e) dst[e] = E::pack(out[2 * e] * inv, out[2 * e + 1] * inv);
          if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.69314718055994531f;
        } else {
#pragma unroll
          for (int e = 0; e < CW; ++e) slot[r * D + lane * CW + e] = out[e];
          if (lane == 0) {
            slot[C::ROWS * D + r] = mx;
            slot[C::ROWS * D + C::ROWS + r] = sum;
          }
        }
      }
      ptx::named_bar_sync(1, C::WARPS * 32);
    }
    if (!w.whole) {
      // whoever leaves the item's last partial joins them all
      __threadfence();
      ptx::named_bar_sync(1, C::WARPS * 32);
      if (threadIdx.x == 0) bars->last = atomicAdd(&p.arrived[2 * head], 1) == w.pieces() - 1;
      ptx::named_bar_sync(1, C::WARPS * 32);
      if (bars->last) {
        __threadfence();
        for (int r = warp; r < rows; r += C::WARPS) paged_join_row<E, D, C::ROWS>(p, head, w.pieces(), r, paged_row(p, it, r));
      }
    }
  }
}

}  // namespace spa
