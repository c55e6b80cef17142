// norm_rope.cuh -- RMS norm of each query and key head with a learned weight,
// then the rotary position rotation, in one pass (forward, backward), and the
// same for new tokens whose keys and values go into a paged cache.
//
// For one head row x (d values), weight w, rotation R(pos) on the first rot
// columns (pairs (i, i + rot/2), or (2i, 2i + 1), turned by an angle whose
// cosine and sine stand in a table row per position):
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  y = R(pos) (w * n).
// Backward, with g = R(pos)^T dy (a rotation's inverse is its transpose):
//   dw = sum over rows of g * n,   dx = r (g w - n mean(g w n)).
//
// Bound by bytes: forward reads x and writes y, backward reads dy and x and
// writes dx.  A row of d values is held by d/8 lanes, 4 pairs each, so that a
// rotation stays within a lane (with 8 neighbouring columns per lane it took
// eight shuffles per lane and row, and the forward of B4 H32 N8192 d128 218
// instead of 186 us, which is 5.8 TB/s); the row sums are shuffles of 3 or 4 steps.  A block
// walks heads of one kind (queries, keys or values): a lane keeps one token's
// table row, with the weight multiplied in where it can be, in registers for
// all of them, and the loads of several heads are issued before the first is
// used.  Arithmetic is in pairs of fp32 (f32x2).  All sums are fp32.
#pragma once

#include "common.cuh"
#include "elem.cuh"

namespace spa {

constexpr int kNrThreads = 128;
constexpr int kNrUnroll = 4;        // head rows in flight per lane group
// Backward: blocks, each one partial of a weight's gradient; 6 per SM, with 80
// registers and 32 to 40 bytes spilled (B1 H32/8 N30001 d128: 174 us, 5.4 TB/s;
// 5 per SM, with up to 96 registers and no spills, 190; 7 per SM 203).
constexpr int kNrMaxBlocks = 888;

struct RowStrides {
  int64_t b, h, n;  // in elements; the d values of a row are contiguous
};

struct NormRopeParams {
  const uint16_t* q;
  const uint16_t* k;
  RowStrides qs, ks;
  const float* wq;
  const float* wk;
  const float2* table;      // [table_len][rot / 2] (cos, sin)
  const int32_t* pos;       // [.., N] or null: the row's own index
  int64_t pos_stride;       // between batches; 0: one row of positions for all
  int64_t table_len;
  int64_t N;
  int64_t tokens;           // B * N
  int Hq, Hk, rot;
  int heads_per_group;      // heads that one lane group walks
  float eps;
  // forward: outputs [B][H][N][d] contiguous
  uint16_t* qo;
  uint16_t* ko;
  // backward: gradients of the outputs, [B][H][N][d] contiguous; of the inputs
  const uint16_t* dqo;
  const uint16_t* dko;
  uint16_t* dq;
  uint16_t* dk;
  RowStrides dqs, dks;
  float* part;              // [blocks][d] partial sums of dwq, then of dwk
  int q_blocks;             // backward: blocks that walk query heads
  float* dwq;
  float* dwk;
};

// The columns of a lane's pairs: a pair's first members stand in columns
// [c0, c0 + 4) and its second members in [c1, c1 + 4), or with neighbouring
// pairs both in turn in [c0, c0 + 8).  Lanes past the rotated columns hold 8
// neighbouring columns in the same form and turn them by nothing.
template <bool NEIGHBOURS>
struct LaneColumns {
  int c0, c1;
  bool turned;
  int pair0;  // its first pair's number
  __device__ __forceinline__ LaneColumns(int sub, int rot) {
    turned = sub < rot / 8;
    pair0 = 4 * sub;
    const bool halves = !NEIGHBOURS && turned;
    c0 = halves ? 4 * sub : 8 * sub;
    c1 = halves ? rot / 2 + 4 * sub : 8 * sub + 4;
  }
};

// 4 pairs of one row: first members a, second members b, two per float2.
struct Pairs4 {
  float2 a[2], b[2];
};

template <bool NEIGHBOURS>
__device__ __forceinline__ uint4 load_pairs(const uint16_t* row, const LaneColumns<NEIGHBOURS>& c) {
  if (NEIGHBOURS) return *reinterpret_cast<const uint4*>(row + c.c0);
  const uint2 u = *reinterpret_cast<const uint2*>(row + c.c0), v = *reinterpret_cast<const uint2*>(row + c.c1);
  return make_uint4(u.x, u.y, v.x, v.y);
}

template <bool NEIGHBOURS>
__device__ __forceinline__ void store_pairs(uint16_t* row, const LaneColumns<NEIGHBOURS>& c, const uint4& v) {
  if (NEIGHBOURS) {
    *reinterpret_cast<uint4*>(row + c.c0) = v;
  } else {
    *reinterpret_cast<uint2*>(row + c.c0) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + c.c1) = make_uint2(v.z, v.w);
  }
}

template <class E, bool NEIGHBOURS>
__device__ __forceinline__ Pairs4 unpack_pairs(const uint4& v) {
  const float2 f0 = E::unpack(v.x), f1 = E::unpack(v.y), f2 = E::unpack(v.z), f3 = E::unpack(v.w);
  if (NEIGHBOURS)
    return {{make_float2(f0.x, f1.x), make_float2(f2.x, f3.x)}, {make_float2(f0.y, f1.y), make_float2(f2.y, f3.y)}};
  return {{f0, f1}, {f2, f3}};
}

template <class E, bool NEIGHBOURS>
__device__ __forceinline__ uint4 pack_pairs(const Pairs4& x) {
  if (NEIGHBOURS)
    return make_uint4(E::pack(x.a[0].x, x.b[0].x), E::pack(x.a[0].y, x.b[0].y), E::pack(x.a[1].x, x.b[1].x),
                      E::pack(x.a[1].y, x.b[1].y));
  return make_uint4(E::pack(x.a[0].x, x.a[0].y), E::pack(x.a[1].x, x.a[1].y), E::pack(x.b[0].x, x.b[0].y),
                    E::pack(x.b[1].x, x.b[1].y));
}

// A lane's fp32 values of a [d] vector, as pairs.
template <bool NEIGHBOURS>
__device__ __forceinline__ Pairs4 vector_pairs(const float* w, const LaneColumns<NEIGHBOURS>& c) {
  const float4 u = *reinterpret_cast<const float4*>(w + c.c0), v = *reinterpret_cast<const float4*>(w + c.c1);
  if (NEIGHBOURS)
    return {{make_float2(u.x, u.z), make_float2(v.x, v.z)}, {make_float2(u.y, u.w), make_float2(v.y, v.w)}};
  return {{make_float2(u.x, u.y), make_float2(u.z, u.w)}, {make_float2(v.x, v.y), make_float2(v.z, v.w)}};
}

// Cosines and sines of a lane's pairs at one position.
struct Turn4 {
  float2 c[2], s[2];
};

template <bool NEIGHBOURS>
__device__ __forceinline__ Turn4 lane_turn(const float2* row, const LaneColumns<NEIGHBOURS>& lc) {
  Turn4 t = {{make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, {make_float2(0.f, 0.f), make_float2(0.f, 0.f)}};
  if (lc.turned) {
    const float4 u = reinterpret_cast<const float4*>(row + lc.pair0)[0];
    const float4 v = reinterpret_cast<const float4*>(row + lc.pair0)[1];
    t.c[0] = make_float2(u.x, u.z);
    t.s[0] = make_float2(u.y, u.w);
    t.c[1] = make_float2(v.x, v.z);
    t.s[1] = make_float2(v.y, v.w);
  }
  return t;
}

__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// Sum over the d / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = D / 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ float dot_pairs(const Pairs4& x, const Pairs4& y) {
  float2 s = __fmul2_rn(x.a[0], y.a[0]);
  s = __ffma2_rn(x.a[1], y.a[1], s);
  s = __ffma2_rn(x.b[0], y.b[0], s);
  s = __ffma2_rn(x.b[1], y.b[1], s);
  return s.x + s.y;
}

// Weight and rotation in one: y_a = r (a ca - b sb), y_b = r (b cb + a sa)
// with ca = c w_a, sb = s w_b, cb = c w_b, sa = s w_a.
struct WeightedTurn {
  float2 ca[2], sb[2], cb[2], sa[2];
  __device__ __forceinline__ WeightedTurn(const Turn4& t, const Pairs4& w) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ca[i] = __fmul2_rn(t.c[i], w.a[i]);
      sb[i] = neg2(__fmul2_rn(t.s[i], w.b[i]));
      cb[i] = __fmul2_rn(t.c[i], w.b[i]);
      sa[i] = __fmul2_rn(t.s[i], w.a[i]);
    }
  }
};

template <class E, int D, bool NEIGHBOURS>
__device__ __forceinline__ uint4 norm_rope_row(const uint4& in, const WeightedTurn& t, float eps) {
  Pairs4 x = unpack_pairs<E, NEIGHBOURS>(in);
  const float r = rsqrtf(row_sum<D>(dot_pairs(x, x)) * (1.f / D) + eps);
  const float2 rr = make_float2(r, r);
  Pairs4 y;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = __fmul2_rn(x.a[i], rr), b = __fmul2_rn(x.b[i], rr);
    y.a[i] = __ffma2_rn(a, t.ca[i], __fmul2_rn(b, t.sb[i]));
    y.b[i] = __ffma2_rn(b, t.cb[i], __fmul2_rn(a, t.sa[i]));
  }
  return pack_pairs<E, NEIGHBOURS>(y);
}

// Position of token (b, n) and whether the table has it.
__device__ __forceinline__ bool token_position(const NormRopeParams& p, int64_t b, int64_t n, int64_t* pos) {
  *pos = p.pos ? (int64_t)p.pos[b * p.pos_stride + n] : n;
  return *pos >= 0 && *pos < p.table_len;
}

// Heads [h0, h1) of one kind that block row `chunk` walks: the chunks of the
// first kind's heads come first, then the second's, then the third's.
struct HeadChunk {
  int kind, h0, h1;
  __device__ __forceinline__ HeadChunk(int chunk, int per, int n0, int n1, int n2 = 0) {
    const int k0 = (n0 + per - 1) / per, k1 = (n1 + per - 1) / per;
    kind = chunk < k0 ? 0 : chunk < k0 + k1 ? 1 : 2;
    const int n = kind == 0 ? n0 : kind == 1 ? n1 : n2;
    h0 = (chunk - (kind > 0 ? k0 : 0) - (kind > 1 ? k1 : 0)) * per;
    h1 = min(h0 + per, n);
  }
};

// Grid: x token tiles, y head chunks (the q heads, then the k heads).
template <class E, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kNrThreads, 8)
    spa_qk_norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int L = D / 8, TOK = kNrThreads / L;
  const LaneColumns<NEIGHBOURS> lc(threadIdx.x % L, p.rot);
  const int64_t tok = (int64_t)blockIdx.x * TOK + threadIdx.x / L;
  const bool live = tok < p.tokens;
  const int64_t tk = live ? tok : p.tokens - 1;
  const int64_t b = tk / p.N, n = tk % p.N;
  int64_t pos;
  const bool known = token_position(p, b, n, &pos);
  const HeadChunk hc(blockIdx.y, p.heads_per_group, p.Hq, p.Hk);
  const bool is_q = hc.kind == 0;
  const WeightedTurn t(lane_turn(p.table + (known ? pos : 0) * (p.rot / 2), lc), vector_pairs(is_q ? p.wq : p.wk, lc));
  const RowStrides rs = is_q ? p.qs : p.ks;
  const uint16_t* src = (is_q ? p.q : p.k) + b * rs.b + n * rs.n;
  uint16_t* dst = (is_q ? p.qo : p.ko) + (b * (is_q ? p.Hq : p.Hk) * p.N + n) * D;
  for (int hb = hc.h0; hb < hc.h1; hb += kNrUnroll) {
    uint4 in[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) in[u] = load_pairs(src + min(hb + u, hc.h1 - 1) * rs.h, lc);
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      uint4 out = norm_rope_row<E, D, NEIGHBOURS>(in[u], t, p.eps);
      if (!known) out = make_uint4(0u, 0u, 0u, 0u);
      if (live && hb + u < hc.h1) store_pairs(dst + (hb + u) * p.N * D, lc, out);
    }
  }
}

// Persistent grid: the first q_blocks blocks walk (token tile, q head chunk),
// the others (token tile, k head chunk).  Each block leaves one partial of
// its weight's gradient; the sum kernel adds them in block order.
template <class E, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kNrThreads, 6)
    spa_qk_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int L = D / 8, TOK = kNrThreads / L;
  __shared__ float s_dw[TOK][D];
  const int grp = threadIdx.x / L;
  const LaneColumns<NEIGHBOURS> lc(threadIdx.x % L, p.rot);
  const bool is_q = (int)blockIdx.x < p.q_blocks;
  const Pairs4 w = vector_pairs(is_q ? p.wq : p.wk, lc);
  const RowStrides rs = is_q ? p.qs : p.ks, ds = is_q ? p.dqs : p.dks;
  const int H = is_q ? p.Hq : p.Hk;
  const int chunks = (H + p.heads_per_group - 1) / p.heads_per_group;
  const int64_t units = ((p.tokens + TOK - 1) / TOK) * chunks;
  const int blocks = is_q ? p.q_blocks : (int)gridDim.x - p.q_blocks;
  Pairs4 dw = {};
  for (int64_t unit = is_q ? blockIdx.x : blockIdx.x - p.q_blocks; unit < units; unit += blocks) {
    const int64_t tok = (unit / chunks) * TOK + grp;
    const bool live = tok < p.tokens;
    const int64_t tk = live ? tok : p.tokens - 1;
    const int64_t b = tk / p.N, n = tk % p.N;
    int64_t pos;
    const bool known = token_position(p, b, n, &pos);
    const Turn4 t = lane_turn(p.table + (known ? pos : 0) * (p.rot / 2), lc);
    const int h0 = (int)(unit % chunks) * p.heads_per_group, h1 = min(h0 + p.heads_per_group, H);
    const uint16_t* src = (is_q ? p.q : p.k) + b * rs.b + n * rs.n;
    const uint16_t* gsrc = (is_q ? p.dqo : p.dko) + (b * H * p.N + n) * D;
    uint16_t* dst = (is_q ? p.dq : p.dk) + b * ds.b + n * ds.n;
    for (int hb = h0; hb < h1; hb += kNrUnroll) {
      uint4 in[kNrUnroll], dy[kNrUnroll];
#pragma unroll
      for (int u = 0; u < kNrUnroll; ++u) {
        const int h = min(hb + u, h1 - 1);
        in[u] = load_pairs(src + h * rs.h, lc);
        dy[u] = load_pairs(gsrc + h * p.N * D, lc);
      }
#pragma unroll
      for (int u = 0; u < kNrUnroll; ++u) {
        const bool store = live && hb + u < h1;
        const Pairs4 x = unpack_pairs<E, NEIGHBOURS>(in[u]), y = unpack_pairs<E, NEIGHBOURS>(dy[u]);
        Pairs4 g, gw;
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // rotated back
          g.a[i] = __ffma2_rn(y.a[i], t.c[i], __fmul2_rn(y.b[i], t.s[i]));
          g.b[i] = __ffma2_rn(y.b[i], t.c[i], neg2(__fmul2_rn(y.a[i], t.s[i])));
          gw.a[i] = __fmul2_rn(g.a[i], w.a[i]);
          gw.b[i] = __fmul2_rn(g.b[i], w.b[i]);
        }
        const float ss = row_sum<D>(dot_pairs(x, x)), dot = row_sum<D>(dot_pairs(gw, x));
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float back = -dot * r * r * (1.f / D);  // -mean(g w n) r
        const float2 rr = make_float2(r, r), bb = make_float2(back, back);
        Pairs4 dx;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          dx.a[i] = __fmul2_rn(rr, __ffma2_rn(x.a[i], bb, gw.a[i]));
          dx.b[i] = __fmul2_rn(rr, __ffma2_rn(x.b[i], bb, gw.b[i]));
        }
        if (known && store) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            dw.a[i] = __ffma2_rn(g.a[i], __fmul2_rn(x.a[i], rr), dw.a[i]);
            dw.b[i] = __ffma2_rn(g.b[i], __fmul2_rn(x.b[i], rr), dw.b[i]);
          }
        }
        uint4 out = pack_pairs<E, NEIGHBOURS>(dx);
        if (!known) out = make_uint4(0u, 0u, 0u, 0u);
        if (store) store_pairs(dst + (hb + u) * ds.h, lc, out);
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  {
    float* row = s_dw[grp];
    const float2 lo0 = NEIGHBOURS ? make_float2(dw.a[0].x, dw.b[0].x) : dw.a[0];
    const float2 lo1 = NEIGHBOURS ? make_float2(dw.a[0].y, dw.b[0].y) : dw.a[1];
    const float2 hi0 = NEIGHBOURS ? make_float2(dw.a[1].x, dw.b[1].x) : dw.b[0];
    const float2 hi1 = NEIGHBOURS ? make_float2(dw.a[1].y, dw.b[1].y) : dw.b[1];
    *reinterpret_cast<float4*>(row + lc.c0) = make_float4(lo0.x, lo0.y, lo1.x, lo1.y);
    *reinterpret_cast<float4*>(row + lc.c1) = make_float4(hi0.x, hi0.y, hi1.x, hi1.y);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kNrThreads) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < TOK; ++i) sum += s_dw[i][c];
    p.part[(int64_t)blockIdx.x * D + c] = sum;
  }
}

// dwq and dwk from the blocks' partials: 32 columns per block, 32 threads per
// column, their sums added in a fixed order.  Grid y: query, key weight.
template <int D>
__global__ void __launch_bounds__(1024) spa_qk_norm_rope_dw_kernel(const float* part, int q_blocks, int blocks,
                                                                   float* dwq, float* dwk) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int i0 = blockIdx.y ? q_blocks : 0, i1 = blockIdx.y ? blocks : q_blocks;
  float sum = 0.f;
  for (int i = i0 + row; i < i1; i += 32) sum += part[(int64_t)i * D + c];
  s[row][lane] = sum;
  __syncthreads();
  float v = s[lane][row];  // column blockIdx.x * 32 + row, partial `lane`
#pragma unroll
  for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  if (lane == 0) (blockIdx.y ? dwk : dwq)[blockIdx.x * 32 + row] = v;
}

// ------------------------------------------------------------------ table
// cos and sin of pos * base^(-2 i / rot), formed in fp64 and rounded once.
__global__ void __launch_bounds__(256) spa_rope_table_kernel(float2* table, int64_t n, int half, double log2_base) {
  for (int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t pos = e / half;
    const int i = (int)(e % half);
    double s, c;
    sincos((double)pos * exp2(-log2_base * (double)i / (double)half), &s, &c);
    table[e] = make_float2((float)c, (float)s);
  }
}

// ------------------------------------------------------------------ append
// The new tokens of B sequences, packed: token rows [cu_q[b], cu_q[b + 1])
// belong to sequence b, whose last new token has position kv_len[b] - 1.
struct AppendParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  RowStrides qs, ks, vs;   // b unused
  const float* wq;
  const float* wk;
  const float2* table;
  int64_t table_len;
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;  // [B][width]
  uint16_t* qo;               // [T][Hq][d]
  uint16_t* k_pages;          // [pages][Hk][page][d]
  uint16_t* v_pages;
  int64_t pages;
  int B, T, Hq, Hk, rot, width, page_shift;
  int heads_per_group;
  float eps;
};

// Number of sequences that end at or before token t, by the L lanes of a
// group: the sequence of t, or B for a row behind the last sequence.
template <int L>
__device__ __forceinline__ int sequence_of(const int32_t* cu_q, int B, int t, int sub) {
  int n = 0;
  for (int i = sub; i < B; i += L) n += cu_q[i + 1] <= t ? 1 : 0;
#pragma unroll
  for (int m = L / 2; m > 0; m /= 2) n += __shfl_xor_sync(0xffffffffu, n, m);
  return n;
}

// Grid: x token tiles, y head chunks (q heads, k heads, v heads).
template <class E, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kNrThreads) spa_paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int L = D / 8, TOK = kNrThreads / L;
  const int sub = threadIdx.x % L;
  const int64_t tok = (int64_t)blockIdx.x * TOK + threadIdx.x / L;
  const int64_t t = min64(tok, p.T - 1);
  const int b = sequence_of<L>(p.cu_q, p.B, (int)t, sub);
  const bool live = tok < p.T && b < p.B && t >= p.cu_q[0];
  int64_t pos = -1, slot = -1;
  if (live) {
    pos = (int64_t)p.kv_len[b] - p.cu_q[b + 1] + t;
    if (pos >= 0 && pos < p.table_len && (pos >> p.page_shift) < p.width) {
      const int64_t page = p.page_table[(int64_t)b * p.width + (pos >> p.page_shift)];
      if (page >= 0 && page < p.pages)
        slot = ((page * p.Hk) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
    }
    // a position without a table row or a page: nothing is cached for it
    if (slot < 0 && sub == 0) report_status(kStatusInval);
  }
  const LaneColumns<NEIGHBOURS> lc(sub, p.rot);
  const HeadChunk hc(blockIdx.y, p.heads_per_group, p.Hq, p.Hk, p.Hk);
  const RowStrides rs = hc.kind == 0 ? p.qs : hc.kind == 1 ? p.ks : p.vs;
  const uint16_t* src = (hc.kind == 0 ? p.q : hc.kind == 1 ? p.k : p.v) + t * rs.n;
  // where head h of this token goes: base + h * step
  uint16_t* dst = hc.kind == 0 ? p.qo + (int64_t)t * p.Hq * D : (hc.kind == 1 ? p.k_pages : p.v_pages) + slot * D;
  const int64_t step = hc.kind == 0 ? D : (int64_t)D << p.page_shift;
  const bool store = live && (hc.kind == 0 || slot >= 0);
  const WeightedTurn turn(lane_turn(p.table + (slot >= 0 ? pos : 0) * (p.rot / 2), lc),
                          vector_pairs(hc.kind == 0 ? p.wq : p.wk, lc));
  for (int hb = hc.h0; hb < hc.h1; hb += kNrUnroll) {
    uint4 in[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) in[u] = load_pairs(src + min(hb + u, hc.h1 - 1) * rs.h, lc);
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      uint4 out = hc.kind == 2 ? in[u] : norm_rope_row<E, D, NEIGHBOURS>(in[u], turn, p.eps);
      if (slot < 0) out = make_uint4(0u, 0u, 0u, 0u);  // a query without a place
      if (store && hb + u < hc.h1) store_pairs(dst + (hb + u) * step, lc, out);
    }
  }
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) report_missing_rows(p.cu_q, p.B, p.T);
}

}  // namespace spa
