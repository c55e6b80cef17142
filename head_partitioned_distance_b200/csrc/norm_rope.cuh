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
// writes dx.  A row of d values is held by d/8 lanes, 16 bytes each, so the
// row sums are shuffles of 3 or 4 steps and a pair's partner is one shuffle
// (or in the lane).  A lane group keeps one token's table row in registers
// for all the heads it walks; loads of several heads are issued before the
// first is used.  All sums are fp32.
#pragma once

#include "common.cuh"
#include "elem.cuh"

namespace spa {

constexpr int kNrThreads = 256;
constexpr int kNrUnroll = 4;        // head rows in flight per lane group
constexpr int kNrMaxBlocks = 592;   // backward: blocks, each one partial of dw

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
  float* part;              // [blocks][2][d] partial sums of dwq, dwk
  float* dwq;
  float* dwk;
};

// What a lane needs to rotate its 8 columns: out = x * c + partner * s, the
// partner in lane `src` of the group (pairs of halves) or next door in the
// lane (neighbouring pairs).  Columns past rot have c = 1, s = 0.
struct LaneTurn {
  float c[8], s[8];
  int src;
};

template <int D, bool NEIGHBOURS>
__device__ __forceinline__ LaneTurn lane_turn(const float2* row, int rot, int sub) {
  LaneTurn t;
  const int col = sub * 8;
  t.src = sub;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t.c[e] = 1.f;
    t.s[e] = 0.f;
  }
  if (col < rot) {
    if (NEIGHBOURS) {
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float4 v = reinterpret_cast<const float4*>(row + col / 2)[e / 2];
        t.c[2 * e] = t.c[2 * e + 1] = v.x;
        t.s[2 * e] = -v.y;
        t.s[2 * e + 1] = v.y;
        t.c[2 * e + 2] = t.c[2 * e + 3] = v.z;
        t.s[2 * e + 2] = -v.w;
        t.s[2 * e + 3] = v.w;
      }
    } else {
      const int half = rot / 2;
      const bool second = col >= half;
      t.src = second ? sub - half / 8 : sub + half / 8;
      const float4* v4 = reinterpret_cast<const float4*>(row + (second ? col - half : col));
      const float sign = second ? 1.f : -1.f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 v = v4[e / 2];
        t.c[e] = v.x;
        t.s[e] = sign * v.y;
        t.c[e + 1] = v.z;
        t.s[e + 1] = sign * v.w;
      }
    }
  }
  return t;
}

// x rotated (dir = 1) or rotated back (dir = -1).
template <int D, bool NEIGHBOURS>
__device__ __forceinline__ void turn8(float (&x)[8], const LaneTurn& t, float dir) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float other = NEIGHBOURS ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], t.src, D / 8);
    y[e] = x[e] * t.c[e] + dir * (other * t.s[e]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = y[e];
}

// Sum over the d / 8 lanes of a row.
template <int D>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = D / 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

template <class E, int D, bool NEIGHBOURS>
__device__ __forceinline__ uint4 norm_rope_row(const uint4& in, const float (&w)[8], const LaneTurn& t, float eps) {
  float x[8];
  unpack8<E>(in, x);
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
  const float r = rsqrtf(row_sum<D>(ss) * (1.f / D) + eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] *= r * w[e];
  turn8<D, NEIGHBOURS>(x, t, 1.f);
  return pack8<E>(x);
}

__device__ __forceinline__ void load_weight8(const float* w, int col, float (&out)[8]) {
  const float4 a = reinterpret_cast<const float4*>(w + col)[0], b = reinterpret_cast<const float4*>(w + col)[1];
  out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
  out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
}

// Position of token (b, n) and whether the table has it.
__device__ __forceinline__ bool token_position(const NormRopeParams& p, int64_t b, int64_t n, int64_t* pos) {
  *pos = p.pos ? (int64_t)p.pos[b * p.pos_stride + n] : n;
  return *pos >= 0 && *pos < p.table_len;
}

// Grid: x token tiles, y head chunks (the q heads, then the k heads).
template <class E, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kNrThreads)
    spa_qk_norm_rope_fwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int L = D / 8, TOK = kNrThreads / L;
  const int sub = threadIdx.x % L, col = sub * 8;
  const int64_t tok = (int64_t)blockIdx.x * TOK + threadIdx.x / L;
  const bool live = tok < p.tokens;
  const int64_t tk = live ? tok : p.tokens - 1;
  const int64_t b = tk / p.N, n = tk % p.N;
  int64_t pos;
  const bool known = token_position(p, b, n, &pos);
  const LaneTurn t = lane_turn<D, NEIGHBOURS>(p.table + (known ? pos : 0) * (p.rot / 2), p.rot, sub);
  float wq[8], wk[8];
  load_weight8(p.wq, col, wq);
  load_weight8(p.wk, col, wk);
  const int h0 = blockIdx.y * p.heads_per_group;
  const int h1 = min(h0 + p.heads_per_group, p.Hq + p.Hk);
  for (int hb = h0; hb < h1; hb += kNrUnroll) {
    uint4 in[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int h = min(hb + u, h1 - 1);
      const uint16_t* src = h < p.Hq ? p.q + b * p.qs.b + h * p.qs.h + n * p.qs.n
                                     : p.k + b * p.ks.b + (h - p.Hq) * p.ks.h + n * p.ks.n;
      in[u] = *reinterpret_cast<const uint4*>(src + col);
    }
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int h = min(hb + u, h1 - 1);
      const bool is_q = h < p.Hq;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = is_q ? wq[e] : wk[e];
      uint4 out = norm_rope_row<E, D, NEIGHBOURS>(in[u], w, t, p.eps);
      if (!known) out = make_uint4(0u, 0u, 0u, 0u);
      uint16_t* dst = is_q ? p.qo + ((b * p.Hq + h) * p.N + n) * D : p.ko + ((b * p.Hk + h - p.Hq) * p.N + n) * D;
      if (live && hb + u < h1) *reinterpret_cast<uint4*>(dst + col) = out;
    }
  }
}

// Persistent grid over (token tile, head chunk); each block leaves one
// partial of dwq and dwk, which the sum kernel adds in block order.
template <class E, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kNrThreads)
    spa_qk_norm_rope_bwd_kernel(const __grid_constant__ NormRopeParams p) {
  constexpr int L = D / 8, TOK = kNrThreads / L;
  __shared__ float s_dw[TOK][2][D];
  const int sub = threadIdx.x % L, col = sub * 8, grp = threadIdx.x / L;
  float wq[8], wk[8], dwq[8], dwk[8];
  load_weight8(p.wq, col, wq);
  load_weight8(p.wk, col, wk);
#pragma unroll
  for (int e = 0; e < 8; ++e) dwq[e] = dwk[e] = 0.f;
  const int chunks = (p.Hq + p.Hk + p.heads_per_group - 1) / p.heads_per_group;
  const int64_t units = ((p.tokens + TOK - 1) / TOK) * chunks;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t tok = (unit / chunks) * TOK + grp;
    const bool live = tok < p.tokens;
    const int64_t tk = live ? tok : p.tokens - 1;
    const int64_t b = tk / p.N, n = tk % p.N;
    int64_t pos;
    const bool known = token_position(p, b, n, &pos);
    const LaneTurn t = lane_turn<D, NEIGHBOURS>(p.table + (known ? pos : 0) * (p.rot / 2), p.rot, sub);
    const int h0 = (int)(unit % chunks) * p.heads_per_group;
    const int h1 = min(h0 + p.heads_per_group, p.Hq + p.Hk);
    for (int hb = h0; hb < h1; hb += kNrUnroll) {
      uint4 in[kNrUnroll], dy[kNrUnroll];
#pragma unroll
      for (int u = 0; u < kNrUnroll; ++u) {
        const int h = min(hb + u, h1 - 1);
        const bool is_q = h < p.Hq;
        const uint16_t* src = is_q ? p.q + b * p.qs.b + h * p.qs.h + n * p.qs.n
                                   : p.k + b * p.ks.b + (h - p.Hq) * p.ks.h + n * p.ks.n;
        const uint16_t* gsrc =
            is_q ? p.dqo + ((b * p.Hq + h) * p.N + n) * D : p.dko + ((b * p.Hk + h - p.Hq) * p.N + n) * D;
        in[u] = *reinterpret_cast<const uint4*>(src + col);
        dy[u] = *reinterpret_cast<const uint4*>(gsrc + col);
      }
#pragma unroll
      for (int u = 0; u < kNrUnroll; ++u) {
        const int h = min(hb + u, h1 - 1);
        const bool is_q = h < p.Hq, store = live && hb + u < h1;
        float x[8], g[8];
        unpack8<E>(in[u], x);
        unpack8<E>(dy[u], g);
        turn8<D, NEIGHBOURS>(g, t, -1.f);
        const bool counts = known && store;
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = is_q ? wq[e] : wk[e];
          ss = fmaf(x[e], x[e], ss);
          dot = fmaf(g[e] * w, x[e], dot);
        }
        ss = row_sum<D>(ss);
        dot = row_sum<D>(dot);
        const float r = rsqrtf(ss * (1.f / D) + p.eps);
        const float back = dot * r * r * (1.f / D);  // mean(g w n) r
        float dx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float w = is_q ? wq[e] : wk[e];
          const float gn = counts ? g[e] * (x[e] * r) : 0.f;
          if (is_q) dwq[e] += gn;
          else dwk[e] += gn;
          dx[e] = r * (g[e] * w - x[e] * back);
        }
        uint16_t* dst = is_q ? p.dq + b * p.dqs.b + h * p.dqs.h + n * p.dqs.n
                             : p.dk + b * p.dks.b + (h - p.Hq) * p.dks.h + n * p.dks.n;
        uint4 out = pack8<E>(dx);
        if (!known) out = make_uint4(0u, 0u, 0u, 0u);
        if (store) *reinterpret_cast<uint4*>(dst + col) = out;
      }
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    s_dw[grp][0][col + e] = dwq[e];
    s_dw[grp][1][col + e] = dwk[e];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * D; c += kNrThreads) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < TOK; ++i) sum += s_dw[i][c / D][c % D];
    p.part[(int64_t)blockIdx.x * 2 * D + c] = sum;
  }
}

// dwq and dwk from the blocks' partials: 32 columns per block, 32 threads per
// column, their sums added in a fixed order.
template <int D>
__global__ void __launch_bounds__(1024) spa_qk_norm_rope_dw_kernel(const float* part, int blocks, float* dwq,
                                                                   float* dwk) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x % 32, row = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float sum = 0.f;
  for (int i = row; i < blocks; i += 32) sum += part[(int64_t)i * 2 * D + c];
  s[row][lane] = sum;
  __syncthreads();
  float v = s[lane][row];  // column blockIdx.x * 32 + row, partial `lane`
#pragma unroll
  for (int m = 16; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  const int cc = blockIdx.x * 32 + row;
  if (lane == 0) (cc < D ? dwq : dwk)[cc % D] = v;
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
  const int sub = threadIdx.x % L, col = sub * 8;
  const int64_t tok = (int64_t)blockIdx.x * TOK + threadIdx.x / L;
  const int t = (int)min64(tok, p.T - 1);
  const int h0 = blockIdx.y * p.heads_per_group;
  const int h1 = min(h0 + p.heads_per_group, p.Hq + 2 * p.Hk);
  const int b = sequence_of<L>(p.cu_q, p.B, t, sub);
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
    if (slot < 0 && sub == 0) atomicExch(&g_spa_status, kStatusInval);
  }
  const LaneTurn turn = lane_turn<D, NEIGHBOURS>(p.table + (slot >= 0 ? pos : 0) * (p.rot / 2), p.rot, sub);
  float wq[8], wk[8];
  load_weight8(p.wq, col, wq);
  load_weight8(p.wk, col, wk);
  for (int hb = h0; hb < h1; hb += kNrUnroll) {
    uint4 in[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int h = min(hb + u, h1 - 1);
      const uint16_t* src = h < p.Hq ? p.q + t * p.qs.n + h * p.qs.h
                            : h < p.Hq + p.Hk ? p.k + t * p.ks.n + (h - p.Hq) * p.ks.h
                                              : p.v + t * p.vs.n + (h - p.Hq - p.Hk) * p.vs.h;
      in[u] = *reinterpret_cast<const uint4*>(src + col);
    }
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int h = min(hb + u, h1 - 1);
      const bool is_q = h < p.Hq, is_v = h >= p.Hq + p.Hk;
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = is_q ? wq[e] : wk[e];
      uint4 out = norm_rope_row<E, D, NEIGHBOURS>(in[u], w, turn, p.eps);
      const bool store = live && hb + u < h1;
      if (store && is_q) {
        if (slot < 0) out = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(p.qo + ((int64_t)t * p.Hq + h) * D + col) = out;
      } else if (store && slot >= 0) {
        const int hk = is_v ? h - p.Hq - p.Hk : h - p.Hq;
        uint16_t* dst = (is_v ? p.v_pages : p.k_pages) + (slot + ((int64_t)hk << p.page_shift)) * D + col;
        *reinterpret_cast<uint4*>(dst) = is_v ? in[u] : out;
      }
    }
  }
}

}  // namespace spa
