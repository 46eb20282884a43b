// Attention over the 8-bit paged KV cache for few query rows a tile (single tokens, blocks, drafts).
//
// The queries of a tile -- (row, query head) pairs of one sequence that share a key/value head -- are the
// 8-wide side of mma.m16n8k16: scores are S^T = K Q^T (16 keys x 8 queries) and the output is
// O^T = V^T P^T, so a single query wastes 7 of 8 columns of a small product instead of 15 of 16 rows of
// a large one, and K and V are the fragments that come straight from the codes in memory:
//   K (A operand): a lane holds, for keys g and g + 8 of a 16-key unit, the channels of its quarter t of the
//     row; the product sums over channels, so which four channels make up a k16 step is free and each lane
//     reads 16-byte pieces;
//   V^T (A operand): a lane holds, for keys 2t, 2t+1, 2t+8, 2t+9, its eighth g of the channels; the byte
//     permute that spreads codes for conversion also pairs two keys, so the transpose costs nothing.
// No shared memory and no barrier stands between memory and the tensor cores; each warp takes 16-key units
// of its own with its own running maximum and sum, the next units' loads in flight while it computes.
// Warps are joined in shared memory, and the CTAs that split a long key axis (a cluster) over distributed
// shared memory, in a fixed order: no workspace, no second launch, no atomics.
#pragma once

#include <cooperative_groups.h>

#include "kv8.cuh"

namespace bltdec {

constexpr int kKv8Warps = 8;
constexpr int kKv8NoPos = 1 << 30;  // position of a unit that is not there: beyond every limit

// Channel of byte group i (4 codes) of a lane's share of a key row: 16-byte (or 8-byte) pieces interleaved
// over the four lanes of a row.
template <int DH>
__host__ __device__ constexpr int kv8_kpiece() { return DH % 64 == 0 ? 16 : 8; }
template <int DH>
__device__ __forceinline__ int kv8_kdim(int i, int t) {
  constexpr int CB = kv8_kpiece<DH>(), PW = CB / 4;
  return (i / PW) * 4 * CB + t * CB + (i % PW) * 4;
}
// Channel of byte b of a lane's share of a value row.
template <int DH>
__host__ __device__ constexpr int kv8_vpiece() { return DH == 96 ? 4 : DH / 8; }
template <int DH>
__device__ __forceinline__ int kv8_vdim(int b, int g) {
  constexpr int VB = kv8_vpiece<DH>();
  return (b / VB) * 8 * VB + g * VB + b % VB;
}

__device__ __forceinline__ uint32_t ldg_u32(const uint8_t* p) {
  uint32_t v;
  asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];\n" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ldg_u64(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];\n" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ldg_u128(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int DH>
__device__ __forceinline__ void kv8_load_krow(uint32_t (&w)[DH / 16], const uint8_t* row, int t) {
  constexpr int CB = kv8_kpiece<DH>();
#pragma unroll
  for (int i = 0; i < DH / 16; i += CB / 4) {
    const uint8_t* p = row + kv8_kdim<DH>(i, t);
    if constexpr (CB == 16) {
      const uint4 x = ldg_u128(p);
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    } else {
      const uint2 x = ldg_u64(p);
      w[i] = x.x, w[i + 1] = x.y;
    }
  }
}
template <int DH>
__device__ __forceinline__ void kv8_load_vrow(uint32_t (&w)[DH / 32], const uint8_t* row, int g) {
  constexpr int VB = kv8_vpiece<DH>();
  if constexpr (VB == 16) {
    const uint4 x = ldg_u128(row + g * 16);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (VB == 8) {
    const uint2 x = ldg_u64(row + g * 8);
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int j = 0; j < DH / 32; ++j) w[j] = ldg_u32(row + j * 32 + g * 4);
  }
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(x));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// P planes of two fp32 values as packed bf16: the sum of the planes has 8 P bits of the value.
template <int P>
__device__ __forceinline__ void kv8_planes(float x0, float x1, uint32_t (&pl)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    pl[i] = f2_to_bf16x2(x0, x1);
    if (i + 1 < P) {
      const float2 f = bf16x2_to_f2(pl[i]);
      x0 -= f.x, x1 -= f.y;
    }
  }
}

template <int DH, int NQ>
struct Kv8Smem {
  static constexpr int OS = DH + 4;  // row stride of a partial output (floats): breaks bank alignment of the rows
  float o[kKv8Warps][8 * NQ][OS];
  float m[kKv8Warps][8 * NQ], l[kKv8Warps][8 * NQ];
  float bo[8 * NQ][OS];  // the CTA's own sums, read by the cluster
  float bm[8 * NQ], bl[8 * NQ];
};

// grid (tiles x CL, key/value heads, sequences), clusters of CL along x.
template <int DH, int FMT, int QP, int PP, int NQ>
__global__ void __launch_bounds__(kKv8Warps * 32) k_kv8_attend(const __grid_constant__ Kv8View c, const __grid_constant__ Kv8AttnArgs a,
                                                                const int CL) {
  constexpr int U = DH <= 64 ? 2 : 1;  // units per step of a warp
  constexpr int KW = DH / 16, VW = DH / 32, MT = DH / 16;
  extern __shared__ float4 kv8_smem4[];
  Kv8Smem<DH, NQ>& sm = *reinterpret_cast<Kv8Smem<DH, NQ>*>(kv8_smem4);
  const int tile = blockIdx.x / CL, rank = blockIdx.x % CL, kvh = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  int r0, r1;
  kv8_rows_of(a.row_off, s, a.n_rows, a.max_rows, c.status, r0, r1);
  const bool sel = a.sel_pages != nullptr;
  // the tile's queries: qbase .. qbase + nq - 1 of the (row, head of the group) pairs from row `row0`
  int row0 = r0, qbase = tile * 8 * NQ, nq = (r1 - r0) * a.G - qbase;
  if (sel) {  // a row's heads share its list, rows do not
    const int tpr = (a.G + 8 * NQ - 1) / (8 * NQ);
    row0 = r0 + tile / tpr;
    qbase = tile % tpr * 8 * NQ;
    nq = row0 < r1 ? a.G - qbase : 0;
  }
  nq = min(nq, 8 * NQ);
  if (nq <= 0) return;  // the same for every CTA of the cluster

  auto row_of = [&](int n) { return row0 + (qbase + n) / a.G; };
  auto head_of = [&](int n) { return kvh * a.G + (qbase + n) % a.G; };
  const int cap = c.max_pages * c.PT;
  int lim_n = 0;  // limit of query `lane`
  if (lane < nq) {
    lim_n = __ldg(a.row_limit + row_of(lane));
    if (lim_n > cap) {
      if (c.status) set_status(c.status, kErrDevice);
      lim_n = cap;
    }
    lim_n = max(lim_n, 0);
  }
  const int maxlim = __reduce_max_sync(0xffffffffu, lim_n);
  const int minlim = __reduce_min_sync(0xffffffffu, lane < nq ? lim_n : INT_MAX);
  int lim[NQ][2];
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) lim[n][e] = __shfl_sync(0xffffffffu, lim_n, n * 8 + 2 * t + e);

  // query fragments (B operand): k16 step i holds the channels of key byte group i
  uint32_t qf[NQ][KW][2][QP];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int qn = n * 8 + g;
    const long long base = qn < nq ? (long long)row_of(qn) * a.qs + (long long)head_of(qn) * a.qhs : 0;
#pragma unroll
    for (int i = 0; i < KW; ++i) {
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (qn < nq) {
        const long long at = base + kv8_kdim<DH>(i, t);
        if (a.q_vec && a.dtype == BLT_T_F32) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at));
          x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = kv8_ld(a.q, a.dtype, at + j);
        }
      }
      kv8_planes<QP>(x[0], x[1], qf[n][i][0]);
      kv8_planes<QP>(x[2], x[3], qf[n][i][1]);
    }
  }

  // this CTA's units: [u0, u1) of nu, its warps taking steps of U units in turn
  const int* list = nullptr;
  int nu = (maxlim + kKv8Block - 1) / kKv8Block;
  if (sel) {
    const size_t li = (size_t)row0 * c.H + kvh;
    list = a.sel_pages + li * a.n_select;
    nu = min(max(__ldg(a.sel_count + li), 0), a.n_select) * c.tpp;
  }
  const int per = ((nu + CL - 1) / CL + U - 1) / U * U;
  const int u0 = min(rank * per, nu), u1 = min(nu, u0 + per);
  const int steps = max(0, (u1 - u0 + U - 1) / U - warp + kKv8Warps - 1) / kKv8Warps;

  float m[NQ][2], l[NQ][2], o[MT][NQ][4];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][n][e] = 0.f;
  }

  // pages and positions of the warp's next 32 units, one per lane
  int c_page = -1, c_pos = kKv8NoPos;
  auto resolve = [&](int it0) {
    const int u = u0 + (warp + kKv8Warps * (it0 + lane / U)) * U + lane % U;
    c_page = -1;
    c_pos = kKv8NoPos;
    if (it0 + lane / U >= steps || u >= u1) return;
    const int e = kv8_div_tpp(c, u);
    int pl = e, pos = u * kKv8Block;
    if (sel) {
      pl = __ldg(list + e);
      const int prev = e > 0 ? __ldg(list + e - 1) : -1;
      if (pl < 0 || pl <= prev || pl >= c.max_pages) return;
      pos = pl * c.PT + (u - e * c.tpp) * kKv8Block;
      if (pos >= maxlim) return;
    }
    c_page = kv8_page(c, s, pl);
    if (c_page >= 0) c_pos = pos;
  };

  struct Stage {
    uint32_t k[U][2][KW], v[U][4][VW];
    int pos[U];
    uint32_t ke[U], ve[U];
  };
  auto load = [&](Stage& st, int it) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int src = (it * U + u) & 31;
      const int page = __shfl_sync(0xffffffffu, c_page, src), pos = __shfl_sync(0xffffffffu, c_pos, src);
      st.pos[u] = pos;
      if (page < 0) {
        st.ke[u] = st.ve[u] = 127;
#pragma unroll
        for (int i = 0; i < KW; ++i) st.k[u][0][i] = st.k[u][1][i] = 0;
#pragma unroll
        for (int i = 0; i < VW; ++i) st.v[u][0][i] = st.v[u][1][i] = st.v[u][2][i] = st.v[u][3][i] = 0;
        continue;
      }
      const int blk = pos / kKv8Block, sub = blk - kv8_div_tpp(c, blk) * c.tpp;
      const size_t at = (size_t)page * c.page_stride + ((size_t)kvh * c.PT + sub * kKv8Block) * DH;
      const size_t ex = (size_t)page * c.exp_stride + kvh * c.tpp + sub;
      const uint8_t *kp = c.k + at, *vp = c.v + at;
      kv8_load_krow<DH>(st.k[u][0], kp + g * DH, t);
      kv8_load_krow<DH>(st.k[u][1], kp + (g + 8) * DH, t);
      kv8_load_vrow<DH>(st.v[u][0], vp + (2 * t) * DH, g);
      kv8_load_vrow<DH>(st.v[u][1], vp + (2 * t + 1) * DH, g);
      kv8_load_vrow<DH>(st.v[u][2], vp + (2 * t + 8) * DH, g);
      kv8_load_vrow<DH>(st.v[u][3], vp + (2 * t + 9) * DH, g);
      st.ke[u] = __ldg(c.ke + ex);
      st.ve[u] = __ldg(c.ve + ex);
    }
  };

  const float cs = a.scale * 1.4426950408889634f;  // scores in units of log 2
  auto compute = [&](const Stage& st) {
    float sc[U][NQ][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][n][e] = 0.f;
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        uint4 f;
        f.x = kv8_pair<FMT>(st.k[u][0][i], 0, kv8_sel<FMT>(0, 1));
        f.y = kv8_pair<FMT>(st.k[u][1][i], 0, kv8_sel<FMT>(0, 1));
        f.z = kv8_pair<FMT>(st.k[u][0][i], 0, kv8_sel<FMT>(2, 3));
        f.w = kv8_pair<FMT>(st.k[u][1][i], 0, kv8_sel<FMT>(2, 3));
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int p = QP - 1; p >= 0; --p) mma16816(sc[u][n], f, qf[n][i][0][p], qf[n][i][1][p]);
      }
      const float ks = kv8_pow2(st.ke[u]) * cs;
      const bool whole = st.pos[u] + kKv8Block <= minlim;
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[u][n][e] *= ks;
          if (!whole && st.pos[u] + g + (e >> 1) * 8 >= lim[n][e & 1]) sc[u][n][e] = -INFINITY;
        }
    }
    bool grow = false;
    float mn[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = m[n][e];
#pragma unroll
        for (int u = 0; u < U; ++u) x = fmaxf(x, fmaxf(sc[u][n][e], sc[u][n][e + 2]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        mn[n][e] = x;
        grow |= x > m[n][e];
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          f[e] = mn[n][e] > m[n][e] ? ex2(m[n][e] - mn[n][e]) : 1.f;  // -inf before the first visible key: 0
          m[n][e] = mn[n][e];
          l[n][e] *= f[e];
        }
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][n][e] *= f[e & 1];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t pf[NQ][2][PP];
      const float vs = kv8_pow2(st.ve[u]);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mx = m[n][e & 1];
          p[e] = ex2(sc[u][n][e] - (mx == -INFINITY ? 0.f : mx));
          l[n][e & 1] += p[e];
          p[e] *= vs;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t pl[PP];
          kv8_planes<PP>(p[2 * e], p[2 * e + 1], pl);  // key g + 8 e, queries 2t, 2t + 1
#pragma unroll
          for (int x = 0; x < PP; ++x) pf[n][e][x] = movmatrix_trans(pl[x]);  // query g, keys 2t + 8 e, 2t + 1 + 8 e
        }
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {  // channels of value bytes 2j and 2j + 1
        constexpr uint32_t s0 = kv8_sel<FMT>(0, 4), s1 = kv8_sel<FMT>(1, 5), s2 = kv8_sel<FMT>(2, 6), s3 = kv8_sel<FMT>(3, 7);
        const int w = j >> 1;
        uint4 f;
        f.x = kv8_pair<FMT>(st.v[u][0][w], st.v[u][1][w], (j & 1) ? s2 : s0);
        f.y = kv8_pair<FMT>(st.v[u][0][w], st.v[u][1][w], (j & 1) ? s3 : s1);
        f.z = kv8_pair<FMT>(st.v[u][2][w], st.v[u][3][w], (j & 1) ? s2 : s0);
        f.w = kv8_pair<FMT>(st.v[u][2][w], st.v[u][3][w], (j & 1) ? s3 : s1);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int p = PP - 1; p >= 0; --p) mma16816(o[j][n], f, pf[n][0][p], pf[n][1][p]);
      }
    }
  };

  if (steps > 0) {
    constexpr int PER = 32 / U;  // steps per resolve
    Stage st[2];
    resolve(0);
    load(st[0], 0);
#pragma unroll 1
    for (int it = 0; it < steps; it += 2) {
      if (it + 1 < steps) load(st[1], it + 1);
      compute(st[0]);
      if (it + 1 >= steps) break;
      if (it + 2 < steps) {
        if ((it + 2) % PER == 0) resolve(it + 2);
        load(st[0], it + 2);
      }
      compute(st[1]);
    }
  }

  // ---- join the warps
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[n][e];
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      const int qn = n * 8 + 2 * t + e;
      if (g == 0) sm.m[warp][qn] = m[n][e], sm.l[warp][qn] = x;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        sm.o[warp][qn][kv8_vdim<DH>(2 * j, g)] = o[j][n][e];
        sm.o[warp][qn][kv8_vdim<DH>(2 * j + 1, g)] = o[j][n][e + 2];
      }
    }
  __syncthreads();
  const float ln2 = 0.6931471805599453f;
  auto finish = [&](int qn, int d, float4 v, float M, float L) {
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // nothing visible: 0; NaN stays
    const long long at = (long long)row_of(qn) * a.os + (long long)head_of(qn) * a.ohs + d;
    kv8_st(a.out, a.dtype, at, v.x * inv);
    kv8_st(a.out, a.dtype, at + 1, v.y * inv);
    kv8_st(a.out, a.dtype, at + 2, v.z * inv);
    kv8_st(a.out, a.dtype, at + 3, v.w * inv);
    if (d == 0 && a.lse) a.lse[(size_t)row_of(qn) * a.Hq + head_of(qn)] = L == 0.f ? -INFINITY : (M + log2f(L)) * ln2;
  };
  for (int i = threadIdx.x; i < nq * (DH / 4); i += kKv8Warps * 32) {
    const int qn = i / (DH / 4), d = i % (DH / 4) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) M = fmaxf(M, sm.m[w][qn]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) {
      const float mw = sm.m[w][qn], f = mw == -INFINITY ? 0.f : ex2(mw - M);
      const float4 x = *reinterpret_cast<const float4*>(&sm.o[w][qn][d]);
      L += f * sm.l[w][qn];
      v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
    }
    if (CL == 1) {
      finish(qn, d, v, M, L);
    } else {
      *reinterpret_cast<float4*>(&sm.bo[qn][d]) = v;
      if (d == 0) sm.bm[qn] = M, sm.bl[qn] = L;
    }
  }
  if (CL == 1) return;
  // ---- join the cluster: each CTA finishes a share of the tile's outputs
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int i = rank * kKv8Warps * 32 + threadIdx.x; i < nq * (DH / 4); i += CL * kKv8Warps * 32) {
    const int qn = i / (DH / 4), d = i % (DH / 4) * 4;
    float M = -INFINITY, L = 0.f;
    for (int r = 0; r < CL; ++r) M = fmaxf(M, *cl.map_shared_rank(&sm.bm[qn], r));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < CL; ++r) {
      const float mr = *cl.map_shared_rank(&sm.bm[qn], r), f = mr == -INFINITY ? 0.f : ex2(mr - M);
      const float4 x = *reinterpret_cast<const float4*>(cl.map_shared_rank(&sm.bo[qn][d], r));
      L += f * *cl.map_shared_rank(&sm.bl[qn], r);
      v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
    }
    finish(qn, d, v, M, L);
  }
  cl.sync();  // the others may still read this CTA's sums
}

template <int DH, int FMT, int QP, int PP, int NQ>
cudaError_t kv8_attend_one(const Kv8View& c, const Kv8AttnArgs& a, int max_keys, int sm_count, cudaStream_t stream) {
  auto kern = k_kv8_attend<DH, FMT, QP, PP, NQ>;
  constexpr int smem = sizeof(Kv8Smem<DH, NQ>);
  const int tpr = (a.G + 8 * NQ - 1) / (8 * NQ);
  const long long tiles = a.sel_pages ? (long long)a.max_rows * tpr : ((long long)a.max_rows * a.G + 8 * NQ - 1) / (8 * NQ);
  long long keys = a.sel_pages ? (long long)a.n_select * c.PT : max_keys;
  keys = max(keys, 1ll);
  // Split the key axis over a cluster while the CTAs do not fill the GPU and each keeps a step per warp.
  int cl = 1;
  while (cl < 16 && tiles * c.H * c.batch * cl < sm_count && keys >= (long long)cl * 2 * kKv8Warps * kKv8Block) cl *= 2;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  if (cl > 8) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * cl), (unsigned)c.H, (unsigned)c.batch);
  cfg.blockDim = dim3(kKv8Warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, c, a, cl);
}

template <int DH, int FMT>
cudaError_t kv8_attend_dh(const Kv8View& c, const Kv8AttnArgs& a, int max_keys, int sm_count, cudaStream_t st) {
  // queries a tile: 8, or 16 where a tile can hold more than 8
  const bool wide = (a.sel_pages ? a.G : (long long)a.max_rows * a.G) > 8;
  if (a.dtype == BLT_T_F32)
    return wide && DH <= 64 ? kv8_attend_one<DH, FMT, 3, 3, (DH <= 64 ? 2 : 1)>(c, a, max_keys, sm_count, st)
                            : kv8_attend_one<DH, FMT, 3, 3, 1>(c, a, max_keys, sm_count, st);
  if (a.dtype == BLT_T_BF16)
    return wide ? kv8_attend_one<DH, FMT, 1, 2, 2>(c, a, max_keys, sm_count, st) : kv8_attend_one<DH, FMT, 1, 2, 1>(c, a, max_keys, sm_count, st);
  return wide ? kv8_attend_one<DH, FMT, 2, 2, 2>(c, a, max_keys, sm_count, st) : kv8_attend_one<DH, FMT, 2, 2, 1>(c, a, max_keys, sm_count, st);
}

}  // namespace bltdec
