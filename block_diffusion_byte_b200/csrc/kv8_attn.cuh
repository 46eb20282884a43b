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
// Codes become f16: both formats are exact in it (int8: 1024 + 128 + c read off the byte, less 1152; e4m3: the
// converter), and a two-plane f16 operand has 22 bits where bf16 has 16.  f16's range is met by powers of two:
// each query is scaled so that its largest channel lies in [2^14, 2^15), and weights times their block's scale are
// taken relative to the largest block scale that the query has seen so far (times 2^14).  What lies 2^38 below the largest
// is cut.
//
// Each warp takes 16-key units of its own with its own running maximum and sum, and copies them (cp.async)
// through a ring of its own in shared memory, kKv8Stages - 1 steps ahead: no barrier stands between the warps, and
// the bytes in flight (two CTAs of eight warps, 8 KB each ahead: 128 KB an SM) cover the memory's latency.
// Warps are joined in shared memory, and the CTAs that split a long key axis (a cluster) over distributed
// shared memory, in a fixed order: no workspace, no second launch, no atomics.
//
// The tensor cores cut sums to fp32 where they do not round them; a warp's chain of products is short (keys / 16 / warps / CTAs
// of the cluster), and fp32 outputs are 4e-7 off at 1028 keys, 8e-7 at 1024 selected ones (plain fp32: 4e-7, 5e-7).
//
// Bound by memory at long contexts: 64 sequences of 4096 to 8192 keys, 8 heads of 128, four query heads each, e4m3: 154 to
// 172 us with the lengths drawn, 5.2 TB/s (0.79 of the measured copy rate); the rest is uneven ends and the dependent work
// of a warp's step (about 340 instructions for 16 keys).  By the chain of lookups at its start (row range, limit, page,
// exponents: about 4 us) when short: 4 rows at 1028 keys, 16 heads of 64, fp32: 6.9 us; one row at 8192: 12.7 us.  Steps on
// the way, on the 64 sequences of one draw: codes as bf16 with the next step in registers, one CTA an SM 282 us; f16 and the
// ring 171 us; queries loaded at once 164 us; pieces moved off shared banks 158 us; keys in halves 150 us; value scales as
// each query sees them 153 us; finite factors 154 us.
#pragma once

#include <cooperative_groups.h>

#include <cfloat>

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

// A unit in shared memory: rows of keys (values) as they come, 16-byte pieces moved about inside each 128 bytes so that
// the lanes of a load meet different banks.  K: lanes read pieces t of rows g; V: pieces g / 2 or g of rows 2t.
template <int DH>
__device__ __forceinline__ int kv8_kplace(int piece) {  // of piece row * DH / 16 + column
  return DH == 128 ? piece ^ ((piece >> 3 & 1) << 2) : piece;
}
template <int DH>
__device__ __forceinline__ int kv8_vplace(int piece) {
  return DH % 64 == 0 ? piece ^ ((piece / (DH / 8) & 3) << 1) : piece;
}
template <int DH>
__device__ __forceinline__ void kv8_load_krow(uint32_t (&w)[DH / 16], const uint8_t* unit, int row, int t) {
  constexpr int CB = kv8_kpiece<DH>();
#pragma unroll
  for (int i = 0; i < DH / 16; i += CB / 4) {
    if constexpr (CB == 16) {
      const uint4 x = *reinterpret_cast<const uint4*>(unit + kv8_kplace<DH>(row * (DH / 16) + kv8_kdim<DH>(i, t) / 16) * 16);
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(unit + row * DH + kv8_kdim<DH>(i, t));
      w[i] = x.x, w[i + 1] = x.y;
    }
  }
}
template <int DH>
__device__ __forceinline__ void kv8_load_vrow(uint32_t (&w)[DH / 32], const uint8_t* unit, int row, int g) {
  constexpr int VB = kv8_vpiece<DH>();
  if constexpr (VB == 16) {
    const uint4 x = *reinterpret_cast<const uint4*>(unit + kv8_vplace<DH>(row * 8 + g) * 16);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
  } else if constexpr (VB == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(unit + kv8_vplace<DH>(row * 4 + (g >> 1)) * 16 + (g & 1) * 8);
    w[0] = x.x, w[1] = x.y;
  } else {
#pragma unroll
    for (int j = 0; j < DH / 32; ++j) w[j] = *reinterpret_cast<const uint32_t*>(unit + row * DH + j * 32 + g * 4);
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

// P planes of two fp32 values as packed f16: the sum of the planes has 11 P bits of the value (|x| < 65504).
template <int P>
__device__ __forceinline__ void kv8_planes(float x0, float x1, uint32_t (&pl)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const __half2 h = __floats2half2_rn(x0, x1);
    pl[i] = *reinterpret_cast<const uint32_t*>(&h);
    if (i + 1 < P) {
      const float2 f = __half22float2(h);
      x0 -= f.x, x1 -= f.y;
    }
  }
}

// The four codes of word w as f16: channels 0, 1 and 2, 3.
template <int FMT>
__device__ __forceinline__ uint2 kv8_half4(uint32_t w) {
  uint2 d;
  if constexpr (FMT == 0) {
    const uint32_t x = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(d.x) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(d.y) : "r"(b), "r"(0x64806480u));
  } else {
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n" : "=r"(d.x), "=r"(d.y) : "r"(w));
  }
  return d;
}
// Codes 2 j and 2 j + 1 of words a and b as f16 pairs (a's in the lower half): channel 2 j, channel 2 j + 1.
template <int FMT>
__device__ __forceinline__ uint2 kv8_half_pairs(uint32_t a, uint32_t b, int j) {
  uint2 d;
  if constexpr (FMT == 0) {
    const uint32_t x = (__byte_perm(a, b, j ? 0x0602 : 0x0400) & 0x00ff00ffu) ^ 0x64806480u;
    const uint32_t y = (__byte_perm(a, b, j ? 0x0703 : 0x0501) & 0x00ff00ffu) ^ 0x64806480u;
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(d.x) : "r"(x), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;\n" : "=r"(d.y) : "r"(y), "r"(0x64806480u));
    return d;
  } else {
    return kv8_half4<1>(__byte_perm(a, b, j ? 0x7362 : 0x5140));
  }
}

// D += A(16x16, f16, row) * B(16x8, f16, col), fp32 accumulate.
__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint4& a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

constexpr int kKv8Stages = 3;
template <int DH>
__host__ __device__ constexpr int kv8_units() { return DH <= 64 ? 2 : 1; }  // units per step: 4 KB (2 KB for DH 32)

template <int DH, int NQ>
struct alignas(16) Kv8WarpSmem {
  static constexpr int OS = DH + 4;  // row stride of a partial output (floats): breaks bank alignment of the rows
  union {
    uint8_t ring[kKv8Stages][kv8_units<DH>()][2][kKv8Block * DH];
    float o[8 * NQ][OS];
  };
  int2 meta[kKv8Stages][kv8_units<DH>()];  // position and exponents (keys' | values' << 8) of a staged unit
  float m[8 * NQ], l[8 * NQ];
};
template <int DH, int NQ>
struct alignas(16) Kv8Smem {
  float bo[8 * NQ][DH + 4];  // the CTA's own sums, read by the cluster
  float bm[8 * NQ], bl[8 * NQ];
  Kv8WarpSmem<DH, NQ> w[1];  // of each warp
};
template <int DH, int NQ>
constexpr size_t kv8_smem(int warps) {
  return sizeof(Kv8Smem<DH, NQ>) + (warps - 1) * sizeof(Kv8WarpSmem<DH, NQ>);
}

// Registers decide the CTAs an SM holds: two where a lane's queries and outputs leave room.
template <int DH, int QP, int NQ>
__host__ __device__ constexpr int kv8_ctas() { return NQ * (DH / 16) * (2 * QP + 4) <= 64 ? 2 : 1; }

// grid (tiles x CL, key/value heads, sequences), clusters of CL along x.
template <int DH, int FMT, int QP, int PP, int NQ>
__global__ void __launch_bounds__(kKv8Warps * 32, kv8_ctas<DH, QP, NQ>()) k_kv8_attend(const __grid_constant__ Kv8View c, const __grid_constant__ Kv8AttnArgs a,
                                                                const int CL) {
  constexpr int U = kv8_units<DH>(), S = kKv8Stages;
  constexpr int KW = DH / 16, VW = DH / 32, MT = DH / 16;
  constexpr int DT = QP == 2 ? BLT_T_F32 : PP == 1 ? BLT_T_BF16 : BLT_T_F16;  // a.dtype
  extern __shared__ float4 kv8_smem4[];
  Kv8Smem<DH, NQ>& sm = *reinterpret_cast<Kv8Smem<DH, NQ>*>(kv8_smem4);
  const int tile = blockIdx.x / CL, rank = blockIdx.x % CL, kvh = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3, W = blockDim.x >> 5;
  Kv8WarpSmem<DH, NQ>& mine = sm.w[warp];

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
  const int steps = max(0, (u1 - u0 + U - 1) / U - warp + W - 1) / W;

  // pages, positions and exponents of the warp's next 32 units, one per lane
  int c_page = -1, c_pos = kKv8NoPos, c_ex = 0;
  auto resolve = [&](int it0) {
    const int u = u0 + (warp + W * (it0 + lane / U)) * U + lane % U;
    c_page = -1;
    c_pos = kKv8NoPos;
    c_ex = 127;
    if (it0 + lane / U >= steps || u >= u1) return;
    const int e = kv8_div_tpp(c, u), sub = u - e * c.tpp;
    int pl = e;
    if (sel) {
      pl = __ldg(list + e);
      const int prev = e > 0 ? __ldg(list + e - 1) : -1;
      if (pl < 0 || pl <= prev || pl >= c.max_pages) return;
    }
    const int pos = pl * c.PT + sub * kKv8Block;
    if (pos >= maxlim) return;
    c_page = kv8_page(c, s, pl);
    if (c_page < 0) return;
    c_pos = pos;
    const size_t ex = (size_t)c_page * c.exp_stride + kvh * c.tpp + sub;
    c_ex = __ldg(c.ke + ex) | __ldg(c.ve + ex) << 8;
  };
  constexpr int PER = 32 / U;  // steps per resolve
  auto issue = [&](int it, int slot) {  // copies of step `it`
    if (it < steps) {
      if (it % PER == 0) resolve(it);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int src = (it * U + u) & 31;
        const int page = __shfl_sync(0xffffffffu, c_page, src), pos = __shfl_sync(0xffffffffu, c_pos, src);
        if (page < 0) continue;
        const int blk = pos / kKv8Block, sub = blk - kv8_div_tpp(c, blk) * c.tpp;
        const size_t at = (size_t)page * c.page_stride + ((size_t)kvh * c.PT + sub * kKv8Block) * DH;
        uint8_t* dst = mine.ring[slot][u][0];
#pragma unroll
        for (int i = lane; i < DH; i += 32) {
          cp_async16(dst + kv8_kplace<DH>(i) * 16, c.k + at + i * 16, 16);
          cp_async16(dst + kKv8Block * DH + kv8_vplace<DH>(i) * 16, c.v + at + i * 16, 16);
        }
      }
    }
    cp_async_commit();
  };
  auto note = [&](int it, int slot) {  // what the copies of step `it` are
    if (it >= steps) return;
    const int src = (it * U + lane) & 31;
    const int pos = __shfl_sync(0xffffffffu, c_pos, src), ex = __shfl_sync(0xffffffffu, c_ex, src);
    if (lane < U) mine.meta[slot][lane] = make_int2(pos, ex);
  };
  for (int i = 0; i < S - 1; ++i) issue(i, i);
  for (int i = 0; i < S - 1; ++i) note(i, i);

  // query fragments (B operand): k16 step i holds the channels of key byte group i.  A query is scaled by a power
  // of two; `qs` undoes it for queries 2t and 2t + 1, times the scale and log2 e: scores are in units of log 2.
  uint32_t qf[NQ][KW][2][QP];
  float qs[NQ][2];
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    const int qn = n * 8 + g;
    const long long base = qn < nq ? (long long)row_of(qn) * a.qs + (long long)head_of(qn) * a.qhs : 0;
    float x[KW][4];
#pragma unroll
    for (int i = 0; i < KW; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = 0.f;
    if (qn < nq && a.q_vec) {
#pragma unroll
      for (int i = 0; i < KW; ++i) kv8_ld4(a.q, DT, base + kv8_kdim<DH>(i, t), true, x[i]);
    } else if (qn < nq) {
#pragma unroll
      for (int i = 0; i < KW; ++i) kv8_ld4(a.q, DT, base + kv8_kdim<DH>(i, t), false, x[i]);
    }
    float big = 0.f;
#pragma unroll
    for (int i = 0; i < KW; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) big = fmaxf(big, fabsf(x[i][j]));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    const int ex = max((int)(__float_as_uint(big) >> 23), 15);
    const float up = copysignf(kv8_pow2(268 - ex), a.scale), down = kv8_pow2(ex - 14);  // the sign of the scale with the query
#pragma unroll
    for (int i = 0; i < KW; ++i) {
      kv8_planes<QP>(x[i][0] * up, x[i][1] * up, qf[n][i][0]);
      kv8_planes<QP>(x[i][2] * up, x[i][3] * up, qf[n][i][1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) qs[n][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4) * fabsf(a.scale) * 1.4426950408889634f;  // in this order: a scale near fp32's largest
  }

  float m[NQ][2], l[NQ][2], o[MT][NQ][4];
  int vref[NQ][2];  // the largest value exponent that the query has seen; its outputs are in units of 2^(vref - 127 - 14)
#pragma unroll
  for (int n = 0; n < NQ; ++n) {
    m[n][0] = m[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
    vref[n][0] = vref[n][1] = kKv8LowExp;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][n][e] = 0.f;
  }

  auto compute = [&](int slot) {
    float sc[U][NQ][4];
    int pos[U], ve[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int2 meta = mine.meta[slot][u];
      pos[u] = meta.x;
      ve[u] = meta.y >> 8;
      const uint8_t* kp = mine.ring[slot][u][0];
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][n][e] = 0.f;
      float odd[4] = {0.f, 0.f, 0.f, 0.f};  // one query group: two chains of products, as no other work stands between them
      uint32_t k0[KW], k1[KW];
      kv8_load_krow<DH>(k0, kp, g, t);
      kv8_load_krow<DH>(k1, kp, g + 8, t);
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const uint2 x = kv8_half4<FMT>(k0[i]), y = kv8_half4<FMT>(k1[i]);
        const uint4 f = make_uint4(x.x, y.x, x.y, y.y);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int p = QP - 1; p >= 0; --p) mma16816_f16(NQ == 1 && (i & 1) ? odd : sc[u][n], f, qf[n][i][0][p], qf[n][i][1][p]);
      }
      if constexpr (NQ == 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[u][0][e] += odd[e];
      }
      const float ks = kv8_pow2(meta.y & 0xff);
      const bool whole = pos[u] + kKv8Block <= minlim;
      float f[NQ][2];  // finite, so that a score of 0 stays 0
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) f[n][e] = fminf(ks * qs[n][e], FLT_MAX);
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[u][n][e] = __fmul_rn(sc[u][n][e], f[n][e & 1]);  // rounded before it meets the maximum, which is
          if (!whole && pos[u] + g + (e >> 1) * 8 >= lim[n][e & 1]) sc[u][n][e] = -INFINITY;
        }
    }
    bool grow = false;
    float mn[NQ][2];
    int vn[NQ][2];
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
        int y = vref[n][e];
#pragma unroll
        for (int u = 0; u < U; ++u) y = max(y, pos[u] < lim[n][e] ? ve[u] : 0);
        vn[n][e] = y;
        grow |= x > m[n][e] || y > vref[n][e];
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
          f[e] *= kv8_pow2(max(127 + vref[n][e] - vn[n][e], 0));  // beyond 2^-126: nothing is left of the sums
          vref[n][e] = vn[n][e];
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
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        float p[4], vs[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) vs[e] = kv8_pow2(min(max(141 + ve[u] - vref[n][e], 0), 141));  // 2^(14 + ve - vref); louder: not seen
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float mx = m[n][e & 1];
          p[e] = ex2(sc[u][n][e] - (mx == -INFINITY ? 0.f : mx));
          l[n][e & 1] += p[e];
          p[e] *= vs[e & 1];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t pl[PP];
          kv8_planes<PP>(p[2 * e], p[2 * e + 1], pl);  // key g + 8 e, queries 2t, 2t + 1
#pragma unroll
          for (int x = 0; x < PP; ++x) pf[n][e][x] = movmatrix_trans(pl[x]);  // query g, keys 2t + 8 e, 2t + 1 + 8 e
        }
      }
      uint32_t v[4][VW];
      const uint8_t* vp = mine.ring[slot][u][1];
#pragma unroll
      for (int r = 0; r < 4; ++r) kv8_load_vrow<DH>(v[r], vp, 2 * t + (r & 1) + (r >> 1) * 8, g);
      if (pos[u] + kKv8Block > maxlim) {  // weight 0, but what lies there may be no number
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (pos[u] + 2 * t + (r & 1) + (r >> 1) * 8 >= maxlim)
#pragma unroll
            for (int i = 0; i < VW; ++i) v[r][i] = 0;
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {  // channels of value bytes 2j and 2j + 1
        const uint2 x = kv8_half_pairs<FMT>(v[0][j >> 1], v[1][j >> 1], j & 1), y = kv8_half_pairs<FMT>(v[2][j >> 1], v[3][j >> 1], j & 1);
        const uint4 f = make_uint4(x.x, x.y, y.x, y.y);
#pragma unroll
        for (int n = 0; n < NQ; ++n)
#pragma unroll
          for (int p = PP - 1; p >= 0; --p) mma16816_f16(o[j][n], f, pf[n][0][p], pf[n][1][p]);
      }
    }
  };

  {
    int slot = 0, fill = S - 1;
#pragma unroll 1
    for (int it = 0; it < steps; ++it) {
      cp_async_wait<S - 2>();
      __syncwarp();  // every lane's copies of this step are there, and the slot to fill has been read by all
      issue(it + S - 1, fill);
      note(it + S - 1, fill);
      compute(slot);
      slot = slot + 1 == S ? 0 : slot + 1;
      fill = fill + 1 == S ? 0 : fill + 1;
    }
    cp_async_wait<0>();
  }
  __syncwarp();  // the ring's memory takes the partial outputs

  // ---- join the warps
#pragma unroll
  for (int n = 0; n < NQ; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[n][e];
      const float vs = kv8_pow2(vref[n][e] - 14);
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      const int qn = n * 8 + 2 * t + e;
      if (g == 0) mine.m[qn] = m[n][e], mine.l[qn] = x;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        mine.o[qn][kv8_vdim<DH>(2 * j, g)] = o[j][n][e] * vs;
        mine.o[qn][kv8_vdim<DH>(2 * j + 1, g)] = o[j][n][e + 2] * vs;
      }
    }
  __syncthreads();
  const float ln2 = 0.6931471805599453f;
  auto finish = [&](int qn, int d, float4 v, float M, float L) {
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);  // nothing visible: 0; NaN stays
    const long long at = (long long)row_of(qn) * a.os + (long long)head_of(qn) * a.ohs + d;
    kv8_st4(a.out, DT, at, a.out_vec, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    if (d == 0 && a.lse) a.lse[(size_t)row_of(qn) * a.Hq + head_of(qn)] = L == 0.f ? -INFINITY : (M + log2f(L)) * ln2;
  };
  for (int i = threadIdx.x; i < nq * (DH / 4); i += W * 32) {
    const int qn = i / (DH / 4), d = i % (DH / 4) * 4;
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w)
      if (w < W) M = fmaxf(M, sm.w[w].m[qn]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kKv8Warps; ++w) {
      if (w >= W) break;
      const float mw = sm.w[w].m[qn], f = mw == -INFINITY ? 0.f : ex2(mw - M);
      const float4 x = *reinterpret_cast<const float4*>(&sm.w[w].o[qn][d]);
      L += f * sm.w[w].l[qn];
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
  for (int i = rank * W * 32 + threadIdx.x; i < nq * (DH / 4); i += CL * W * 32) {
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
  const int tpr = (a.G + 8 * NQ - 1) / (8 * NQ);
  const long long tiles = a.sel_pages ? (long long)a.max_rows * tpr : ((long long)a.max_rows * a.G + 8 * NQ - 1) / (8 * NQ);
  const long long ctas = tiles * c.H * c.batch;
  long long keys = a.sel_pages ? (long long)a.n_select * c.PT : max_keys;
  keys = max(keys, 1ll);
  // Split the key axis over a cluster while the CTAs do not fill the GPU and each keeps a step per warp (one byte at 8192
  // keys, 16 heads: 38.5 us whole, 13 us in eighths), and where CTAs are long enough that their end is uneven (64 sequences
  // of 4096 to 8192 keys, 8 heads: 158 us whole, 149 us in halves; 16 of 4096, 16 heads: 32 and 36 us).
  int cl = 1;
  while (cl < 8 && ((ctas * cl < sm_count && keys >= (long long)cl * 2 * kKv8Warps * kKv8Block) ||
                    (ctas * cl < 8 * sm_count && keys >= (long long)cl * 6144)))
    cl *= 2;
  // Eight warps a CTA, or four where many short CTAs wait for one another's start (1024 CTAs of 1024 selected keys: 43 us
  // with eight warps, 36 us with four; 16 x 16 CTAs of 4096 keys: 32 and 36 us).
  const int warps = ctas * cl >= 4 * sm_count && keys <= 2048 ? kKv8Warps / 2 : kKv8Warps;
  const int smem = (int)kv8_smem<DH, NQ>(warps);
  const cudaError_t e = kv8_allow_smem<k_kv8_attend<DH, FMT, QP, PP, NQ>>((int)kv8_smem<DH, NQ>(kKv8Warps));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * cl), (unsigned)c.H, (unsigned)c.batch);
  cfg.blockDim = dim3(warps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1;
  return cudaLaunchKernelEx(&cfg, kern, c, a, cl);
}

template <int DH, int FMT>
cudaError_t kv8_tile_dh(const Kv8View& c, const Kv8AttnArgs& a, long long tiles, int max_keys, int sm_count, cudaStream_t st);

template <int DH, int FMT>
cudaError_t kv8_attend_dh(const Kv8View& c, const Kv8AttnArgs& a, int max_keys, int sm_count, cudaStream_t st) {
  // Many rows against many keys: tiles of 128 queries on tcgen05.  Such a CTA takes longer to start and to end (20 us), and a
  // tile of few rows is mostly idle.  Few-row kernel / tiles, us, 16 heads of 64, bf16: 64 rows at 8192 keys 27 / 32, 96
  // rows 45 / 31; 256 rows at 1024 keys 16 / 21; 8 sequences of 4096 keys, 64 rows 68 / 58, 48 rows 53 / 62.  8 heads of
  // 128, f16: 48 rows at 8192 keys 35 / 33, 64 rows 51 / 33; 256 rows at 1024 keys 24 / 28.
  const long long queries = (long long)a.max_rows * a.G, tiles = (queries + 127) / 128;
  if (!a.sel_pages && queries >= 64 && queries * max_keys >= 3 << 17 && tiles * c.H * c.batch <= INT_MAX / 8)
    return kv8_tile_dh<DH, FMT>(c, a, tiles, max_keys, sm_count, st);
  // queries a tile: 8, or 16 where a tile can hold more than 8
  const bool wide = (a.sel_pages ? a.G : (long long)a.max_rows * a.G) > 8;
  // planes (11 bits each) of the queries and of the weights: fp32 two and two; bf16 and f16 queries fit one; weights one
  // for bf16 (its own step is 16 times coarser) and two for f16
  if (a.dtype == BLT_T_F32)
    return wide ? kv8_attend_one<DH, FMT, 2, 2, 2>(c, a, max_keys, sm_count, st) : kv8_attend_one<DH, FMT, 2, 2, 1>(c, a, max_keys, sm_count, st);
  if (a.dtype == BLT_T_BF16)
    return wide ? kv8_attend_one<DH, FMT, 1, 1, 2>(c, a, max_keys, sm_count, st) : kv8_attend_one<DH, FMT, 1, 1, 1>(c, a, max_keys, sm_count, st);
  return wide ? kv8_attend_one<DH, FMT, 1, 2, 2>(c, a, max_keys, sm_count, st) : kv8_attend_one<DH, FMT, 1, 2, 1>(c, a, max_keys, sm_count, st);
}

}  // namespace bltdec
