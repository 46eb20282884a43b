// Attention over the 8-bit paged KV cache for many query rows (prompts): 128 queries against tiles of keys on the
// 5th-generation tensor cores.
//
// A CTA takes 128 queries -- (row, query head) pairs of one sequence that share a key/value head -- and walks its
// keys in tiles of N.  Per tile  S = Q K^T  (128 x N, fp32 in tensor memory),  P = exp2(S c - m),  O += P V  with P read
// from tensor memory, so neither S nor P passes through shared memory.  Three roles:
//   warps 0-3  a thread a query: S from tensor memory, running maximum and sum, P back into tensor memory;
//   warps 4-6  codes to f16 operands in shared memory (128-byte swizzle: K as rows of channels, V as rows of channels
//              too, taken MN-major), a few tiles deep.  The codes of a block of 16 positions are one bulk copy into the
//              place of the operand, converted there;
//   warp 7     one thread issues the products.
// Two CTAs share an SM (heads of up to 64; one where a tile's operands take 32 KB), so one's products run under the
// other's exponentials.  Codes are exact in f16 and enter as they are.  A block's key scale joins the factor of its
// scores, its value scale the weights, relative to the largest one that the row itself sees: a loud block takes nothing
// from its neighbours' keys, nor anything from rows that do not see it.  O is corrected only when a row's maximum has grown
// by more than 2^6 (weights carry 2^8 as room above f16's least) or a louder value scale comes.
// Every wait is bounded; one that runs out ends the CTA with BLT_ERR_DEVICE in the status word, and no CTA of its cluster
// stores the tile's rows.
//
// Bound by the weights' work: one exponential each on the 16-a-clock unit (512 clocks a tile) and, in a thread, the chain
// score -> maximum -> exponential -> f16 -> tensor memory (about 1000 clocks a tile and CTA, two CTAs an SM); the
// products take 350 clocks a tile (one f16 plane each) and never wait.  Four causal prompts of 2048, 16 heads of 64, bf16:
// 100 us, 344 TFLOP/s; 1024 fp32 rows at 8192 keys (two planes of q and of the weights): 111 us, 290 TFLOP/s.  Steps on
// the way (the two in turn): 128-key tiles, S and P in one place 195, 327 us; masked and whole tiles apart 123, 186;
// 64-key tiles with the next tile's S under this one's weights 105, 146; bulk copies converted in place, a warp a tile,
// three S tiles 95, 132 (with one barrier for the weights of all tiles, which was wrong; 100 with one a tile); keys split
// over a cluster where tiles are few -, 100; fp32 sums in chains of 8 tiles -, 105; scales of blocks in the scores and weights
// instead of the operands, scores of any size 100, 111.
#pragma once

#include <cfloat>
#include <cstddef>

#include "kv8.cuh"
#include "kv8_attn.cuh"

namespace bltdec {

constexpr int kKvtQ = 128;                            // queries a tile (tensor memory lanes)
constexpr int kKvtThreads = 256;                      // 16 warps of two CTAs leave 128 registers a thread
constexpr int kKvtLoaders = 3;                        // warps that convert, a tile each in turn
constexpr long long kKvtWaitClocks = 2000000000ll;    // about a second
constexpr long long kKvtStallClocks = 20000000ll;     // where the waits are to run out
constexpr float kKvtLargeScore = 1048576.f;           // 2^20 (log 2): half a step of fp32 is 2^-4 there
// 2^-60: a product is at most 2^31, so that a score below this scale is 2^-29 at most and may as well be of this scale; and
// scores of up to 2^67 are within fp32's range in its units
constexpr float kKvtLeastScale = 8.673617379884035e-19f;
constexpr float kKvtGrow = 6.f;                       // growth of the maximum (log 2) that is let stand
constexpr int kKvtShift = 8;                          // weights are at most 2^(kKvtGrow + kKvtShift) < 65504
// Least power of two that a weight is taken times: in f16 a weight (at most 2^kKvtGrow) rounds to 0 then, and l still has it.
constexpr int kKvtLeast = -40;

constexpr int kKvtN = 64;                             // keys a tile
// Tiles of operands in shared memory: four and two CTAs an SM, or one CTA where a tile takes 32 KB.
template <int DH, int QP>
__host__ __device__ constexpr int kvt_slots() { return DH > 64 && QP == 1 ? 5 : 4; }
// The tensor cores cut each sum to fp32 instead of rounding it, so a long chain of products drifts (fp32 outputs at 8192
// keys: 8.2e-6 off).  fp32 rows end the chain after this many tiles and add it to a total with rounding (1.7e-6, plain fp32
// 1.7e-6); 0: one chain, for bf16 and f16 rows, whose own rounding is up to 2^-9 and 2^-12 of a number (the drift grows with
// the keys: at this rate it is that of f16 at about 200000).
template <int QP>
__host__ __device__ constexpr int kvt_fold() { return QP == 2 ? 8 : 0; }
template <int DH, int QP>
__host__ __device__ constexpr int kvt_bufs() { return DH <= 64 && kvt_fold<QP>() ? 2 : 3; }  // tiles of S in tensor memory
template <int DH>
__host__ __device__ constexpr int kvt_cols() { return DH <= 64 ? 64 : 128; }  // columns of O (whole swizzle atoms of V)

template <int DH, int QP>
struct KvtSmem {
  static constexpr int HALVES = DH > 64 ? 2 : 1;  // swizzle atoms of 64 channels
  uint8_t q[QP][HALVES][kKvtQ * 128];
  static constexpr int SLOTS = kvt_slots<DH, QP>();
  uint8_t k[SLOTS][HALVES][kKvtN * 128];
  uint8_t v[SLOTS][HALVES][kKvtN * 128];
  int4 meta[SLOTS];  // a tile's key exponents and value exponents (a byte a block), missing blocks (bits), largest key << 8 | value exponent
  uint64_t q_full, drained, raw_full[SLOTS], kv_full[SLOTS], kv_empty[SLOTS], s_full[kvt_bufs<DH, QP>()], p_full[kvt_bufs<DH, QP>()], o_done[kvt_bufs<DH, QP>()];
  uint32_t tmem;
  int max_lim, ok;
};
template <int DH>
struct KvtSums {  // a CTA's sums, in place of the operands
  float o[kKvtQ][DH + 4];
  float2 ml[kKvtQ];
};
template <int DH, int QP>
__host__ __device__ constexpr size_t kvt_smem() { return sizeof(KvtSmem<DH, QP>) + 1024; }

// ------------------------------------------------------------------------ primitives
// Shared-memory operand of 128-byte rows with 128-byte swizzle, 8-row groups 1024 bytes apart.  `lead`: bytes between
// atoms of 64 channels for an MN-major operand (unused for a K-major one).
__device__ __forceinline__ uint64_t kvt_desc(uint32_t saddr, uint32_t lead) {
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lead >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
// f16 x f16 -> fp32, M 128, N n; A K-major; B K-major or MN-major.
__host__ __device__ constexpr uint32_t kvt_idesc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kKvtQ >> 4) << 24);
}
__device__ __forceinline__ void kvt_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void kvt_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b),
      "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ bool kvt_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void kvt_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void kvt_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void kvt_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void kvt_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void kvt_ld_wait(float (&v)[32]) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));  // the values are read after the wait
}
__device__ __forceinline__ void kvt_ld16(uint32_t taddr, uint32_t (&r)[16]) {  // waited for
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void kvt_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]),
      "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void kvt_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void kvt_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// A whole warp waits for phase `parity` of a barrier; false for all its lanes once `clocks` are over.  (The SM's clock, not
// the global timer, whose reading takes as long as a product.)
__device__ __forceinline__ bool kvt_wait(uint64_t* b, unsigned parity, long long clocks) {
  bool done = mbar_try(b, parity);
  if (__all_sync(0xffffffffu, done)) return true;
  const long long t0 = clock64();
  while (true) {
    done = done || mbar_try(b, parity);
    if (__all_sync(0xffffffffu, done)) return true;
    if (__any_sync(0xffffffffu, clock64() - t0 > clocks)) return false;
  }
}
// Chunk c (16 bytes, 8 f16) of a 128-byte row in the 128-byte swizzle.
__device__ __forceinline__ int kvt_swz(int row, int c) { return row * 128 + ((c ^ (row & 7)) << 4); }

// grid: query tiles x sequences x key/value heads, flat, the tile slowest and the last tile (the most keys of a causal
// prompt) first, so that long CTAs start early.
template <int DH, int FMT, int QP, int PP>
__global__ void __launch_bounds__(kKvtThreads, kvt_smem<DH, QP>() <= 113 * 1024 ? 2 : 1)
    k_kv8_tile(const __grid_constant__ Kv8View c, const __grid_constant__ Kv8AttnArgs a, const int n_tiles, const int CL) {
  constexpr int N = kKvtN, NV = kvt_cols<DH>(), NB = N / kKv8Block, SLOTS = kvt_slots<DH, QP>(), BUFS = kvt_bufs<DH, QP>();
  constexpr int FOLD = kvt_fold<QP>();
  // tensor memory: tiles of S (P's planes in place, N / 2 columns each), O, the total of the chains before
  constexpr int COL_O = BUFS * N, COL_T = COL_O + NV, COLS = COL_T + (FOLD ? NV : 0) <= 256 ? 256 : 512;
  static_assert(COLS == 256 || kvt_smem<DH, QP>() > 113 * 1024, "two CTAs share an SM's 512 columns");
  constexpr int DT = QP == 2 ? BLT_T_F32 : PP == 1 ? BLT_T_BF16 : BLT_T_F16;  // a.dtype
  extern __shared__ uint8_t kvt_raw[];
  KvtSmem<DH, QP>& sm = *reinterpret_cast<KvtSmem<DH, QP>*>((reinterpret_cast<uintptr_t>(kvt_raw) + 1023) & ~(uintptr_t)1023);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x % CL, item = blockIdx.x / CL;
  auto wait = [&](uint64_t* b, unsigned parity) { return kvt_wait(b, parity, a.stall ? kKvtStallClocks : kKvtWaitClocks); };
  const int kvh = item % c.H, s = item / c.H % c.batch, tile = n_tiles - 1 - item / c.H / c.batch;
  int r0, r1;
  kv8_rows_of(a.row_off, s, a.n_rows, a.max_rows, c.status, r0, r1);
  const int qbase = tile * kKvtQ, nq = min((r1 - r0) * a.G - qbase, kKvtQ);
  if (nq <= 0) return;  // the same for every CTA of a cluster

  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, kKvtQ);
    mbar_init(&sm.drained, 1);
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(sm.raw_full + i, 1);
      mbar_init(sm.kv_full + i, 32);
      mbar_init(sm.kv_empty + i, 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(sm.s_full + i, 1);
      mbar_init(sm.p_full + i, kKvtQ);  // one a buffer: a warp may be done with the next tile before another with this
      mbar_init(sm.o_done + i, 1);
    }
    sm.max_lim = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 7) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sm.tmem)), "r"(COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
  }
  int lim = 0;
  const int cap = c.max_pages * c.PT;
  const int qrow = r0 + (qbase + (int)threadIdx.x) / a.G, qhead = kvh * a.G + (qbase + (int)threadIdx.x) % a.G;
  if (warp < 4 && (int)threadIdx.x < nq) {
    lim = __ldg(a.row_limit + qrow);
    if (lim > cap) {
      if (c.status) set_status(c.status, kErrDevice);
      lim = cap;
    }
    lim = max(lim, 0);
  }
  __syncthreads();
  if (warp < 4) {
    const int wl = __reduce_max_sync(0xffffffffu, lim);
    if (lane == 0) atomicMax(&sm.max_lim, wl);
  }
  kvt_before();
  __syncthreads();
  kvt_after();
  const uint32_t tmem = sm.tmem;
  // this CTA's tiles: j0 .. j0 + nt - 1 of the keys' (the loops below count from 0)
  const int max_lim = sm.max_lim, all_tiles = (max_lim + N - 1) / N, per = (all_tiles + CL - 1) / CL;
  const int j0 = min(rank * per, all_tiles), nt = min(per, all_tiles - j0);
  bool ok = true;
  KvtSums<DH>& sums = *reinterpret_cast<KvtSums<DH>*>(&sm);

  if (warp < 4) {
    // ------------------------------------------------------------------ a thread a query
    const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
    const bool mine = (int)threadIdx.x < nq;
    // the query scaled so that its largest channel lies in [2^14, 2^15), the sign of the scale with it
    const long long qat = mine ? (long long)qrow * a.qs + (long long)qhead * a.qhs : 0;
    constexpr int QC = DH <= 64 ? DH : 32;  // channels in registers at once (all loads of a row in flight where they fit)
    float x[QC];
    float big = 0.f;
    auto fetch = [&](int c0) {
      if (a.q_vec) {
#pragma unroll
        for (int i = 0; i < QC; i += 8) {
          float y[8] = {};
          if (mine) kv8_ld8(a.q, DT, qat + c0 + i, true, y);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[i + e] = y[e];
        }
      } else {
#pragma unroll
        for (int i = 0; i < QC; ++i) x[i] = mine ? kv8_ld(a.q, DT, qat + c0 + i) : 0.f;
      }
    };
#pragma unroll
    for (int c0 = 0; c0 < DH; c0 += QC) {
      fetch(c0);
#pragma unroll
      for (int i = 0; i < QC; ++i) big = fmaxf(big, fabsf(x[i]));
    }
    const int ex = max((int)(__float_as_uint(big) >> 23), 15);
    const float up = a.scale == 0.f ? 0.f : copysignf(kv8_pow2(268 - ex), a.scale);
    const float qs = a.scale == 0.f ? 1.f : kv8_pow2(ex - 14) * fabsf(a.scale) * 1.4426950408889634f;  // in this order: a scale near fp32's largest
#pragma unroll
    for (int c0 = 0; c0 < DH; c0 += QC) {
      if (nt == 0) break;  // the memory is the sums' at once
      if (QC < DH) fetch(c0);
#pragma unroll
      for (int i = 0; i < QC; i += 8) {
        uint32_t w[4][QP];
#pragma unroll
        for (int e = 0; e < 4; ++e) kv8_planes<QP>(x[i + 2 * e] * up, x[i + 2 * e + 1] * up, w[e]);
#pragma unroll
        for (int p = 0; p < QP; ++p)
          *reinterpret_cast<uint4*>(&sm.q[p][(c0 + i) / 64][kvt_swz(threadIdx.x, (c0 + i) % 64 / 8)]) =
              make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
      }
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    mbar_arrive(&sm.q_full);

    float m = -INFINITY, l = 0.f;
    int vrun = kKv8LowExp;
    for (int j = 0; j < nt; ++j) {
      const int slot = j % SLOTS;
      if (!wait(sm.s_full + j % BUFS, (j / BUFS) & 1) || !wait(sm.kv_full + slot, (j / SLOTS) & 1)) {  // products, meta
        ok = false;
        break;
      }
      kvt_after();
      const uint32_t sp = lane_base + j % BUFS * N;
      float v[N / 32][32];
#pragma unroll
      for (int i = 0; i < N / 32; ++i) kvt_ld32(sp + i * 32, v[i]);
      const int4 meta = sm.meta[slot];
      const int pos0 = (j0 + j) * N;
      // Scales of the blocks' scores: at least kKvtLeastScale, as a zero query or zero keys take them below fp32's range, where
      // a masked score, -inf, times it is NaN; and finite, so that a score of 0 stays 0.
      float ks[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) ks[b] = fminf(fmaxf(kv8_pow2(meta.x >> 8 * b & 255) * qs, kKvtLeastScale), FLT_MAX);
      // A product is at most DH 2^15 top: no score of the tile is above kKvtLargeScore
      const bool small = kv8_pow2(meta.w >> 8) * qs <= kKvtLargeScore / (DH * 32768.f * (FMT == 0 ? 128.f : 512.f));
      const bool whole = __all_sync(0xffffffffu, pos0 + N <= lim && meta.z == 0 && small);
      float ref = 0.f;  // what the scores and m have been lessened by
#pragma unroll
      for (int i = 0; i < N / 32; ++i) kvt_ld_wait(v[i]);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (pos0 + i >= lim || (meta.z >> (i / kKv8Block) & 1)) v[i / 32][i % 32] = -INFINITY;
        if (__any_sync(0xffffffffu, !small)) {
          // Large scores: the fused products below are not rounded, and could exceed the rounded maximum by more than a
          // weight has room for.  Round the scores here and take them relative to the maximum that comes out, in the
          // products' own units, so that the rest stays as it is.
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < N; ++i) top = fmaxf(top, __fmul_rn(v[i / 32][i % 32], ks[i / kKv8Block]));
          ref = top > m + kKvtGrow || m == -INFINITY ? top : m;
          ref = ref == -INFINITY ? 0.f : ref;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float k = ks[i / kKv8Block];
            v[i / 32][i % 32] = (__fmul_rn(v[i / 32][i % 32], k) - ref) * (1.f / k);
          }
          m -= ref;
        }
      }
      float mxb[NB], mx = -INFINITY;
#pragma unroll
      for (int b = 0; b < NB; ++b) mxb[b] = -INFINITY;
#pragma unroll
      for (int i = 0; i < N; ++i) mxb[i / kKv8Block] = fmaxf(mxb[i / kKv8Block], v[i / 32][i % 32]);
#pragma unroll
      for (int b = 0; b < NB; ++b) mx = fmaxf(mx, mxb[b] * ks[b]);
      // correction: a maximum that has grown too far, or louder values
      float f = 1.f;
      if (mx > m + kKvtGrow || (m == -INFINITY && mx > m)) {
        f = ex2(m - mx);
        m = mx;
      }
      int vnew = max(vrun, whole ? meta.w & 255 : 0);
      if (!whole) {  // the blocks that this row sees
#pragma unroll
        for (int b = 0; b < NB; ++b)
          if (pos0 + b * kKv8Block < lim && !(meta.z >> b & 1)) vnew = max(vnew, meta.y >> 8 * b & 255);
      }
      l *= f;
      f *= kv8_pow2(max(127 + vrun - vnew, 0));
      vrun = vnew;
      const bool fold = FOLD && j > 0 && j % max(FOLD, 1) == 0;  // this tile's product begins a chain
      if (j > 0 && (fold || __any_sync(0xffffffffu, f != 1.f))) {
        if (!wait(sm.o_done + (j - 1) % BUFS, ((j - 1) / BUFS) & 1)) {
          ok = false;
          break;
        }
        kvt_after();
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 16) {
          uint32_t x[16], y[16];
          kvt_ld16(lane_base + COL_O + c0, x);
          if (FOLD && j > FOLD) {
            kvt_ld16(lane_base + COL_T + c0, y);
            if (fold) {
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) + __uint_as_float(y[i]));
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
              kvt_st16(lane_base + COL_T + c0, y);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
          kvt_st16(lane_base + (fold ? COL_T : COL_O) + c0, x);
        }
      }
      // weights, times 2^(kKvtShift + the block's value exponent below the row's reference)
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int shift = min(max(kKvtShift + (meta.y >> 8 * b & 255) - vrun, kKvtLeast), kKvtShift);
        const float off = (float)shift - base;
        float s0 = 0.f, s1 = 0.f;
        uint32_t w[PP][8];
#pragma unroll
        for (int e = 0; e < kKv8Block; e += 2) {
          const int i = b * kKv8Block + e;
          const float p0 = ex2(fmaf(v[i / 32][i % 32], ks[b], off)), p1 = ex2(fmaf(v[i / 32][i % 32 + 1], ks[b], off));
          s0 += p0;
          s1 += p1;
          uint32_t pl[PP];
          kv8_planes<PP>(p0, p1, pl);
#pragma unroll
          for (int p = 0; p < PP; ++p) w[p][e >> 1] = pl[p];
        }
        l += (s0 + s1) * kv8_pow2(127 - shift);
#pragma unroll
        for (int p = 0; p < PP; ++p) kvt_st8(sp + p * (N / 2) + b * 8, w[p]);
      }
      m += ref;
      kvt_st_wait();
      kvt_before();
      mbar_arrive(sm.p_full + j % BUFS);
    }
    // ---- the CTA's own sums
    if (nt > 0 && ok && !wait(sm.o_done + (nt - 1) % BUFS, ((nt - 1) / BUFS) & 1)) ok = false;
    kvt_after();
    auto total = [&](int c0, float (&v)[32]) {  // and the chains before
      if (!FOLD || nt <= FOLD) return;
      float y[32];
      kvt_ld32(lane_base + COL_T + c0, y);
      kvt_ld_wait(y);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += y[i];
    };
    if (ok && CL == 1) {  // out = O / l
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // nothing visible: 0; NaN stays
      const float unit = inv * kv8_pow2(vrun - kKvtShift);
      const long long at = (long long)qrow * a.os + (long long)qhead * a.ohs;
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += 32) {
        float v[32];
        if (nt > 0) {
          kvt_ld32(lane_base + COL_O + c0, v);
          kvt_ld_wait(v);
          total(c0, v);
        }
        if (mine) {
#pragma unroll
          for (int i = 0; i < 32; i += 8) {
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = l == 0.f ? 0.f : v[i + e] * unit;
            kv8_st8(a.out, DT, at + c0 + i, a.out_vec, y);
          }
        }
      }
      if (mine && a.lse) a.lse[(size_t)qrow * a.Hq + qhead] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    } else if (ok) {
      // for the cluster: over the operands' memory, every product has been made
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      const float unit = kv8_pow2(vrun - kKvtShift);
      if (nt > 0) {
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 32) {
          float v[32];
          kvt_ld32(lane_base + COL_O + c0, v);
          kvt_ld_wait(v);
          total(c0, v);
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<float4*>(&sums.o[threadIdx.x][c0 + i]) = make_float4(v[i] * unit, v[i + 1] * unit, v[i + 2] * unit, v[i + 3] * unit);
        }
      }
      sums.ml[threadIdx.x] = make_float2(m, l);
    }
  } else if (warp < 7) {
    // ------------------------------------------------------------------ codes to operands
    // A warp takes whole tiles, every third one: its copies are in flight while the others convert.
    constexpr int CPR = DH / 16;         // 16-byte pieces of a row
    constexpr int PC = N * CPR / 32;     // pieces of K (and of V) a lane has in a tile
    const int first = warp - 4;
    // lane b < NB: the table's entry for the tile's block b, INT_MIN if it has none.  The entry is looked at when the
    // codes are asked for, a tile later: looking at it here would wait for it.
    auto entry_of = [&](int j) {
      const int blk = (j0 + j) * NB + lane;
      if (j >= nt || lane >= NB || blk * kKv8Block >= max_lim) return INT_MIN;
      return __ldg(c.table + (size_t)s * c.max_pages + kv8_div_tpp(c, blk));
    };
    // Where block b's codes are put: in the operand's own place, such that a part (all keys, or with two swizzle atoms
    // the first and the second 32) is read whole before anything is written over it.
    constexpr int PARTS = KvtSmem<DH, QP>::HALVES, PCH = PC / PARTS, BP = NB / PARTS;
    auto raw_of = [&](uint8_t (*dst)[N * 128], int b) {
      return PARTS == 1 ? dst[0] + b * kKv8Block * DH : dst[b / BP] + N * 64 + b % BP * kKv8Block * DH;
    };
    // The tile's codes as f16.  Blocks that are not `held`, and rows from `rows` on (they may be no numbers), become 0.
    auto convert = [&](uint8_t (*dst)[N * 128], unsigned held, int rows) {
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        uint4 w[PCH];
        const uint4* raw = reinterpret_cast<const uint4*>(raw_of(dst, h * BP));
#pragma unroll
        for (int i = 0; i < PCH; ++i) w[i] = raw[i * 32 + lane];
        __syncwarp();
        if (held != (1u << NB) - 1 || rows < N) {
#pragma unroll
          for (int i = 0; i < PCH; ++i) {
            const int key = h * (N / PARTS) + (i * 32 + lane) / CPR;
            if (!(held >> (key / kKv8Block) & 1) || key >= rows) w[i] = make_uint4(0, 0, 0, 0);
          }
        }
#pragma unroll
        for (int i = 0; i < PCH; ++i) {
          const int pc = i * 32 + lane, key = h * (N / PARTS) + pc / CPR, ch = pc % CPR * 16;
          const uint2 x0 = kv8_half4<FMT>(w[i].x), x1 = kv8_half4<FMT>(w[i].y), x2 = kv8_half4<FMT>(w[i].z), x3 = kv8_half4<FMT>(w[i].w);
          uint8_t* d = dst[ch / 64];
          *reinterpret_cast<uint4*>(d + kvt_swz(key, ch % 64 / 8)) = make_uint4(x0.x, x0.y, x1.x, x1.y);
          *reinterpret_cast<uint4*>(d + kvt_swz(key, ch % 64 / 8 + 1)) = make_uint4(x2.x, x2.y, x3.x, x3.y);
        }
        if (PARTS > 1) __syncwarp();
      }
    };
    const bool stall = a.stall && item == 0 && rank == 0 && first == 0;  // the tiles of this warp never come
    int entry = entry_of(first);
    for (int j = first; j < nt && !stall; j += kKvtLoaders) {
      const int slot = j % SLOTS;
      // The slot's last tile is done with.  (A barrier tells two phases apart, and this warp saw tile j - 3 - SLOTS done.)
      static_assert(SLOTS > kKvtLoaders, "the slot's tile before last came no later than that");
      if (j >= SLOTS && !wait(sm.kv_empty + slot, (j / SLOTS - 1) & 1)) {
        ok = false;
        break;
      }
      const bool there = (unsigned)entry < (unsigned)c.n_pages;
      if (!there && entry != INT_MIN && c.status) set_status(c.status, kErrDevice);
      const unsigned held = __ballot_sync(0xffffffffu, there);
      if (lane == 0) mbar_expect_tx(sm.raw_full + slot, __popc(held) * 2 * kKv8Block * DH);
      __syncwarp();
      int ke = -1, ve = -1;
      if (there) {
        const int blk = (j0 + j) * NB + lane, sub = blk - kv8_div_tpp(c, blk) * c.tpp;
        const size_t at = (size_t)entry * c.page_stride + ((size_t)kvh * c.PT + sub * kKv8Block) * DH;
        bulk_g2s(raw_of(sm.k[slot], lane), c.k + at, kKv8Block * DH, sm.raw_full + slot);
        bulk_g2s(raw_of(sm.v[slot], lane), c.v + at, kKv8Block * DH, sm.raw_full + slot);
        const size_t e = (size_t)entry * c.exp_stride + kvh * c.tpp + sub;
        ke = __ldg(c.ke + e);
        ve = __ldg(c.ve + e);
      }
      entry = entry_of(j + kKvtLoaders);
      if (!wait(sm.raw_full + slot, (j / SLOTS) & 1)) {
        ok = false;
        wait(sm.raw_full + slot, (j / SLOTS) & 1);  // the copies in flight
        break;
      }
      const unsigned kes = __reduce_or_sync(0xffffffffu, there ? (unsigned)ke << 8 * lane : 0u);
      const unsigned ves = __reduce_or_sync(0xffffffffu, there ? (unsigned)ve << 8 * lane : 0u);
      const int kmax = max(__reduce_max_sync(0xffffffffu, ke), 0), vmax = max(__reduce_max_sync(0xffffffffu, ve), 0);
      const int rows = min(max_lim - (j0 + j) * N, N), nb = (rows + kKv8Block - 1) / kKv8Block;
      // blocks before the end of the keys that have no page (blocks behind it are masked by the limits)
      if (lane == 0) sm.meta[slot] = make_int4((int)kes, (int)ves, (int)(~held & ((1u << nb) - 1)), kmax << 8 | vmax);
      convert(sm.k[slot], held, N);
      convert(sm.v[slot], held, rows);
      asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
      mbar_arrive(sm.kv_full + slot);
    }
  } else if (nt > 0) {
    // ------------------------------------------------------------------ products: the warp together, one lane issuing
    constexpr uint32_t is = kvt_idesc(N, false), io = kvt_idesc(NV, true);
    constexpr uint32_t QSTEP = kKvtQ * 128 / 16, KSTEP = N * 128 / 16, KSLOT = KvtSmem<DH, QP>::HALVES * KSTEP;  // in descriptors' units
    const bool lead = kvt_elect();
    const uint64_t qd = kvt_desc(smem_u32(sm.q), 16), kd = kvt_desc(smem_u32(sm.k), 16), vd = kvt_desc(smem_u32(sm.v), N * 128);
    auto scores = [&](int j) {
      const int slot = j % SLOTS, buf = j % BUFS;
      if (!wait(sm.kv_full + slot, (j / SLOTS) & 1)) return false;
      kvt_after();
      if (lead) {
        const uint64_t kj = kd + (uint32_t)slot * KSLOT;
        const uint32_t d = tmem + buf * N;
#pragma unroll
        for (int p = 0; p < QP; ++p)
#pragma unroll
          for (int k0 = 0; k0 < DH; k0 += 16)  // 16 channels: 32 bytes inside the swizzle atom
            kvt_mma_ss(d, qd + (p * KvtSmem<DH, QP>::HALVES + k0 / 64) * QSTEP + k0 % 64 / 8, kj + k0 / 64 * KSTEP + k0 % 64 / 8, is,
                       p > 0 || k0 > 0);
        kvt_commit(sm.s_full + buf);
      }
      __syncwarp();
      return true;
    };
    ok = wait(&sm.q_full, 0) && scores(0);
    for (int j = 0; ok && j < nt; ++j) {
      // the next tile's scores run under this tile's weights; their columns held P of a tile whose product is done
      const int b = j + 1 - BUFS;
      if ((b >= 0 && !wait(sm.o_done + b % BUFS, (b / BUFS) & 1)) || (j + 1 < nt && !scores(j + 1)) || !wait(sm.p_full + j % BUFS, (j / BUFS) & 1)) {
        ok = false;
        break;
      }
      kvt_after();
      const int slot = j % SLOTS, buf = j % BUFS;
      if (lead) {
        const uint64_t vj = vd + (uint32_t)slot * KSLOT;
        const uint32_t pa = tmem + buf * N;
        const bool going = FOLD ? j % max(FOLD, 1) > 0 : j > 0;  // the chain goes on
#pragma unroll
        for (int p = PP - 1; p >= 0; --p)
#pragma unroll
          for (int k0 = 0; k0 < N; k0 += 16)  // 16 keys: two 8-row groups of V
            kvt_mma_ts(tmem + COL_O, pa + p * (N / 2) + k0 / 2, vj + k0 * 8, io, going || p < PP - 1 || k0 > 0);
        kvt_commit(sm.o_done + buf);
        kvt_commit(sm.kv_empty + slot);
      }
      __syncwarp();
    }
    // nothing is in flight when the memory goes
    if (ok) ok = wait(sm.o_done + (nt - 1) % BUFS, ((nt - 1) / BUFS) & 1);
    if (!ok) {
      if (lead) kvt_commit(&sm.drained);
      __syncwarp();
      wait(&sm.drained, 0);
    }
  }
  kvt_before();
  const bool all_ok = __syncthreads_and(ok) != 0;
  if (warp == 7) {
    kvt_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(COLS));
  }
  if (threadIdx.x == 0) {
    if (!all_ok && c.status) set_status(c.status, kErrDevice);
    sm.ok = all_ok;
  }
  if (CL == 1) return;
  // ---- join the cluster and store: each CTA finishes a share of the rows, four channels a thread
  namespace cg = cooperative_groups;
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  bool every = true;  // no CTA's sums are missing
  for (int r = 0; r < CL; ++r) every = every && *cl.map_shared_rank(&sm.ok, r);
  const int share = kKvtQ / CL;
  for (int i = threadIdx.x; every && i < share * (DH / 4); i += kKvtThreads) {
    const int qn = rank * share + i / (DH / 4), d = i % (DH / 4) * 4;
    if (qn >= nq) break;
    float M = -INFINITY, L = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < CL; ++r) M = fmaxf(M, cl.map_shared_rank(&sums.ml[qn], r)->x);
    for (int r = 0; r < CL; ++r) {
      const float2 ml = *cl.map_shared_rank(&sums.ml[qn], r);
      if (ml.y == 0.f) continue;  // saw nothing
      const float f = ml.x == M ? 1.f : ex2(ml.x - M);
      const float4 x = *reinterpret_cast<const float4*>(cl.map_shared_rank(&sums.o[qn][d], r));
      L += f * ml.y;
      v.x += f * x.x, v.y += f * x.y, v.z += f * x.z, v.w += f * x.w;
    }
    const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
    const int row = r0 + (qbase + qn) / a.G, head = kvh * a.G + (qbase + qn) % a.G;
    kv8_st4(a.out, DT, (long long)row * a.os + (long long)head * a.ohs + d, a.out_vec, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    if (d == 0 && a.lse) a.lse[(size_t)row * a.Hq + head] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  }
  cl.sync();  // the others may still read this CTA's sums
}

template <int DH, int FMT, int QP, int PP>
cudaError_t kv8_tile_one(const Kv8View& c, const Kv8AttnArgs& a, long long tiles, int max_keys, int sm_count, cudaStream_t stream) {
  using Smem = KvtSmem<DH, QP>;
  static_assert(sizeof(KvtSums<DH>) <= offsetof(Smem, meta), "the sums fit in the operands' memory");
  auto kern = k_kv8_tile<DH, FMT, QP, PP>;
  constexpr int smem = (int)kvt_smem<DH, QP>();
  const long long ctas = tiles * c.H * c.batch;
  // Split the keys over a cluster while all CTAs still run at once and each keeps 16 tiles.  Heads of 128, bf16, 8192 keys,
  // one CTA an SM, us: 20 CTAs 59 in eighths (two waves), 45 in quarters; 64 CTAs 89 in quarters, 76 in halves; 128 CTAs 150
  // in halves, 127 whole.  Of clusters of 8 with an SM a CTA, 12 run at once and 16 do not (59 us, 45 in quarters).
  constexpr int per_sm = kvt_smem<DH, QP>() <= 113 * 1024 ? 2 : 1;
  int cl = 1;
  while (cl < 8 && ctas * cl * 2 <= (long long)per_sm * sm_count && (per_sm == 2 || cl < 4 || ctas <= 12) && max_keys >= cl * 2 * 16 * kKvtN) cl *= 2;
  const cudaError_t e = kv8_allow_smem<k_kv8_tile<DH, FMT, QP, PP>>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(ctas * cl));
  cfg.blockDim = dim3(kKvtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cl;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cl > 1;
  return cudaLaunchKernelEx(&cfg, kern, c, a, (int)tiles, cl);
}

template <int DH, int FMT>
cudaError_t kv8_tile_dh(const Kv8View& c, const Kv8AttnArgs& a, long long tiles, int max_keys, int sm_count, cudaStream_t st) {
  if (a.dtype == BLT_T_F32) return kv8_tile_one<DH, FMT, 2, 2>(c, a, tiles, max_keys, sm_count, st);
  if (a.dtype == BLT_T_BF16) return kv8_tile_one<DH, FMT, 1, 1>(c, a, tiles, max_keys, sm_count, st);
  return kv8_tile_one<DH, FMT, 1, 2>(c, a, tiles, max_keys, sm_count, st);
}

}  // namespace bltdec
