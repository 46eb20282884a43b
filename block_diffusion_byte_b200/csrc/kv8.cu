// The 8-bit paged KV cache: storing, reading back, choosing pages, and the C ABI of bltkv8.h.
#include "kv8.cuh"

#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace bltdec {

cudaError_t kv8_attend_d32(int, const Kv8View&, const Kv8AttnArgs&, int, int, cudaStream_t);
cudaError_t kv8_attend_d64(int, const Kv8View&, const Kv8AttnArgs&, int, int, cudaStream_t);
cudaError_t kv8_attend_d96(int, const Kv8View&, const Kv8AttnArgs&, int, int, cudaStream_t);
cudaError_t kv8_attend_d128(int, const Kv8View&, const Kv8AttnArgs&, int, int, cudaStream_t);

struct Kv8RowsArgs {
  void *k, *v;
  int dtype, n_rows, max_rows, vec;
  long long rs, hs;
  const int *row_off, *start;
};

constexpr int kKv8RowThreads = 256;  // of append and read, at most

// ------------------------------------------------------------------------ append
// One CTA per touched page of a sequence and one or more heads (grid.y of them share the heads), one warp per (block of
// 16 positions, K or V): a lane keeps DH / 16 groups of 8 channels in registers, so a block's rows are read once, its
// amax is a warp reduction, and the codes leave as 8-byte pieces.  Bound by memory for prompts (four of 8192 bf16 rows, 16
// heads of 64: 53 us, 3.8 TB/s of the rows read and codes written once), by its four dependent lookups for few rows (one
// row: 3.7 us).
template <int DH, int FMT, int DT>
__global__ void __launch_bounds__(kKv8RowThreads, 4) k_kv8_append(const __grid_constant__ Kv8View c, const __grid_constant__ Kv8RowsArgs a) {
  constexpr int GPR = DH / 8, NG = DH / 16;  // groups per row; groups per lane
  const int s = blockIdx.z, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  int r0, r1;
  kv8_rows_of(a.row_off, s, a.n_rows, a.max_rows, c.status, r0, r1);
  if (r1 <= r0) return;
  const int start = __ldg(a.start + s);
  const long long cap = (long long)c.max_pages * c.PT;
  if (start < 0 || start + (long long)(r1 - r0) > cap) {
    if (c.status && threadIdx.x == 0) set_status(c.status, kErrDevice);
    return;
  }
  const int end = start + (r1 - r0), pi = start / c.PT + blockIdx.x, p0 = pi * c.PT;
  if (p0 >= end) return;
  const int page = kv8_page(c, s, pi);
  if (page < 0) return;
  const int b0 = max(start - p0, 0) / kKv8Block, b1 = (min(end - p0, c.PT) + kKv8Block - 1) / kKv8Block;  // blocks that take rows
  __shared__ float lo[16][DH], hi[16][DH];
  __shared__ float s_amax[kKv8RowThreads / 32];
#pragma unroll 1
  for (int h = blockIdx.y; h < c.H; h += gridDim.y) {
    const size_t at = (size_t)page * c.page_stride + (size_t)h * c.PT * DH;
    const size_t ex = (size_t)page * c.exp_stride + (size_t)h * c.tpp;
    for (int i = warp; i < 2 * (b1 - b0); i += nw) {
      const bool val = i & 1;
      const int b = b0 + (i >> 1), q0 = p0 + b * kKv8Block;
      uint8_t* codes = (val ? c.v : c.k) + at + (size_t)b * kKv8Block * DH;
      uint8_t* exps = (val ? c.ve : c.ke) + ex + b;
      const void* src = val ? a.v : a.k;
      float x[NG][8];
      float old = 0.f;
      if (q0 < start) old = kv8_pow2(*exps);  // kept rows: all lanes read the exponent before lane 0 writes it
      if (q0 >= start && q0 + kKv8Block <= end && a.vec) {  // a block of new rows: all its loads at once
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int gi = j * 32 + lane;
          kv8_ld8(src, DT, (long long)(r0 + (q0 - start) + gi / GPR) * a.rs + (long long)h * a.hs + gi % GPR * 8, true, x[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          const int gi = j * 32 + lane, pos = q0 + gi / GPR, ch = gi % GPR * 8;
          if (pos < start) {
            kv8_decode8<FMT>(*reinterpret_cast<const uint2*>(codes + gi * 8), x[j]);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              // beyond fp32's range: an infinity where the code is the largest, else a number near the range's end
              const float y = x[j][e] * old;
              x[j][e] = fabsf(y) > FLT_MAX && fabsf(x[j][e]) < (FMT == 0 ? 127.f : 448.f) ? copysignf(FLT_MAX, y) : y;
            }
          } else if (pos < end) {
            kv8_ld8(src, DT, (long long)(r0 + (pos - start)) * a.rs + (long long)h * a.hs + ch, a.vec, x[j]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[j][e] = 0.f;
          }
        }
      }
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, kv8_mag(x[j][e]));
      amax = warp_max(amax);
      const int e = kv8_exponent<FMT>(amax);
      const float inv = kv8_pow2(254 - e);
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const int gi = j * 32 + lane, pos = q0 + gi / GPR;
        if (pos < end) {
          uint2 w;
          w.x = kv8_encode4<FMT>(x[j][0], x[j][1], x[j][2], x[j][3], inv);
          w.y = kv8_encode4<FMT>(x[j][4], x[j][5], x[j][6], x[j][7], inv);
          *reinterpret_cast<uint2*>(codes + gi * 8) = w;
        }
      }
      __syncwarp();
      if (lane == 0) *exps = (uint8_t)e;
    }
    if (!c.kmin) continue;
    // ---- the page's summary over every position it holds now
    __syncthreads();  // the codes and exponents of this page are the CTA's own writes
    const int held = min(end - p0, c.PT);
    {
      // thread: channels 8 (i % GPR) .., positions i / GPR, i / GPR + step, ...
      const int lanes = min((int)blockDim.x / GPR, 16), row = threadIdx.x / GPR, ch = threadIdx.x % GPR * 8;
      if (row < lanes) {
        float mn[8], mx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mn[e] = INFINITY, mx[e] = -INFINITY;
        for (int p = row; p < held; p += lanes) {
          float y[8];
          kv8_decode8<FMT>(*reinterpret_cast<const uint2*>(c.k + at + (size_t)p * DH + ch), y);
          const float sc = kv8_pow2(c.ke[ex + p / kKv8Block]);
#pragma unroll
          for (int e = 0; e < 8; ++e) mn[e] = fminf(mn[e], y[e] * sc), mx[e] = fmaxf(mx[e], y[e] * sc);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) lo[row][ch + e] = mn[e], hi[row][ch + e] = mx[e];
      }
      __syncthreads();
      float amax = 0.f;
      for (int d = threadIdx.x; d < DH; d += blockDim.x) {
        float mn = lo[0][d], mx = hi[0][d];
        for (int r = 1; r < lanes; ++r) mn = fminf(mn, lo[r][d]), mx = fmaxf(mx, hi[r][d]);
        // a code's value can lie beyond fp32 where a block holds magnitudes near 3e38: it counts as fp32's largest
        mn = fminf(fmaxf(mn, -FLT_MAX), FLT_MAX), mx = fminf(fmaxf(mx, -FLT_MAX), FLT_MAX);
        lo[0][d] = mn, hi[0][d] = mx;
        amax = fmaxf(amax, fmaxf(fabsf(mn), fabsf(mx)));
      }
      amax = warp_max(amax);
      if (lane == 0) s_amax[warp] = amax;
      __syncthreads();
      amax = s_amax[0];
      for (int w = 1; w < nw; ++w) amax = fmaxf(amax, s_amax[w]);
      const int e = kv8_exponent<0>(amax);
      const float inv = kv8_pow2(254 - e);
      for (int d = threadIdx.x; d < DH; d += blockDim.x) {
        const size_t o = (size_t)page * c.sum_stride + (size_t)h * DH + d;
        c.kmin[o] = (int8_t)__float2int_rn(lo[0][d] * inv);
        c.kmax[o] = (int8_t)__float2int_rn(hi[0][d] * inv);
      }
      if (threadIdx.x == 0) c.ksexp[(size_t)page * c.sexp_stride + h] = (uint8_t)e;
      __syncthreads();  // the next head writes the shared arrays
    }
  }
}

// ------------------------------------------------------------------------ read
// The same grid; a thread takes pieces of 8 codes, four in flight (the same prompts: 48 us, 4.2 TB/s; one row: 2.3 us).
template <int DH, int FMT, int DT>
__global__ void __launch_bounds__(kKv8RowThreads, 4) k_kv8_read(const __grid_constant__ Kv8View c, const __grid_constant__ Kv8RowsArgs a) {
  constexpr int GPR = DH / 8, UN = 4;
  const int s = blockIdx.z;
  int r0, r1;
  kv8_rows_of(a.row_off, s, a.n_rows, a.max_rows, c.status, r0, r1);
  if (r1 <= r0) return;
  const int start = __ldg(a.start + s);
  const long long cap = (long long)c.max_pages * c.PT;
  if (start < 0 || start + (long long)(r1 - r0) > cap) {
    if (c.status && threadIdx.x == 0) set_status(c.status, kErrDevice);
    return;
  }
  const int end = start + (r1 - r0), pi = start / c.PT + blockIdx.x, p0 = pi * c.PT;
  if (p0 >= end) return;
  const int page = kv8_page(c, s, pi);
  const int q0 = max(p0, start), n = min(end, p0 + c.PT) - q0, half = n * GPR;
#pragma unroll 1
  for (int h = blockIdx.y; h < c.H; h += gridDim.y) {
    const size_t at = (size_t)page * c.page_stride + (size_t)h * c.PT * DH, ex = (size_t)page * c.exp_stride + (size_t)h * c.tpp;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < 2 * half; i0 += UN * blockDim.x) {
      uint2 w[UN];
      int e[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + u * blockDim.x;
        w[u] = make_uint2(0, 0);
        e[u] = 127;
        if (page >= 0 && i < 2 * half) {
          const bool val = i >= half;
          const int gi = val ? i - half : i, in = q0 + gi / GPR - p0;
          w[u] = __ldg(reinterpret_cast<const uint2*>((val ? c.v : c.k) + at + (size_t)in * DH + gi % GPR * 8));
          e[u] = __ldg((val ? c.ve : c.ke) + ex + in / kKv8Block);
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + u * blockDim.x;
        if (i >= 2 * half) break;
        const bool val = i >= half;
        const int gi = val ? i - half : i;
        float x[8];
        kv8_decode8<FMT>(w[u], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= kv8_pow2(e[u]);
        kv8_st8(val ? a.v : a.k, DT, (long long)(r0 + (q0 - start) + gi / GPR) * a.rs + (long long)h * a.hs + gi % GPR * 8, a.vec, x);
      }
    }
  }
}

// ------------------------------------------------------------------------ select
struct Kv8SelArgs {
  const void* q;
  int dtype, Hq, G, n_rows, max_rows, n_select, n_sink, n_local, cap_pages;
  long long qs, qhs;
  const int *row_off, *row_limit;
  int *pages, *count;
};

constexpr int kKv8SelThreads = 512;  // at most

// One CTA per (row, key/value head).  Scores: four lanes share a page's minima and maxima; a query channel
// is either >= 0 or < 0, so max(q lo, q hi) is q's positive part times the maximum plus its negative part
// times the minimum -- two byte dot products (dp4a), exact.  The chosen set: the n-th largest score by
// radix descent over order-preserving keys, then the lowest pages among its equals; written in order.  Bound by its
// dependent lookups and the descent's barriers: 16 CTAs of 512 pages 9 us, 1024 CTAs of 128 pages 15.6 us.
template <int DH>
__global__ void __launch_bounds__(kKv8SelThreads) k_kv8_select(const __grid_constant__ Kv8View c, const __grid_constant__ Kv8SelArgs a) {
  constexpr int QW = DH / 4, LW = DH / 16;  // words of a row; words of a lane
  constexpr int NWMAX = kKv8SelThreads / 32;
  constexpr int BATCH = DH <= 64 ? 4 : 2;  // pages a lane has in flight
  extern __shared__ uint32_t sel_smem[];
  __shared__ uint32_t hist[256];
  __shared__ int warp_n[NWMAX][2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const int s = blockIdx.z, kvh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = blockDim.x, NW = T >> 5;
  int r0, r1;
  kv8_rows_of(a.row_off, s, a.n_rows, a.max_rows, c.status, r0, r1);
  const int row = r0 + blockIdx.x;
  if (row >= r1) return;
  uint32_t* qpos = sel_smem;                                    // [G][QW] positive parts
  uint32_t* qneg = qpos + a.G * QW;                             // [G][QW] negative parts
  float* qsc = reinterpret_cast<float*>(qneg + a.G * QW);       // [G] scales
  uint32_t* key = reinterpret_cast<uint32_t*>(qsc + ((a.G + 3) & ~3));  // [pages]
  int lim = __ldg(a.row_limit + row);
  if (lim > c.max_pages * c.PT) {
    if (c.status && threadIdx.x == 0) set_status(c.status, kErrDevice);
    lim = c.max_pages * c.PT;
  }
  const int nb = (int)(((long long)max(lim, 0) + c.PT - 1) / c.PT);
  int* out = a.pages + ((size_t)row * c.H + kvh) * a.n_select;
  if (threadIdx.x == 0) a.count[(size_t)row * c.H + kvh] = min(nb, a.n_select);
  if (nb <= a.n_select) {
    for (int i = threadIdx.x; i < a.n_select; i += T) out[i] = i < nb ? i : -1;
    return;
  }
  // the first pages' table entries are on their way while the queries are made
  const int t = lane & 3, stride = NW * 8;
  auto entry = [&](int p) { return p < nb && !(p < a.n_sink || p >= nb - a.n_local) ? __ldg(c.table + (size_t)s * c.max_pages + p) : INT_MIN; };
  int next[BATCH];
#pragma unroll
  for (int k = 0; k < BATCH; ++k) next[k] = entry(warp * 8 + (lane >> 2) + k * stride);
  // ---- the group's queries in 8 bits: a warp a head
  for (int g = warp; g < a.G; g += NW) {
    const long long base = (long long)row * a.qs + (long long)(kvh * a.G + g) * a.qhs;
    float x[4] = {0.f, 0.f, 0.f, 0.f};
    float amax = 0.f;
    if (lane < QW) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = kv8_ld(a.q, a.dtype, base + lane * 4 + e);
        amax = fmaxf(amax, kv8_mag(x[e]));
      }
    }
    amax = warp_max(amax);
    const int e = kv8_exponent<0>(amax);
    if (lane < QW) {
      const uint32_t w = kv8_encode4<0>(x[0], x[1], x[2], x[3], kv8_pow2(254 - e));
      const uint32_t neg = (w & 0x80808080u) >> 7, mask = neg * 0xffu;  // bytes below 0
      qpos[g * QW + lane] = w & ~mask;
      qneg[g * QW + lane] = w & mask;
    }
    if (lane == 0) qsc[g] = kv8_pow2(e);
  }
  __syncthreads();
  // ---- scores
  for (int p0 = warp * 8 + (lane >> 2); p0 - (lane >> 2) < nb; p0 += BATCH * stride) {
    uint32_t lo[BATCH][LW], hi[BATCH][LW];
    float es[BATCH];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int page = next[k];
      const bool there = (unsigned)page < (unsigned)c.n_pages;
      es[k] = -1.f;  // no page
#pragma unroll
      for (int i = 0; i < LW; ++i) lo[k][i] = hi[k][i] = 0;
      if (there) {
        const size_t o = (size_t)page * c.sum_stride + (size_t)kvh * DH + t * (DH / 4);
#pragma unroll
        for (int i = 0; i < LW; i += 2) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(c.kmin + o + i * 4)), y = __ldg(reinterpret_cast<const uint2*>(c.kmax + o + i * 4));
          lo[k][i] = x.x, lo[k][i + 1] = x.y, hi[k][i] = y.x, hi[k][i + 1] = y.y;
        }
        es[k] = kv8_pow2(__ldg(c.ksexp + (size_t)page * c.sexp_stride + kvh));
      } else if (page != INT_MIN && c.status) {
        set_status(c.status, kErrDevice);
      }
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) next[k] = entry(p0 + (BATCH + k) * stride);
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int p = p0 + k * stride;
      float best = -INFINITY;
      for (int g = 0; g < a.G; ++g) {
        int dot = 0;
#pragma unroll
        for (int i = 0; i < LW; ++i) {
          dot = __dp4a((int)qpos[g * QW + t * LW + i], (int)hi[k][i], dot);
          dot = __dp4a((int)qneg[g * QW + t * LW + i], (int)lo[k][i], dot);
        }
        dot += __shfl_xor_sync(0xffffffffu, dot, 1);
        dot += __shfl_xor_sync(0xffffffffu, dot, 2);
        // The smaller scale first: what is in fp32's range stays there.  Clamped to that range, so that only pages that are
        // always chosen have an infinite score.
        best = fmaxf(best, fminf(fmaxf((float)dot * fminf(qsc[g], es[k]) * fmaxf(qsc[g], es[k]), -FLT_MAX), FLT_MAX));
      }
      if (t == 0 && p < nb) {
        if (p < a.n_sink || p >= nb - a.n_local) best = INFINITY;
        else if (es[k] < 0.f) best = -INFINITY;
        const uint32_t u = __float_as_uint(best + 0.f);  // -0 counts as 0
        key[p] = u & 0x80000000u ? ~u : u | 0x80000000u;
      }
    }
  }
  // ---- the key of the n_select-th page: 8 bits at a time
  if (threadIdx.x == 0) s_prefix = 0, s_left = a.n_select;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = threadIdx.x; i < 256; i += T) hist[i] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int p = threadIdx.x; p - threadIdx.x < nb; p += T) {
      const bool in = p < nb && (shift == 24 || key[p] >> (shift + 8) == prefix >> (shift + 8));
      const unsigned bin = in ? (key[p] >> shift) & 255u : 256u;
      const unsigned same = __match_any_sync(0xffffffffu, bin);  // one atomic per distinct value of a warp
      if (in && (int)(__ffs(same) - 1) == lane) atomicAdd(&hist[bin], (unsigned)__popc(same));
    }
    __syncthreads();
    if (warp == 0) {  // the bin that holds the s_left-th key from the top: lane l sums bins 255 - 8 l ..
      unsigned n = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) n += hist[255 - lane * 8 - i];
      unsigned above = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned y = __shfl_up_sync(0xffffffffu, above, d);
        if (lane >= d) above += y;
      }
      const unsigned left = s_left;
      above -= n;  // keys in higher lanes' bins
      __syncwarp();
      if (above < left && left <= above + n) {
        for (int i = 0; i < 8; ++i) {
          const unsigned b = 255 - lane * 8 - i, k = hist[b];
          if (above + k >= left) {
            s_prefix = prefix | (b << shift);
            s_left = (int)(left - above);
            break;
          }
          above += k;
        }
      }
    }
    __syncthreads();
  }
  // ---- pages above the key, and the first s_left equal to it, in order
  const uint32_t kth = s_prefix;
  const int ties = s_left;
  int n_out = 0, n_tie = 0;
  for (int p0 = 0; p0 < nb; p0 += T) {
    const int p = p0 + threadIdx.x;
    const uint32_t k = p < nb ? key[p] : 0;
    const bool eq = p < nb && k == kth, gt = p < nb && k > kth;
    const unsigned meq = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) warp_n[warp][0] = __popc(meq);
    __syncthreads();
    int tie = n_tie + __popc(meq & ((1u << lane) - 1)), all_eq = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) tie += warp_n[w][0];
      all_eq += warp_n[w][0];
    }
    const bool take = gt || (eq && tie < ties);
    const unsigned mt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) warp_n[warp][1] = __popc(mt);
    __syncthreads();
    int at = n_out + __popc(mt & ((1u << lane) - 1)), all = 0;
    for (int w = 0; w < NW; ++w) {
      if (w < warp) at += warp_n[w][1];
      all += warp_n[w][1];
    }
    if (take) out[at] = p;
    n_out += all;
    n_tie += all_eq;
    __syncthreads();
  }
}

// ------------------------------------------------------------------------ host
namespace {

thread_local char g_err[256] = "";

int bad(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int bad(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof g_err, fmt, ap);
  va_end(ap);
  return code;
}
int cuda_bad(const char* what, cudaError_t e) { return bad(BLT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e)); }

// The device of the cache's keys is current for the life of this.
struct DeviceScope {
  int back = -1;
  ~DeviceScope() {
    if (back >= 0) cudaSetDevice(back);
  }
  int enter(const void* p) {
    cudaPointerAttributes at{};
    cudaError_t e = cudaPointerGetAttributes(&at, p);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_bad("cudaPointerGetAttributes", e);
    }
    if (at.type != cudaMemoryTypeDevice && at.type != cudaMemoryTypeManaged)
      return bad(BLT_ERR_INVALID_ARG, "the cache is not in device memory");
    int cur = 0;
    if ((e = cudaGetDevice(&cur)) != cudaSuccess) return cuda_bad("cudaGetDevice", e);
    if (at.type == cudaMemoryTypeDevice && cur != at.device) {
      if ((e = cudaSetDevice(at.device)) != cudaSuccess) return cuda_bad("cudaSetDevice", e);
      back = cur;
    }
    return BLT_OK;
  }
};

bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int check_cache(const blt_kv8_cache* c, Kv8View& v) {
  if (!c) return bad(BLT_ERR_INVALID_ARG, "the cache is NULL");
  if (c->format != BLT_KV8_INT8 && c->format != BLT_KV8_E4M3) return bad(BLT_ERR_INVALID_ARG, "format %d", c->format);
  if (c->head_dim != 32 && c->head_dim != 64 && c->head_dim != 96 && c->head_dim != 128)
    return bad(BLT_ERR_INVALID_ARG, "head_dim %d is not 32, 64, 96 or 128", c->head_dim);
  if (c->page_tokens < 16 || c->page_tokens % 16 || c->page_tokens > 256)
    return bad(BLT_ERR_INVALID_ARG, "page_tokens %d is not a multiple of 16 up to 256", c->page_tokens);
  if (c->n_heads < 1 || c->n_heads > 65535 || c->n_pages < 1 || c->batch < 1 || c->batch > 65535 || c->max_pages < 1 ||
      (long long)c->max_pages * c->page_tokens >= (1ll << 30))
    return bad(BLT_ERR_INVALID_ARG, "n_heads %d, n_pages %d, batch %d, max_pages %d", c->n_heads, c->n_pages, c->batch, c->max_pages);
  if (!c->k || !c->v || !c->k_exp || !c->v_exp || !c->page_table) return bad(BLT_ERR_INVALID_ARG, "a NULL pointer in the cache");
  const long long ps = (long long)c->n_heads * c->page_tokens * c->head_dim, es = (long long)c->n_heads * (c->page_tokens / 16),
                  ss = (long long)c->n_heads * c->head_dim;
  v.page_stride = c->page_stride ? c->page_stride : ps;
  v.exp_stride = c->exp_stride ? c->exp_stride : es;
  v.sum_stride = c->sum_stride ? c->sum_stride : ss;
  v.sexp_stride = c->sexp_stride ? c->sexp_stride : c->n_heads;
  if (v.page_stride < ps || v.page_stride % 16 || v.exp_stride < es || v.sum_stride < ss || v.sum_stride % 8 || v.sexp_stride < c->n_heads)
    return bad(BLT_ERR_INVALID_ARG, "a page stride is too small or misaligned");
  if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_min, 8) || misaligned(c->k_max, 8) || misaligned(c->page_table, 4) ||
      misaligned(c->status, 4))
    return bad(BLT_ERR_INVALID_ARG, "a misaligned pointer in the cache");
  if ((c->k_min != nullptr) != (c->k_max != nullptr) || (c->k_min != nullptr) != (c->k_sexp != nullptr))
    return bad(BLT_ERR_INVALID_ARG, "k_min, k_max and k_sexp come together");
  v.k = c->k, v.v = c->v, v.ke = c->k_exp, v.ve = c->v_exp;
  v.kmin = c->k_min, v.kmax = c->k_max, v.ksexp = c->k_sexp;
  v.table = c->page_table, v.status = c->status;
  v.H = c->n_heads, v.PT = c->page_tokens, v.tpp = c->page_tokens / 16;
  v.tpp_magic = v.tpp == 1 ? 0u : (unsigned)((1ull << 32) / v.tpp + 1);
  v.n_pages = c->n_pages, v.batch = c->batch, v.max_pages = c->max_pages;
  return BLT_OK;
}

size_t dtype_size(int dtype) { return dtype == BLT_T_F32 ? 4 : 2; }

int check_rows(const blt_kv8_cache* c, const blt_kv8_rows* r, Kv8RowsArgs& a) {
  if (!r) return bad(BLT_ERR_INVALID_ARG, "rows is NULL");
  if (r->dtype < BLT_T_F32 || r->dtype > BLT_T_F16) return bad(BLT_ERR_INVALID_ARG, "dtype %d", r->dtype);
  if (r->n_rows < 0 || r->max_rows < 0) return bad(BLT_ERR_INVALID_ARG, "n_rows %d, max_rows %d", r->n_rows, r->max_rows);
  a.n_rows = r->n_rows;
  a.max_rows = r->max_rows < r->n_rows ? r->max_rows : r->n_rows;
  if (a.max_rows == 0) return BLT_OK;
  if (!r->k || !r->v || !r->row_offsets || !r->start) return bad(BLT_ERR_INVALID_ARG, "a NULL pointer in rows");
  const size_t es = dtype_size(r->dtype);
  if (misaligned(r->k, es) || misaligned(r->v, es) || misaligned(r->row_offsets, 4) || misaligned(r->start, 4))
    return bad(BLT_ERR_INVALID_ARG, "a misaligned pointer in rows");
  if (r->row_stride < 0 || r->head_stride < 0) return bad(BLT_ERR_INVALID_ARG, "a negative stride in rows");
  a.k = r->k, a.v = r->v, a.dtype = r->dtype, a.rs = r->row_stride, a.hs = r->head_stride;
  a.row_off = r->row_offsets, a.start = r->start;
  a.vec = !misaligned(r->k, 16) && !misaligned(r->v, 16) && r->row_stride * es % 16 == 0 && r->head_stride * es % 16 == 0;
  return BLT_OK;
}

// Whether two of the rows x heads pieces of `dim` elements that are to be written share an element: two offsets
// i * row_stride + j * head_stride closer than dim.  Where one stride steps over the whole of the other axis, it is the other
// one that counts; else each difference along the shorter axis is held against the nearest multiples of the other's stride.
bool overlap(int rows, long long row_stride, int heads, long long head_stride, int dim) {
  if ((rows > 1 && row_stride < dim) || (heads > 1 && head_stride < dim)) return true;
  if (rows <= 1 || heads <= 1 || row_stride / heads >= head_stride || head_stride / rows >= row_stride) return false;
  const bool by_row = rows < heads;
  const long long n = by_row ? rows : heads, step = by_row ? row_stride : head_stride;
  const long long others = by_row ? heads : rows, other = by_row ? head_stride : row_stride;
  for (long long i = 1; i < n; ++i) {
    const long long k = i * step / other, d = i * step - k * other;
    if ((k < others && d < dim) || (k + 1 < others && other - d < dim)) return true;
  }
  return false;
}

template <class F>
int by_dim(int dh, int fmt, F f) {
  if (dh == 32) return fmt == BLT_KV8_INT8 ? f.template operator()<32, 0>() : f.template operator()<32, 1>();
  if (dh == 64) return fmt == BLT_KV8_INT8 ? f.template operator()<64, 0>() : f.template operator()<64, 1>();
  if (dh == 96) return fmt == BLT_KV8_INT8 ? f.template operator()<96, 0>() : f.template operator()<96, 1>();
  return fmt == BLT_KV8_INT8 ? f.template operator()<128, 0>() : f.template operator()<128, 1>();
}

// Streaming multiprocessors of the current device (asked once per device; the same answer every time, from any thread).
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) n = 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

cudaError_t kv8_attend_launch(int fmt, int dh, const Kv8View& c, const Kv8AttnArgs& a, int max_keys, cudaStream_t st) {
  const int sms = sm_count();
  switch (dh) {
    case 32: return kv8_attend_d32(fmt, c, a, max_keys, sms, st);
    case 64: return kv8_attend_d64(fmt, c, a, max_keys, sms, st);
    case 96: return kv8_attend_d96(fmt, c, a, max_keys, sms, st);
    default: return kv8_attend_d128(fmt, c, a, max_keys, sms, st);
  }
}

}  // namespace bltdec

using namespace bltdec;

namespace {

// Queues a kernel.  The error is this launch's own: cudaGetLastError() could report what an earlier call of the thread left.
template <class... P, class... A>
int launch(const char* what, void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e == cudaSuccess) return BLT_OK;
  cudaGetLastError();
  return cuda_bad(what, e);
}

struct AppendLaunch {
  const Kv8View& v;
  const Kv8RowsArgs& a;
  dim3 grid;
  int threads;
  cudaStream_t st;
  template <int DH, int FMT>
  int operator()() const {
    auto go = [&](auto kern) { return launch("blt_kv8_append", kern, grid, threads, 0, st, v, a); };
    return a.dtype == BLT_T_F32 ? go(k_kv8_append<DH, FMT, BLT_T_F32>)
                                : a.dtype == BLT_T_BF16 ? go(k_kv8_append<DH, FMT, BLT_T_BF16>) : go(k_kv8_append<DH, FMT, BLT_T_F16>);
  }
};
struct ReadLaunch {
  const Kv8View& v;
  const Kv8RowsArgs& a;
  dim3 grid;
  int threads;
  cudaStream_t st;
  template <int DH, int FMT>
  int operator()() const {
    auto go = [&](auto kern) { return launch("blt_kv8_read", kern, grid, threads, 0, st, v, a); };
    return a.dtype == BLT_T_F32 ? go(k_kv8_read<DH, FMT, BLT_T_F32>)
                                : a.dtype == BLT_T_BF16 ? go(k_kv8_read<DH, FMT, BLT_T_BF16>) : go(k_kv8_read<DH, FMT, BLT_T_F16>);
  }
};
struct SelectLaunch {
  const Kv8View& v;
  const Kv8SelArgs& a;
  dim3 grid;
  int threads;
  size_t smem;
  cudaStream_t st;
  template <int DH, int FMT>
  int operator()() const {
    const cudaError_t e = kv8_allow_smem<k_kv8_select<DH>>(kKv8MaxSelPages * 4 + 64 * (DH / 4 * 8 + 4));
    if (e != cudaSuccess) {
      cudaGetLastError();
      return cuda_bad("blt_kv8_select", e);
    }
    return launch("blt_kv8_select", k_kv8_select<DH>, grid, threads, smem, st, v, a);
  }
};

int store_or_read(const blt_kv8_cache* c, const blt_kv8_rows* rows, void* stream, bool store) {
  g_err[0] = 0;
  Kv8View v{};
  Kv8RowsArgs a{};
  if (int rc = check_cache(c, v)) return rc;
  if (int rc = check_rows(c, rows, a)) return rc;
  if (a.max_rows == 0) return BLT_OK;
  if (!store && overlap(a.n_rows, a.rs, c->n_heads, a.hs, c->head_dim)) return bad(BLT_ERR_INVALID_ARG, "rows to be written overlap");
  DeviceScope dev;
  if (int rc = dev.enter(c->k)) return rc;
  // rows at any position touch at most this many pages
  const long long pages = ((long long)a.max_rows + 2ll * c->page_tokens - 2) / c->page_tokens;
  const long long px = pages < c->max_pages ? pages : c->max_pages;
  // Heads share CTAs once there would be more than 16 CTAs an SM: the lookups of a CTA then serve more rows (four prompts
  // of 8192 rows, 16 heads: append 61 us with a CTA a head, 53 us so; 64 sequences of 16 rows: 8.3 us, 10.5 us with 8 an SM).
  long long gy = c->n_heads;
  while (gy > 1 && px * c->batch * gy > 16ll * sm_count()) gy = (gy + 1) / 2;
  const dim3 grid((unsigned)px, (unsigned)gy, (unsigned)c->batch);
  const int blocks = c->page_tokens / 16, touched = (int)((a.max_rows + 30ll) / 16);
  int warps = 2 * (blocks < touched ? blocks : touched);
  warps = warps < 4 ? 4 : warps > kKv8RowThreads / 32 ? kKv8RowThreads / 32 : warps;
  return store ? by_dim(c->head_dim, c->format, AppendLaunch{v, a, grid, warps * 32, (cudaStream_t)stream})
               : by_dim(c->head_dim, c->format, ReadLaunch{v, a, grid, warps * 32, (cudaStream_t)stream});
}

}  // namespace

extern "C" {

int blt_kv8_append(const blt_kv8_cache* c, const blt_kv8_rows* rows, void* stream) { return store_or_read(c, rows, stream, true); }

int blt_kv8_read(const blt_kv8_cache* c, const blt_kv8_rows* rows, void* stream) { return store_or_read(c, rows, stream, false); }

int blt_kv8_attend(const blt_kv8_cache* c, const blt_kv8_attention* t, void* stream) {
  g_err[0] = 0;
  Kv8View v{};
  if (int rc = check_cache(c, v)) return rc;
  if (!t) return bad(BLT_ERR_INVALID_ARG, "the attention is NULL");
  if (t->dtype < BLT_T_F32 || t->dtype > BLT_T_F16) return bad(BLT_ERR_INVALID_ARG, "dtype %d", t->dtype);
  if (t->n_q_heads < 1 || t->n_q_heads % c->n_heads) return bad(BLT_ERR_INVALID_ARG, "n_q_heads %d for %d heads", t->n_q_heads, c->n_heads);
  if (t->n_rows < 0 || t->max_rows < 0 || t->max_keys < 0)
    return bad(BLT_ERR_INVALID_ARG, "n_rows %d, max_rows %d, max_keys %d", t->n_rows, t->max_rows, t->max_keys);
  if (!std::isfinite(t->scale)) return bad(BLT_ERR_INVALID_ARG, "scale is not finite");
  const int max_rows = t->max_rows < t->n_rows ? t->max_rows : t->n_rows;
  if (max_rows == 0) return BLT_OK;
  if (!t->q || !t->out || !t->row_offsets || !t->row_limit) return bad(BLT_ERR_INVALID_ARG, "a NULL pointer in the attention");
  const size_t es = dtype_size(t->dtype);
  if (misaligned(t->q, es) || misaligned(t->out, es) || misaligned(t->lse, 4) || misaligned(t->row_offsets, 4) || misaligned(t->row_limit, 4) ||
      misaligned(t->sel_pages, 4) || misaligned(t->sel_count, 4))
    return bad(BLT_ERR_INVALID_ARG, "a misaligned pointer in the attention");
  if (t->q_row_stride < 0 || t->q_head_stride < 0 || t->out_row_stride < 0 || t->out_head_stride < 0)
    return bad(BLT_ERR_INVALID_ARG, "a negative stride in the attention");
  if (overlap(t->n_rows, t->out_row_stride, t->n_q_heads, t->out_head_stride, c->head_dim)) return bad(BLT_ERR_INVALID_ARG, "rows of out overlap");
  if ((t->sel_pages != nullptr) != (t->sel_count != nullptr)) return bad(BLT_ERR_INVALID_ARG, "sel_pages and sel_count come together");
  if (t->sel_pages && (t->n_select < 1 || (long long)t->n_select * c->page_tokens >= (1ll << 30)))
    return bad(BLT_ERR_INVALID_ARG, "n_select %d", t->n_select);
  if (t->flags & ~BLT_KV8_TEST_STALL) return bad(BLT_ERR_INVALID_ARG, "flags %d", t->flags);
  if ((long long)max_rows * t->n_q_heads >= (1ll << 26)) return bad(BLT_ERR_INVALID_ARG, "%d rows of %d heads", max_rows, t->n_q_heads);
  DeviceScope dev;
  if (int rc = dev.enter(c->k)) return rc;
  Kv8AttnArgs a{};
  a.q = t->q, a.out = t->out, a.lse = t->lse, a.dtype = t->dtype;
  a.Hq = t->n_q_heads, a.G = t->n_q_heads / c->n_heads, a.n_rows = t->n_rows, a.max_rows = max_rows, a.scale = t->scale;
  a.qs = t->q_row_stride, a.qhs = t->q_head_stride, a.os = t->out_row_stride, a.ohs = t->out_head_stride;
  a.row_off = t->row_offsets, a.row_limit = t->row_limit;
  a.sel_pages = t->sel_pages, a.sel_count = t->sel_count, a.n_select = t->n_select;
  a.stall = (t->flags & BLT_KV8_TEST_STALL) != 0;
  a.q_vec = !misaligned(t->q, 16) && t->q_row_stride * es % 16 == 0 && t->q_head_stride * es % 16 == 0;
  a.out_vec = !misaligned(t->out, 16) && t->out_row_stride * es % 16 == 0 && t->out_head_stride * es % 16 == 0;
  const cudaError_t e = kv8_attend_launch(c->format, c->head_dim, v, a, t->max_keys, (cudaStream_t)stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return cuda_bad("blt_kv8_attend", e);
  }
  return BLT_OK;
}

int blt_kv8_select(const blt_kv8_cache* c, const blt_kv8_selection* t, void* stream) {
  g_err[0] = 0;
  Kv8View v{};
  if (int rc = check_cache(c, v)) return rc;
  if (!t) return bad(BLT_ERR_INVALID_ARG, "the selection is NULL");
  if (!c->k_min) return bad(BLT_ERR_INVALID_ARG, "the cache has no summaries");
  if (c->max_pages > kKv8MaxSelPages) return bad(BLT_ERR_INVALID_ARG, "max_pages %d above %d", c->max_pages, kKv8MaxSelPages);
  if (t->dtype < BLT_T_F32 || t->dtype > BLT_T_F16) return bad(BLT_ERR_INVALID_ARG, "dtype %d", t->dtype);
  if (t->n_q_heads < 1 || t->n_q_heads % c->n_heads || t->n_q_heads / c->n_heads > 64)
    return bad(BLT_ERR_INVALID_ARG, "n_q_heads %d for %d heads (at most 64 a head)", t->n_q_heads, c->n_heads);
  if (t->n_rows < 0 || t->max_rows < 0 || t->max_keys < 0)
    return bad(BLT_ERR_INVALID_ARG, "n_rows %d, max_rows %d, max_keys %d", t->n_rows, t->max_rows, t->max_keys);
  if (t->n_select < 1 || t->n_sink < 0 || t->n_local < 0 || (long long)t->n_sink + t->n_local > t->n_select)
    return bad(BLT_ERR_INVALID_ARG, "n_select %d, n_sink %d, n_local %d", t->n_select, t->n_sink, t->n_local);
  const int max_rows = t->max_rows < t->n_rows ? t->max_rows : t->n_rows;
  if (max_rows == 0) return BLT_OK;
  if (!t->q || !t->row_offsets || !t->row_limit || !t->sel_pages || !t->sel_count) return bad(BLT_ERR_INVALID_ARG, "a NULL pointer in the selection");
  if (misaligned(t->q, dtype_size(t->dtype)) || misaligned(t->row_offsets, 4) || misaligned(t->row_limit, 4) || misaligned(t->sel_pages, 4) ||
      misaligned(t->sel_count, 4))
    return bad(BLT_ERR_INVALID_ARG, "a misaligned pointer in the selection");
  if (t->q_row_stride < 0 || t->q_head_stride < 0) return bad(BLT_ERR_INVALID_ARG, "a negative stride in the selection");
  DeviceScope dev;
  if (int rc = dev.enter(c->k)) return rc;
  Kv8SelArgs a{};
  a.q = t->q, a.dtype = t->dtype, a.Hq = t->n_q_heads, a.G = t->n_q_heads / c->n_heads;
  a.n_rows = t->n_rows, a.max_rows = max_rows, a.n_select = t->n_select, a.n_sink = t->n_sink, a.n_local = t->n_local;
  a.qs = t->q_row_stride, a.qhs = t->q_head_stride, a.row_off = t->row_offsets, a.row_limit = t->row_limit;
  a.pages = t->sel_pages, a.count = t->sel_count;
  const size_t smem = (size_t)a.G * (c->head_dim / 4) * 8 + ((a.G + 3) & ~3) * 4 + (size_t)c->max_pages * 4;
  const dim3 grid((unsigned)max_rows, (unsigned)c->n_heads, (unsigned)c->batch);
  // a thread for each expected page, 128 to 512: short lists leave room for more CTAs on an SM (64 rows x 16 heads of 128
  // pages: 25 us with 512 threads)
  const int want = (t->max_keys + c->page_tokens - 1) / c->page_tokens;
  const int threads = want <= 128 ? 128 : want <= 256 ? 256 : kKv8SelThreads;
  return by_dim(c->head_dim, c->format, SelectLaunch{v, a, grid, threads, smem, (cudaStream_t)stream});
}

const char* blt_kv8_last_error(void) { return g_err; }

}  // extern "C"
