// Device pieces of the 8-bit paged KV cache (include/bltkv8.h).
//
// A code c of a block with exponent e stands for c * 2^(e - 127).  Both int8 and e4m3 codes, and their products with a power
// of two, are exact in bf16 (storing and reading back go through it) and, as bare codes, in f16 (attention's operands).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <limits.h>

#include <atomic>

#include "bltkv8.h"
#include "common.cuh"

namespace bltdec {

constexpr int kKv8Block = 16;      // positions that share an exponent (one k16 step of the value product)
constexpr int kKv8LowExp = 16;     // least exponent: e4m3's smallest step, 2^-9 2^(16 - 127), is normal in bf16
constexpr int kKv8MaxSelPages = 49152;  // blt_kv8_select keeps a score per page in shared memory

// What the kernels need of a blt_kv8_cache, by value.
struct Kv8View {
  uint8_t *k, *v, *ke, *ve;
  int8_t *kmin, *kmax;
  uint8_t* ksexp;
  long long page_stride, exp_stride, sum_stride, sexp_stride;
  const int* table;
  int* status;
  int H, PT, tpp;     // tpp: 16-position blocks per page
  unsigned tpp_magic; // floor(2^32 / tpp) + 1: x / tpp == umulhi(x, magic) for x < 2^28 (tpp <= 16)
  int n_pages, batch, max_pages;
};

__device__ __forceinline__ int kv8_div_tpp(const Kv8View& c, int x) {
  return c.tpp == 1 ? x : (int)__umulhi((unsigned)x, c.tpp_magic);
}

// Pool page of a sequence's page, -1 (and the status word set) if there is none.
__device__ __forceinline__ int kv8_page(const Kv8View& c, int s, int pi) {
  const int p = (pi >= 0 && pi < c.max_pages) ? __ldg(c.table + (size_t)s * c.max_pages + pi) : -1;
  if (p < 0 || p >= c.n_pages) {
    if (c.status) set_status(c.status, kErrDevice);
    return -1;
  }
  return p;
}

// Rows of sequence s: [r0, r1), cut to the arrays and to max_rows.
__device__ __forceinline__ void kv8_rows_of(const int* off, int s, int n_rows, int max_rows, int* status, int& r0, int& r1) {
  r0 = __ldg(off + s);
  r1 = __ldg(off + s + 1);
  const int a = min(max(r0, 0), n_rows), b = min(max(r1, a), a + min(n_rows - a, max_rows));
  if ((a != r0 || b != r1) && status) set_status(status, kErrDevice);
  r0 = a;
  r1 = b;
}

__device__ __forceinline__ float kv8_pow2(int e) { return __int_as_float(e << 23); }  // 2^(e - 127), 1 <= e <= 254

// Least e >= kKv8LowExp with amax <= top * 2^(e - 127); amax finite.  FMT 0: top 127 = 1.984375 * 2^6;
// FMT 1: top 448 = 1.75 * 2^8.
template <int FMT>
__device__ __forceinline__ int kv8_exponent(float amax) {
  const unsigned u = __float_as_uint(amax);
  const int ex = (int)(u >> 23);
  const unsigned frac = u & 0x7fffffu;
  const int e = FMT == 0 ? ex - 6 + (frac > 0x7e0000u) : ex - 8 + (frac > 0x600000u);
  return max(e, kKv8LowExp);
}

// x with NaN as 0; infinities are left to the caller's clamp.
__device__ __forceinline__ float kv8_finite(float x) {
  return x != x ? 0.f : x;
}
__device__ __forceinline__ float kv8_mag(float x) {  // |x| if finite, else 0
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// Four codes of x0..x3 at scale inv = 2^(127 - e), to nearest even.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_encode4(float x0, float x1, float x2, float x3, float inv) {
  if constexpr (FMT == 0) {
    // 1.5 * 2^23 + y: the sum's rounding is y's, and its low byte the code (the conversion unit is four times slower)
    auto one = [inv](float x) { return __float_as_uint(fminf(fmaxf(kv8_finite(x) * inv, -127.f), 127.f) + 12582912.f); };
    return __byte_perm(__byte_perm(one(x0), one(x1), 0x0040), __byte_perm(one(x2), one(x3), 0x0040), 0x5410);
  } else {
    auto two = [inv](float a, float b) {
      const float2 y = make_float2(fminf(fmaxf(kv8_finite(a) * inv, -448.f), 448.f), fminf(fmaxf(kv8_finite(b) * inv, -448.f), 448.f));
      return (uint32_t)__nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
    };
    return two(x0, x1) | (two(x2, x3) << 16);
  }
}

// Codes in bytes (sel & 0xf) and (sel >> 8 & 0xf) of (hi:lo) as two bf16 (lower half first).  `sel` is a
// byte-permute selector that puts the first code into bytes 0 and 1 and the second into 2 and 3.
// int8: with l the low 7 bits and n the sign bit the value is l - 128 n = (128 + l) - (128 + 128 n),
//   both exact bf16 numbers with exponent bits 0x4300 / 0x4380.
// e4m3: sign | 4 exponent | 3 mantissa bits moved into a bf16's places read as value * 2^-120 (the
//   exponent bias is 7 there and 127 here; subnormals included), times 2^120.
template <int FMT>
__device__ __forceinline__ uint32_t kv8_pair(uint32_t lo, uint32_t hi, uint32_t sel) {
  const uint32_t y = __byte_perm(lo, hi, sel);
  if constexpr (FMT == 0) {
    const uint32_t a = (y & 0x007f007fu) | 0x43004300u, b = (y & 0x00800080u) | 0x43004300u;
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(b));
    return d;
  } else {
    const uint32_t a = (y & 0x80008000u) | ((y >> 4) & 0x07f007f0u);
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;\n" : "=r"(d) : "r"(a), "r"(0x7b807b80u));
    return d;
  }
}
// Selector for codes i and j of the eight bytes (hi:lo).
__host__ __device__ constexpr uint32_t kv8_sel(int i, int j) { return (uint32_t)(i | (i << 4) | (j << 8) | (j << 12)); }

__device__ __forceinline__ float2 bf16x2_to_f2(uint32_t p) {
  return make_float2(__uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
}
__device__ __forceinline__ uint32_t f2_to_bf16x2(float x0, float x1) {  // x0 in the lower half
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(d) : "f"(x1), "f"(x0));
  return d;
}

// Element i of an array of BLT_T_* type.
__device__ __forceinline__ float kv8_ld(const void* p, int dtype, long long i) {
  if (dtype == BLT_T_F32) return __ldg(static_cast<const float*>(p) + i);
  if (dtype == BLT_T_BF16) return __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
  return __half2float(__ldg(static_cast<const __half*>(p) + i));
}
__device__ __forceinline__ void kv8_st(void* p, int dtype, long long i, float v) {
  if (dtype == BLT_T_F32) static_cast<float*>(p)[i] = v;
  else if (dtype == BLT_T_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else static_cast<__half*>(p)[i] = __float2half_rn(v);
}
// Four elements from i; vec: 16-byte aligned rows (i a multiple of 4).
__device__ __forceinline__ void kv8_ld4(const void* p, int dtype, long long i, bool vec, float (&x)[4]) {
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = kv8_ld(p, dtype, i + j);
  } else if (dtype == BLT_T_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  } else {
    const uint2 a = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i));
    const float2 f = dtype == BLT_T_BF16 ? bf16x2_to_f2(a.x) : __half22float2(*reinterpret_cast<const __half2*>(&a.x));
    const float2 h = dtype == BLT_T_BF16 ? bf16x2_to_f2(a.y) : __half22float2(*reinterpret_cast<const __half2*>(&a.y));
    x[0] = f.x, x[1] = f.y, x[2] = h.x, x[3] = h.y;
  }
}
// Four elements to i; vec: 16-byte aligned rows (i a multiple of 4).
__device__ __forceinline__ void kv8_st4(void* p, int dtype, long long i, bool vec, float x, float y, float z, float w) {
  if (!vec) {
    kv8_st(p, dtype, i, x), kv8_st(p, dtype, i + 1, y), kv8_st(p, dtype, i + 2, z), kv8_st(p, dtype, i + 3, w);
  } else if (dtype == BLT_T_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(x, y, z, w);
  } else if (dtype == BLT_T_BF16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(f2_to_bf16x2(x, y), f2_to_bf16x2(z, w));
  } else {
    const __half2 a = __floats2half2_rn(x, y), b = __floats2half2_rn(z, w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}
// Eight elements from i; vec: 16-byte aligned.
__device__ __forceinline__ void kv8_ld8(const void* p, int dtype, long long i, bool vec, float (&x)[8]) {
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = kv8_ld(p, dtype, i + j);
  } else if (dtype == BLT_T_F32) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i));
    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + i) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = dtype == BLT_T_BF16 ? bf16x2_to_f2(w[j]) : __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      x[2 * j] = f.x, x[2 * j + 1] = f.y;
    }
  }
}
__device__ __forceinline__ void kv8_st8(void* p, int dtype, long long i, bool vec, const float (&x)[8]) {
  if (!vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) kv8_st(p, dtype, i + j, x[j]);
  } else if (dtype == BLT_T_F32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    o[0] = make_float4(x[0], x[1], x[2], x[3]);
    o[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (dtype == BLT_T_BF16) {
        w[j] = f2_to_bf16x2(x[2 * j], x[2 * j + 1]);
      } else {
        const __half2 h = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// Eight codes (lo: the first four) as floats, without the scale.
template <int FMT>
__device__ __forceinline__ void kv8_decode8(uint2 w, float (&x)[8]) {
  const uint32_t v[2] = {w.x, w.y};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 2 * (j & 1);
    const float2 f = bf16x2_to_f2(kv8_pair<FMT>(v[j >> 1], 0, kv8_sel(i, i + 1)));
    x[2 * j] = f.x, x[2 * j + 1] = f.y;
  }
}

// ------------------------------------------------------------------------ attention arguments
struct Kv8AttnArgs {
  const void* q;
  void* out;
  float* lse;
  int dtype, Hq, G, n_rows, max_rows;
  float scale;
  long long qs, qhs, os, ohs;
  const int *row_off, *row_limit;
  const int *sel_pages, *sel_count;
  int n_select;
  int q_vec, out_vec;  // rows of q (out) allow 16-byte loads (stores)
  int stall;           // BLT_KV8_TEST_STALL
};
// Allows a kernel `bytes` of dynamic shared memory on the current device: asked of the driver once a device.
template <auto KERN>
cudaError_t kv8_allow_smem(int bytes) {
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

cudaError_t kv8_attend_launch(int fmt, int dh, const Kv8View& c, const Kv8AttnArgs& a, int max_keys, cudaStream_t st);

}  // namespace bltdec
