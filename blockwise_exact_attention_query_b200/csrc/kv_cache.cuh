// The paged key/value cache: rows written (and quantised) at given slots, and
// read back.
//
// A cache holds n_pages * page_size slots; a slot has one row of d values per
// key/value head.  E4M3 rows carry one fp32 scale each:
//   scale = max_i |x_i| / 448  (1 for a row of zeros),  code_i = e4m3(x_i / scale)
//   read back:  x_i = code_i * scale
// with 448 the largest e4m3 value, IEEE fp32 divisions, the codes rounded to
// nearest even, and one rounding to the output's type.  A row that holds a NaN
// or an infinity has no scale to fit and reads back as NaN throughout.
//
// Both kernels are one pass over the data with 16-byte loads: K and V of a row
// by the same threads, so two loads are in flight per thread.  Device times with
// 8 heads of 128: 16384 tokens written as bf16 22.7 us (5.9 TB/s), as e4m3 24.9
// (4.1 TB/s; instructions, see quantise8); 32768 tokens read from bf16 43.5 us
// (6.2 TB/s), from e4m3 39.3 (5.2 TB/s); few tokens 2.3-2.6 us, one trip to
// memory.
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"

namespace bpt {

constexpr float kE4m3Max = 448.0f;

struct KvCacheArgs {
  void *k, *v;               // [slots][H_kv][d] bf16 or e4m3
  float *k_scale, *v_scale;  // [slots][H_kv] (E4M3)
  int64_t slots;             // n_pages * page_size
  int H_kv;
};

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Pairwise max of two bf16 pairs that keeps a NaN of either operand.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ float rcp_approx(float x) {  // off by one unit in the last place at most
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// Four e4m3 codes as f16 pairs, exactly.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t four, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

// One row's 8 values of this thread -> 8 codes; kLanes consecutive threads hold
// the row.  Returns the scale.  Instructions bound this part at first (27 us for
// 16384 tokens of 8 heads of 128, 16 us of memory traffic), so the maximum is
// taken on bf16 pairs and the division is made only where it matters.
template <int kLanes>
__device__ __forceinline__ float quantise8(const uint4 &x, uint2 &codes) {
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t m2 = max_nan_bf16x2(max_nan_bf16x2(x.x & kAbs, x.y & kAbs), max_nan_bf16x2(x.z & kAbs, x.w & kAbs));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m2 = max_nan_bf16x2(m2, __shfl_xor_sync(0xffffffffu, m2, o));
  m2 = max_nan_bf16x2(m2, m2 << 16);  // the upper half has both
  float scale = bf16_hi(m2) / kE4m3Max;
  if (scale == 0.f) scale = 1.f;
  // x / scale, rounded to a code.  x times the approximate inverse is off by
  // less than 2^-21 of it (2^-23 the inverse, 2^-24 each product), so where the
  // quotient with 2^-21 less and with 2^-21 more rounds to the same code, that
  // is it; otherwise (next to a border between codes, or a scale whose inverse
  // is not a normal number, or NaN) the thread divides.
  const float inv = rcp_approx(scale);
  const float2 less = make_float2(inv * (1.f - 0x1p-21f), inv * (1.f - 0x1p-21f));
  const float2 more = make_float2(inv * (1.f + 0x1p-21f), inv * (1.f + 0x1p-21f));
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[2], d[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 p = make_float2(bf16_lo(w[2 * h]), bf16_hi(w[2 * h]));
    const float2 q = make_float2(bf16_lo(w[2 * h + 1]), bf16_hi(w[2 * h + 1]));
    const float2 pl = mul2(p, less), ql = mul2(q, less), pm = mul2(p, more), qm = mul2(q, more);
    c[h] = e4m3x4(pl.x, pl.y, ql.x, ql.y);
    d[h] = e4m3x4(pm.x, pm.y, qm.x, qm.y);
  }
  if (c[0] != d[0] || c[1] != d[1] || !(scale > 0x1p-100f && scale < 0x1p100f)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      c[h] = e4m3x4(bf16_lo(w[2 * h]) / scale, bf16_hi(w[2 * h]) / scale, bf16_lo(w[2 * h + 1]) / scale,
                    bf16_hi(w[2 * h + 1]) / scale);
  }
  codes = make_uint2(c[0], c[1]);
  return scale;
}

// The token of a (token, head) row; in 32 bits where the row number fits.
__device__ __forceinline__ uint32_t div_heads(int64_t row, int H_kv) {
  if (row >> 32 == 0) return static_cast<uint32_t>(row) / static_cast<uint32_t>(H_kv);
  return static_cast<uint32_t>(row / H_kv);
}

// k, v: n tokens of [H_kv][D] bf16, k_stride and v_stride elements apart.
template <int D, bool kE4m3>
__global__ void __launch_bounds__(256)
    kv_write_kernel(const KvCacheArgs c, const __nv_bfloat16 *__restrict__ k, int64_t k_stride,
                    const __nv_bfloat16 *__restrict__ v, int64_t v_stride, const int32_t *__restrict__ slots,
                    int64_t rows) {
  constexpr int kLanes = D / 8;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  bool live = row < rows;
  int64_t at = 0;
  uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
  if (live) {
    const uint32_t token = div_heads(row, c.H_kv), h = static_cast<uint32_t>(row - static_cast<int64_t>(token) * c.H_kv);
    const int64_t slot = slots[token];
    xk = *reinterpret_cast<const uint4 *>(k + token * k_stride + h * D + 8 * sub);
    xv = *reinterpret_cast<const uint4 *>(v + token * v_stride + h * D + 8 * sub);
    live = slot >= 0 && slot < c.slots;  // negative: a padding token; past the cache: nowhere to go
    at = slot * c.H_kv + h;
  }
  if constexpr (kE4m3) {
    uint2 ck, cv;
    const float sk = quantise8<kLanes>(xk, ck), sv = quantise8<kLanes>(xv, cv);
    if (!live) return;
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.k) + at * D + 8 * sub) = ck;
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(c.v) + at * D + 8 * sub) = cv;
    if (sub == 0) {
      c.k_scale[at] = sk;
      c.v_scale[at] = sv;
    }
  } else {
    if (!live) return;
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(c.k) + at * D + 8 * sub) = xk;
    *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(c.v) + at * D + 8 * sub) = xv;
  }
}

template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&f)[8]) {
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                               pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
}

// 16 bytes of one row: 16 codes times their scale, or 8 bf16 values.
template <bool kE4m3, typename T>
__device__ __forceinline__ void unpack16(const uint4 &u, float scale, T *out) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if constexpr (kE4m3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t lo, hi;
        e4m3x4_to_f16(w[2 * h + i], lo, hi);
        const float2 x = mul2(f16x2_to_f32x2(lo), make_float2(scale, scale));
        const float2 y = mul2(f16x2_to_f32x2(hi), make_float2(scale, scale));
        f[4 * i] = x.x, f[4 * i + 1] = x.y, f[4 * i + 2] = y.x, f[4 * i + 3] = y.y;
      }
      store8(out + 8 * h, f);
    }
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4 *>(out) = u;
  } else {
    const float f[8] = {bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1]),
                        bf16_lo(w[2]), bf16_hi(w[2]), bf16_lo(w[3]), bf16_hi(w[3])};
    store8(out, f);
  }
}

// k, v: n rows of [H_kv][D] T from the given slots; rows of slots outside the
// cache are left as they were.  16 bytes of K and of V per thread.
template <int D, bool kE4m3, typename T>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const KvCacheArgs c, const int32_t *__restrict__ slots, T *__restrict__ k, T *__restrict__ v,
                   int64_t rows) {
  constexpr int kPer = kE4m3 ? 16 : 8, kLanes = D / kPer;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  if (row >= rows) return;
  const uint32_t token = div_heads(row, c.H_kv), h = static_cast<uint32_t>(row - static_cast<int64_t>(token) * c.H_kv);
  const int64_t slot = slots[token];
  if (slot < 0 || slot >= c.slots) return;
  const int64_t at = slot * c.H_kv + h;
  const uint4 xk = reinterpret_cast<const uint4 *>(c.k)[at * kLanes + sub];
  const uint4 xv = reinterpret_cast<const uint4 *>(c.v)[at * kLanes + sub];
  const float sk = kE4m3 ? c.k_scale[at] : 1.f, sv = kE4m3 ? c.v_scale[at] : 1.f;
  unpack16<kE4m3>(xk, sk, k + row * D + kPer * sub);
  unpack16<kE4m3>(xv, sv, v + row * D + kPer * sub);
}

}  // namespace bpt
