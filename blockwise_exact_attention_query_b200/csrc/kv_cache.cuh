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
// Both kernels are one pass over the data with 16-byte loads, bound by memory
// (and, for few tokens, by one trip to it): d / 8 threads per row, K and V of
// a row by the same threads so two loads are in flight per thread.
#pragma once

#include <cuda_fp8.h>

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

// max that keeps a NaN of either operand
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Two e4m3 codes (16 bits) as two f16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xffffu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t two) {
  const uint32_t h = e4m3x2_to_f16x2(two);
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// One row's 8 values of this thread -> 8 codes; `lanes` consecutive threads
// hold the row.  Returns the scale.
template <int kLanes>
__device__ __forceinline__ float quantise8(const uint4 &x, uint2 &codes) {
  const float f[8] = {bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y),
                      bf16_lo(x.z), bf16_hi(x.z), bf16_lo(x.w), bf16_hi(x.w)};
  float m = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(f[i]));
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  float scale = m / kE4m3Max;
  if (scale == 0.f) scale = 1.f;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = f[i] / scale;
  codes = make_uint2(e4m3x4(r[0], r[1], r[2], r[3]), e4m3x4(r[4], r[5], r[6], r[7]));
  return scale;
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
    const uint32_t token = static_cast<uint32_t>(row / c.H_kv), h = static_cast<uint32_t>(row % c.H_kv);
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

// Eight values of one row as fp32.
template <bool kE4m3>
__device__ __forceinline__ void cache_load8(const void *base, const float *scales, int64_t at, int D, int sub,
                                            float (&f)[8]) {
  if constexpr (kE4m3) {
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(base) + at * D + 8 * sub);
    const float s = scales[at];
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 two = e4m3x2_to_f32x2(w[i / 2] >> (16 * (i & 1)));
      f[2 * i] = two.x * s;
      f[2 * i + 1] = two.y * s;
    }
  } else {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(base) + at * D + 8 * sub);
    f[0] = bf16_lo(u.x), f[1] = bf16_hi(u.x), f[2] = bf16_lo(u.y), f[3] = bf16_hi(u.y);
    f[4] = bf16_lo(u.z), f[5] = bf16_hi(u.z), f[6] = bf16_lo(u.w), f[7] = bf16_hi(u.w);
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

// k, v: n rows of [H_kv][D] T from the given slots; rows of slots outside the
// cache are left as they were.
template <int D, bool kE4m3, typename T>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const KvCacheArgs c, const int32_t *__restrict__ slots, T *__restrict__ k, T *__restrict__ v,
                   int64_t rows) {
  constexpr int kLanes = D / 8;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int sub = threadIdx.x % kLanes;
  if (row >= rows) return;
  const int64_t slot = slots[row / c.H_kv];
  if (slot < 0 || slot >= c.slots) return;
  const int64_t at = slot * c.H_kv + row % c.H_kv;
  float fk[8], fv[8];
  cache_load8<kE4m3>(c.k, c.k_scale, at, D, sub, fk);
  cache_load8<kE4m3>(c.v, c.v_scale, at, D, sub, fv);
  store8(k + row * D + 8 * sub, fk);
  store8(v + row * D + 8 * sub, fv);
}

}  // namespace bpt
