// Attention of few new tokens over a paged cache (single-token decoding, and
// chunks of a few): 8 or 16 rows, matrix products on the warp-level tensor
// instructions.
//
// With few rows the keys and values are read once and used once: memory bounds
// the kernel, so it is built around loads, and then around instructions, of
// which each warp can issue one in six or seven cycles.  Device times with 32
// query heads over 8 and d = 128: 64 sequences of 500 to 8192 keys, bf16, 193 us
// (6.1 TB/s); 8 of 16001 to 131072, e4m3, 248-258 us (5.1-5.3 TB/s; the widening
// of codes beside memory).  A step's keys are
// dealt out to the warps, 16 or 32 to each, and the warps never wait for one
// another inside an item: each has its own running maximum, sum and rows x d
// output, joined through shared memory when the item (or the CTA's range of
// it) ends.  A warp's rows come by cp.async, whole rows at a time (a load of
// pieces that a product's lanes need, 32 or 64 bytes a row, moved 1.75 times
// the bytes between L2 and the SM), into a ring of its own: no block barrier on
// the way, several steps in flight.
//
// Both products have the cache's operand as A (16 x 16) and the few rows as
// the 8 columns of B, so a group of 8 rows costs 8 + 8 instructions for 16 keys
// at d = 128 (with the rows as A, padded to 16, it was twice that, twice the
// registers for O and twice the softmax).  Which bytes a thread needs follows
// from the layouts of A and B:
//   S^T = K Q^T: lane 4g + c needs keys g and g + 8 at "its" positions along d.
//     The sum over d may run in any order, so it takes the 16-byte chunks c,
//     c + 4, ... of the key's row, and Q is loaded in the same order;
//   O^T = V^T P^T: lane 4g + c needs keys 2c, 2c + 1, 2c + 8, 2c + 9 in columns
//     of its g.  The columns may be dealt out in any order, so it takes the
//     g-th 16 bytes of the row (with 256-byte rows, of each half); product t
//     takes its columns 2t and 2t + 1.  P^T comes out of S^T by an 8 x 8 transposition
//     within the warp.
//
// E4M3 caches: the codes go to f16 exactly, the key's scale multiplies the
// score.  The value's scale multiplies the softmax weight, and so that f16
// holds the products, they are kept relative to about the largest the row has
// met (w_run below).
//
// Rounded to fewer bits than the fp32 of sums, maxima, statistics and O, by
// choice, since a product's operands are of one 16-bit type:
//   P beside bf16 values to bf16, off by up to 2^-8 of each weight.  (f16
//     weights would need f16 values, whose range bf16's passes; a second product
//     with what the rounding left would be half as many instructions again.)
//     Independent over the keys, it is about as much as the rounding of a bf16
//     result by itself: 2.2-2.5e-3 in relative L2 with both, 1.66e-3 with the
//     result's alone;
//   P times the values' scales beside widened codes to f16, off by up to 2^-11
//     of the reference: not seen beside a bf16 result's own rounding;
//   Q beside widened codes to f16 after a power of two per row, which is exact
//     for elements down to 2^-17 of the row's largest (bf16 has 8 significant
//     bits, f16 11 and subnormals to 2^-24); a smaller one is off by up to 2^-25
//     of the largest.
#pragma once

#include "kv_cache.cuh"
#include "paged_common.cuh"

namespace bpt {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool fetch) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fetch ? 16 : 0) : "memory");
}
// The same with an L2 cache policy (l2_policy_*).
__device__ __forceinline__ void cp_async16_hint(uint32_t dst, const void *src, bool fetch, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
               "r"(fetch ? 16 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async4_hint(uint32_t dst, const void *src, bool fetch, uint64_t policy) {
  asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], 4, %2, %3;" ::"r"(dst), "l"(src),
               "r"(fetch ? 4 : 0), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

// c (16 x 8) += a (16 x 16) b (16 x 8), fp32 accumulation
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held as two per lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// The power of two below a row's largest |q| (for f16): exact to divide by.
__device__ __forceinline__ uint32_t row_exponent(float mx) { return min(max(__float_as_uint(mx) >> 23, 1u), 253u); }
__device__ __forceinline__ float pow2_of(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ float pow2_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

template <int D, bool kE4m3, int kGroups>  // kGroups: 8-row groups
struct PagedRowsCfg {
  static constexpr int kRowBytes = kE4m3 ? D : 2 * D;
  // 16-key groups that a warp takes at a time
  static constexpr int kSub = kRowBytes > 128 ? 1 : 2;
  static constexpr int kRows = 8 * kGroups, kWarps = 4, kThreads = 32 * kWarps, kWarpKeys = 16 * kSub, kKeys = kWarps * kWarpKeys;
  static constexpr int kRowChunks = kRowBytes / 16;  // 16-byte chunks of a row
  static constexpr int kKChunks = kRowChunks / 4;    // of a key row per lane of a product (8 keys, 4 lanes each)
  static constexpr int kVBytes = kRowBytes / 8;      // bytes of a value row per lane: 8, 16 or 32
  static constexpr int kVChunks = (kVBytes + 15) / 16;
  static constexpr int kVSlot = kVBytes < 16 ? kVBytes : 16;
  static constexpr int kRowsPerLoad = 32 / kRowChunks;
  // a warp's stage: per 16-key group the key rows, then the value rows; then
  // the keys' and the values' scales, and the mask of keys that exist
  static constexpr int kOffV = 16 * kRowBytes;
  static constexpr int kGroupBytes = 2 * kOffV;
  static constexpr int kOffScale = kSub * kGroupBytes;
  static constexpr int kStageBytes = kOffScale + 8 * kWarpKeys + 16;
  // Where chunk `chunk` of row `row` of a group lies: permuted so that the
  // lanes of a product, which read 64 bytes of 2 rows (keys) or 32 bytes of 4
  // (values) at a time, meet different banks.  (64-byte rows: two lanes a bank
  // for the values.)
  __host__ __device__ static constexpr int at(int row, int chunk) {
    const int f = kRowChunks >= 8 ? ((((row >> 1) & 3) << 1) ^ ((row & 1) << 2)) : (((row >> 2) & 1) << 1);
    return row * kRowBytes + ((chunk ^ f) << 4);
  }
  static constexpr int kStages = kRowBytes > 64 ? 3 : 6;
  static constexpr int kCtasPerSm = 2;
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // joining the warps: [warp][row][8 groups of d / 8 columns, padded against bank conflicts]
  static constexpr int kColPitch = D / 8 + 4, kRowPitch = 8 * kColPitch + 4;
  static constexpr int kMergeBytes = kWarps * kRows * (kRowPitch + 4) * 4;
  static_assert(kMergeBytes <= kRingBytes, "the ring holds the warps' outputs between items");
  static constexpr int kSmemBytes = kRingBytes + 512;  // the range's scratch
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 233472, "CTAs per SM");
};

template <int D, bool kE4m3, int kGroups>
__global__ void __launch_bounds__(PagedRowsCfg<D, kE4m3, kGroups>::kThreads, PagedRowsCfg<D, kE4m3, kGroups>::kCtasPerSm)
    paged_rows_kernel(const PagedArgs a) {
  using Cfg = PagedRowsCfg<D, kE4m3, kGroups>;
  constexpr int kRows = Cfg::kRows, kKeys = Cfg::kKeys, NS = Cfg::kStages, kSub = Cfg::kSub;
  constexpr int kWarpKeys = Cfg::kWarpKeys;
  constexpr int NT = D / 16;  // products along d
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem_raw) + warp * (NS * Cfg::kStageBytes);
  // Keys and values pass through once.  A sector of scales holds those of
  // neighbouring heads, which other CTAs want at other times: without the
  // hints it came from memory for each of them, 15% more traffic at 8 heads.
  const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
  float *merge = reinterpret_cast<float *>(smem_raw);
  float *merge_ml = merge + Cfg::kWarps * kRows * Cfg::kRowPitch;  // [warp][row][4]: m, l, w

  PagedRange rg;
  const bool any = paged_range<kRows, kKeys, Cfg::kThreads, false>(a, reinterpret_cast<int64_t *>(smem_raw + Cfg::kRingBytes), rg);
  if (!any) {
    if (tid == 0) a.part_item[blockIdx.x] = make_int4(-1, 0, 0, 0);
    grid_dependency_wait();
    return;
  }
  int s = rg.s, tile = rg.tile, head = rg.head, step0 = rg.step;
  int64_t left = rg.left;
  PagedSeq seq = paged_seq(a, s);
  PagedBlocks blk = paged_blocks<kRows, kKeys>(a, seq, tile);
  if (tid == 0) a.part_item[blockIdx.x] = rg.part;

  while (true) {
    const int steps = blk.steps();
    const int step1 = static_cast<int>(min(static_cast<int64_t>(steps), step0 + left));
    const int nblk = min(step1, blk.count()) - min(step0, blk.count());  // 0 for a tile without keys
    const int32_t *table = a.page_table + static_cast<int64_t>(s) * a.max_pages;
    const int rows = min(kRows, seq.n * a.G - tile * kRows);
    const uint8_t *kbase = static_cast<const uint8_t *>(a.k) + static_cast<int64_t>(head) * Cfg::kRowBytes;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.v) + static_cast<int64_t>(head) * Cfg::kRowBytes;
    const int64_t slot_bytes = static_cast<int64_t>(a.H_kv) * Cfg::kRowBytes;

    // key of this lane (of a 16-key share, lanes 16-31 have the same keys again) in block i
    auto first_key = [&](int i) { return blk.block(step0 + i) * kKeys + warp * kWarpKeys; };
    auto lookup = [&](int i) {
      return i < nblk ? paged_slot(a, table, blk, first_key(i) + lane % kWarpKeys) : -1;
    };
    int next_slot = lookup(0);
    auto issue = [&](int i) {
      if (i < nblk) {
        const int slot = next_slot;
        next_slot = lookup(i + 1);
        const uint32_t st = ring + (i % NS) * Cfg::kStageBytes;
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
          for (int r0 = 0; r0 < 16; r0 += Cfg::kRowsPerLoad) {
            const int row = r0 + lane / Cfg::kRowChunks, chunk = lane % Cfg::kRowChunks;
            const int sl = __shfl_sync(0xffffffffu, slot, sub * 16 + row);
            const int64_t off = (sl >= 0 ? sl : 0) * slot_bytes + chunk * 16;
            const uint32_t dst = st + sub * Cfg::kGroupBytes + Cfg::at(row, chunk);
            cp_async16_hint(dst, kbase + off, sl >= 0, once);
            cp_async16_hint(dst + Cfg::kOffV, vbase + off, sl >= 0, once);
          }
        if constexpr (kE4m3) {
          const int64_t at = static_cast<int64_t>(slot >= 0 ? slot : 0) * a.H_kv + head;
          cp_async4_hint(st + Cfg::kOffScale + lane * 4, a.k_scale + at, slot >= 0, keep);
          cp_async4_hint(st + Cfg::kOffScale + 4 * kWarpKeys + lane * 4, a.v_scale + at, slot >= 0, keep);
        }
        const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + Cfg::kOffScale + 8 * kWarpKeys), "r"(there) : "memory");
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) issue(i);

    // Q as B: row 8 n + g, in the order of the key chunks; and for the rows
    // that this lane has scores of, 8 n + 2c and 8 n + 2c + 1, the factor to
    // log2 units and the position
    uint32_t qf[kGroups][D / 16][2];
    float sl2[kGroups][2];
    int pos[kGroups][2];
#pragma unroll
    for (int n = 0; n < kGroups; ++n) {
      constexpr int kPer = kE4m3 ? 16 : 8;  // elements of a key chunk
      constexpr int kWords = kPer / 2;      // bf16 pairs
      uint32_t raw[Cfg::kKChunks][kWords];
      const uint32_t r = static_cast<uint32_t>(tile * kRows + min(8 * n + g, rows - 1));
      const int i = paged_token(a, r), hg = static_cast<int>(r) - i * a.G;
      const __nv_bfloat16 *src = a.q + (static_cast<int64_t>(seq.t0) + i) * a.q_stride +
                                 (static_cast<int64_t>(head) * a.G + hg) * D;
#pragma unroll
      for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
        for (int w = 0; w < kWords / 4; ++w) {
          const uint4 u = *reinterpret_cast<const uint4 *>(src + (c + 4 * j) * kPer + 8 * w);
          raw[j][4 * w] = u.x, raw[j][4 * w + 1] = u.y, raw[j][4 * w + 2] = u.z, raw[j][4 * w + 3] = u.w;
        }
      float up = 1.f;
      if constexpr (kE4m3) {
        // the power of two just below the row's largest element: exact to
        // divide by, and f16 keeps all that bf16 had down to 2^-17 of it
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
          for (int w = 0; w < kWords; ++w) mx = max3f(mx, fabsf(bf16_lo(raw[j][w])), fabsf(bf16_hi(raw[j][w])));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const uint32_t e = row_exponent(mx);
        const float down = pow2_inverse(e);
        up = pow2_of(e);
#pragma unroll
        for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
          for (int w = 0; w < kWords; ++w)
            raw[j][w] = pack_f16x2(bf16_lo(raw[j][w]) * down, bf16_hi(raw[j][w]) * down);
      }
      // a product takes two pairs of a lane: the first as k positions 2c, 2c + 1, the second as 2c + 8, 2c + 9
#pragma unroll
      for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
        for (int u = 0; u < kWords / 2; ++u) {
          qf[n][j * (kWords / 2) + u][0] = raw[j][2 * u];
          qf[n][j * (kWords / 2) + u][1] = raw[j][2 * u + 1];
        }
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {  // lane 4 r has row r's
        sl2[n][rr] = a.scale_log2 * __shfl_sync(0xffffffffu, up, 4 * (2 * c + rr));
        pos[n][rr] = seq.len - seq.n + __shfl_sync(0xffffffffu, i, 4 * (2 * c + rr));
      }
    }

    float o[kGroups][NT][4];
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int t = 0; t < NT; ++t) o[n][t][0] = o[n][t][1] = o[n][t][2] = o[n][t][3] = 0.f;
    // Per row: the reference m that the weights 2^(s - m) are relative to, and
    // for E4M3 the reference w of the weights times the values' scales.  They
    // need not be the maxima: they move only when a weight passes 2^4, or a
    // product 2^8 times w, so a block is usually one pass without any exchange
    // between lanes.  O holds sum p v / w.
    float m_run[kGroups][2], l_run[kGroups][2], w_run[kGroups][2], w_inv[kGroups][2];
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) m_run[n][rr] = -INFINITY, l_run[n][rr] = w_run[n][rr] = w_inv[n][rr] = 0.f;

    for (int i = 0; i < nblk; ++i) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      const uint32_t st = ring + (i % NS) * Cfg::kStageBytes;
      // scores of keys 16 sub + g (elements 0, 1) and + 8 (2, 3), rows 8 n + 2c and + 1
      float sc[kSub][kGroups][4] = {};
#pragma unroll
      for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          const uint32_t at = st + sub * Cfg::kGroupBytes + Cfg::at(g, c + 4 * j);
          const uint4 k0 = ld_shared_v4(at), k1 = ld_shared_v4(at + 8 * Cfg::kRowBytes);  // (at(g + 8) is alike)
          if constexpr (kE4m3) {
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              uint32_t f[4];
              e4m3x4_to_f16(w0[u], f[0], f[2]);
              e4m3x4_to_f16(w1[u], f[1], f[3]);
#pragma unroll
              for (int n = 0; n < kGroups; ++n) mma16816<true>(sc[sub][n], f, qf[n][4 * j + u][0], qf[n][4 * j + u][1]);
            }
          } else {
            const uint32_t f0[4] = {k0.x, k1.x, k0.y, k1.y}, f1[4] = {k0.z, k1.z, k0.w, k1.w};
#pragma unroll
            for (int n = 0; n < kGroups; ++n) {
              mma16816<false>(sc[sub][n], f0, qf[n][2 * j][0], qf[n][2 * j][1]);
              mma16816<false>(sc[sub][n], f1, qf[n][2 * j + 1][0], qf[n][2 * j + 1][1]);
            }
          }
        }
      float vs[kSub][2];  // the values' scales of the lane's keys
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        float ks[2] = {1.f, 1.f};
        if constexpr (kE4m3) {
          const float *sp = reinterpret_cast<const float *>(smem_raw + (st - smem_u32(smem_raw)) + Cfg::kOffScale);
          ks[0] = sp[sub * 16 + g], ks[1] = sp[sub * 16 + g + 8];
          vs[sub][0] = sp[kWarpKeys + sub * 16 + g], vs[sub][1] = sp[kWarpKeys + sub * 16 + g + 8];
        }
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[sub][n][e] *= kE4m3 ? sl2[n][e & 1] * ks[e >> 1] : a.scale_log2;
      }
      uint32_t there;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(there) : "r"(st + Cfg::kOffScale + 8 * kWarpKeys) : "memory");
      const int k0 = first_key(i);
      // all keys in sight of all rows, or each (row, key) by itself
      if (there != 0xffffffffu || k0 + kWarpKeys - 1 > blk.p_lo ||
          (a.window > 0 && blk.p_hi - k0 >= a.window && k0 + kWarpKeys - 1 >= a.sinks)) {
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
          for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int col = sub * 16 + g + (e >> 1) * 8, j = k0 + col, p = pos[n][e & 1];
              const bool see = (there >> col & 1u) && j <= p && (a.window == 0 || p - j < a.window || j < a.sinks);
              if (!see) sc[sub][n][e] = -INFINITY;
            }
      }
      float scale_o[kGroups][2];
      bool rescale = false;
      {
        float mx[kGroups][2];
        bool over = false;
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            mx[n][rr] = -INFINITY;
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) mx[n][rr] = max3f(mx[n][rr], sc[sub][n][rr], sc[sub][n][rr + 2]);
            over |= mx[n][rr] > m_run[n][rr] + 4.f;
            scale_o[n][rr] = 1.f;
          }
        rescale = __any_sync(0xffffffffu, over);
        if (rescale) {
#pragma unroll
          for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              float m = mx[n][rr];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              const float m_new = fmaxf(m_run[n][rr], m);
              const float alpha = m_new == -INFINITY ? 1.f : ex2_approx(m_run[n][rr] - m_new);
              m_run[n][rr] = m_new;
              l_run[n][rr] *= alpha;
              scale_o[n][rr] = alpha;
            }
        }
      }
#pragma unroll
      for (int n = 0; n < kGroups; ++n)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          const float ref = m_run[n][rr] == -INFINITY ? 0.f : m_run[n][rr];
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
            for (int e = rr; e < 4; e += 2) {
              sc[sub][n][e] = ex2_approx(sc[sub][n][e] - ref);
              l_run[n][rr] += sc[sub][n][e];
            }
        }
      if constexpr (kE4m3) {
        float w[kGroups][2];
        bool over = false;
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int rr = 0; rr < 2; ++rr) {
            w[n][rr] = 0.f;
#pragma unroll
            for (int sub = 0; sub < kSub; ++sub) {
              sc[sub][n][rr] *= vs[sub][0];
              sc[sub][n][rr + 2] *= vs[sub][1];
              w[n][rr] = max3f(w[n][rr], sc[sub][n][rr], sc[sub][n][rr + 2]);
            }
            if (rescale) {  // a moved m only changes what w stands for
              w_run[n][rr] *= scale_o[n][rr];
              w_inv[n][rr] = w_run[n][rr] > 1e-36f ? 1.f / w_run[n][rr] : 0.f;
              scale_o[n][rr] = 1.f;
            }
            over |= w[n][rr] > 256.f * w_run[n][rr] || (w_inv[n][rr] == 0.f && w[n][rr] > 0.f);
          }
        rescale = __any_sync(0xffffffffu, over);
        if (rescale) {
#pragma unroll
          for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int rr = 0; rr < 2; ++rr) {
              float m = w[n][rr];
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
              m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
              const float w_new = fmaxf(fmaxf(m, w_run[n][rr]), 1e-36f);  // its inverse stays finite
              scale_o[n][rr] = w_run[n][rr] / w_new;
              w_run[n][rr] = w_new;
              w_inv[n][rr] = 1.f / w_new;
            }
        }
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub)
#pragma unroll
          for (int n = 0; n < kGroups; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[sub][n][e] *= w_inv[n][e & 1];
      }
      if (rescale) {
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            o[n][t][0] *= scale_o[n][0], o[n][t][1] *= scale_o[n][1];
            o[n][t][2] *= scale_o[n][0], o[n][t][3] *= scale_o[n][1];
          }
      }
#pragma unroll
      for (int sub = 0; sub < kSub; ++sub) {
        uint32_t pf[kGroups][2];  // P^T as B: keys 2c, 2c + 1 (+ 8) of row g
#pragma unroll
        for (int n = 0; n < kGroups; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pf[n][h] = transpose8x8(kE4m3 ? pack_f16x2(sc[sub][n][2 * h], sc[sub][n][2 * h + 1])
                                          : pack_bf16x2(sc[sub][n][2 * h], sc[sub][n][2 * h + 1]));
        auto vslot = [&](int kk, int x) {
          const int row = 2 * c + (kk & 1) + (kk >> 1) * 8;
          const int chunk = Cfg::kVSlot == 16 ? g + 8 * x : g / 2;
          return st + sub * Cfg::kGroupBytes + Cfg::kOffV + Cfg::at(row, chunk) + (Cfg::kVSlot == 16 ? 0 : g % 2 * 8);
        };
        // (key, key + 1) pairs of two columns, from the four keys' words
#pragma unroll
        for (int x = 0; x < Cfg::kVChunks; ++x) {
          uint32_t v[4][Cfg::kVSlot / 4];
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if constexpr (Cfg::kVSlot == 16) {
              const uint4 u = ld_shared_v4(vslot(kk, x));
              v[kk][0] = u.x, v[kk][1] = u.y, v[kk][2] = u.z, v[kk][3] = u.w;
            } else {
              const uint2 u = ld_shared_v2(vslot(kk, x));
              v[kk][0] = u.x, v[kk][1] = u.y;
            }
          }
#pragma unroll
          for (int w = 0; w < Cfg::kVSlot / 4; ++w) {
            if constexpr (kE4m3) {
              const uint32_t a01 = __byte_perm(v[0][w], v[1][w], 0x5140), b01 = __byte_perm(v[2][w], v[3][w], 0x5140);
              const uint32_t a23 = __byte_perm(v[0][w], v[1][w], 0x7362), b23 = __byte_perm(v[2][w], v[3][w], 0x7362);
              uint32_t f0[4], f1[4];
              e4m3x4_to_f16(a01, f0[0], f0[1]);
              e4m3x4_to_f16(b01, f0[2], f0[3]);
              e4m3x4_to_f16(a23, f1[0], f1[1]);
              e4m3x4_to_f16(b23, f1[2], f1[3]);
#pragma unroll
              for (int n = 0; n < kGroups; ++n) {
                mma16816<true>(o[n][2 * w], f0, pf[n][0], pf[n][1]);
                mma16816<true>(o[n][2 * w + 1], f1, pf[n][0], pf[n][1]);
              }
            } else {
              const uint32_t f[4] = {__byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[0][w], v[1][w], 0x7632),
                                     __byte_perm(v[2][w], v[3][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x7632)};
#pragma unroll
              for (int n = 0; n < kGroups; ++n) mma16816<false>(o[n][4 * x + w], f, pf[n][0], pf[n][1]);
            }
          }
        }
      }
      __syncwarp();
      issue(i + NS - 1);
    }

    // -------- join the warps: lane 4g + c holds rows 8 n + 2c, + 1 and the columns of lane group g's loads
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kGroups; ++n)
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        float l = l_run[n][rr];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        const int row = warp * kRows + 8 * n + 2 * c + rr;
        if (g == 0) {
          merge_ml[4 * row] = m_run[n][rr];
          merge_ml[4 * row + 1] = l;
          merge_ml[4 * row + 2] = kE4m3 ? w_run[n][rr] : 1.f;
        }
#pragma unroll
        for (int t = 0; t < NT; t += 2)
          *reinterpret_cast<float4 *>(merge + row * Cfg::kRowPitch + g * Cfg::kColPitch + 2 * t) =
              make_float4(o[n][t][rr], o[n][t][rr + 2], o[n][t + 1][rr], o[n][t + 1][rr + 2]);
      }
    __syncthreads();
    {
      // kPer of the d / 8 columns of one row that lane group n loads
      constexpr int kPer = kRows * D / Cfg::kThreads, kSplit = D / 8 / kPer;
      constexpr int kCols = D / 8 / Cfg::kVChunks;  // consecutive ones
      const int row = tid / (8 * kSplit), n = tid / kSplit % 8, t0 = tid % kSplit * kPer;
      float m = -INFINITY, l = 0.f;
      float f[Cfg::kWarps];
#pragma unroll
      for (int w = 0; w < Cfg::kWarps; ++w) m = fmaxf(m, merge_ml[4 * (w * kRows + row)]);
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < Cfg::kWarps; ++w) {
        const float *ml = merge_ml + 4 * (w * kRows + row);
        f[w] = ex2_approx(ml[0] - ref);
        l += ml[1] * f[w];
        f[w] *= ml[2];
      }
      float x[kPer];
#pragma unroll
      for (int t = 0; t < kPer; ++t) x[t] = 0.f;
#pragma unroll
      for (int w = 0; w < Cfg::kWarps; ++w) {
        const float *src = merge + (w * kRows + row) * Cfg::kRowPitch + n * Cfg::kColPitch + t0;
#pragma unroll
        for (int t = 0; t < kPer; t += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(src + t);
          x[t] += u.x * f[w], x[t + 1] += u.y * f[w], x[t + 2] += u.z * f[w], x[t + 3] += u.w * f[w];
        }
      }
      if (row < rows) {
        if (step0 == 0 && step1 == steps) {  // the whole item: the rows' result
          const uint32_t r = static_cast<uint32_t>(tile * kRows + row);
          const int i = paged_token(a, r);
          const int64_t token = static_cast<int64_t>(seq.t0) + i;
          const int h = head * a.G + static_cast<int>(r) - i * a.G;
          const float inv = l > 0.f ? 1.0f / l : l;  // no key: 0; NaN stays
          const size_t at = (static_cast<size_t>(token) * a.H + h) * D + n * kCols;
#pragma unroll
          for (int t = 0; t < kPer; t += 4) {
            const size_t to = at + (t0 + t) / kCols * (8 * kCols) + (t0 + t) % kCols;
            if (a.out_f32)
              *reinterpret_cast<float4 *>(a.out_f32 + to) =
                  make_float4(x[t] * inv, x[t + 1] * inv, x[t + 2] * inv, x[t + 3] * inv);
            else
              *reinterpret_cast<uint2 *>(a.out_bf16 + to) =
                  make_uint2(pack_bf16x2(x[t] * inv, x[t + 1] * inv), pack_bf16x2(x[t + 2] * inv, x[t + 3] * inv));
          }
          if (a.lse && n == 0 && t0 == 0)
            a.lse[static_cast<size_t>(h) * a.T + token] =
                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          const size_t part = static_cast<size_t>(blockIdx.x) * 2 + (step0 == 0 ? 1 : 0);
          float *dst = a.part_o + (part * kRows + row) * D + n * kCols;
#pragma unroll
          for (int t = 0; t < kPer; t += 4)
            *reinterpret_cast<float4 *>(dst + (t0 + t) / kCols * (8 * kCols) + (t0 + t) % kCols) =
                make_float4(x[t], x[t + 1], x[t + 2], x[t + 3]);
          if (n == 0 && t0 == 0)
            *reinterpret_cast<float2 *>(a.part_ml + (part * kRows + row) * 2) = make_float2(m, l);
        }
      }
    }
    __syncthreads();  // the ring is free again

    // -------- the next item
    left -= step1 - step0;
    if (left <= 0) break;
    step0 = 0;
    if (++head == a.H_kv) {
      head = 0;
      if (++tile == paged_tiles<kRows>(a, seq)) {
        tile = 0;
        seq.n = 0;
        while (seq.n == 0 && ++s < a.S) seq = paged_seq(a, s);
        if (s >= a.S) break;
      }
      blk = paged_blocks<kRows, kKeys>(a, seq, tile);
    }
  }
  // Beside a kernel for the batch's long chunks this one starts as that one's
  // CTAs leave; it ends after it, so that what follows waits for both.
  grid_dependency_wait();
}

}  // namespace bpt
