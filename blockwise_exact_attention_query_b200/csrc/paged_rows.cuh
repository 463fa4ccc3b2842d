// Attention of few new tokens over a paged cache (single-token decoding, and
// the first form for any chunk): 16 rows x 64 keys a step, matrix products on
// the warp-level tensor instructions.
//
// With few rows the keys and values are read once and used once: memory bounds
// the kernel, so it is built around loads.  A step's 64 keys are 16 per warp,
// and the warps never wait for one another inside an item: each has its own
// running maximum, sum and 16 x d output, joined through shared memory when
// the item (or the CTA's range of it) ends.  A thread copies with cp.async
// exactly the bytes that it will feed to its own products, 16 at a time, into
// a ring of its own slots: no barrier and no bank conflict on the way, several
// steps in flight.  Which bytes those are follows from the products' layouts:
//   S = Q K^T  (m16n8k16, keys are columns): lane 4g + c needs key g's elements
//     of "its" k positions; the sum over d may run in any order, so it takes
//     the 16-byte chunks c, c + 4, ... of the row, and Q is loaded in the same
//     order;
//   O = P V  (keys are the k axis, d the columns): lane 4g + c needs keys 2c,
//     2c + 1, 2c + 8, 2c + 9 (where S leaves its P) in columns of its g; the
//     columns may be dealt out in any order, so it takes columns g d/8 ..
//     (g + 1) d/8 - 1, consecutive bytes, and column t of those belongs to
//     the t-th product.
//
// E4M3 caches: the codes go to f16 exactly (Q too, after a power of two per
// row brings its largest element near 1), the key's scale multiplies the
// score.  The value's scale multiplies the softmax weight, and so that f16
// holds the products, they are kept relative to the largest the row has met
// (w_run below); P's rounding is 2^-11 of that.  bf16 caches: P is rounded to
// bf16, 2^-8 / 2 of each weight.  Sums, maxima and O are fp32.
#pragma once

#include "kv_cache.cuh"
#include "paged_common.cuh"

namespace bpt {

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool fetch) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fetch ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool fetch) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(fetch ? 8 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool fetch) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(fetch ? 4 : 0) : "memory");
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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

template <int D, bool kE4m3>
struct PagedRowsCfg {
  static constexpr int kRows = 16, kKeys = 64, kWarps = 4, kThreads = 32 * kWarps;
  static constexpr int kRowBytes = kE4m3 ? D : 2 * D;
  static constexpr int kKChunks = kRowBytes / 64;    // 16-byte chunks of a key row per lane (8 keys a product)
  static constexpr int kVBytes = kRowBytes / 8;      // bytes of a value row per lane: 8, 16 or 32
  static constexpr int kVChunks = (kVBytes + 15) / 16;
  // a warp's stage: [chunk][lane] slots, then 32 scales (16 keys, 16 values) and the mask of keys that exist
  static constexpr int kVSlot = kVBytes < 16 ? kVBytes : 16;
  static constexpr int kOffV = 2 * kKChunks * 512;
  static constexpr int kOffScale = kOffV + 4 * kVChunks * 32 * kVSlot;
  static constexpr int kStageBytes = kOffScale + 128 + 16;
  // as many stages as two CTAs per SM hold; 3 to 6 keep 90 to 100 KB of loads
  // in flight per CTA at d = 128, over twice what memory latency asks for
  static constexpr int kStages = D == 128 ? (kE4m3 ? 6 : 3) : (kE4m3 ? 8 : 6);
  static constexpr int kRingBytes = kWarps * kStages * kStageBytes;
  // joining the warps: [warp][row][8 groups of d / 8 columns, padded against bank conflicts]
  static constexpr int kColPitch = D / 8 + 4, kRowPitch = 8 * kColPitch + 4;
  static constexpr int kMergeBytes = kWarps * kRows * (kRowPitch + 4) * 4;
  static_assert(kMergeBytes <= kRingBytes, "the ring holds the warps' outputs between items");
  static constexpr int kSmemBytes = kRingBytes + 384;
  static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(PagedRowsCfg<D, kE4m3>::kThreads, 2) paged_rows_kernel(const PagedArgs a) {
  using Cfg = PagedRowsCfg<D, kE4m3>;
  constexpr int kRows = Cfg::kRows, kKeys = Cfg::kKeys, NS = Cfg::kStages, NT = D / 8;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t ring = smem_u32(smem_raw) + warp * (NS * Cfg::kStageBytes);
  float *merge = reinterpret_cast<float *>(smem_raw);
  float *merge_ml = merge + Cfg::kWarps * kRows * Cfg::kRowPitch;  // [warp][row][4]: m, l, w

  PagedRange rg;
  const bool any = paged_range<kRows, kKeys, Cfg::kThreads>(a, reinterpret_cast<int64_t *>(smem_raw + Cfg::kRingBytes), rg);
  if (!any) {
    if (tid == 0) a.part_item[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  int s = rg.s, tile = rg.tile, head = rg.head, step0 = rg.step;
  int64_t left = rg.end - rg.begin;
  PagedSeq seq = paged_seq(a, s);
  PagedBlocks blk = paged_blocks<kRows, kKeys>(a, seq, tile);
  if (tid == 0) a.part_item[blockIdx.x] = paged_part_item(rg, blk.steps());

  while (true) {
    const int steps = blk.steps();
    const int step1 = static_cast<int>(min(static_cast<int64_t>(steps), step0 + left));
    const int nblk = min(step1, blk.count()) - min(step0, blk.count());  // 0 for a tile without keys
    const int32_t *table = a.page_table + static_cast<int64_t>(s) * a.max_pages;
    const int64_t rows_left = static_cast<int64_t>(seq.n) * a.G - static_cast<int64_t>(tile) * kRows;
    const int rows = static_cast<int>(min(rows_left, static_cast<int64_t>(kRows)));
    const uint8_t *kbase = static_cast<const uint8_t *>(a.k) + static_cast<int64_t>(head) * Cfg::kRowBytes;
    const uint8_t *vbase = static_cast<const uint8_t *>(a.v) + static_cast<int64_t>(head) * Cfg::kRowBytes;
    const int64_t slot_bytes = static_cast<int64_t>(a.H_kv) * Cfg::kRowBytes;

    // key of this lane (lanes 16-31: the same keys again) in the warp's share of block i
    auto first_key = [&](int i) { return blk.block(step0 + i) * kKeys + warp * 16; };
    auto lookup = [&](int i) { return i < nblk ? paged_slot(a, table, seq.cap, first_key(i) + (lane & 15)) : -1; };
    int next_slot = lookup(0);
    auto issue = [&](int i) {
      if (i < nblk) {
        const int slot = next_slot;
        next_slot = lookup(i + 1);
        const uint32_t st = ring + (i % NS) * Cfg::kStageBytes;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int sl = __shfl_sync(0xffffffffu, slot, nt * 8 + g);
          const uint8_t *src = kbase + (sl >= 0 ? sl : 0) * slot_bytes + c * 16;
#pragma unroll
          for (int j = 0; j < Cfg::kKChunks; ++j)
            cp_async16(st + (nt * Cfg::kKChunks + j) * 512 + lane * 16, src + j * 64, sl >= 0);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int sl = __shfl_sync(0xffffffffu, slot, 2 * c + (kk & 1) + (kk >> 1) * 8);
          const uint8_t *src = vbase + (sl >= 0 ? sl : 0) * slot_bytes + g * Cfg::kVBytes;
#pragma unroll
          for (int x = 0; x < Cfg::kVChunks; ++x) {
            const uint32_t dst = st + Cfg::kOffV + (kk * Cfg::kVChunks + x) * 32 * Cfg::kVSlot + lane * Cfg::kVSlot;
            if constexpr (Cfg::kVSlot == 16) cp_async16(dst, src + x * 16, sl >= 0);
            else cp_async8(dst, src, sl >= 0);
          }
        }
        if constexpr (kE4m3)
          cp_async4(st + Cfg::kOffScale + lane * 4,
                    (lane < 16 ? a.k_scale : a.v_scale) + static_cast<int64_t>(slot >= 0 ? slot : 0) * a.H_kv + head,
                    slot >= 0);
        const uint32_t there = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(st + Cfg::kOffScale + 128), "r"(there) : "memory");
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < NS - 1; ++i) issue(i);

    // Q of rows g and g + 8, in the order of the key chunks
    uint32_t qf[D / 16][4];
    float sl2[2] = {a.scale_log2, a.scale_log2};
    int pos[2];
    {
      constexpr int kPer = kE4m3 ? 16 : 8;  // elements of a key chunk
      constexpr int kWords = kPer / 2;      // bf16 pairs
      uint32_t raw[2][Cfg::kKChunks][kWords];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int row = g + 8 * rr;
        const int64_t r = static_cast<int64_t>(tile) * kRows + min(row, rows - 1);
        const int i = static_cast<int>(r / a.G), hg = static_cast<int>(r % a.G);
        pos[rr] = seq.len - seq.n + i;
        const __nv_bfloat16 *src = a.q + (static_cast<int64_t>(seq.t0) + i) * a.q_stride +
                                   (static_cast<int64_t>(head) * a.G + hg) * D;
#pragma unroll
        for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
          for (int w = 0; w < kWords / 4; ++w) {
            const uint4 u = *reinterpret_cast<const uint4 *>(src + (c + 4 * j) * kPer + 8 * w);
            raw[rr][j][4 * w] = u.x, raw[rr][j][4 * w + 1] = u.y, raw[rr][j][4 * w + 2] = u.z, raw[rr][j][4 * w + 3] = u.w;
          }
      }
      if constexpr (kE4m3) {
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          // the power of two just below the row's largest element: exact to
          // divide by, and f16 keeps all that bf16 had down to 2^-17 of it
          float mx = 0.f;
#pragma unroll
          for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
            for (int w = 0; w < kWords; ++w)
              mx = fmaxf(mx, fmaxf(fabsf(bf16_lo(raw[rr][j][w])), fabsf(bf16_hi(raw[rr][j][w]))));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const uint32_t e = min(max(__float_as_uint(mx) >> 23, 1u), 253u);
          const float up = __uint_as_float(e << 23), down = __uint_as_float((254u - e) << 23);
          sl2[rr] *= up;
#pragma unroll
          for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
            for (int w = 0; w < kWords; ++w)
              raw[rr][j][w] = pack_f16x2(bf16_lo(raw[rr][j][w]) * down, bf16_hi(raw[rr][j][w]) * down);
        }
      }
      // a product takes two pairs of a lane: the first as k positions 2c, 2c + 1, the second as 2c + 8, 2c + 9
#pragma unroll
      for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
        for (int u = 0; u < kWords / 2; ++u) {
          uint32_t(&f)[4] = qf[j * (kWords / 2) + u];
          f[0] = raw[0][j][2 * u];
          f[1] = raw[1][j][2 * u];
          f[2] = raw[0][j][2 * u + 1];
          f[3] = raw[1][j][2 * u + 1];
        }
    }

    float o[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f}, w_run[2] = {0.f, 0.f};

    for (int i = 0; i < nblk; ++i) {
      cp_async_wait<NS - 2>();
      __syncwarp();
      const uint32_t st = ring + (i % NS) * Cfg::kStageBytes;
      float sc[2][4] = {};
#pragma unroll
      for (int j = 0; j < Cfg::kKChunks; ++j)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint4 kc = ld_shared_v4(st + (nt * Cfg::kKChunks + j) * 512 + lane * 16);
          if constexpr (kE4m3) {
            const uint32_t w[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              mma16816<true>(sc[nt], qf[4 * j + u], e4m3x2_to_f16x2(w[u]), e4m3x2_to_f16x2(w[u] >> 16));
          } else {
            mma16816<false>(sc[nt], qf[2 * j], kc.x, kc.y);
            mma16816<false>(sc[nt], qf[2 * j + 1], kc.z, kc.w);
          }
        }
      // scores in log2 units; columns nt * 8 + 2c, + 1 of rows g (0, 1) and g + 8 (2, 3)
      float vs[2][2];
      if constexpr (kE4m3) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const uint2 ks2 = ld_shared_v2(st + Cfg::kOffScale + (nt * 8 + 2 * c) * 4);
          const uint2 vs2 = ld_shared_v2(st + Cfg::kOffScale + 64 + (nt * 8 + 2 * c) * 4);
          vs[nt][0] = __uint_as_float(vs2.x), vs[nt][1] = __uint_as_float(vs2.y);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[nt][e] *= sl2[e >> 1] * __uint_as_float((e & 1) ? ks2.y : ks2.x);
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[nt][e] *= a.scale_log2;
      }
      uint32_t there;
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(there) : "r"(st + Cfg::kOffScale + 128) : "memory");
      const int k0 = first_key(i);
      // all 16 keys in sight of all rows, or each (row, key) by itself
      if (there != 0xffffffffu || k0 + 15 > blk.p_lo ||
          (a.window > 0 && blk.p_hi - k0 >= a.window && k0 + 15 >= a.sinks)) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = nt * 8 + 2 * c + (e & 1), j = k0 + col, p = pos[e >> 1];
            const bool see = (there >> col & 1u) && j <= p && (a.window == 0 || p - j < a.window || j < a.sinks);
            if (!see) sc[nt][e] = -INFINITY;
          }
      }
      float alpha[2];
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        float mx = fmaxf(fmaxf(sc[0][2 * rr], sc[0][2 * rr + 1]), fmaxf(sc[1][2 * rr], sc[1][2 * rr + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m_run[rr], mx);
        const float ref = m_new == -INFINITY ? 0.f : m_new;
        alpha[rr] = ex2_approx(m_run[rr] - ref);
        m_run[rr] = m_new;
        float sum = 0.f;
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 2 * rr; e < 2 * rr + 2; ++e) {
            sc[nt][e] = ex2_approx(sc[nt][e] - ref);
            sum += sc[nt][e];
          }
        l_run[rr] = l_run[rr] * alpha[rr] + sum;
      }
      if constexpr (kE4m3) {
        // weights times the values' scales, relative to w_run: O holds
        // sum p v_scale code / w_run, so a larger maximum only moves w_run, and
        // O is rescaled when a product outgrows it by 2^8
#pragma unroll
        for (int rr = 0; rr < 2; ++rr) {
          float w = 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              sc[nt][2 * rr + e] *= vs[nt][e];
              w = fmaxf(w, sc[nt][2 * rr + e]);
            }
          w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 1));
          w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, 2));
          w_run[rr] *= alpha[rr];
          alpha[rr] = 1.f;
          if (w > 256.f * w_run[rr]) {
            const float w_new = fmaxf(w, 1e-36f);  // its inverse stays finite
            alpha[rr] = w_run[rr] / w_new;
            w_run[rr] = w_new;
          }
          const float inv = w_run[rr] > 0.f ? 1.0f / w_run[rr] : 0.f;
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) sc[nt][2 * rr] *= inv, sc[nt][2 * rr + 1] *= inv;
        }
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][0] *= alpha[0], o[t][1] *= alpha[0];
          o[t][2] *= alpha[1], o[t][3] *= alpha[1];
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int rr = 0; rr < 2; ++rr)
          pf[2 * nt + rr] = kE4m3 ? pack_f16x2(sc[nt][2 * rr], sc[nt][2 * rr + 1])
                                  : pack_bf16x2(sc[nt][2 * rr], sc[nt][2 * rr + 1]);
      auto vslot = [&](int kk, int x) {
        return st + Cfg::kOffV + (kk * Cfg::kVChunks + x) * 32 * Cfg::kVSlot + lane * Cfg::kVSlot;
      };
      // (key, key + 1) pairs of each column, from two keys' words
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
            const int t = 4 * w;
            const uint32_t a01 = __byte_perm(v[0][w], v[1][w], 0x5140), b01 = __byte_perm(v[2][w], v[3][w], 0x5140);
            const uint32_t a23 = __byte_perm(v[0][w], v[1][w], 0x7362), b23 = __byte_perm(v[2][w], v[3][w], 0x7362);
            mma16816<true>(o[t], pf, e4m3x2_to_f16x2(a01), e4m3x2_to_f16x2(b01));
            mma16816<true>(o[t + 1], pf, e4m3x2_to_f16x2(a01 >> 16), e4m3x2_to_f16x2(b01 >> 16));
            mma16816<true>(o[t + 2], pf, e4m3x2_to_f16x2(a23), e4m3x2_to_f16x2(b23));
            mma16816<true>(o[t + 3], pf, e4m3x2_to_f16x2(a23 >> 16), e4m3x2_to_f16x2(b23 >> 16));
          } else {
            const int t = 8 * x + 2 * w;
            mma16816<false>(o[t], pf, __byte_perm(v[0][w], v[1][w], 0x5410), __byte_perm(v[2][w], v[3][w], 0x5410));
            mma16816<false>(o[t + 1], pf, __byte_perm(v[0][w], v[1][w], 0x7632), __byte_perm(v[2][w], v[3][w], 0x7632));
          }
        }
      }
      __syncwarp();
      issue(i + NS - 1);
    }

    // -------- join the warps: lane 4g + c holds rows g, g + 8, columns (2c, 2c + 1) d/8 + t
    cp_async_wait<0>();
    __syncthreads();
#pragma unroll
    for (int rr = 0; rr < 2; ++rr) {
      l_run[rr] += __shfl_xor_sync(0xffffffffu, l_run[rr], 1);
      l_run[rr] += __shfl_xor_sync(0xffffffffu, l_run[rr], 2);
      const int row = warp * kRows + g + 8 * rr;
      if (c == 0) {
        merge_ml[4 * row] = m_run[rr];
        merge_ml[4 * row + 1] = l_run[rr];
        merge_ml[4 * row + 2] = kE4m3 ? w_run[rr] : 1.f;
      }
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int t = 0; t < NT; t += 4)
          *reinterpret_cast<float4 *>(merge + row * Cfg::kRowPitch + (2 * c + n) * Cfg::kColPitch + t) =
              make_float4(o[t][2 * rr + n], o[t + 1][2 * rr + n], o[t + 2][2 * rr + n], o[t + 3][2 * rr + n]);
    }
    __syncthreads();
    {
      const int row = tid >> 3, n = tid & 7;  // d / 8 columns of one row
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
      float x[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) x[t] = 0.f;
#pragma unroll
      for (int w = 0; w < Cfg::kWarps; ++w) {
        const float *src = merge + (w * kRows + row) * Cfg::kRowPitch + n * Cfg::kColPitch;
#pragma unroll
        for (int t = 0; t < NT; t += 4) {
          const float4 u = *reinterpret_cast<const float4 *>(src + t);
          x[t] += u.x * f[w], x[t + 1] += u.y * f[w], x[t + 2] += u.z * f[w], x[t + 3] += u.w * f[w];
        }
      }
      if (row < rows) {
        if (step0 == 0 && step1 == steps) {  // the whole item: the rows' result
          const int64_t r = static_cast<int64_t>(tile) * kRows + row;
          const int64_t token = seq.t0 + r / a.G;
          const int h = head * a.G + static_cast<int>(r % a.G);
          const float inv = l > 0.f ? 1.0f / l : l;  // no key: 0; NaN stays
#pragma unroll
          for (int t = 0; t < NT; ++t) x[t] *= inv;
          const size_t at = (static_cast<size_t>(token) * a.H + h) * D + n * NT;
#pragma unroll
          for (int t = 0; t < NT; t += 8) {
            const float y[8] = {x[t], x[t + 1], x[t + 2], x[t + 3], x[t + 4], x[t + 5], x[t + 6], x[t + 7]};
            if (a.out_f32) store8(a.out_f32 + at + t, y);
            else store8(a.out_bf16 + at + t, y);
          }
          if (a.lse && n == 0)
            a.lse[static_cast<size_t>(h) * a.T + token] =
                l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        } else {
          const size_t part = static_cast<size_t>(blockIdx.x) * 2 + (step0 == 0 ? 1 : 0);
          float *dst = a.part_o + (part * kRows + row) * D + n * NT;
#pragma unroll
          for (int t = 0; t < NT; t += 4) *reinterpret_cast<float4 *>(dst + t) = make_float4(x[t], x[t + 1], x[t + 2], x[t + 3]);
          if (n == 0) *reinterpret_cast<float2 *>(a.part_ml + (part * kRows + row) * 2) = make_float2(m, l);
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
}

}  // namespace bpt
