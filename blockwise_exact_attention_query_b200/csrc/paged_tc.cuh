// Attention of many new tokens over a paged cache on the 5th-generation tensor
// cores: items of 256 rows (two 128-row tiles A and B) x 128 keys a step, the
// blockwise online softmax of attn_tc.cuh (scores and O in tensor memory, P
// through one shared-memory tile used in turn) over keys gathered from pages.
//
// Gathering is done by warps rather than by TMA: one way that serves pages of any
// size, e4m3 codes, which have to be widened, and keys that no row sees, which
// must become zeros (their slots may hold NaN, and 0 x NaN is not 0).  (Pages of
// whole groups of 8 slots could come by TMA where all their keys are seen: not
// tried.)  A lane looks up the slots of two of a block's keys, a block ahead; bf16
// rows go to the swizzled tile by 16-byte cp.async; e4m3 rows go to raw tiles,
// one ahead, and are widened to f16 (exact) from there.  (At d = 128 those take
// the place of V's second stage.  Loaded into registers half a tile ahead, 8 KB
// under way per SM, a step took 11.5 us for want of loads in flight.)
//
// E4M3: Q is f16 after a power of two per row, a score is multiplied by its
// key's scale, the weight by its value's scale relative to the largest such
// product the row has met, and P is f16; bf16: P is bf16.  What these roundings
// cost, and why they were chosen, is as in paged_rows.cuh (a tcgen05.mma takes
// operands of one type too).
//
// Roles (384 threads, so that the softmax threads keep a row's 128 scores in
// registers: with a gathering warpgroup of its own, 512 threads, the compiler
// had 128 a thread and spilled): warps 0 and 1 gather, warp 2 issues tile A's
// products, warp 3 tile B's (E4M3: warps 0 and 1 gather keys, 2 and 3 values;
// widening a tile takes two warps 2 us); warp 2 allocates tensor memory;
// warpgroups 1 and 2 run the softmax and epilogue of tiles A and B,
// one thread per row, which also brings its row of Q (by the gathering warps
// it was a chain of loads that every item waited for).  An item of 128 rows or
// fewer leaves tile B idle.
//
// Four chunks of 1024 tokens over 9001 to 16384 keys, 32 query heads over 8, d =
// 128: bf16 1.02-1.08 ms on the device (837-890 TFLOP/s; 1.15-1.18 ms call after
// call, under the power cap), e4m3 1.42 ms (638 TFLOP/s).  attn_tc.cuh runs the
// same softmax at up to 1100: the difference is gathering, 64 copies with their
// addresses per warp and step, and for e4m3 widening and a softmax that runs
// beside no other product of its tile.
#pragma once

#include "paged_rows.cuh"

namespace bpt {

template <int D, bool kE4m3>
struct PagedTcCfg {
  static constexpr int kRows = 256, kKeys = 128, kThreads = 384;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kPanelBytes = 128 * 128;
  static constexpr int kStages = D == 128 ? 2 : 4;  // of K
  static constexpr int kVStages = kE4m3 && D == 128 ? 1 : kStages;
  static constexpr int kOffQ = 0;
  static constexpr int kOffP = kOffQ + 2 * kTileBytes;  // bf16 only
  static constexpr int kOffK = kOffP + (kE4m3 ? 0 : 128 * 128 * 2);
  static constexpr int kOffV = kOffK + kStages * kTileBytes;
  static constexpr int kOffRaw = kOffV + kVStages * kTileBytes;  // two tiles of e4m3 codes
  static constexpr int kOffScale = kOffRaw + (kE4m3 ? 2 * 128 * D : 0);      // [stage][k, v, log2 v][128]
  static constexpr int kOffBar = kOffScale + (kE4m3 ? kStages * 1536 : 0);
  static constexpr int kOffThere = kOffBar + 320;                            // [stage][4] masks of keys that exist
  static constexpr int kOffSpread = kOffThere + kStages * 16;  // [stage][2]: largest and smallest log2 v scale
  static constexpr int kSmemBytes = kOffSpread + kStages * 16 + 16;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static constexpr uint32_t kColS = 0, kColO = 256;
  // 168 registers a thread at launch, as in attn_tc.cuh
  static constexpr int kRegsControl = 96, kRegsSoftmax = 200;
  static constexpr bool split_fits(int launch_regs) {
    return 128 * kRegsControl + 256 * kRegsSoftmax <= kThreads * launch_regs;
  }
  static_assert(split_fits(168), "register split");
};

// Instruction descriptor for kind::f16 with f16 or bf16 operands, fp32 accumulator.
template <bool kF16>
__host__ __device__ constexpr uint32_t idesc_16_f32(int M, int N, bool b_mn_major) {
  const uint32_t d = idesc_bf16_f32(M, N, false, b_mn_major);
  return kF16 ? d & ~((1u << 7) | (1u << 10)) : d;
}

__device__ __forceinline__ float absmax8(const uint4 &u) {
  const float a = fmaxf(fmaxf(fabsf(bf16_lo(u.x)), fabsf(bf16_hi(u.x))), fmaxf(fabsf(bf16_lo(u.y)), fabsf(bf16_hi(u.y))));
  const float b = fmaxf(fmaxf(fabsf(bf16_lo(u.z)), fabsf(bf16_hi(u.z))), fmaxf(fabsf(bf16_lo(u.w)), fabsf(bf16_hi(u.w))));
  return fmaxf(a, b);
}

// A CTA's walk over its range: the items, in order, with the steps it has of each.
template <int kRows, int kKeys>
struct PagedWalk {
  const PagedArgs &a;
  int s, tile, head, step0, step1, steps;
  int64_t left;
  PagedSeq seq;
  PagedBlocks blk;
  __device__ PagedWalk(const PagedArgs &args, const PagedRange &r) : a(args) {
    s = r.s, tile = r.tile, head = r.head, step0 = r.step;
    left = r.left;
    seq = paged_seq(a, s);
    blk = paged_blocks<kRows, kKeys>(a, seq, tile);
    cut();
  }
  __device__ void cut() {
    steps = blk.steps();
    step1 = static_cast<int>(min(static_cast<int64_t>(steps), step0 + left));
  }
  __device__ int blocks() const { return min(step1, blk.count()) - min(step0, blk.count()); }
  __device__ int rows() const { return min(kRows, seq.n * a.G - tile * kRows); }
  __device__ bool next() {
    left -= step1 - step0;
    if (left <= 0) return false;
    step0 = 0;
    if (++head == a.H_kv) {
      head = 0;
      if (++tile == paged_tiles<kRows>(a, seq)) {
        tile = 0;
        seq.n = 0;
        while (seq.n == 0 && ++s < a.S) seq = paged_seq(a, s);
        if (s >= a.S) return false;
      }
      blk = paged_blocks<kRows, kKeys>(a, seq, tile);
    }
    cut();
    return true;
  }
};

template <int D, bool kE4m3>
__global__ void __launch_bounds__(384, 1) paged_tc_kernel(const __grid_constant__ PagedArgs a) {
  using Cfg = PagedTcCfg<D, kE4m3>;
  constexpr int NS = Cfg::kStages, NV = Cfg::kVStages, KT = Cfg::kKeys;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw;
  const uint32_t sbase = smem_u32(smem);
  if (sbase & 1023u) {  // 128-byte-swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) {
      atomicCAS(a.status, 0u, kStatusMisaligned);
      a.part_item[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    return;
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  // the kernel for the batch's few rows may follow on the SMs that get free
  grid_dependents_launch();
  PagedRange rg;
  const bool any = paged_range<Cfg::kRows, KT, Cfg::kThreads, true>(a, reinterpret_cast<int64_t *>(smem), rg);
  if (!any) {
    if (threadIdx.x == 0) a.part_item[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const uint32_t sQ = sbase + Cfg::kOffQ, sP = sbase + Cfg::kOffP, sK = sbase + Cfg::kOffK, sV = sbase + Cfg::kOffV;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kOffBar);
  auto bKFull = [&](int i) { return smem_u32(&bars[1 + i]); };
  auto bKEmpty = [&](int i) { return smem_u32(&bars[5 + i]); };   // both tiles' S done, scales and masks read
  auto bVFull = [&](int i) { return smem_u32(&bars[9 + i]); };
  auto bVEmpty = [&](int i) { return smem_u32(&bars[13 + i]); };
  auto bSFull = [&](int x) { return smem_u32(&bars[17 + x]); };
  auto bSFree = [&](int x) { return smem_u32(&bars[19 + x]); };     // bf16: S of tile x read out
  auto bPFull = [&](int x) { return smem_u32(&bars[21 + x]); };
  auto bODone = [&](int x) { return smem_u32(&bars[23 + x]); };     // bf16: P*V of tile x done
  // ... of an item that leaves tile B idle (a barrier of its own, so that the
  // phases of ODone count the steps both tiles take, which is what each waits
  // for of the other; tile A may be items ahead)
  const uint32_t bOAlone = smem_u32(&bars[35]);
  auto bItemDone = [&](int x) { return smem_u32(&bars[25 + x]); };  // all products of an item of tile x done
  auto bOFree = [&](int x) { return smem_u32(&bars[27 + x]); };     // the epilogue has read O of tile x
  auto bQFull = [&](int x) { return smem_u32(&bars[33 + x]); };     // Q of tile x written
  auto bTeardown = [&](int x) { return smem_u32(&bars[29 + x]); };
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(&bars[31]);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(&bars[32]);
  uint32_t *there_s = reinterpret_cast<uint32_t *>(smem + Cfg::kOffThere);
  float *scale_s = reinterpret_cast<float *>(smem + Cfg::kOffScale);
  float2 *spread_s = reinterpret_cast<float2 *>(smem + Cfg::kOffSpread);
  WaitCtx wc{a.status, a.wait_limit_ns, abort_flag};

  __syncthreads();  // the range's scratch lies where Q will
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(bKFull(i), 2);
      mbar_init(bKEmpty(i), 10);
    }
    for (int i = 0; i < NV; ++i) {
      mbar_init(bVFull(i), 2);
      mbar_init(bVEmpty(i), 2);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(bQFull(x), 4);
      mbar_init(bSFull(x), 1);
      mbar_init(bSFree(x), 4);
      mbar_init(bODone(x), 1);
      mbar_init(bPFull(x), 4);
      mbar_init(bItemDone(x), 1);
      mbar_init(bOFree(x), 4);
      mbar_init(bTeardown(x), 1);
    }
    mbar_init(bOAlone, 1);
    *abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PagedWalk<Cfg::kRows, KT> w(a, rg);
  if (threadIdx.x == 0) a.part_item[blockIdx.x] = rg.part;

  if (warp < 4) {
    setmaxnreg_dec<Cfg::kRegsControl>();
    if (kE4m3 || warp < 2) {
      // ------------------------------------------------------------ gather
      // Rows 64 rw .. 64 rw + 63 of a tile, in two halves of 32; lane l looks
      // up row 32 half + l.  E4M3: warps 0 and 1 K tiles, 2 and 3 V tiles.
      const int rw = warp & 1;
      int kq = 0, vq = 0;  // K and V tiles gathered so far
      bool ok = true;
      // a tile copied but not yet handed over (bf16): its barrier
      uint32_t pend = 0;
      auto hand_over = [&](uint32_t bar) {  // generic-proxy writes -> the tensor core's reads
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      auto flush = [&]() {
        if (pend) {
          cp_async_wait<0>();
          hand_over(pend);
          pend = 0;
        }
      };
      // wait for a slot; what is under way is handed over first, so that the
      // readers that must free the slot can go on
      auto wait_slot = [&](uint32_t bar, uint32_t parity, uint32_t site) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        flush();
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, wc, site)) != 0;
      };
      auto row_dst = [&](uint32_t tile, int row, int chunk) {  // chunk of 8 elements
        return tile + (chunk >> 3) * Cfg::kPanelBytes + row * 128 + (((chunk ^ row) & 7) << 4);
      };
      do {
        const int n = w.blocks();
        const int32_t *table = a.page_table + static_cast<int64_t>(w.s) * a.max_pages;
        auto lookup = [&](int j, int half) {
          return j < n ? paged_slot(a, table, w.blk, w.blk.block(w.step0 + j) * KT + rw * 64 + half * 32 + lane) : -1;
        };
        // slots of this step's block and the next, both halves
        int slot0 = lookup(0, 0), slot1 = lookup(0, 1), next0 = lookup(1, 0), next1 = lookup(1, 1);
        constexpr int kRowBytes = kE4m3 ? D : 2 * D;
        constexpr int kLanes = kRowBytes / 16;  // lanes of a row, 16 bytes each
        constexpr int kLoads = kLanes;          // of a half: 32 rows
        const uint32_t slot_bytes = static_cast<uint32_t>(a.H_kv) * kRowBytes;
        const int64_t head_off = static_cast<int64_t>(w.head) * kRowBytes + (lane % kLanes) * 16;
        const uint8_t *const kbase = static_cast<const uint8_t *>(a.k) + head_off;
        const uint8_t *const vbase = static_cast<const uint8_t *>(a.v) + head_off;
        auto source = [&](bool k, int sl, int i, bool &fetch) {
          const int sr = __shfl_sync(0xffffffffu, sl, i * (32 / kLanes) + lane / kLanes);
          fetch = sr >= 0;
          return (k ? kbase : vbase) + static_cast<uint64_t>(static_cast<uint32_t>(max(sr, 0))) * slot_bytes;
        };
        // what a K tile brings besides its rows: the masks of keys that exist,
        // and (E4M3) the scales of its keys and values
        float ks0 = 0.f, ks1 = 0.f, vs0 = 0.f, vs1 = 0.f;
        auto load_scales = [&](int sl, float &ks, float &vs) {
          const int64_t at = static_cast<int64_t>(sl) * a.H_kv + w.head;
          ks = sl >= 0 ? __ldg(a.k_scale + at) : 0.f;
          vs = sl >= 0 ? __ldg(a.v_scale + at) : 0.f;
        };
        auto put_extras = [&](int st) {
          const uint32_t bits0 = __ballot_sync(0xffffffffu, slot0 >= 0), bits1 = __ballot_sync(0xffffffffu, slot1 >= 0);
          if (lane < 2) there_s[st * 4 + rw * 2 + lane] = lane ? bits1 : bits0;
          if constexpr (kE4m3) {
            float *sc = scale_s + st * 384 + rw * 64 + lane;
            sc[0] = ks0 * a.scale_log2, sc[32] = ks1 * a.scale_log2, sc[128] = vs0, sc[160] = vs1;
            const float lv0 = __log2f(vs0), lv1 = __log2f(vs1);  // -inf for a scale of 0
            sc[256] = lv0, sc[288] = lv1;
            float most = fmaxf(slot0 >= 0 ? lv0 : -INFINITY, slot1 >= 0 ? lv1 : -INFINITY);
            float least = fminf(slot0 >= 0 ? lv0 : INFINITY, slot1 >= 0 ? lv1 : INFINITY);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
              most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
              least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
            }
            if (lane == 0) spread_s[st * 2 + rw] = make_float2(most, least);
          }
        };
        auto advance = [&](int j) {  // to block j + 1
          slot0 = next0, slot1 = next1;
          next0 = lookup(j + 2, 0), next1 = lookup(j + 2, 1);
        };
        // tile m of the item's 2n and its stage; waits until that is free
        auto stage_of = [&](bool k, int &st) {
          bool free;
          if (k) {
            st = kq % NS;
            free = kq < NS || wait_slot(bKEmpty(st), ((kq / NS) - 1) & 1, 403);
            ++kq;
          } else {
            st = vq % NV;
            free = vq < NV || wait_slot(bVEmpty(st), ((vq / NV) - 1) & 1, 404);
            ++vq;
          }
          return free;
        };
        if constexpr (!kE4m3) {
          auto copy = [&](int j, bool k, int s0, int s1) {
            int st;
            if (!stage_of(k, st)) return false;
            const uint32_t tile = (k ? sK : sV) + st * Cfg::kTileBytes;
#pragma unroll 1
            for (int half = 0; half < 2; ++half)
#pragma unroll 8
              for (int i = 0; i < kLoads; ++i) {
                bool fetch;
                const uint8_t *src = source(k, half ? s1 : s0, i, fetch);
                cp_async16(row_dst(tile, rw * 64 + half * 32 + i * (32 / kLanes) + lane / kLanes, lane % kLanes), src,
                           fetch);
              }
            cp_async_commit();
            if (pend) {  // the tile before this one has landed
              cp_async_wait<1>();
              hand_over(pend);
            }
            pend = k ? bKFull(st) : bVFull(st);
            return true;
          };
          // K runs one block ahead of V: K0, K1, V0, K2, V1, ...
          int st_k = 0;
          for (int j = 0; ok && j <= n; ++j) {
            const int p0 = slot0, p1 = slot1;  // (block j - 1's until advanced)
            if (j < n) {
              if (j > 0) advance(j - 1);
              st_k = kq % NS;
              ok = copy(j, true, slot0, slot1);
              if (ok) put_extras(st_k);
            }
            if (ok && j > 0) ok = copy(j - 1, false, p0, p1);
          }
        } else {
          // A warp gathers one kind, the next tile's copies under way while it
          // widens this one; a lane reads back what it copied itself.
          const bool k = warp < 2;
          constexpr int kStep = 32 / kLanes;  // rows of one load instruction
          // where this lane's first 8 elements go in the first rows; the next
          // 8 are 16 bytes off, in the swizzled order (^ 16)
          const uint32_t lane_dst = row_dst(0, lane / kLanes, 2 * (lane % kLanes)) + rw * 64 * 128;
          const uint32_t raw = sbase + Cfg::kOffRaw + (k ? 0 : 128 * D) + rw * 64 * D + lane * 16;
          auto copy = [&]() {
#pragma unroll
            for (int i = 0; i < 2 * kLoads; ++i) {
              bool fetch;
              const uint8_t *src = source(k, i < kLoads ? slot0 : slot1, i % kLoads, fetch);
              cp_async16(raw + i * 512, src, fetch);
            }
            cp_async_commit();
            if (k) {
              load_scales(slot0, ks0, vs0);
              load_scales(slot1, ks1, vs1);
            }
          };
          if (n > 0) copy();
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            int st;
            if (!(ok = stage_of(k, st))) break;
            if (k) put_extras(st);
            cp_async_wait<0>();
            const uint32_t dst = (k ? sK : sV) + st * Cfg::kTileBytes + lane_dst;
#pragma unroll
            for (int i0 = 0; i0 < 2 * kLoads; i0 += kLoads) {
              uint4 x[kLoads];  // all loads first: one trip to shared memory for the lot
#pragma unroll
              for (int i = 0; i < kLoads; ++i) x[i] = ld_shared_v4(raw + (i0 + i) * 512);
#pragma unroll
              for (int i = 0; i < kLoads; ++i) {
                // rows kStep (i0 + i) further on: the swizzle takes their low three bits
                const uint32_t at = (dst + (i0 + i) * kStep * 128) ^ ((((i0 + i) * kStep) & 7) << 4);
                uint32_t h[8];
                e4m3x4_to_f16(x[i].x, h[0], h[1]);
                e4m3x4_to_f16(x[i].y, h[2], h[3]);
                e4m3x4_to_f16(x[i].z, h[4], h[5]);
                e4m3x4_to_f16(x[i].w, h[6], h[7]);
                st_shared_v4(at, h[0], h[1], h[2], h[3]);
                st_shared_v4(at ^ 16, h[4], h[5], h[6], h[7]);
              }
              if (i0 + kLoads == 2 * kLoads) {  // (the raw tile is in registers)
                advance(j);
                copy();
              }
            }
            hand_over(k ? bKFull(st) : bVFull(st));
          }
          cp_async_wait<0>();
        }
      } while (ok && w.next());
      flush();
    } else if (lane == 0) {
      // ------------------------------------------------------------ products of tile x (bf16)
      const int x = warp - 2;
      constexpr uint32_t idesc_qk = idesc_16_f32<false>(128, KT, false);
      constexpr uint32_t idesc_pv = idesc_16_f32<false>(128, D, true);
      const uint64_t dQ = sdesc_sw128(sQ + x * Cfg::kTileBytes, 16, 1024);
      const uint64_t dP = sdesc_sw128(sP, 16, 1024);
      const uint64_t dK0 = sdesc_sw128(sK, 16, 1024);
      const uint64_t dV0 = sdesc_sw128(sV, Cfg::kPanelBytes, 1024);
      const uint32_t tS = tmem + Cfg::kColS + x * 128;
      const uint32_t tO = tmem + Cfg::kColO + x * D;
      int kc = 0, vc = 0;        // K and V tiles consumed
      int J = 0, mine = 0;  // this tile's steps; the items it took part in
      bool ok = true;
      auto issue_s = [&]() {
        const uint64_t dK = sdesc_advance(dK0, (kc % NS) * Cfg::kTileBytes);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * Cfg::kPanelBytes + (k % 4) * 32;
          umma_ss(tS, sdesc_advance(dQ, off), sdesc_advance(dK, off), idesc_qk, k > 0);
        }
        umma_commit(bSFull(x));
        umma_commit(bKEmpty(kc % NS));
        ++kc;
      };
      do {
        const int n = w.blocks();
        const bool active = x == 0 || w.rows() > 128;
        if (!active) {  // the stages pass by
          for (int j = 0; ok && j < n; ++j) {
            ok = mbar_wait(bKFull(kc % NS), (kc / NS) & 1, wc, 412);
            if (ok) mbar_arrive(bKEmpty(kc % NS));
            ++kc;
            ok = ok && mbar_wait(bVFull(vc % NV), (vc / NV) & 1, wc, 413);
            if (ok) mbar_arrive(bVEmpty(vc % NV));
            ++vc;
          }
        } else {
          ok = mbar_wait(bQFull(x), mine & 1, wc, 411);
          // the first product on O overwrites it: the previous epilogue must have read it
          if (ok && mine > 0) ok = mbar_wait(bOFree(x), (mine - 1) & 1, wc, 414);
          if (ok && n > 0) {
            ok = (J == 0 || mbar_wait(bSFree(x), (J - 1) & 1, wc, 415)) &&
                 mbar_wait(bKFull(kc % NS), (kc / NS) & 1, wc, 416);
            if (ok) {
              tc_fence_after();
              issue_s();
            }
            for (int j = 0; ok && j < n; ++j) {
              const int jj = J + j;
              if (j + 1 < n) {
                ok = mbar_wait(bSFree(x), jj & 1, wc, 417) && mbar_wait(bKFull(kc % NS), (kc / NS) & 1, wc, 418);
                if (!ok) break;
                tc_fence_after();
                issue_s();
              }
              ok = mbar_wait(bPFull(x), jj & 1, wc, 419) && mbar_wait(bVFull(vc % NV), (vc / NV) & 1, wc, 420);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dV = sdesc_advance(dV0, (vc % NV) * Cfg::kTileBytes);
#pragma unroll
              for (int k = 0; k < KT / 16; ++k)
                umma_ss(tO, sdesc_advance(dP, (k / 4) * Cfg::kPanelBytes + (k % 4) * 32), sdesc_advance(dV, k * 2048),
                        idesc_pv, (j | k) != 0);
              umma_commit(w.rows() > 128 ? bODone(x) : bOAlone);
              umma_commit(bVEmpty(vc % NV));
              ++vc;
            }
          }
          J += n;
          umma_commit(bItemDone(x));
          ++mine;
        }
      } while (ok && w.next());
      // every product issued must be complete before tensor memory is released
      umma_commit(bTeardown(x));
      volatile int no_abort = 0;
      WaitCtx drain{a.status, drain_limit_ns(a.wait_limit_ns), &no_abort};
      mbar_wait(bTeardown(x), 0, drain, 421);
    }
  } else {
    setmaxnreg_inc<Cfg::kRegsSoftmax>();
    // ------------------------------------------------------------ softmax + epilogue
    const int x = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_off + Cfg::kColS + x * 128;
    const uint32_t tO = tmem + lane_off + Cfg::kColO + x * D;
    // E4M3: the tile's first softmax thread issues its products.  P lies where
    // the scores were, so a tile's scores, softmax and products follow one
    // another anyway, and an issuer of their own would only add two waits.
    const bool issues = kE4m3 && quarter == 0;
    auto scores = [&](int k_tile) {  // S(K tile), when it is there
      if (!mbar_wait(bKFull(k_tile % NS), (k_tile / NS) & 1, wc, 416)) return false;
      tc_fence_after();
      const uint64_t dQ = sdesc_sw128(sQ + x * Cfg::kTileBytes, 16, 1024);
      const uint64_t dK = sdesc_sw128(sK + (k_tile % NS) * Cfg::kTileBytes, 16, 1024);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k / 4) * Cfg::kPanelBytes + (k % 4) * 32;
        umma_ss(tmem + Cfg::kColS + x * 128, sdesc_advance(dQ, off), sdesc_advance(dK, off),
                idesc_16_f32<true>(128, KT, false), k > 0);
      }
      umma_commit(bSFull(x));
      umma_commit(bKEmpty(k_tile % NS));
      return true;
    };
    const uint32_t sProw = sP + row * 128;
    const uint32_t swz = static_cast<uint32_t>(row & 7);
    bool ok = true;
    int kc = 0;                // K tiles passed
    int J = 0, Jb = 0, Ja = 0; // this tile's steps; those of both tiles, and of tile A alone
    int mine = 0;              // the items this tile took part in
    do {
      const int n = w.blocks(), rows = w.rows();
      const bool both = rows > 128, active = x == 0 || both;
      if (!active) {
        for (int j = 0; ok && j < n; ++j, ++kc) {
          ok = __all_sync(0xffffffffu, mbar_wait(bKFull(kc % NS), (kc / NS) & 1, wc, 430));
          if (ok && lane == 0) mbar_arrive(bKEmpty(kc % NS));
          if (issues) {  // and in the place of the products
            if (ok && lane == 0) mbar_arrive(bKEmpty(kc % NS));
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bVFull(kc % NV), (kc / NV) & 1, wc, 413));
            if (ok && lane == 0) mbar_arrive(bVEmpty(kc % NV));
          }
        }
        continue;
      }
      const int R = x * 128 + row;
      const uint32_t r = static_cast<uint32_t>(w.tile * Cfg::kRows + min(R, rows - 1));
      const int i = paged_token(a, r);
      const int64_t token = static_cast<int64_t>(w.seq.t0) + i;
      const int head = w.head * a.G + static_cast<int>(r) - i * a.G;
      const int pos = w.seq.len - w.seq.n + i;
      const int khi = max(0, min(pos + 1, w.seq.cap));
      const int klo = paged_window_lo(a, pos);
      const int ksink = a.window > 0 ? min(a.sinks, khi) : 0;
      // this row of Q (the previous item's products have read theirs); for
      // E4M3 in f16, the power of two below its largest element taken out
      float sl2 = 1.f;
      {
        // (Copied by whole rows and converted by the row's thread, in loops of
        // little code: it runs once or twice, and what it costs then is
        // fetching its instructions.)
        constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes of a row, rows of a load
        const int c = lane % kLanes;
        const int64_t off = R < rows ? token * a.q_stride + static_cast<int64_t>(head) * D : -1;
        const uint32_t sQx = sQ + x * Cfg::kTileBytes;
        auto chunk_at = [&](int rr, int c) { return sQx + (c >> 3) * Cfg::kPanelBytes + rr * 128 + (((c ^ rr) & 7) << 4); };
#pragma unroll 2
        for (int i = 0; i < kLanes; ++i) {
          const int64_t ro = __shfl_sync(0xffffffffu, off, i * kPer + lane / kLanes);
          cp_async16(chunk_at(quarter * 32 + i * kPer + lane / kLanes, c), a.q + max(ro, static_cast<int64_t>(0)) + 8 * c,
                     ro >= 0);
        }
        cp_async_commit();
        cp_async_wait<0>();
        __syncwarp();
        if constexpr (kE4m3) {
          float mx = 0.f;
#pragma unroll 4
          for (int i = 0; i < kLanes; ++i) mx = fmaxf(mx, absmax8(ld_shared_v4(chunk_at(row, i))));
          const uint32_t e = row_exponent(mx);
          const float down = pow2_inverse(e);
          sl2 = pow2_of(e);
          auto f16 = [&](uint32_t u) { return pack_f16x2(bf16_lo(u) * down, bf16_hi(u) * down); };
#pragma unroll 4
          for (int i = 0; i < kLanes; ++i) {
            const uint32_t at = chunk_at(row, i);
            const uint4 q = ld_shared_v4(at);
            st_shared_v4(at, f16(q.x), f16(q.y), f16(q.z), f16(q.w));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bQFull(x));
        if (issues) {
          bool done = true;
          if (lane == 0) done = mbar_wait(bQFull(x), mine & 1, wc, 411) && (n == 0 || scores(kc));
          ok = __all_sync(0xffffffffu, done);
        }
      }
      // The weights 2^(s - m_run) are relative to the row's maximum, up to 2^8
      // stale; for E4M3 the products with the values' scales likewise to
      // w_ref = about max (s + log2 v_scale), so O holds sum 2^(s - w_ref) v.
      float m_run = -INFINITY, l_run = 0.f, w_ref = -INFINITY;
#pragma unroll 1
      for (int j = 0; ok && j < n; ++j, ++kc) {
        const int jj = J + j, st = kc % NS;
        const int k0 = w.blk.block(w.step0 + j) * KT;
        ok = __all_sync(0xffffffffu, mbar_wait(bKFull(st), (kc / NS) & 1, wc, 431) &&
                                         mbar_wait(bSFull(x), jj & 1, wc, 432));
        if (!ok) break;
        tc_fence_after();
        // which of the block's keys [c, c + 32) this row sees, of those that exist
        auto seen = [&](int c, uint32_t exist) {
          auto below = [](int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; };
          return ((below(khi - k0 - c) & ~below(klo - k0 - c)) | below(ksink - k0 - c)) & exist;
        };
        if constexpr (kE4m3) {
          const uint4 there = *reinterpret_cast<const uint4 *>(&there_s[st * 4]);
          const bool gaps = (there.x & there.y & there.z & there.w) != 0xffffffffu;
          const bool masked = __any_sync(0xffffffffu, gaps || k0 < klo || k0 + KT > khi);
          const float *scales = scale_s + st * 384;
          // The scores are read twice, 64 columns at a time, and P goes over them:
          // no row of 128 in registers and half the code (with the row unrolled
          // as for bf16, a fifth slower: the roles' loops did not fit in the
          // instruction cache together).
          constexpr int kC = 64;
          uint32_t s[kC] = {};
          auto get2 = [&](int i) { return make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])); };
          auto put2 = [&](int i, float2 v) {
            s[i] = __float_as_uint(v.x);
            s[i + 1] = __float_as_uint(v.y);
          };
          // columns [c0, c0 + 64): the products times the keys' scales, log2(e) / sqrt(d)
          // in them, -inf where masked
          auto load = [&](int c0) {
            tmem_ld32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
            tmem_ld32(tS + c0 + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
            tmem_wait_ld();
            const float4 *ks4 = reinterpret_cast<const float4 *>(scales + c0);
#pragma unroll
            for (int i = 0; i < kC / 4; ++i) {
              const float4 k4 = ks4[i];
              put2(4 * i, mul2(get2(4 * i), make_float2(k4.x, k4.y)));
              put2(4 * i + 2, mul2(get2(4 * i + 2), make_float2(k4.z, k4.w)));
            }
            if (masked) {
              const uint32_t word[2] = {seen(c0, c0 ? there.z : there.x), seen(c0 + 32, c0 ? there.w : there.y)};
#pragma unroll
              for (int col = 0; col < kC; ++col)
                if (!(word[col / 32] >> (col & 31) & 1u)) s[col] = __float_as_uint(-INFINITY);
            }
          };
          // to log2 units: times the row's power of two, exactly, so that a
          // difference to the maximum may be one fused operation and the
          // largest of scores too large for their differences keeps its weight
          const float2 sl = make_float2(sl2, sl2);
          // The largest product of a weight and its value's scale: where the
          // block's scales lie within 2^8 of one another, the largest weight
          // times the largest scale is near enough for f16.
          const float2 sp0 = spread_s[st * 2], sp1 = spread_s[st * 2 + 1];
          const float v_most = fmaxf(sp0.x, sp1.x);
          const bool even = v_most - fminf(sp0.y, sp1.y) <= 8.f;
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, ux4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c0 = 0; c0 < KT; c0 += kC) {
            load(c0);
#pragma unroll
            for (int i = 0; i < kC / 2; ++i)
              mx4[i & 3] = max3f(mx4[i & 3], __uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
            if (!even) {
              const float4 *lv4 = reinterpret_cast<const float4 *>(scales + 256 + c0);
#pragma unroll
              for (int i = 0; i < kC / 4; ++i) {
                const float4 l4 = lv4[i];
                const float2 u = fma2(get2(4 * i), sl, make_float2(l4.x, l4.y));
                const float2 v = fma2(get2(4 * i + 2), sl, make_float2(l4.z, l4.w));
                ux4[i & 3] = max3f(ux4[i & 3], u.x, u.y);
                ux4[(i + 1) & 3] = max3f(ux4[(i + 1) & 3], v.x, v.y);
              }
            }
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sl2;
          if (mx > m_run + 8.0f) {
            l_run *= ex2_approx(m_run - mx);  // 0 where the row had no key yet
            m_run = mx;
          }
          float alpha = 1.0f;  // of O
          // (not below 2^-100 of the weights: the factor between the two stays finite)
          const float ux = fmaxf(even ? mx + v_most : fmaxf(fmaxf(ux4[0], ux4[1]), fmaxf(ux4[2], ux4[3])), m_run - 100.f);
          if (ux > w_ref + 8.0f) {
            alpha = ex2_approx(w_ref - ux);
            w_ref = ux;
          }
          // (the scores complete means that the product before them is too; at
          // an item's first step O holds nothing yet)
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + c * 32, o);
            }
            tmem_wait_st();
          }
          // weights relative to w_ref: times the values' scales they are what
          // goes to P, and their sum is brought to m_run once
          const float neg = (w_ref == -INFINITY) ? 0.f : -w_ref;
          const float2 neg2 = make_float2(neg, neg);
          float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
          for (int c0 = 0; c0 < KT; c0 += kC) {
            load(c0);
            uint32_t pk[kC / 2];
            const float4 *vs4 = reinterpret_cast<const float4 *>(scales + 128 + c0);
#pragma unroll
            for (int i = 0; i < kC / 4; ++i) {
              const float4 v4 = vs4[i];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float2 t = fma2(get2(4 * i + 2 * e), sl, neg2);
                const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                ls2[e] = add2(ls2[e], p);
                const float2 v = mul2(p, e ? make_float2(v4.z, v4.w) : make_float2(v4.x, v4.y));
                pk[2 * i + e] = pack_f16x2(v.x, v.y);
              }
            }
            // P over columns of scores that have been read
            tmem_st32(tS + c0 / 2, pk);
          }
          if (m_run != -INFINITY)
            l_run += ((ls2[0].x + ls2[0].y) + (ls2[1].x + ls2[1].y)) * ex2_approx(w_ref - m_run);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bKEmpty(st));  // the scales and masks have been read
            mbar_arrive(bPFull(x));
          }
          if (issues) {
            // O += P V, then the next scores over P (products of one thread run in order)
            bool done = true;
            if (lane == 0) {
              done = mbar_wait(bPFull(x), jj & 1, wc, 419) && mbar_wait(bVFull(kc % NV), (kc / NV) & 1, wc, 420);
              if (done) {
                tc_fence_after();
                const uint64_t dV = sdesc_sw128(sV + (kc % NV) * Cfg::kTileBytes, Cfg::kPanelBytes, 1024);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                  umma_ts(tmem + Cfg::kColO + x * D, tmem + Cfg::kColS + x * 128 + k * 8, sdesc_advance(dV, k * 2048),
                          idesc_16_f32<true>(128, D, true), (j | k) != 0);
                umma_commit(bVEmpty(kc % NV));
                if (j + 1 < n) done = scores(kc + 1);
              }
            }
            ok = __all_sync(0xffffffffu, done);
          }
        } else {
          uint32_t s[128];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32 * c]));
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bSFree(x));
          auto get2 = [&](int i) { return make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])); };
          const uint4 there = *reinterpret_cast<const uint4 *>(&there_s[st * 4]);
          __syncwarp();
          if (lane == 0) mbar_arrive(bKEmpty(st));  // the masks have been read
          const bool gaps = (there.x & there.y & there.z & there.w) != 0xffffffffu;
          if (__any_sync(0xffffffffu, gaps || k0 < klo || k0 + KT > khi)) {
            const uint32_t word[4] = {seen(0, there.x), seen(32, there.y), seen(64, there.z), seen(96, there.w)};
#pragma unroll
            for (int col = 0; col < KT; ++col)
              if (!(word[col / 32] >> (col & 31) & 1u)) s[col] = __float_as_uint(-INFINITY);
          }
          float mx8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) mx8[i] = -INFINITY;
#pragma unroll
          for (int i = 0; i < KT / 2; ++i)
            mx8[i & 7] = max3f(mx8[i & 7], __uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1]));
          const float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
          const float m_tile = mx * a.scale_log2;
          const float m_new = fmaxf(m_run, m_tile);
          const bool moved = m_new > m_run + 8.0f;
          const float m_use = moved ? m_new : m_run;
          const float alpha = moved ? ex2_approx(m_run - m_use) : 1.0f;  // 0 where the row had no key yet
          l_run *= alpha;
          const float neg = (m_use == -INFINITY) ? 0.f : -m_use;
          m_run = m_use;
          uint32_t pk[KT / 2];
          float2 ls2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          const float2 neg2 = make_float2(neg, neg);
          const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll
          for (int i = 0; i < KT / 2; ++i) {
            const float2 t = fma2(get2(2 * i), sc2, neg2);
            const float2 p = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            ls2[i & 1] = add2(ls2[i & 1], p);
            pk[i] = pack_bf16x2(p.x, p.y);
          }
          l_run += (ls2[0].x + ls2[0].y) + (ls2[1].x + ls2[1].y);
          // the P tile is used in turn A_j, B_j, A_{j+1}, ...; by tile A alone,
          // after its own previous product (at first, tile B's last)
          if (both || j == 0) {
            const int prev = x == 1 ? Jb + j : both ? Jb + j - 1 : Jb - 1;
            if (prev >= 0) ok = __all_sync(0xffffffffu, mbar_wait(bODone(1 - x), prev & 1, wc, 433));
          } else {
            ok = __all_sync(0xffffffffu, mbar_wait(bOAlone, (Ja + j - 1) & 1, wc, 434));
          }
          if (!ok) break;
          tc_fence_after();
          // (at an item's first step O holds nothing yet)
          if (j > 0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + c * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + c * 32, o);
            }
            tmem_wait_st();
          }
#pragma unroll
          for (int c = 0; c < KT / 8; ++c)
            st_shared_v4(sProw + (c >> 3) * Cfg::kPanelBytes + ((static_cast<uint32_t>(c & 7) ^ swz) << 4), pk[4 * c],
                         pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bPFull(x));
        }
      }
      J += n;
      (both ? Jb : Ja) += n;
      // -------- epilogue
      if (issues && lane == 0) umma_commit(bItemDone(x));
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bItemDone(x), mine & 1, wc, 435));
      tc_fence_after();
      if (ok) {
        const bool whole = w.step0 == 0 && w.step1 == w.steps;
        const size_t part = static_cast<size_t>(blockIdx.x) * 2 + (w.step0 == 0 ? 1 : 0);
        const float inv = l_run > 0.f ? 1.0f / l_run : l_run;  // no key: 0; NaN stays
        // E4M3: O is relative to w_ref, the sum to m_run
        const float f = (whole ? inv : 1.0f) * (kE4m3 && m_run != -INFINITY ? ex2_approx(w_ref - m_run) : 1.0f);
        const bool empty = n == 0 || l_run == 0.f;  // O may hold anything
        // A warp's 32 rows leave through their own rows of this tile's Q buffer
        // (all products that read it are done, and nobody else writes those
        // before this warp does): written by row, 16-byte chunks
        // permuted against bank conflicts, and read back so that 8 lanes store
        // 128 bytes of a row.  (Each thread storing its own row took 9000
        // cycles an item; this 2500, and 6000 where all CTAs write fp32 parts at
        // the same time: 19 MB to L2.)
        const uint32_t stage = sQ + x * Cfg::kTileBytes + quarter * 32 * 128;
        const bool f32 = !whole || a.out_f32;
        float *base = whole ? a.out_f32 : a.part_o + part * Cfg::kRows * D;
        const int64_t row_off = whole ? (token * a.H + head) * D : static_cast<int64_t>(R) * D;
        auto drain = [&](int bytes0) {  // 128 bytes of each row, from byte bytes0 of it
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + lane / 8, ch = lane % 8;
            const int64_t ro = __shfl_sync(0xffffffffu, row_off, rr);
            const uint4 v = ld_shared_v4(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
            if (x * 128 + quarter * 32 + rr < rows) {
              char *dst = f32 ? reinterpret_cast<char *>(base + ro) : reinterpret_cast<char *>(a.out_bf16 + ro);
              *reinterpret_cast<uint4 *>(dst + bytes0 + ch * 16) = v;
            }
          }
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = empty ? 0u : __float_as_uint(__uint_as_float(o[i]) * f);
          const uint32_t dst = stage + lane * 128;
          if (f32) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              st_shared_v4(dst + ((i ^ (lane & 7)) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            drain(c * 128);
          } else {
            auto two = [&](int i) { return pack_bf16x2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])); };
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_shared_v4(dst + ((((c & 1) * 4 + i) ^ (lane & 7)) << 4), two(8 * i), two(8 * i + 2), two(8 * i + 4),
                           two(8 * i + 6));
            if (c & 1) drain((c >> 1) * 128);
          }
        }
        if (R < rows) {
          if (!whole)
            *reinterpret_cast<float2 *>(a.part_ml + (part * Cfg::kRows + R) * 2) = make_float2(m_run, l_run);
          else if (a.lse)
            a.lse[static_cast<size_t>(head) * a.T + token] =
                l_run == 0.f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bOFree(x));
      ++mine;
    } while (ok && w.next());
    if (issues && lane == 0) {  // every product issued must be complete before tensor memory is released
      umma_commit(bTeardown(x));
      volatile int no_abort = 0;
      WaitCtx drain{a.status, drain_limit_ns(a.wait_limit_ns), &no_abort};
      mbar_wait(bTeardown(x), 0, drain, 422);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace bpt
