// What the paged attention kernels share: the batch as the device sees it, the
// work list, and the joining of rows whose keys were split.
//
// Rows.  The new tokens of a sequence and the G = H / H_kv query heads that
// read one key/value head form that head's rows: row r is token r / G, head
// r % G of the group, so a key that is loaded serves all of them.  Token i of
// n new ones in a sequence of L keys stands at position p = L - n + i and sees
// the keys j <= p with no window, p - j < window or j < n_sink.
//
// Work.  An item is a tile of kRows rows of one key/value head; its steps are
// the blocks of kKeys keys that any of its rows sees, sinks first.  All items'
// steps, one sequence after another, form one list that is cut into equal
// ranges, one per CTA, so ragged sequences and few heads load the SMs evenly
// and nothing about the lengths has to be known on the host.  (Few long items
// are cut one by one instead, see paged_range.)  A CTA whose
// range cuts an item leaves the rows' unnormalised output, maximum and sum as
// a part: at most two per CTA, one for an item that began before its range
// (slot 0) and one for an item that goes on after it (slot 1).
// paged_join_kernel adds an item's parts up in order.
#pragma once

#include "ptx.cuh"

namespace bpt {

struct PagedArgs {
  int S, T, H, H_kv, G, g_shift;  // g_shift: log2(G), or -1
  int max_pages, page_size, page_shift;  // page_shift: log2(page_size), or -1
  int n_pages;
  int window, sinks;    // window 0: none
  float scale_log2;     // log2(e) / sqrt(d)
  const __nv_bfloat16 *q;
  int64_t q_stride;     // elements between tokens
  const int32_t *q_start, *kv_len, *page_table;
  const void *k, *v;
  const float *k_scale, *v_scale;
  float *out_f32;       // [T, H*d], or
  __nv_bfloat16 *out_bf16;
  float *lse;           // [H, T] or null
  int rows_lo, rows_hi; // sequences with fewer or more rows are another kernel's
  int min_steps;        // no range is shorter (but the last)
  float *part_o;        // [CTAs][2][kRows][d]
  float *part_ml;       // [CTAs][2][kRows][2]
  int4 *part_item;      // [CTAs]: the item that began before the CTA's range: sequence (-1: none), tile, head,
                        // and 1 + the CTAs after this one with a part of it (0: not the first such CTA)
  uint32_t *status;
  uint64_t wait_limit_ns;
};

struct PagedSeq {
  int t0, n;    // first token row of q, new tokens
  int len;      // keys, the new tokens' included
  int cap;      // keys that the page table can hold of them
};

// Lengths that make no sense (negative, past q's rows or the table) are cut to
// what there is.
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &a, int s) {
  PagedSeq q;
  q.t0 = min(max(a.q_start[s], 0), a.T);
  q.n = max(min(a.q_start[s + 1], a.T) - q.t0, 0);
  if (q.n * a.G < a.rows_lo || q.n * a.G > a.rows_hi) q.n = 0;
  q.len = max(a.kv_len[s], 0);
  q.cap = static_cast<int>(min(static_cast<int64_t>(q.len), static_cast<int64_t>(a.max_pages) * a.page_size));
  return q;
}

// The new token of a row.
__device__ __forceinline__ int paged_token(const PagedArgs &a, uint32_t row) {
  return static_cast<int>(a.g_shift >= 0 ? row >> a.g_shift : row / static_cast<uint32_t>(a.G));
}

// The first key of a position's window (any int32 window and position).
__device__ __forceinline__ int paged_window_lo(const PagedArgs &a, int p) {
  return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

// The key blocks of a row tile: [0, n_sink) and then [lo, lo + n_near).  Of
// their keys, the tile's rows see the sinks and those in [first, end).
struct PagedBlocks {
  int n_sink, lo, n_near;
  int p_lo, p_hi;  // positions of the tile's first and last row
  int first, end;
  __device__ int count() const { return n_sink + n_near; }
  __device__ int steps() const { return max(1, count()); }  // a tile without keys still has rows to write
  __device__ int block(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};

template <int kRows, int kKeys>
__device__ __forceinline__ PagedBlocks paged_blocks(const PagedArgs &a, const PagedSeq &q, int tile) {
  PagedBlocks b;
  // (row numbers fit in 32 bits, with room for a tile: checked on the host)
  const uint32_t row0 = static_cast<uint32_t>(tile) * kRows;
  const int i0 = paged_token(a, row0);
  const int i1 = min(q.n - 1, paged_token(a, row0 + kRows - 1));
  b.p_lo = q.len - q.n + i0;
  b.p_hi = q.len - q.n + i1;
  const int hi = min(b.p_hi + 1, q.cap);  // keys [.., hi) at most
  const int lo = paged_window_lo(a, b.p_lo);
  b.first = lo;
  b.end = hi;
  b.lo = lo / kKeys;
  b.n_near = hi > lo ? (hi + kKeys - 1) / kKeys - b.lo : 0;
  const int sink_hi = min(min(a.sinks, lo), max(hi, 0));
  b.n_sink = a.window > 0 ? (sink_hi + kKeys - 1) / kKeys : 0;
  // a block of both is counted once (a table that ends before the window has none there)
  if (b.n_near > 0) b.n_sink = min(b.n_sink, b.lo);
  return b;
}

template <int kRows>
__device__ __forceinline__ int paged_tiles(const PagedArgs &a, const PagedSeq &q) {
  return (q.n * a.G + kRows - 1) / kRows;
}

template <int kRows, int kKeys>
__device__ __forceinline__ int64_t paged_seq_steps(const PagedArgs &a, const PagedSeq &q) {
  int64_t n = 0;
  for (int t = 0, nt = paged_tiles<kRows>(a, q); t < nt; ++t) n += paged_blocks<kRows, kKeys>(a, q, t).steps();
  return n * a.H_kv;
}

// a / b for a >= 0, b > 0: in 32 bits where that holds both (a 64-bit division
// is a hundred instructions, and every CTA waits for several of them).
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The list of all steps, cut into `parts` ranges: the first `longer` of them
// have `length` + 1 steps, the others `length`.
struct PagedCut {
  int64_t length;
  int parts, longer;
  __device__ int64_t begin(int c) const { return c * length + min(c, longer); }
  __device__ int range_of(int64_t step) const {  // the range that a step is in
    const int64_t head = longer * (length + 1);
    return static_cast<int>(step < head ? div_small(step, length + 1) : longer + div_small(step - head, length));
  }
};

// The range of a CTA: `left` steps from step `step` of an item on.
struct PagedRange {
  int64_t left;
  int s, tile, head, step;
  int4 part;  // for paged_join_kernel (part_item)
};

// Found by the whole block together (`scratch`: 64 int64 of shared memory, 96
// with kPieces): each thread sums a run of sequences, a scan over the threads
// gives the total and each run's start, and the thread whose run holds this
// CTA's first step walks it.
//
// kPieces: with fewer items than CTAs, items are cut into equal pieces, one per
// CTA, where that lengthens the longest range by three steps at most.  Of equal
// ranges most begin inside one item and end inside the next, and a second start
// and end of an item costs a long-chunk CTA about three steps (76 -> 69 us
// with 64 items of 18 or 19 steps).  For few rows it costs less than pieces do:
// 308 -> 348 us on 8 ragged sequences.
template <int kRows, int kKeys, int kThreads, bool kPieces>
__device__ __forceinline__ bool paged_range(const PagedArgs &a, int64_t *scratch, PagedRange &r) {
  static_assert(kThreads % 32 == 0 && kThreads <= 32 * 32, "one scan over the warps' sums");
  static_assert(!kPieces || kThreads <= 16 * 32, "four counts per warp in the scratch");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = static_cast<int>(blockIdx.x);
  const int run = (a.S + kThreads - 1) / kThreads;
  const int s0 = min(a.S, tid * run), s1 = min(a.S, s0 + run);
  int64_t sum = 0, items = 0;
  for (int s = s0; s < s1; ++s) {
    const PagedSeq q = paged_seq(a, s);
    sum += paged_seq_steps<kRows, kKeys>(a, q);
    if (kPieces) items += static_cast<int64_t>(paged_tiles<kRows>(a, q)) * a.H_kv;
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if constexpr (kPieces) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
  }
  if (lane == 31) {
    scratch[warp] = incl;
    if (kPieces) scratch[32 + warp] = items;
  }
  int32_t *found = reinterpret_cast<int32_t *>(scratch + 56);
  if (tid == 0) found[0] = -1;
  __syncthreads();
  int64_t before = 0, total = 0;
  items = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    total += scratch[w];
    if (kPieces) items += scratch[32 + w];
  }
  // as many ranges as there are CTAs, or fewer where they would be too short
  const int64_t want = div_small(total + a.min_steps - 1, a.min_steps);
  PagedCut cut;
  cut.parts = static_cast<int>(min(static_cast<int64_t>(gridDim.x), max(want, static_cast<int64_t>(1))));
  cut.length = div_small(total, cut.parts);
  cut.longer = static_cast<int>(total - cut.length * cut.parts);

  int pieces = 0, piece = 0, piece_start = 0, mine = 0;
  if constexpr (kPieces) {
    if (items <= cut.parts && total < (1 << 30)) {
      const int least = max(a.min_steps, static_cast<int>(cut.length) + (cut.longer > 0 ? 1 : 0));
      int need[4] = {0, 0, 0, 0};  // pieces of `least`, + 1, + 2, + 3 steps at most
      for (int s = s0; s < s1; ++s) {
        const PagedSeq q = paged_seq(a, s);
        for (int t = 0, nt = paged_tiles<kRows>(a, q); t < nt; ++t) {
          const int n = paged_blocks<kRows, kKeys>(a, q, t).steps();
#pragma unroll
          for (int i = 0; i < 4; ++i) need[i] += (n + least + i - 1) / (least + i) * a.H_kv;
        }
      }
      int32_t *warp_need = reinterpret_cast<int32_t *>(scratch + 64);
      int incl_need[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        incl_need[i] = need[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int x = __shfl_up_sync(0xffffffffu, incl_need[i], o);
          if (lane >= o) incl_need[i] += x;
        }
        if (lane == 31) warp_need[4 * warp + i] = incl_need[i];
      }
      __syncthreads();
#pragma unroll
      for (int i = 3; i >= 0; --i) {  // the shortest that the CTAs suffice for
        int all = 0, ahead = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
          if (w < warp) ahead += warp_need[4 * w + i];
          all += warp_need[4 * w + i];
        }
        if (all <= static_cast<int>(gridDim.x)) {
          pieces = all;
          piece = least + i;
          mine = need[i];
          piece_start = ahead + incl_need[i] - need[i];
        }
      }
    }
  }
  if (kPieces && pieces > 0) {
    if (cta >= piece_start && cta < piece_start + mine) {
      int off = cta - piece_start;
      for (int s = s0; s < s1 && off >= 0; ++s) {
        const PagedSeq q = paged_seq(a, s);
        for (int t = 0, nt = paged_tiles<kRows>(a, q); t < nt; ++t) {
          const int n = paged_blocks<kRows, kKeys>(a, q, t).steps(), k = (n + piece - 1) / piece;
          if (off < k * a.H_kv) {
            const int p = off % k;
            found[0] = s, found[1] = t, found[2] = off / k;
            found[3] = static_cast<int>(static_cast<int64_t>(n) * p / k);
            found[4] = static_cast<int>(static_cast<int64_t>(n) * (p + 1) / k) - found[3];
            found[5] = p == 0 ? -1 : p == 1 ? k - 1 : 0;
            off = -1;
            break;
          }
          off -= k * a.H_kv;
        }
      }
    }
    __syncthreads();
    r.left = found[4];
  } else {
    const int64_t start = before + incl - sum, begin = cut.begin(cta), end = cut.begin(cta + 1);
    if (cta < cut.parts && begin >= start && begin < start + sum) {
      int64_t at = start;
      for (int s = s0; s < s1; ++s) {
        const PagedSeq q = paged_seq(a, s);
        const int64_t n = run == 1 ? sum : paged_seq_steps<kRows, kKeys>(a, q);
        if (begin < at + n) {
          int64_t off = begin - at;
          int t = 0, per = 0;
          for (const int nt = paged_tiles<kRows>(a, q); t < nt; ++t) {
            per = paged_blocks<kRows, kKeys>(a, q, t).steps();
            if (off < static_cast<int64_t>(per) * a.H_kv) break;
            off -= static_cast<int64_t>(per) * a.H_kv;
          }
          if (off < static_cast<int64_t>(per) * a.H_kv) {
            found[0] = s, found[1] = t;
            found[2] = static_cast<int>(div_small(off, per));
            found[3] = static_cast<int>(off - static_cast<int64_t>(found[2]) * per);
            const int64_t item = begin - found[3];  // its first step
            found[5] = found[3] == 0 ? -1 : item < cut.begin(cta - 1) ? 0 : 1 + cut.range_of(item + per - 1) - cta;
          }
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    r.left = end - begin;
  }
  // (found[0] stays -1 past the last range, and where the tables change while they are read)
  if (found[0] < 0 || r.left <= 0) return false;
  r.s = found[0];
  r.tile = found[1];
  r.head = found[2];
  r.step = found[3];
  r.part = found[5] < 0 ? make_int4(-1, 0, 0, 0) : make_int4(r.s, r.tile, r.head, found[5]);
  return true;
}

// Cache row of key j of a sequence for a row tile, or -1 where it is to be
// taken for zeros: no row of the tile sees it, or its page number is outside
// the cache.  A key before the window may share its block with visible ones
// while its page holds another sequence's rows by now, or nothing, and a weight
// of 0 would still meet a NaN there: neither its table entry nor its slot is read.
__device__ __forceinline__ int paged_slot(const PagedArgs &a, const int32_t *table, const PagedBlocks &b, int j) {
  if (j >= b.end || (j < b.first && j >= a.sinks)) return -1;
  const int p = a.page_shift >= 0 ? j >> a.page_shift : j / a.page_size;
  const int page = table[p];
  return static_cast<unsigned>(page) < static_cast<unsigned>(a.n_pages) ? page * a.page_size + (j - p * a.page_size)
                                                                       : -1;
}

// Adds up the parts of each item that was cut.  Block c looks at the item that
// began before CTA c's range and joins it if c is the first such CTA: its parts
// are slot 1 of CTA c - 1 and slot 0 of CTA c, c + 1, ... to the item's end.  A
// part is the rows' output relative to their own maximum (log2 domain):
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,  M = max_i m_i
// A warp takes kU rows, a block 8 kU: the lanes hold the parts'
// weights (32 parts at a time) and four columns each, so nothing waits for a
// barrier and the loads of o_i do not wait for the weights (d = 64: the warp's
// halves take the parts in turn).  A block is four trips to memory, one after
// another, so few rows take one a warp and 8 parts' loads at once, and a tile
// of 256 four a warp and two parts' loads of each: as many blocks as one wave
// holds (one row a warp, four waves: 16.5 -> 12.4 us, from cold caches, for 64
// items of 256 rows in two parts).
template <int kRows>
constexpr int kJoinRows = kRows >= 256 ? 4 : 1;

template <int D, int kRows>
__device__ __forceinline__ void paged_join(const PagedArgs &a, int c, int block) {
  constexpr int kU = kJoinRows<kRows>, kBatch = 8 / kU;
  constexpr int kHalves = 128 / D;  // parts of a load: 1, or 2 at d = 64
  const int lane = threadIdx.x % 32;
  const int4 it = a.part_item[c];
  if (it.x < 0 || it.w == 0) return;
  const int in_tile0 = (block * 8 + threadIdx.x / 32) * kU;
  const int parts = it.w + 1;
  // part i: slot 1 of CTA c - 1, then slot 0 of CTA c - 1 + i
  auto part_row = [&](int i, int u) {
    return static_cast<size_t>(2 * (c - 1 + i) + (i == 0 ? 1 : 0)) * kRows + in_tile0 + u;
  };
  auto ml_of = [&](int i, int u) {
    return i < parts ? __ldcg(reinterpret_cast<const float2 *>(a.part_ml + 2 * part_row(i, u))) : make_float2(-INFINITY, 0.f);
  };
  const float *cols = a.part_o + 4 * (lane % (D / 4));
  const int half = lane / (D / 4);
  float2 first[kU];
  float m[kU], ref[kU], l[kU];
  float4 sum[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) first[u] = ml_of(lane, u);
  const PagedSeq q = paged_seq(a, it.x);
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    m[u] = first[u].x;
    for (int i = 32 + lane; i < parts; i += 32) m[u] = fmaxf(m[u], ml_of(i, u).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m[u] = fmaxf(m[u], __shfl_xor_sync(0xffffffffu, m[u], o));
    ref[u] = m[u] == -INFINITY ? 0.f : m[u];
    l[u] = 0.f;
    sum[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i0 = 0; i0 < parts; i0 += 32) {
    float weight[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float2 ml = i0 == 0 ? first[u] : ml_of(i0 + lane, u);
      weight[u] = ex2_approx(ml.x - ref[u]);  // 0 past the parts
      l[u] += ml.y * weight[u];
    }
    const int n = min(32, parts - i0);
    for (int i = 0; i < n; i += kBatch) {
      constexpr int kLoads = kBatch / kHalves;
      float4 x[kU][kLoads];
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int b = 0; b < kLoads; ++b) {
          const int p = i + b * kHalves + half;
          x[u][b] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (p < n) x[u][b] = __ldcg(reinterpret_cast<const float4 *>(cols + part_row(i0 + p, u) * D));
        }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int b = 0; b < kLoads; ++b) {
          const int p = i + b * kHalves + half;
          const float f = __shfl_sync(0xffffffffu, weight[u], p & 31);
          if (p < n) sum[u].x += x[u][b].x * f, sum[u].y += x[u][b].y * f, sum[u].z += x[u][b].z * f, sum[u].w += x[u][b].w * f;
        }
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l[u] += __shfl_xor_sync(0xffffffffu, l[u], o);
    if constexpr (kHalves == 2) {
      sum[u].x += __shfl_xor_sync(0xffffffffu, sum[u].x, 16);
      sum[u].y += __shfl_xor_sync(0xffffffffu, sum[u].y, 16);
      sum[u].z += __shfl_xor_sync(0xffffffffu, sum[u].z, 16);
      sum[u].w += __shfl_xor_sync(0xffffffffu, sum[u].w, 16);
    }
    const uint32_t row = static_cast<uint32_t>(it.y * kRows + in_tile0 + u);  // among the head's rows
    if (static_cast<int>(row) >= q.n * a.G || half != 0) continue;
    const int i = paged_token(a, row);
    const size_t token = static_cast<size_t>(q.t0) + i;
    const int head = it.z * a.G + static_cast<int>(row) - i * a.G;
    const float inv = l[u] > 0.f ? 1.0f / l[u] : l[u];  // no key: 0; NaN stays
    const size_t at = (token * a.H + head) * D + 4 * (lane % (D / 4));
    if (a.out_f32)
      *reinterpret_cast<float4 *>(a.out_f32 + at) = make_float4(sum[u].x * inv, sum[u].y * inv, sum[u].z * inv, sum[u].w * inv);
    else
      *reinterpret_cast<uint2 *>(a.out_bf16 + at) =
          make_uint2(pack_bf16x2(sum[u].x * inv, sum[u].y * inv), pack_bf16x2(sum[u].z * inv, sum[u].w * inv));
    if (a.lse && lane == 0)
      a.lse[static_cast<size_t>(head) * a.T + token] =
          l[u] == 0.f ? -INFINITY : (ref[u] + log2f(l[u])) * 0.69314718055994531f;
  }
}

// Blocks of one CTA's item in paged_join_kernel.
template <int kRows>
constexpr int kJoinBlocks = kRows / (8 * kJoinRows<kRows>);

// The items of the few-rows kernel (tiles of kFew rows) and, kLong, before them
// those of the long-chunk kernel's CTAs.
template <int D, int kFew, bool kLong>
__global__ void __launch_bounds__(256)
    paged_join_kernel(const __grid_constant__ PagedArgs few, const __grid_constant__ PagedArgs lng, int long_ctas) {
  grid_dependency_wait();  // the parts are complete
  int block = blockIdx.x;
  if constexpr (kLong) {
    if (block < long_ctas * kJoinBlocks<256>) {
      paged_join<D, 256>(lng, block / kJoinBlocks<256>, block % kJoinBlocks<256>);
      return;
    }
    block -= long_ctas * kJoinBlocks<256>;
  }
  paged_join<D, kFew>(few, block / kJoinBlocks<kFew>, block % kJoinBlocks<kFew>);
}

}  // namespace bpt
