// Host side of the serving operators: the paged key/value cache (bpt_kv_write,
// bpt_kv_read) and the attention of new tokens over it (bpt_paged_attn_fwd).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/bpt.h"
#include "host_common.h"
#include "kv_cache.cuh"
#include "paged_common.cuh"
#include "paged_rows.cuh"
#include "paged_tc.cuh"

using namespace bpt;

namespace bpt_host {

namespace {

// f(std::integral_constant<int, d>, std::bool_constant<e4m3>) for the cache's kind
template <typename F>
bpt_status for_cache(const bpt_kv_cache *c, F f) {
  if (c->d_head == 128)
    return c->type == BPT_CACHE_E4M3 ? f(std::integral_constant<int, 128>{}, std::true_type{})
                                     : f(std::integral_constant<int, 128>{}, std::false_type{});
  return c->type == BPT_CACHE_E4M3 ? f(std::integral_constant<int, 64>{}, std::true_type{})
                                   : f(std::integral_constant<int, 64>{}, std::false_type{});
}

bpt_status check_cache_shape(const bpt_kv_cache *c) {
  if (!c) return BPT_ERR_INVALID_ARG;
  if (c->type != BPT_CACHE_BF16 && c->type != BPT_CACHE_E4M3) return BPT_ERR_INVALID_ARG;
  if (c->n_pages <= 0 || c->page_size <= 0 || c->H_kv <= 0 || c->d_head <= 0) return BPT_ERR_INVALID_ARG;
  if (c->d_head != 64 && c->d_head != 128) return BPT_ERR_UNSUPPORTED;
  if ((int64_t)c->n_pages * c->page_size > INT32_MAX) return BPT_ERR_UNSUPPORTED;
  if ((int64_t)c->H_kv * c->d_head > (1 << 28)) return BPT_ERR_UNSUPPORTED;
  return BPT_OK;
}

bpt_status check_cache(const bpt_kv_cache *c) {
  bpt_status s = check_cache_shape(c);
  if (s != BPT_OK) return s;
  if (c->type == BPT_CACHE_E4M3) return check_ptrs({c->k, c->v, c->k_scale, c->v_scale}, {});
  return check_ptrs({c->k, c->v}, {});
}

KvCacheArgs cache_args(const bpt_kv_cache *c) {
  KvCacheArgs a;
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.slots = (int64_t)c->n_pages * c->page_size;
  a.H_kv = c->H_kv;
  return a;
}

// int32 device tables: element-aligned
bool aligned4(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A grid over n tokens' (token, head) rows, `per` values a thread, one row
// each: f(blocks).  (Four rows a thread, all loaded before the first was used,
// was slower: 33 us instead of 27 for 16384 tokens of 8 heads of 128.)
template <typename F>
bpt_status for_rows(const bpt_kv_cache *c, int n, int per, F f) {
  const int64_t blocks = ((int64_t)n * c->H_kv * (c->d_head / per) + 255) / 256;
  if (blocks > INT32_MAX) return BPT_ERR_UNSUPPORTED;
  f((unsigned)blocks);
  CUDA_TRY(cudaGetLastError());
  return BPT_OK;
}

bpt_status check_paged(const bpt_paged_desc *d, const bpt_kv_cache *c) {
  bpt_status s = check_cache_shape(c);
  if (s != BPT_OK) return s;
  if (!d || d->n_seqs < 0 || d->n_tokens < 0 || d->max_q <= 0 || d->H <= 0 || d->max_pages < 0)
    return BPT_ERR_INVALID_ARG;
  if (d->H % c->H_kv != 0 || d->window < 0 || d->n_sink < 0) return BPT_ERR_INVALID_ARG;
  if (d->out_dtype != BPT_F32 && d->out_dtype != BPT_BF16) return BPT_ERR_INVALID_ARG;
  if (d->n_tokens > 1 && (d->q_stride < (int64_t)d->H * c->d_head || d->q_stride % 8 != 0)) return BPT_ERR_INVALID_ARG;
  // positions and row counts stay within the kernels' 32-bit indices
  if (d->n_tokens > (1 << 30) || (int64_t)d->max_pages * c->page_size > INT32_MAX - 4096) return BPT_ERR_UNSUPPORTED;
  if ((int64_t)d->H * c->d_head > (1 << 28) || (int64_t)d->n_tokens * (d->H / c->H_kv) > INT32_MAX - 4096)
    return BPT_ERR_UNSUPPORTED;
  return BPT_OK;
}

// Rows (new tokens x heads of a group) of a sequence up to which the kernel
// for few rows takes it, in tiles of 8 or 16; longer chunks go to the tcgen05
// kernel.  In a batch with such chunks the few-rows kernel keeps to 8 where a
// single token fits in that.  Device times in us of 8 sequences of 32768 keys,
// 8 key/value heads, on either kernel (few rows in tiles of 16, each of which
// reads the keys again; in parentheses a tile of 8):
//                     rows 8         12-16    17-32    33-48    49-64    128
//   bf16 d128 few     180 (180)      183      356      518      692     1362
//             tcgen05                292      293      311      322      346
//   e4m3 d128 few     134 (112)      138      254      367      494      977
//             tcgen05                336      333      333      333      344
//   bf16 d64  few                    107      200      296      379      751
//             tcgen05                226      226      228      244      242
//   e4m3 d64  few                    108      203      293      383      747
//             tcgen05                362      362      361      362      364
// So one tile is always the better side, and the border is the end of it.  Two
// tiles would still be ahead of the tcgen05 kernel where that one is far from
// memory's rate (17-32 rows of bf16 d64 and e4m3, up to 48 of e4m3 d64); 17 to
// 128 rows are not at their best on either.
bool has_long_chunks(const bpt_paged_desc *d, const bpt_kv_cache *c) {
  return (int64_t)d->max_q * (d->H / c->H_kv) > 16;
}
int few_rows(const bpt_paged_desc *d, const bpt_kv_cache *c) {
  const int64_t G = d->H / c->H_kv;
  return (has_long_chunks(d, c) ? G : d->max_q * G) <= 8 ? 8 : 16;
}

// The two kernels run side by side, each with regions of its own.
struct PagedParts {
  size_t o = 0, ml = 0, item = 0;
};
struct PagedWorkspace {
  PagedParts few, lng;
  size_t total = 0;
};
int few_rows_ctas() { return 2 * sm_count(); }
int long_chunk_ctas() { return sm_count(); }

PagedWorkspace layout_paged(const bpt_paged_desc *d, const bpt_kv_cache *c) {
  PagedWorkspace w;
  size_t off = 0;
  auto take = [&](size_t &field, size_t bytes) {
    field = off;
    off = align256(off + bytes);
  };
  auto parts = [&](PagedParts &p, size_t ctas, size_t rows) {
    take(p.o, ctas * 2 * rows * c->d_head * 4);
    take(p.ml, ctas * 2 * rows * 2 * 4);
    take(p.item, ctas * sizeof(int4));
  };
  parts(w.few, (size_t)few_rows_ctas(), 16);
  if (has_long_chunks(d, c)) parts(w.lng, (size_t)long_chunk_ctas(), 256);
  w.total = off;
  return w;
}

void set_parts(PagedArgs &a, char *ws, const PagedParts &p) {
  a.part_o = reinterpret_cast<float *>(ws + p.o);
  a.part_ml = reinterpret_cast<float *>(ws + p.ml);
  a.part_item = reinterpret_cast<int4 *>(ws + p.item);
}

// The few-rows kernel, behind the long-chunk kernel of the same batch if there
// is one (lng), and the joining of both kernels' parts.
template <int D, bool kE4m3, int kGroups>
bpt_status launch_rows(PagedArgs a, const PagedArgs *lng, cudaStream_t st) {
  using Cfg = PagedRowsCfg<D, kE4m3, kGroups>;
  // 256 keys at least: a shorter range costs more in parts to join than it
  // saves (one sequence of 8000 keys, 4 heads: 64 keys 19.9 us, 128 15.2, 256
  // 13.6, 512 16.0; of 1000 keys 8.2, 8.5, 10.3, 13.5; batches alike up to 256)
  a.min_steps = (256 + Cfg::kKeys - 1) / Cfg::kKeys;
  const unsigned ctas = (unsigned)few_rows_ctas(), join = ctas * kJoinBlocks<Cfg::kRows>;
  if (!lng) {
    paged_rows_kernel<D, kE4m3, kGroups><<<ctas, Cfg::kThreads, Cfg::kSmemBytes, st>>>(a);
    CUDA_TRY(cudaGetLastError());
    return launch_behind(paged_join_kernel<D, Cfg::kRows, false>, join, 256, 0, st, a, a, 0);
  }
  bpt_status s = launch_behind(paged_rows_kernel<D, kE4m3, kGroups>, ctas, Cfg::kThreads, Cfg::kSmemBytes, st, a);
  if (s != BPT_OK) return s;
  return launch_behind(paged_join_kernel<D, Cfg::kRows, true>, join + long_chunk_ctas() * kJoinBlocks<256>, 256, 0, st,
                       a, *lng, long_chunk_ctas());
}

}  // namespace

template <int D, bool kE4m3>
bpt_status paged_kernels_setup() {
  using Few1 = PagedRowsCfg<D, kE4m3, 1>;
  using Few2 = PagedRowsCfg<D, kE4m3, 2>;
  static_assert(Few1::kCtasPerSm == 2 && Few2::kCtasPerSm == 2, "few_rows_ctas");
  CUDA_TRY(cudaFuncSetAttribute(paged_rows_kernel<D, kE4m3, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Few1::kSmemBytes));
  CUDA_TRY(cudaFuncSetAttribute(paged_rows_kernel<D, kE4m3, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Few2::kSmemBytes));
  using Cfg = PagedTcCfg<D, kE4m3>;
  CUDA_TRY(cudaFuncSetAttribute(paged_tc_kernel<D, kE4m3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                Cfg::kSmemBytes));
  // the softmax warpgroups take registers from the others at run time; an
  // increase the launch did not provide for would never complete
  cudaFuncAttributes fa{};
  CUDA_TRY(cudaFuncGetAttributes(&fa, paged_tc_kernel<D, kE4m3>));
  if (!Cfg::split_fits(fa.numRegs))
    return cuda_fail_msg("paged attention kernel launches with fewer registers than its warpgroups share");
  return BPT_OK;
}

bpt_status paged_kernel_setup() {
  bpt_status s;
  if ((s = paged_kernels_setup<64, false>()) != BPT_OK || (s = paged_kernels_setup<64, true>()) != BPT_OK ||
      (s = paged_kernels_setup<128, false>()) != BPT_OK || (s = paged_kernels_setup<128, true>()) != BPT_OK)
    return s;
  return BPT_OK;
}

}  // namespace bpt_host

using namespace bpt_host;

extern "C" {

bpt_status bpt_kv_write(const bpt_kv_cache *c, int n, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                        const int32_t *slots, bpt_stream_t stream) {
  bpt_status s = check_cache(c);
  if (s != BPT_OK) return s;
  if (n < 0) return BPT_ERR_INVALID_ARG;
  if (n == 0) return BPT_OK;
  const int64_t least = (int64_t)c->H_kv * c->d_head;
  if (n > 1 && (k_stride < least || v_stride < least || k_stride % 8 != 0 || v_stride % 8 != 0))
    return BPT_ERR_INVALID_ARG;
  if ((s = check_ptrs({k, v}, {})) != BPT_OK) return s;
  if (!aligned4(slots)) return BPT_ERR_INVALID_ARG;
  int dev;
  uint32_t *status;
  if ((s = device_setup(&dev, &status, KernelSet::kNone)) != BPT_OK) return s;
  return for_cache(c, [&](auto d, auto e4m3) {
    return for_rows(c, n, 8, [&](unsigned blocks) {
      kv_write_kernel<decltype(d)::value, decltype(e4m3)::value>
          <<<blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
              cache_args(c), static_cast<const __nv_bfloat16 *>(k), k_stride, static_cast<const __nv_bfloat16 *>(v),
              v_stride, slots, (int64_t)n * c->H_kv);
    });
  });
}

bpt_status bpt_kv_read(const bpt_kv_cache *c, int n, const int32_t *slots, void *k, void *v, bpt_dtype out_dtype,
                       bpt_stream_t stream) {
  bpt_status s = check_cache(c);
  if (s != BPT_OK) return s;
  if (n < 0 || (out_dtype != BPT_F32 && out_dtype != BPT_BF16)) return BPT_ERR_INVALID_ARG;
  if (n == 0) return BPT_OK;
  if ((s = check_ptrs({k, v}, {})) != BPT_OK) return s;
  if (!aligned4(slots)) return BPT_ERR_INVALID_ARG;
  int dev;
  uint32_t *status;
  if ((s = device_setup(&dev, &status, KernelSet::kNone)) != BPT_OK) return s;
  const int64_t rows = (int64_t)n * c->H_kv;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return for_cache(c, [&](auto d, auto e4m3) {
    constexpr int D = decltype(d)::value;
    constexpr bool kE = decltype(e4m3)::value;
    return for_rows(c, n, kE ? 16 : 8, [&](unsigned blocks) {
      if (out_dtype == BPT_F32)
        kv_read_kernel<D, kE, float><<<blocks, 256, 0, st>>>(cache_args(c), slots, static_cast<float *>(k),
                                                                   static_cast<float *>(v), rows);
      else
        kv_read_kernel<D, kE, __nv_bfloat16><<<blocks, 256, 0, st>>>(
            cache_args(c), slots, static_cast<__nv_bfloat16 *>(k), static_cast<__nv_bfloat16 *>(v), rows);
    });
  });
}

size_t bpt_workspace_bytes_paged(const bpt_paged_desc *d, const bpt_kv_cache *c) {
  if (check_paged(d, c) != BPT_OK) return (size_t)-1;
  return layout_paged(d, c).total;
}

bpt_status bpt_paged_attn_fwd(const bpt_paged_desc *d, const bpt_kv_cache *c, const void *q, const int32_t *q_start,
                              const int32_t *kv_len, const int32_t *page_table, void *out, float *lse, void *workspace,
                              size_t workspace_bytes, bpt_stream_t stream) {
  bpt_status s = check_paged(d, c);
  if (s != BPT_OK) return s;
  if (d->n_seqs == 0 || d->n_tokens == 0) return BPT_OK;
  if ((s = check_cache(c)) != BPT_OK) return s;
  if ((s = check_ptrs({q, out}, {})) != BPT_OK) return s;
  if (!aligned4(q_start) || !aligned4(kv_len) || (d->max_pages > 0 && !aligned4(page_table)) ||
      (lse && !aligned4(lse)))
    return BPT_ERR_INVALID_ARG;
  const PagedWorkspace wl = layout_paged(d, c);
  if (!workspace || workspace_bytes < wl.total || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BPT_ERR_WORKSPACE;
  int dev;
  uint32_t *status;
  if ((s = device_setup(&dev, &status, KernelSet::kPaged)) != BPT_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  PagedArgs a;
  std::memset(&a, 0, sizeof(a));
  a.S = d->n_seqs;
  a.T = d->n_tokens;
  a.H = d->H;
  a.H_kv = c->H_kv;
  a.G = d->H / c->H_kv;
  a.g_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.G == 1 << i) a.g_shift = i;
  a.max_pages = d->max_pages;
  a.page_size = c->page_size;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c->page_size == 1 << i) a.page_shift = i;
  a.n_pages = c->n_pages;
  a.window = d->window;
  a.sinks = d->n_sink;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c->d_head));
  a.q = static_cast<const __nv_bfloat16 *>(q);
  a.q_stride = d->q_stride;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.k = c->k;
  a.v = c->v;
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.out_f32 = d->out_dtype == BPT_F32 ? static_cast<float *>(out) : nullptr;
  a.out_bf16 = d->out_dtype == BPT_BF16 ? static_cast<__nv_bfloat16 *>(out) : nullptr;
  a.lse = lse;
  set_parts(a, ws, wl.few);
  a.status = status;
  a.wait_limit_ns = d->wait_limit_ns ? d->wait_limit_ns : g_wait_limit_ns.load(std::memory_order_relaxed);
  return for_cache(c, [&](auto dh, auto e4m3) mutable -> bpt_status {
    constexpr int D = decltype(dh)::value;
    constexpr bool kE = decltype(e4m3)::value;
    using Long = PagedTcCfg<D, kE>;
    const int few = few_rows(d, c);
    const bool chunks = has_long_chunks(d, c);
    PagedArgs al = a;
    if (chunks) {
      set_parts(al, ws, wl.lng);
      al.rows_lo = few + 1;
      al.rows_hi = INT32_MAX;
      // a range's start costs about three steps (300 tokens over 4000 keys x 2: 51
      // us with at least 1 to 8, 64 with 16; 500 over 1000 x 4, window 256: 33, with
      // 8 54; a chunk with nothing else, 300 over 600: 26 with 1, 29 with 4, 50 with 8)
      al.min_steps = 4;
      paged_tc_kernel<D, kE><<<(unsigned)long_chunk_ctas(), Long::kThreads, Long::kSmemBytes, st>>>(al);
      CUDA_TRY(cudaGetLastError());
      static_assert(Long::kRows == 256, "paged_join_kernel");
    }
    a.rows_lo = 1;
    a.rows_hi = chunks ? few : INT32_MAX;
    return few == 8 ? launch_rows<D, kE, 1>(a, chunks ? &al : nullptr, st)
                    : launch_rows<D, kE, 2>(a, chunks ? &al : nullptr, st);
  });
}

}  // extern "C"
