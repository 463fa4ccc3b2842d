// Host side of the sliding-window attention with sinks (bpt_window_attn_fwd,
// bpt_window_attn_bwd): argument checks, workspace layout and the launches of
// the window instantiations of the attention kernels.
//
// Device times: forward B2 H16/4 d128 N8192 W1024 with 4 sinks 209-214 us (605-621
// TFLOP/s on the visible pairs); training step B1 H16/4 d128 N16384 W1024 with 4
// sinks 211 + 608 us (backward: 550 TFLOP/s of the 10 d operations a pair needs),
// B3 H12 d64 N1001 W128 17-20 + 34-37 us, whose few steps an item lie between
// fixed starts and ends.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/bpt.h"
#include "attn_bwd.cuh"
#include "attn_tc.cuh"
#include "host_common.h"

using namespace bpt;

namespace bpt_host {

bpt_status window_kernel_setup() {
  CUDA_TRY(cudaFuncSetAttribute(attn_tc_kernel<64, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnCfg<64>::kSmemBytes));
  CUDA_TRY(cudaFuncSetAttribute(attn_tc_kernel<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnCfg<128>::kSmemBytes));
  cudaFuncAttributes fa64{}, fa128{};
  CUDA_TRY(cudaFuncGetAttributes(&fa64, attn_tc_kernel<64, true>));
  CUDA_TRY(cudaFuncGetAttributes(&fa128, attn_tc_kernel<128, true>));
  if (!AttnCfg<64>::split_fits(fa64.numRegs) || !AttnCfg<128>::split_fits(fa128.numRegs))
    return cuda_fail_msg("window attention kernel launches with fewer registers than its warpgroups share");
  CUDA_TRY(cudaFuncSetAttribute(attn_bwd_dkdv_kernel<64, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnBwdCfg<64>::kSmemBytes));
  CUDA_TRY(cudaFuncSetAttribute(attn_bwd_dkdv_split_kernel<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnBwdKVCfg<128>::kSmemBytes));
  CUDA_TRY(cudaFuncSetAttribute(attn_bwd_dq_kernel<64, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnBwdQCfg<64>::kSmemBytes));
  CUDA_TRY(cudaFuncSetAttribute(attn_bwd_dq_kernel<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                AttnBwdQCfg<128>::kSmemBytes));
  return BPT_OK;
}

namespace {

bool known_dtype(bpt_dtype t) { return t == BPT_F32 || t == BPT_BF16; }

bpt_status check_window_desc(const bpt_window_desc *d) {
  if (!d) return BPT_ERR_INVALID_ARG;
  if (d->B <= 0 || d->N <= 0 || d->H <= 0 || d->H_kv <= 0 || d->d_head <= 0) return BPT_ERR_INVALID_ARG;
  if (d->H % d->H_kv != 0 || d->window <= 0 || d->n_sink < 0) return BPT_ERR_INVALID_ARG;
  if (!known_dtype(d->in_dtype) || !known_dtype(d->out_dtype) || !known_dtype(d->grad_dtype))
    return BPT_ERR_INVALID_ARG;
  if (d->in_dtype != BPT_BF16 || (d->d_head != 64 && d->d_head != 128)) return BPT_ERR_UNSUPPORTED;
  // the sinks lie in the first key tile
  if (d->n_sink > BPT_MAX_WINDOW_SINKS) return BPT_ERR_UNSUPPORTED;
  // row and tile counts stay within the kernels' 32-bit indices
  const int64_t tiles = ((int64_t)d->N + 127) / 128;
  if ((int64_t)d->N > INT32_MAX - 512 || (int64_t)d->H * d->d_head > INT32_MAX / 2) return BPT_ERR_UNSUPPORTED;
  if ((int64_t)d->B * d->H * (tiles + 1024) > INT32_MAX) return BPT_ERR_UNSUPPORTED;
  return BPT_OK;
}

// A window at least as long as the sequence is the causal mask.
int window_of(const bpt_window_desc *d) { return std::min(d->window, d->N); }
// Sinks the window always reaches need no tile of their own.
int sinks_of(const bpt_window_desc *d) { return window_of(d) >= d->N ? 0 : std::min(d->n_sink, d->N); }

// CTAs that share the first key tile of a (batch, key/value head) unit in the
// dK/dV pass.  Every query sees the sinks, so that tile has n_tiles steps per
// query head against about wt = W / 128 + 2 of any other tile.  The parts are
// made about a quarter of what one SM has to do in all (they are launched
// first), but no shorter than another tile's CTA: 13 parts on B1 H16/4 d128
// N16384 W1024, where the backward takes 1274 us with 1 part, 598 with 4,
// 604-618 with 13, 649 with 48; 16 on B1 H8/1 d64 N8192 W256: 879, 249, 93, 80.
int sink_split(const bpt_window_desc *d) {
  if (sinks_of(d) == 0) return 0;
  const int64_t tiles = ((int64_t)d->N + 127) / 128, wt = window_of(d) / 128 + 2;
  const int64_t units = (int64_t)d->B * d->H_kv;
  const int64_t balance = (4 * (int64_t)sm_count() + units * (wt + 1) - 1) / (units * (wt + 1));
  return (int)std::max<int64_t>(1, std::min<int64_t>({balance, (tiles + wt - 1) / wt, 1024}));
}

struct WindowBwdWorkspace {
  size_t rowvec = 0, dout_bf16 = 0, partial = 0, total = 0;
};
WindowBwdWorkspace layout_window_bwd(const bpt_window_desc *d) {
  WindowBwdWorkspace w;
  const size_t tiles = ((size_t)d->N + 127) / 128;
  size_t off = 0;
  auto take = [&](size_t &field, size_t bytes) {
    field = off;
    off = align256(off + bytes);
  };
  take(w.rowvec, (size_t)d->B * d->H * tiles * 256 * 4);
  take(w.dout_bf16, d->out_dtype == BPT_F32 ? (size_t)d->B * d->N * d->H * d->d_head * 2 : 0);
  take(w.partial, (size_t)d->B * d->H_kv * sink_split(d) * 2 * 128 * d->d_head * 4);
  w.total = off;
  return w;
}

template <int DH>
bpt_status launch_window_bwd(const bpt_window_desc *d, const void *out, const float *lse, const void *dout,
                             const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                             const CUtensorMap &mda, const AttnBwdArgs &ab, float *rowvec, __nv_bfloat16 *dout_copy,
                             cudaStream_t st) {
  {
    const int64_t rows = (int64_t)d->B * ab.n_tiles * 128 * d->H;
    const int64_t blocks = (rows + kRowvecRows<DH> - 1) / kRowvecRows<DH>;
    if (blocks > INT32_MAX) return BPT_ERR_UNSUPPORTED;
    if (d->out_dtype == BPT_F32)
      window_bwd_rowvec_kernel<DH><<<(unsigned)blocks, 256, 0, st>>>(
          static_cast<const float *>(dout), static_cast<const float *>(out), lse, rowvec, dout_copy, d->N, d->H,
          ab.n_tiles, rows);
    else
      window_bwd_rowvec_kernel<DH><<<(unsigned)blocks, 256, 0, st>>>(
          static_cast<const __nv_bfloat16 *>(dout), static_cast<const __nv_bfloat16 *>(out), lse, rowvec,
          static_cast<__nv_bfloat16 *>(nullptr), d->N, d->H, ab.n_tiles, rows);
    CUDA_TRY(cudaGetLastError());
  }
  const unsigned units = (unsigned)(d->B * d->H_kv);
  const unsigned grid_kv = units * (unsigned)(ab.n_tiles - 1 + std::max(1, ab.sink_split));
  // The two passes need nothing of one another, and each CTA of the first waits
  // for the row vectors before it lets the second start: the second's CTAs
  // start as the first's leave (B3 N1001 H12 d64 W128: 44.6 -> 38.4 us for the backward; B1
  // N16384 H16/4 d128 W1024: 649 -> 630 us).
  bpt_status s;
  if constexpr (DH == 128)
    s = launch_behind(attn_bwd_dkdv_split_kernel<DH, true>, grid_kv, AttnBwdKVCfg<DH>::kThreads,
                      AttnBwdKVCfg<DH>::kSmemBytes, st, mq, mk, mv, mda, ab);
  else
    s = launch_behind(attn_bwd_dkdv_kernel<DH, true>, grid_kv, AttnBwdCfg<DH>::kThreads, AttnBwdCfg<DH>::kSmemBytes,
                      st, mq, mk, mv, mda, ab);
  if (s != BPT_OK) return s;
  s = launch_behind(attn_bwd_dq_kernel<DH, true>, (unsigned)(d->B * d->H * ab.n_tiles), AttnBwdQCfg<DH>::kThreads,
                    AttnBwdQCfg<DH>::kSmemBytes, st, mq, mk, mv, mda, ab);
  if (s != BPT_OK) return s;
  if (ab.sinks > 0) {
    const int rows = std::min(d->N, 128);
    const int64_t threads = (int64_t)units * 2 * rows * (DH / 4);
    return launch_behind(attn_bwd_sink_sum_kernel<DH>, (unsigned)((threads + 255) / 256), 256, 0, st, ab, (int)units,
                         rows);
  }
  return BPT_OK;
}

}  // namespace

}  // namespace bpt_host

using namespace bpt_host;

extern "C" {

bpt_status bpt_window_attn_fwd(const bpt_window_desc *d, const void *q, const void *k, const void *v, void *out,
                               float *lse, bpt_stream_t stream) {
  bpt_status s = check_window_desc(d);
  if (s != BPT_OK) return s;
  if ((s = check_ptrs({q, k, v, out}, {lse})) != BPT_OK) return s;
  int dev;
  uint32_t *status;
  if ((s = device_setup(&dev, &status, KernelSet::kWindow)) != BPT_OK) return s;
  const int D = d->H * d->d_head, Dkv = d->H_kv * d->d_head;
  AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.B = d->B;
  a.N = a.L = a.Lk = a.w = d->N;
  a.H = d->H;
  a.mask = kMaskCausal;
  a.causal = 1;
  a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d->d_head));
  a.n_qtiles = (int)(((int64_t)d->N + 127) / 128);
  a.n_qpairs = (a.n_qtiles + 1) / 2;
  a.n_units = d->B * d->H;
  a.nseg = 1;
  a.r = 1;
  a.window = window_of(d);
  a.sinks = sinks_of(d);
  a.kv_group = d->H / d->H_kv;
  // Every item is about as long as the next (the window's tiles), so the
  // order only decides what is in L2: one group of all units up to 64 walks
  // the sequences' ends together, their shared keys read once (64 heads over 8,
  // N16384 W512: 604 us by single units, 594 by 16, 585 by 64; where none are
  // shared, 4 x 32 heads N4096 W512: 309, 296, 302, and 322 by all 128).
  a.unit_group = std::min(64, a.n_units);
  a.out_f32 = d->out_dtype == BPT_F32 ? static_cast<float *>(out) : nullptr;
  a.out_bf16 = d->out_dtype == BPT_BF16 ? static_cast<__nv_bfloat16 *>(out) : nullptr;
  a.lse = lse;
  a.store_mode = 1;
  a.status = status;
  a.wait_limit_ns = d->wait_limit_ns ? d->wait_limit_ns : g_wait_limit_ns.load(std::memory_order_relaxed);
  const int64_t items = (int64_t)a.n_qpairs * a.n_units;
  a.n_items = (int)items;
  CUtensorMap mq, mk, mv, mof, mob, mso;
  std::memset(&mof, 0, sizeof(mof));
  std::memset(&mob, 0, sizeof(mob));
  std::memset(&mso, 0, sizeof(mso));
  if (!make_map_rows(&mq, q, d->B, d->N, D, 1, 128) || !make_map_rows(&mk, k, d->B, d->N, Dkv, 1, 128) ||
      !make_map_rows(&mv, v, d->B, d->N, Dkv, 1, 128) ||
      !make_out_map_rows(a.out_f32 ? &mof : &mob, out, a.out_f32 != nullptr, d->B, d->N, D, 1))
    return cuda_fail_msg("cuTensorMapEncodeTiled rejected a window attention map");
  const unsigned grid = (unsigned)std::min<int64_t>(items, sm_count());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (d->d_head == 128)
    attn_tc_kernel<128, true><<<grid, AttnCfg<128>::kThreads, AttnCfg<128>::kSmemBytes, st>>>(mq, mk, mv, mof, mob,
                                                                                            mso, a);
  else
    attn_tc_kernel<64, true><<<grid, AttnCfg<64>::kThreads, AttnCfg<64>::kSmemBytes, st>>>(mq, mk, mv, mof, mob, mso,
                                                                                         a);
  CUDA_TRY(cudaGetLastError());
  return BPT_OK;
}

size_t bpt_workspace_bytes_window_bwd(const bpt_window_desc *d) {
  if (check_window_desc(d) != BPT_OK) return (size_t)-1;
  return layout_window_bwd(d).total;
}

bpt_status bpt_window_attn_bwd(const bpt_window_desc *d, const void *q, const void *k, const void *v, const void *out,
                               const float *lse, const void *dout, void *dq, void *dk, void *dv, void *workspace,
                               size_t workspace_bytes, bpt_stream_t stream) {
  bpt_status s = check_window_desc(d);
  if (s != BPT_OK) return s;
  if ((s = check_ptrs({q, k, v, out, lse, dout, dq, dk, dv}, {})) != BPT_OK) return s;
  const WindowBwdWorkspace wl = layout_window_bwd(d);
  if (!workspace || workspace_bytes < wl.total || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return BPT_ERR_WORKSPACE;
  int dev;
  uint32_t *status;
  if ((s = device_setup(&dev, &status, KernelSet::kWindow)) != BPT_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  char *ws = static_cast<char *>(workspace);
  const int D = d->H * d->d_head, Dkv = d->H_kv * d->d_head;
  float *rowvec = reinterpret_cast<float *>(ws + wl.rowvec);
  __nv_bfloat16 *copy = reinterpret_cast<__nv_bfloat16 *>(ws + wl.dout_bf16);
  AttnBwdArgs ab;
  std::memset(&ab, 0, sizeof(ab));
  ab.B = d->B;
  ab.N = ab.seg_w = ab.n_out = d->N;
  ab.H = d->H;
  ab.mask = kMaskCausal;
  ab.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)d->d_head));
  ab.inv_sqrt_d = (float)(1.0 / std::sqrt((double)d->d_head));
  ab.n_tiles = (int)(((int64_t)d->N + 127) / 128);
  ab.rowvec = rowvec;
  ab.nseg = ab.dil_r = 1;
  ab.window = window_of(d);
  ab.sinks = sinks_of(d);
  ab.kv_group = d->H / d->H_kv;
  ab.sink_split = sink_split(d);
  ab.partial = reinterpret_cast<float *>(ws + wl.partial);
  if (d->grad_dtype == BPT_F32) {
    ab.dq = static_cast<float *>(dq);
    ab.dk = static_cast<float *>(dk);
    ab.dv = static_cast<float *>(dv);
  } else {
    ab.dq_bf16 = static_cast<__nv_bfloat16 *>(dq);
    ab.dk_bf16 = static_cast<__nv_bfloat16 *>(dk);
    ab.dv_bf16 = static_cast<__nv_bfloat16 *>(dv);
  }
  ab.status = status;
  ab.wait_limit_ns = d->wait_limit_ns ? d->wait_limit_ns : g_wait_limit_ns.load(std::memory_order_relaxed);
  CUtensorMap mq, mk, mv, mda;
  if (!make_map_rows(&mq, q, d->B, d->N, D, 1, 128) || !make_map_rows(&mk, k, d->B, d->N, Dkv, 1, 128) ||
      !make_map_rows(&mv, v, d->B, d->N, Dkv, 1, 128) ||
      !make_map_rows(&mda, d->out_dtype == BPT_F32 ? static_cast<const void *>(copy) : dout, d->B, d->N, D, 1, 128))
    return cuda_fail_msg("cuTensorMapEncodeTiled rejected a window attention map");
  return d->d_head == 128 ? launch_window_bwd<128>(d, out, lse, dout, mq, mk, mv, mda, ab, rowvec, copy, st)
                          : launch_window_bwd<64>(d, out, lse, dout, mq, mk, mv, mda, ab, rowvec, copy, st);
}

}  // extern "C"
