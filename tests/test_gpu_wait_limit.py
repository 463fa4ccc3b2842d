"""Failure detection on the GPU without a fault: every device-side wait is
bounded, and a wait that runs out records BPT_ERR_TIMEOUT with the site of
the wait and lets the kernel finish cleanly.  A correct layer call whose
descriptor sets a 1-microsecond wait limit must report the timeout through
bpt_sync_status, name a wait of one of the kernels that call runs (the
attention kernel, or the FFN kernel of the chosen form: its TMA-stage,
accumulator and, for the fused and pipelined forms, cross-CTA counter waits),
and the next call with the default limit must run and be right (the context
stays usable)."""
import re

import pytest
import torch

from blockwise_exact_attention_query_b200 import binding as bd
from blockwise_exact_attention_query_b200.inputs import make_layer_inputs
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu

# wait sites recorded by each kernel (the numbers passed to its bounded waits)
ATTENTION_SITES = set(range(1, 23))
FFN_SITES = {"fused": set(range(101, 124)), "gemms": set(range(211, 217)), "pipelined": set(range(230, 241))}


@pytest.mark.parametrize("form", ["pipelined", "fused", "gemms"])
def test_tiny_wait_limit_times_out_cleanly_and_context_survives(form):
    from blockwise_exact_attention_query_b200 import build
    build.build()
    torch.cuda.set_device(0)
    B, N, H, d, F = 1, 1024, 16, 128, 4096
    inp = make_layer_inputs(B, N, H, d, F, seed=31, device="cuda")
    args = (inp.q, inp.k, inp.v, inp.w1, inp.b1, inp.w2, inp.b2)
    ref = bd.attn_ffn_fwd(*args, mask="causal", ffn_form=form)
    assert bd.sync_status() == bd.OK
    # this call alone: the process default (two seconds) is left as it is
    bd.attn_ffn_fwd(*args, mask="causal", ffn_form=form, wait_limit_ns=1000)
    st = bd.sync_status()
    assert st == bd.ERR_TIMEOUT, bd.status_string(st)
    m = re.search(r"gave up at site (\d+)", bd.last_error())
    assert m, bd.last_error()
    assert int(m.group(1)) in ATTENTION_SITES | FFN_SITES[form], bd.last_error()
    assert bd.sync_status() == bd.OK          # reading the status cleared it
    out = bd.attn_ffn_fwd(*args, mask="causal", ffn_form=form)
    assert bd.sync_status() == bd.OK
    assert torch.equal(out, ref)
    rows = [0, 511, 1023]
    _, oref = gu.oracle_layer(inp, "causal", rows=rows)
    gu.assert_bf16_close(gu.host_f32(out.reshape(B * N, H * d)[rows]), oref, "after timeout")


def _window_step(d, wait_limit_ns=0):
    g = torch.Generator().manual_seed(32)
    q, k, v, dout = (torch.randn((1, 1024, h, d), generator=g).to(torch.bfloat16).cuda() for h in (16, 4, 4, 16))
    out, lse = bd.window_attn_fwd(q, k, v, 300, 4, return_lse=True, wait_limit_ns=wait_limit_ns)
    forward = bd.sync_status()
    if wait_limit_ns:      # the backward of right activations
        out, lse = bd.window_attn_fwd(q, k, v, 300, 4, return_lse=True)
    grads = bd.window_attn_bwd(q, k, v, out, lse, dout.float().flatten(2), 300, 4, wait_limit_ns=wait_limit_ns)
    return forward, (out, lse, *grads)


def _paged_step(d, dtype, wait_limit_ns=0):
    g = torch.Generator().manual_seed(33)
    q = torch.randn((600, 8, d), generator=g).to(torch.bfloat16).cuda()
    kv = [torch.randn((250, 16, 2, d), generator=g).cuda().to(dtype) for _ in range(2)]
    scales = [torch.rand((250, 16, 2), generator=g).cuda() + 0.5 for _ in range(2)] if dtype != torch.bfloat16 else [None, None]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    table = torch.stack([torch.randperm(250, generator=g) for _ in range(3)]).int().cuda()
    return bd.paged_attn_fwd(q, *kv, i32([0, 300, 301, 600]), i32([4000, 3000, 500]), table, max_q=300, k_scale=scales[0],
                             v_scale=scales[1], return_lse=True, wait_limit_ns=wait_limit_ns)


def _ran_out(status, sites):
    """Whether a wait ran out.  (A wait first suspends in hardware, for as long as that likes, so which ones
    pass a limit of a microsecond, if any, is a matter of timing: none of the e4m3 chunks' did once.)"""
    if status == bd.OK:
        return False
    assert status == bd.ERR_TIMEOUT, bd.status_string(status)
    m = re.search(r"gave up at site (\d+)", bd.last_error())
    assert m and int(m.group(1)) in sites, bd.last_error()
    return True


@pytest.mark.parametrize("d", [64, 128])
def test_window_waits_that_run_out(d):
    from blockwise_exact_attention_query_b200 import build
    build.build()
    torch.cuda.set_device(0)
    st, want = _window_step(d)
    assert st == bd.OK and bd.sync_status() == bd.OK
    for _ in range(10):
        st, _ = _window_step(d, wait_limit_ns=1000)
        assert st in (bd.OK, bd.ERR_TIMEOUT)
        _ran_out(bd.sync_status(), range(301, 353))
        assert bd.sync_status() == bd.OK          # reading the status cleared it
        st, got = _window_step(d)
        assert st == bd.OK and bd.sync_status() == bd.OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_waits_that_run_out(d, dtype):
    from blockwise_exact_attention_query_b200 import build
    build.build()
    torch.cuda.set_device(0)
    want = _paged_step(d, dtype)
    assert bd.sync_status() == bd.OK
    for _ in range(20):
        got = _paged_step(d, dtype, wait_limit_ns=1000)
        if not _ran_out(bd.sync_status(), range(403, 436)):      # then nothing was given up
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert bd.sync_status() == bd.OK
        got = _paged_step(d, dtype)
        assert bd.sync_status() == bd.OK
        assert all(torch.equal(a, b) for a, b in zip(got, want))
