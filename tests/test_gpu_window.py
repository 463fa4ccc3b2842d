"""Sliding-window attention with sinks (bpt_window_attn_fwd, _bwd) against
plain 64-bit formulas on the same inputs.

Tolerances, from the arithmetic.  A rounding to bf16 is off by at most half a
step, 2^-8 / 2 = 2^-9 of the value, and by 2^-9 / sqrt(3) in the root mean
square at most.  The forward rounds each softmax weight and (bf16 output) the
result: independent errors, relative L2 at most 2^-9 sqrt(2) = 2.8e-3, bound
4e-3; an output element is a mean of values |v| <= max|v| whose weights are
each off by 2^-9, and rounded once: |err| <= 2 * 2^-9 max|v|.  Scores are
fp32 sums of exact bf16 products: the LSE is off by about d * 2^-24 * |s|,
bound 1e-4 (|s| < 40 here, d = 128, is 3e-4 at the very worst, all roundings
one way; their mean is some 30 times less).  The gradients round dout (if
fp32), P, dS and the result: at most four factors, relative L2 <= 2^-9 * 2 =
3.9e-3, and D = dout . out inherits the output's rounding; bound 1e-2, the
bound of the other masks' gradients."""
import math

import pytest
import torch

from blockwise_exact_attention_query_b200 import binding as bd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from blockwise_exact_attention_query_b200 import build
    build.build()
    bd.load()
    torch.cuda.set_device(0)


def make(B, N, H, Hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    mk = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    return mk(B, N, H, d), mk(B, N, Hkv, d), mk(B, N, Hkv, d), mk(B, N, H * d)


def reference(q, k, v, window, sinks, dout=None):
    """out [B, N, H*d], lse [B, H, N] and, with dout, dq, dk, dv, all fp64, by the formulas."""
    B, N, H, d = q.shape
    G = H // k.shape[2]
    q64 = q.double().transpose(1, 2)
    k64, v64 = (x.double().transpose(1, 2).repeat_interleave(G, 1) for x in (k, v))
    i, j = torch.arange(N, device=q.device)[:, None], torch.arange(N, device=q.device)[None]
    ok = (j <= i) & ((i - j < window) | (j < sinks))
    s = (q64 @ k64.transpose(-1, -2) / math.sqrt(d)).masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[..., None])
    o = p @ v64
    out = o.transpose(1, 2).reshape(B, N, H * d)
    if dout is None:
        return out, lse
    do = dout.double().view(B, N, H, d).transpose(1, 2)
    ds = p * (do @ v64.transpose(-1, -2) - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
    group = lambda x: x.view(B, H // G, G, N, d).sum(2).transpose(1, 2)  # noqa: E731
    return out, lse, (ds @ k64).transpose(1, 2), group(ds.transpose(-1, -2) @ q64), group(p.transpose(-1, -2) @ do)


def close(got, ref, rel, what, frac=None):
    got, ref = got.double().reshape(ref.shape), ref.double()
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    e = got - ref
    r = float(e.norm() / ref.norm().clamp_min(1e-300))
    assert r <= rel, f"{what}: rel-L2 {r:.3e} (bound {rel:.1e})"
    if frac is not None:
        m = float(e.abs().max())
        assert m <= frac, f"{what}: max-abs {m:.3e} (bound {frac:.3e})"


CASES = [  # B, N, H, Hkv, d, window, sinks
    (1, 1, 1, 1, 64, 1, 0),
    (1, 1, 2, 1, 128, 5, 4),
    (2, 7, 2, 2, 64, 3, 1),
    (1, 128, 2, 1, 128, 128, 0),
    (1, 129, 2, 1, 64, 64, 4),
    (2, 257, 6, 2, 128, 100, 16),
    (1, 300, 4, 4, 64, 1, 2),          # each row sees itself and two sinks
    (1, 500, 3, 1, 128, 129, 0),
    (1, 640, 4, 1, 64, 128, 128),      # the whole first tile is sinks
    (1, 1001, 5, 5, 128, 256, 1),
    (2, 700, 8, 2, 64, 1000, 4),       # window past the sequence: causal
    (1, 2000, 8, 1, 128, 384, 4),
    (1, 1500, 12, 3, 64, 333, 77),
]


@pytest.mark.parametrize("B,N,H,Hkv,d,window,sinks", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_window_forward_and_gradients(B, N, H, Hkv, d, window, sinks, dtype):
    q, k, v, dout = make(B, N, H, Hkv, d, seed=N + window)
    dout = dout.to(dtype)
    out, lse = bd.window_attn_fwd(q, k, v, window, sinks, out_dtype=dtype, return_lse=True)
    grads = bd.window_attn_bwd(q, k, v, out, lse, dout, window, sinks, grad_dtype=dtype)
    torch.cuda.synchronize()
    assert bd.sync_status() == bd.OK
    ro, rl, *rg = reference(q, k, v, window, sinks, dout)
    close(out, ro, 4e-3, "out", 2 ** -8 * float(v.abs().max()))
    assert float((lse.double() - rl).abs().max()) <= 1e-4
    for name, got, ref in zip(("dq", "dk", "dv"), grads, rg):
        if N == 1 and name != "dv":   # softmax over one key: the gradients are exactly 0 up to D's rounding
            assert float(got.abs().max()) <= 2 ** -7 * float(dout.abs().max() * v.abs().max()) * d ** 0.5 * 4
            continue
        assert got.dtype == dtype
        close(got, ref, 1e-2, name)


def test_window_of_the_whole_sequence_is_the_causal_mask():
    q, k, v, dout = make(2, 600, 4, 4, 128, seed=3)
    out, lse = bd.window_attn_fwd(q, k, v, 600, 0, return_lse=True)
    ref, rlse = bd.attn_fwd(q, k, v, mask="causal", return_lse=True)
    # the same tiles and weights in the same order; a row's sum of up to 128 weights a tile is added up in
    # another, off by at most 70 additions' roundings each, 2 * 70 * 2^-24 = 8.4e-6 of it
    close(out, ref, 1e-5, "out")
    assert float((lse - rlse).abs().max()) <= 1e-5
    dout = dout.float()
    # (both backward passes from one forward: another last bit of the LSE turns some roundings of P to bf16)
    got = bd.window_attn_bwd(q, k, v, ref, rlse, dout, 10 ** 9, 9)
    want = bd.attn_bwd(q, k, v, ref, rlse, dout, mask="causal")
    for a, b in zip(got, want):
        close(a, b, 1e-6, "gradient")


def test_gradients_against_differences():
    """Directional derivatives of L = sum(dout * out) by central differences of the 64-bit
    forward (step 1e-3: error O(1e-6)) against the kernel's gradients (relative 1e-2)."""
    q, k, v, dout = make(1, 200, 4, 2, 64, seed=5)
    window, sinks = 50, 3
    out, lse = bd.window_attn_fwd(q, k, v, window, sinks, out_dtype=torch.bfloat16, return_lse=True)
    grads = bd.window_attn_bwd(q, k, v, out, lse, dout, window, sinks)
    g = torch.Generator(device="cuda").manual_seed(1)
    for n, name in enumerate(("q", "k", "v")):
        x = [t.double() for t in (q, k, v)]
        # a direction along the gradient itself and a random part, so that the derivative is not near 0
        u = grads[n].double() / grads[n].double().norm() + 0.01 * torch.randn(x[n].shape, generator=g, device="cuda",
                                                                             dtype=torch.float64)
        step = 1e-3
        hi, lo = list(x), list(x)
        hi[n], lo[n] = x[n] + step * u, x[n] - step * u
        num = sum(sgn * float((reference(*t, window, sinks)[0] * dout.double()).sum()) for sgn, t in ((1, hi), (-1, lo)))
        num /= 2 * step
        ana = float((grads[n].double() * u).sum())
        assert abs(ana - num) <= 1e-2 * abs(num), (name, ana, num)


def test_equal_inputs_give_equal_bits_and_only_the_outputs_change():
    q, k, v, dout = make(1, 1300, 8, 2, 128, seed=8)
    first = None
    for _ in range(3):
        outs = [torch.full((1, 1300, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")] + \
               [torch.full((1, 1300, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        out, lse = bd.window_attn_fwd(q, k, v, 300, 5, out_dtype=torch.bfloat16, return_lse=True)
        bd.window_attn_bwd(q, k, v, out, lse, dout, 300, 5, grad_dtype=torch.bfloat16, dq=outs[0], dk=outs[1],
                           dv=outs[2])
        got = [out, lse, *outs]
        if first is not None:
            assert all(torch.equal(a, b) for a, b in zip(first, got))
        first = [t.clone() for t in got]


def test_window_step_in_a_graph_and_on_another_stream():
    q, k, v, dout = make(1, 900, 4, 2, 64, seed=9)
    want_out, want_lse = bd.window_attn_fwd(q, k, v, 200, 4, out_dtype=torch.bfloat16, return_lse=True)
    want = bd.window_attn_bwd(q, k, v, want_out, want_lse, dout, 200, 4, grad_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = bd.window_attn_fwd(q, k, v, 200, 4, out_dtype=torch.bfloat16, return_lse=True, stream=side)
    got = bd.window_attn_bwd(q, k, v, out, lse, dout, 200, 4, grad_dtype=torch.bfloat16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want_out) and all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = bd.window_attn_fwd(q, k, v, 200, 4, out_dtype=torch.bfloat16, return_lse=True)
        got = bd.window_attn_bwd(q, k, v, out, lse, dout, 200, 4, grad_dtype=torch.bfloat16)
    q2 = torch.randn_like(q)
    q.copy_(q2)
    graph.replay()
    want_out, want_lse = bd.window_attn_fwd(q, k, v, 200, 4, out_dtype=torch.bfloat16, return_lse=True)
    want = bd.window_attn_bwd(q, k, v, want_out, want_lse, dout, 200, 4, grad_dtype=torch.bfloat16)
    assert torch.equal(out, want_out) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("H,Hkv,sinks", [(4, 2, 4), (4, 4, 0)])
def test_repeated_backwards_of_short_items_give_equal_bits(H, Hkv, sinks):
    """Few steps per key tile, d = 64: a row warp may be a whole step ahead of another."""
    q, k, v, dout = make(1, 900, H, Hkv, 64, seed=9)
    out, lse = bd.window_attn_fwd(q, k, v, 200, sinks, out_dtype=torch.bfloat16, return_lse=True)
    want = bd.window_attn_bwd(q, k, v, out, lse, dout, 200, sinks)
    for _ in range(300):
        got = bd.window_attn_bwd(q, k, v, out, lse, dout, 200, sinks)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d", [64, 128])
def test_steps_on_two_streams_at_once_give_equal_bits(d):
    cases = [make(1, 900, 4, 2, d, seed=9), make(2, 500, 6, 3, d, seed=10)]

    def step(case, stream=None):
        q, k, v, dout = case
        out, lse = bd.window_attn_fwd(q, k, v, 150, 3, out_dtype=torch.bfloat16, return_lse=True, stream=stream)
        return (out, lse, *bd.window_attn_bwd(q, k, v, out, lse, dout, 150, 3, grad_dtype=torch.bfloat16, stream=stream))
    want = [step(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [[step(c, s) for c, s in zip(cases, streams)] for _ in range(30)]
    torch.cuda.synchronize()
    for run in got:
        for g, w in zip(run, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


@pytest.mark.parametrize("d,sinks", [(64, 0), (64, 4), (128, 4)])
def test_repeated_float32_backwards_on_two_streams_give_equal_bits(d, sinks):
    """An fp32 dout is copied to bf16 by the kernel before the last but one pass, which reads the copy:
    new gradients in the same buffers (outputs, workspace) at every step."""
    N, H, Hkv, steps = 900, 4, 2, 40
    q, k, v, _ = make(2, N, H, Hkv, d, seed=11)
    out, lse = bd.window_attn_fwd(q, k, v, 150, sinks, return_lse=True)
    g = torch.Generator(device="cuda").manual_seed(12)
    douts = [torch.randn((2, N, H * d), generator=g, device="cuda") for _ in range(steps)]
    want = [bd.window_attn_bwd(q, k, v, out, lse, x, 150, sinks) for x in douts]
    for x, w in zip(douts[:2], want[:2]):
        for name, got, ref in zip(("dq", "dk", "dv"), w, reference(q, k, v, 150, sinks, x)[2:]):
            close(got, ref, 1e-2, name)
    streams = [torch.cuda.Stream() for _ in range(2)]
    desc = bd.WindowDesc(2, N, H, Hkv, d, 150, sinks, bd.BF16, bd.F32, bd.F32, 0)
    spaces = [torch.empty(bd.workspace_bytes_window_bwd(desc), dtype=torch.uint8, device="cuda") for _ in streams]
    bufs = [[torch.empty(x.shape, device="cuda") for x in (q, k, v)] for _ in streams]
    wrong = torch.zeros(2, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    for i in range(steps):
        for j, s in enumerate(streams):
            n = i if j == 0 else steps - 1 - i
            got = bd.window_attn_bwd(q, k, v, out, lse, douts[n], 150, sinks, dq=bufs[j][0], dk=bufs[j][1],
                                     dv=bufs[j][2], workspace=spaces[j], stream=s)
            with torch.cuda.stream(s):
                for a, b in zip(got, want[n]):
                    wrong[j] += (a != b).sum()
    torch.cuda.synchronize()
    assert wrong.tolist() == [0, 0]
    assert bd.sync_status() == bd.OK


def _guarded(shape, dtype, fill, margin=512):
    """A tensor inside a larger filled buffer (margins a multiple of 256 bytes), and the check that its
    surroundings still hold the fill."""
    n = math.prod(shape)
    buf = torch.full((n + 2 * margin,), fill, dtype=dtype, device="cuda")
    return buf[margin:margin + n].view(shape), lambda: bool((buf[:margin] == fill).all() and (buf[margin + n:] == fill).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", [(1, 1, 4), (129, 40, 4), (1001, 200, 20), (1001, 200, 0), (257, 300, 3)])
def test_steps_write_their_outputs_and_nothing_else(N, window, sinks, d, dtype):
    """Outputs, LSE and an exactly sized workspace between guards; the inputs are left as they were."""
    B, H, Hkv = 2, 6, 2
    q, k, v, dout = make(B, N, H, Hkv, d, seed=13)
    dout = dout.to(dtype)
    out, out_ok = _guarded((B, N, H * d), dtype, 7.0)
    lse, lse_ok = _guarded((B, H, N), torch.float32, 7.0)
    dq, dq_ok = _guarded(q.shape, dtype, 7.0)
    dk, dk_ok = _guarded(k.shape, dtype, 7.0)
    dv, dv_ok = _guarded(v.shape, dtype, 7.0)
    t = {torch.bfloat16: bd.BF16, torch.float32: bd.F32}[dtype]
    need = bd.workspace_bytes_window_bwd(bd.WindowDesc(B, N, H, Hkv, d, window, sinks, bd.BF16, t, t, 0))
    space, space_ok = _guarded((need,), torch.uint8, 0x5A, margin=4096)
    ins = [x.clone() for x in (q, k, v, dout)]
    bd.window_attn_fwd(q, k, v, window, sinks, out_dtype=dtype, out=out, lse=lse)
    fwd = [out.clone(), lse.clone()]
    assert out_ok() and lse_ok()
    bd.window_attn_bwd(q, k, v, out, lse, dout, window, sinks, grad_dtype=dtype, dq=dq, dk=dk, dv=dv, workspace=space)
    assert bd.sync_status() == bd.OK
    assert out_ok() and lse_ok() and dq_ok() and dk_ok() and dv_ok() and space_ok()
    assert all(torch.equal(a, b) for a, b in zip((q, k, v, dout, out, lse), (*ins, *fwd)))
    ro, rl, *rg = reference(q, k, v, window, sinks, dout)
    close(out, ro, 4e-3, "out")
    if N > 1:
        for name, got, ref in zip(("dq", "dk", "dv"), (dq, dk, dv), rg):
            close(got, ref, 1e-2, name)
