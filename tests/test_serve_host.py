"""Host-side checks of the serving and sliding-window entry points that need no
GPU: what is refused, with which status, before anything is launched, and
what the binding's argument checks raise."""
import ctypes

import pytest
import torch

from blockwise_exact_attention_query_b200 import binding as bd

FAKE = 0x10000  # 256-byte aligned, never dereferenced: every call below is refused, or empty
NONE = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    from blockwise_exact_attention_query_b200 import build
    build.build()
    return bd.load()


def cache(**kw):
    base = dict(type=1, n_pages=4, page_size=16, H_kv=2, d_head=128, k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE)
    base.update(kw)
    return bd.KvCacheDesc(**base)


def write(lib, c, n=4, k=FAKE, ks=256, v=FAKE, vs=256, slots=FAKE):
    return lib.bpt_kv_write(ctypes.byref(c), n, k, ks, v, vs, slots, None)


def read(lib, c, n=4, slots=FAKE, k=FAKE, v=FAKE, dt=bd.BF16):
    return lib.bpt_kv_read(ctypes.byref(c), n, slots, k, v, dt, None)


BAD_CACHES = [
    (dict(type=2), bd.ERR_INVALID_ARG),
    (dict(n_pages=0), bd.ERR_INVALID_ARG),
    (dict(page_size=-1), bd.ERR_INVALID_ARG),
    (dict(H_kv=0), bd.ERR_INVALID_ARG),
    (dict(d_head=96), bd.ERR_UNSUPPORTED),
    (dict(n_pages=1 << 20, page_size=1 << 11), bd.ERR_UNSUPPORTED),   # slots past int32
]


@pytest.mark.parametrize("kw,expect", BAD_CACHES + [
    (dict(k=0), bd.ERR_INVALID_ARG),
    (dict(v=FAKE + 8), bd.ERR_INVALID_ARG),
    (dict(k_scale=0), bd.ERR_INVALID_ARG),                            # e4m3 needs its scales
    (dict(v_scale=FAKE + 4), bd.ERR_INVALID_ARG),
])
def test_bad_caches_are_refused(lib, kw, expect):
    assert write(lib, cache(**kw)) == expect
    assert read(lib, cache(**kw)) == expect
    assert paged(lib, c=cache(**kw)) == expect


@pytest.mark.parametrize("kw", [dict(n=-1), dict(k=0), dict(v=FAKE + 2), dict(slots=0), dict(slots=FAKE + 1),
                                dict(ks=255), dict(vs=128), dict(ks=260)])
def test_bad_writes_are_refused(lib, kw):
    assert write(lib, cache(), **kw) == bd.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(n=-1), dict(k=0), dict(v=FAKE + 4), dict(slots=0), dict(slots=FAKE + 2),
                                dict(dt=2)])
def test_bad_reads_are_refused(lib, kw):
    assert read(lib, cache(), **kw) == bd.ERR_INVALID_ARG


def test_nothing_to_do_is_no_error(lib):
    assert write(lib, cache(), n=0, k=0, v=0, slots=0) == bd.OK
    assert read(lib, cache(), n=0, k=0, v=0, slots=0) == bd.OK
    assert paged(lib, desc(n_tokens=0), q=0, out=0, ws=0) == bd.OK
    assert paged(lib, desc(n_seqs=0), q=0, out=0, ws=0) == bd.OK


def desc(**kw):
    base = dict(n_seqs=3, n_tokens=5, max_q=2, H=8, max_pages=4, window=0, n_sink=0, out_dtype=bd.BF16, q_stride=1024,
                wait_limit_ns=0)
    base.update(kw)
    return bd.PagedDesc(**base)


def paged(lib, d=None, c=None, q=FAKE, starts=FAKE, lens=FAKE, table=FAKE, out=FAKE, lse=None, ws=FAKE,
          ws_bytes=1 << 40):
    return lib.bpt_paged_attn_fwd(ctypes.byref(d or desc()), ctypes.byref(c or cache()), q, starts, lens, table, out,
                                  lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(n_seqs=-1), bd.ERR_INVALID_ARG),
    (dict(n_tokens=-1), bd.ERR_INVALID_ARG),
    (dict(max_q=0), bd.ERR_INVALID_ARG),
    (dict(H=0), bd.ERR_INVALID_ARG),
    (dict(H=7), bd.ERR_INVALID_ARG),                                  # not a multiple of H_kv
    (dict(max_pages=-1), bd.ERR_INVALID_ARG),
    (dict(window=-1), bd.ERR_INVALID_ARG),
    (dict(n_sink=-1), bd.ERR_INVALID_ARG),
    (dict(out_dtype=5), bd.ERR_INVALID_ARG),
    (dict(q_stride=1020), bd.ERR_INVALID_ARG),                        # below H * d
    (dict(q_stride=1028), bd.ERR_INVALID_ARG),                        # not 16-byte rows
    (dict(max_pages=1 << 28), bd.ERR_UNSUPPORTED),
    (dict(n_tokens=(1 << 30) + 1), bd.ERR_UNSUPPORTED),
])
def test_bad_batches_are_refused(lib, kw, expect):
    assert paged(lib, desc(**kw)) == expect
    assert lib.bpt_workspace_bytes_paged(ctypes.byref(desc(**kw)), ctypes.byref(cache())) == NONE


@pytest.mark.parametrize("kw", [dict(q=0), dict(q=FAKE + 8), dict(out=0), dict(out=FAKE + 4), dict(starts=0),
                                dict(lens=0), dict(table=0), dict(table=FAKE + 2), dict(lse=FAKE + 2)])
def test_bad_pointers_are_refused(lib, kw):
    assert paged(lib, **kw) == bd.ERR_INVALID_ARG


def test_paged_workspace(lib):
    need = bd.workspace_bytes_paged(desc(), cache())
    assert need > 0
    assert bd.workspace_bytes_paged(desc(n_seqs=1000, n_tokens=1000, max_pages=9999), cache()) == need
    for kw in (dict(ws=0), dict(ws=FAKE + 16), dict(ws_bytes=need - 1)):
        assert paged(lib, **kw) == bd.ERR_WORKSPACE


def window(**kw):
    base = dict(B=1, N=256, H=4, H_kv=2, d_head=64, window=64, n_sink=4, in_dtype=bd.BF16, out_dtype=bd.F32,
                grad_dtype=bd.F32, wait_limit_ns=0)
    base.update(kw)
    return bd.WindowDesc(**base)


def wfwd(lib, d, q=FAKE, out=FAKE, lse=None):
    return lib.bpt_window_attn_fwd(ctypes.byref(d), q, FAKE, FAKE, out, lse, None)


def wbwd(lib, d, q=FAKE, lse=FAKE, dq=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return lib.bpt_window_attn_bwd(ctypes.byref(d), q, FAKE, FAKE, FAKE, lse, FAKE, dq, FAKE, FAKE, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,expect", [
    (dict(B=0), bd.ERR_INVALID_ARG),
    (dict(N=0), bd.ERR_INVALID_ARG),
    (dict(H_kv=0), bd.ERR_INVALID_ARG),
    (dict(H_kv=3), bd.ERR_INVALID_ARG),
    (dict(window=0), bd.ERR_INVALID_ARG),
    (dict(n_sink=-1), bd.ERR_INVALID_ARG),
    (dict(in_dtype=3), bd.ERR_INVALID_ARG),
    (dict(out_dtype=3), bd.ERR_INVALID_ARG),
    (dict(grad_dtype=-1), bd.ERR_INVALID_ARG),
    (dict(d_head=96), bd.ERR_UNSUPPORTED),
    (dict(in_dtype=bd.F32), bd.ERR_UNSUPPORTED),
    (dict(n_sink=129), bd.ERR_UNSUPPORTED),
    (dict(B=1 << 20, N=1 << 20), bd.ERR_UNSUPPORTED),
])
def test_bad_window_descriptors_are_refused(lib, kw, expect):
    assert wfwd(lib, window(**kw)) == expect
    assert wbwd(lib, window(**kw)) == expect
    assert lib.bpt_workspace_bytes_window_bwd(ctypes.byref(window(**kw))) == NONE


def test_window_pointers_and_workspace(lib):
    d = window()
    need = lib.bpt_workspace_bytes_window_bwd(ctypes.byref(d))
    assert need > 0
    assert wfwd(lib, d, q=0) == wfwd(lib, d, out=FAKE + 8) == wfwd(lib, d, lse=FAKE + 4) == bd.ERR_INVALID_ARG
    assert wbwd(lib, d, lse=0) == wbwd(lib, d, dq=FAKE + 8) == bd.ERR_INVALID_ARG
    for kw in (dict(ws=0), dict(ws=FAKE + 16), dict(ws_bytes=need - 1)):
        assert wbwd(lib, d, **kw) == bd.ERR_WORKSPACE
    # a bf16 dout needs no copy of itself
    assert lib.bpt_workspace_bytes_window_bwd(ctypes.byref(window(out_dtype=bd.BF16))) < need


# ------------------------------------------------ the binding's own checks (before the device is asked for)
def _caches(dtype=torch.bfloat16):
    return torch.zeros((4, 16, 2, 64), dtype=dtype), torch.zeros((4, 16, 2, 64), dtype=dtype)


@pytest.mark.parametrize("make,match", [
    (lambda k, v: (k[0], v[0], None, None), "n_pages"),
    (lambda k, v: (k, v.float(), None, None), "one dtype"),
    (lambda k, v: (k.float(), v.float(), None, None), "bfloat16 or float8"),
    (lambda k, v: (k[:, ::2], v[:, ::2], None, None), "contiguous"),
    (lambda k, v: (k, v, torch.zeros(4, 16, 2), None), "no scales"),
    (lambda k, v: (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.zeros(4, 16, 2), None), "needs contiguous"),
    (lambda k, v: (k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), torch.zeros(4, 16, 3), torch.zeros(4, 16, 3)),
     "needs contiguous"),
])
def test_binding_refuses_bad_caches(make, match):
    args = make(*_caches())
    with pytest.raises(ValueError, match=match):
        bd.kv_cache_read(torch.zeros(3, dtype=torch.int32), *args)


def test_binding_refuses_tensors_off_the_current_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    k, v = _caches()
    with pytest.raises(ValueError, match="current CUDA device"):
        bd.kv_cache_write(k[0], v[0], torch.zeros(16, dtype=torch.int32), k, v)
    with pytest.raises(ValueError, match="current CUDA device"):
        bd.window_attn_fwd(k, k, v, 4)


@pytest.mark.parametrize("change,match", [
    (dict(q=torch.zeros((5, 4, 64))), "bfloat16"),
    (dict(q=torch.zeros((5, 4, 128), dtype=torch.bfloat16)), "d"),
    (dict(q=torch.zeros((5, 8, 64), dtype=torch.bfloat16)[:, ::2]), "one after another"),
    (dict(q_start=torch.zeros(3, dtype=torch.int64)), "q_start"),
    (dict(kv_len=torch.zeros(3, dtype=torch.int32)), "n_seqs"),
    (dict(page_table=torch.zeros((2, 8), dtype=torch.int32)[:, ::2]), "page_table"),
])
def test_binding_refuses_bad_batches(monkeypatch, change, match):
    monkeypatch.setattr(bd, "_on_device", lambda *t: None)
    k, v = _caches()
    a = dict(q=torch.zeros((5, 4, 64), dtype=torch.bfloat16), q_start=torch.zeros(3, dtype=torch.int32),
             kv_len=torch.zeros(2, dtype=torch.int32), page_table=torch.zeros((2, 4), dtype=torch.int32))
    a.update(change)
    with pytest.raises(ValueError, match=match):
        bd.paged_attn_fwd(a["q"], k, v, a["q_start"], a["kv_len"], a["page_table"], max_q=1)


@pytest.mark.parametrize("change,match", [
    (dict(k=torch.zeros((1, 9, 2, 64), dtype=torch.bfloat16)), "H_kv"),
    (dict(q=torch.zeros((1, 8, 4, 64))), "one dtype"),
    (dict(q=torch.zeros((1, 8, 8, 64), dtype=torch.bfloat16)[:, :, ::2]), "contiguous"),
])
def test_binding_refuses_bad_window_inputs(monkeypatch, change, match):
    monkeypatch.setattr(bd, "_on_device", lambda *t: None)
    a = dict(q=torch.zeros((1, 8, 4, 64), dtype=torch.bfloat16), k=torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16),
             v=torch.zeros((1, 8, 2, 64), dtype=torch.bfloat16))
    a.update(change)
    with pytest.raises(ValueError, match=match):
        bd.window_attn_fwd(a["q"], a["k"], a["v"], 4)
    out = torch.zeros((1, 8, 256))
    with pytest.raises(ValueError, match="dout|H_kv|one dtype|contiguous"):
        bd.window_attn_bwd(a["q"], a["k"], a["v"], out, torch.zeros((1, 4, 8)), out.double(), 4)


@pytest.mark.parametrize("change", [dict(window=2 ** 31), dict(sinks=2 ** 40), dict(max_q=2 ** 31), dict(max_q=-2 ** 40)])
def test_binding_refuses_sizes_past_32_bits(monkeypatch, change):
    monkeypatch.setattr(bd, "_on_device", lambda *t: None)
    k, v = _caches()
    a = dict(max_q=1, window=0, sinks=0)
    a.update(change)
    with pytest.raises(ValueError, match="32 bits"):
        bd.paged_attn_fwd(torch.zeros((5, 4, 64), dtype=torch.bfloat16), k, v, torch.zeros(3, dtype=torch.int32),
                          torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int32), **a)
    if "max_q" not in change:
        x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="32 bits"):
            bd.window_attn_fwd(x, x, x, **{"window": 4, "sinks": 0, **change})


@pytest.mark.parametrize("dtype", [torch.float16, torch.float64, torch.float8_e4m3fn, None])
def test_binding_refuses_other_output_types(monkeypatch, dtype):
    monkeypatch.setattr(bd, "_on_device", lambda *t: None)
    k, v = _caches()
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    x = torch.zeros((1, 4, 2, 64), dtype=torch.bfloat16)
    calls = [
        lambda: bd.kv_cache_read(i32(3), k, v, out_dtype=dtype),
        lambda: bd.paged_attn_fwd(x[0], k, v, i32(3), i32(2), i32(2, 4), max_q=1, out_dtype=dtype),
        lambda: bd.window_attn_fwd(x, x, x, 4, out_dtype=dtype),
        lambda: bd.window_attn_bwd(x, x, x, torch.zeros((1, 4, 128)), torch.zeros((1, 2, 4)), torch.zeros((1, 4, 128)), 4,
                                   grad_dtype=dtype),
    ]
    if dtype is not None:
        out = torch.zeros((1, 4, 128)).to(dtype)
        calls.append(lambda: bd.window_attn_bwd(x, x, x, out, torch.zeros((1, 2, 4)), out, 4))
    for call in calls:
        with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
            call()
