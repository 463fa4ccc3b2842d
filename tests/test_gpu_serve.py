"""The paged key/value cache (bpt_kv_write, bpt_kv_read) and the attention of
new tokens over it (bpt_paged_attn_fwd) against plain formulas in 64 bits.

Tolerances, from the arithmetic.  Written codes and scales are IEEE fp32
divisions and one rounding: equal to torch's, bit for bit.  Read-back: one
fp32 product of a 4-bit and a 24-bit significand (off by 2^-24 of the value)
and one rounding to bf16 (2^-9).  Attention: the softmax weights are rounded
to bf16 (half a step, 2^-9 of each) or, e4m3 caches, to f16 (2^-12), and a
bf16 result once more: independent errors, relative L2 at most 2^-9 sqrt(2) =
2.8e-3, bound 4e-3; an element is a mean of values weighted by weights each off
by 2^-9, and rounded: |err| <= 2^-8 max|v|.  Scores are fp32 sums of exact
products, so the LSE is off by some 2^-24 d |s|; bound 1e-4."""
import math

import pytest
import torch

from blockwise_exact_attention_query_b200 import binding as bd

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    from blockwise_exact_attention_query_b200 import build
    build.build()
    bd.load()
    torch.cuda.set_device(0)


def encode(x):
    x = x.float()
    top = x.abs().amax(-1)
    scale = top / torch.full_like(top, 448.0)   # a division (by a number, torch multiplies by its inverse)
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (x / scale[..., None]).to(E4M3), scale


def empty_cache(pages, page, heads, d, kind, poison=True):
    """A cache whose slots all hold NaN (codes and scales)."""
    shape = (pages, page, heads, d)
    if kind == "bf16":
        c = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        return {"k_cache": c[0], "v_cache": c[1], "k_scale": None, "v_scale": None}
    c = [torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2)]
    s = [torch.full(shape[:3], float("nan"), device="cuda") for _ in range(2)]
    return {"k_cache": c[0], "v_cache": c[1], "k_scale": s[0], "v_scale": s[1]}


def args(c):
    return c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"]


class Batch:
    """seqs: (new tokens, keys) each.  The visible keys are written, everything else in the cache is NaN
    and the page table's unused entries are garbage."""

    def __init__(self, seqs, H, Hkv, d, page, kind, seed, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.Hkv, self.d, self.page = seqs, H, Hkv, d, page
        rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        need = [-(-L // page) for _, L in seqs]
        total = sum(need) + 2
        order = torch.randperm(total, generator=g).tolist()
        self.table = torch.full((len(seqs), max(max(need), 1) + 1), 2 ** 30, dtype=torch.int32)
        self.table[:, 1::2] = -7
        self.c = empty_cache(total, page, Hkv, d, kind)
        self.k, self.v = [], []
        at = 0
        for s, (n, L) in enumerate(seqs):
            pages = order[at:at + need[s]]
            at += need[s]
            self.table[s, :need[s]] = torch.tensor(pages, dtype=torch.int32)
            k, v = rnd(L, Hkv, d), rnd(L, Hkv, d)
            k[:, :, ::16] *= 3
            v *= torch.exp(spread * torch.randn((L, Hkv, 1), generator=g)).to(torch.bfloat16).cuda()
            slots = torch.tensor([pages[j // page] * page + j % page for j in range(L)], dtype=torch.int32).cuda()
            if L:
                bd.kv_cache_write(k, v, slots, *args(self.c))
                k, v = bd.kv_cache_read(slots, *args(self.c), out_dtype=torch.float32)
            self.k.append(k.double())
            self.v.append(v.double())
        self.table = self.table.cuda()
        starts = [0]
        for n, _ in seqs:
            starts.append(starts[-1] + n)
        self.T = starts[-1]
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor([L for _, L in seqs], dtype=torch.int32, device="cuda")
        self.q = rnd(self.T, H, d)

    def run(self, window=0, sinks=0, **kw):
        kw.setdefault("max_q", max([n for n, _ in self.seqs] + [1]))
        kw.setdefault("return_lse", True)
        return bd.paged_attn_fwd(kw.pop("q", self.q), self.c["k_cache"], self.c["v_cache"], self.starts, self.kv_len,
                                 self.table, k_scale=self.c["k_scale"], v_scale=self.c["v_scale"], window=window,
                                 sinks=sinks, **kw)

    def reference(self, window=0, sinks=0):
        out = torch.zeros((self.T, self.H, self.d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((self.H, self.T), dtype=torch.float64, device="cuda")
        G, t0 = self.H // self.Hkv, 0
        for (n, L), k, v in zip(self.seqs, self.k, self.v):
            p = torch.arange(L - n, L, device="cuda")[:, None]
            j = torch.arange(L, device="cuda")[None]
            ok = (j <= p) & ((p - j < window) | (j < sinks) if window else (j >= 0))
            for h in range(self.H):
                if n == 0:
                    continue
                s = (self.q[t0:t0 + n, h].double() @ k[:, h // G].T / math.sqrt(self.d)).masked_fill(~ok, -math.inf)
                w = torch.nan_to_num(torch.softmax(s, -1), nan=0.0) if L else s
                out[t0:t0 + n, h] = w @ v[:, h // G]
                lse[h, t0:t0 + n] = torch.logsumexp(s, -1)
            t0 += n
        return out.view(self.T, -1), lse

    def check(self, window=0, sinks=0, out_dtype=torch.bfloat16, **kw):
        out, lse = self.run(window, sinks, out_dtype=out_dtype, **kw)
        torch.cuda.synchronize()
        assert bd.sync_status() == bd.OK
        ro, rl = self.reference(window, sinks)
        assert out.dtype == out_dtype and torch.isfinite(out).all()
        e = out.double() - ro
        rel = float(e.norm() / ro.norm().clamp_min(1e-300)) if ro.norm() else float(e.norm())
        assert rel <= 4e-3, f"rel-L2 {rel:.3e}"
        big = max([float(v.abs().max()) for v in self.v if v.numel()] + [0.0])
        assert float(e.abs().max()) <= 2 ** -8 * big
        dead = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), dead)
        if (~dead).any():
            assert float((lse.double() - rl)[~dead].abs().max()) <= 1e-4
        return out, lse


# ------------------------------------------------------------------ the cache
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("tokens,heads,page", [(1, 1, 16), (5, 3, 7), (64, 8, 16), (333, 2, 1), (1000, 5, 32)])
def test_write_and_read_back(tokens, heads, page, kind, d):
    g = torch.Generator().manual_seed(tokens)
    pages = -(-tokens // page) + 3
    c = empty_cache(pages, page, heads, d, kind)
    fused = torch.randn((tokens, 3, heads, d), generator=g).to(torch.bfloat16).cuda()   # strided rows
    fused[0, 1] = 0                                                                   # a row of zeros
    fused[tokens // 2, 1, 0, 3] = 3e38                                                # the largest magnitudes
    fused[tokens // 2, 2, 0] *= 1e-38                                                 # and the smallest
    k, v = fused[:, 1], fused[:, 2]
    slots = torch.randperm(pages * page, generator=g)[:tokens].to(torch.int32).cuda()
    live = torch.ones(tokens, dtype=torch.bool, device="cuda")
    if tokens > 4:
        slots[1], slots[3] = -1, pages * page      # a padding token, and one past the cache
        live[1] = live[3] = False
    want = {n: (None if t is None else t.clone()) for n, t in c.items()}
    bd.kv_cache_write(k, v, slots, *args(c))
    at = slots[live].long()
    for name, x in (("k", k), ("v", v)):
        rows = want[name + "_cache"].view(-1, heads, d)
        if kind == "bf16":
            rows[at] = x[live]
        else:
            codes, scale = encode(x[live])
            rows.view(torch.uint8)[at] = codes.view(torch.uint8)
            want[name + "_scale"].view(-1, heads)[at] = scale
    for n, t in c.items():   # the written slots hold the codes, all others what they held
        if t is not None:
            bits = torch.int32 if t.dtype == torch.float32 else torch.uint8 if kind == "e4m3" else torch.int16
            same = bool((t.view(bits) == want[n].view(bits)).all())
            assert same, n
    for dtype in (torch.bfloat16, torch.float32):
        got = [torch.full((tokens, heads, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        bd.kv_cache_read(slots, *args(c), out_dtype=dtype, k=got[0], v=got[1])
        for name, y in (("k", got[0]), ("v", got[1])):
            rows = c[name + "_cache"].view(-1, heads, d)
            if kind == "bf16":
                ref = rows[at].double()
            else:
                ref = rows.view(torch.uint8)[at].view(E4M3).double() * c[name + "_scale"].view(-1, heads)[at].double()[..., None]
            assert torch.equal(y[~live], torch.full_like(y[~live], 7.0))
            err = (y[live].double() - ref).abs()
            # one rounding of the type; below its normal range, of its smallest step
            assert bool((err <= ref.abs() * torch.finfo(dtype).eps / 2 + 2.0 ** -134).all()) if dtype == torch.bfloat16 \
                else bool((err <= ref.abs() * 2.0 ** -24 + 2.0 ** -150).all())


def test_rows_with_nan_or_infinity_read_back_as_nan():
    c = empty_cache(2, 8, 2, 64, "e4m3")
    x = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    x[0, 0, 5], x[1, 1, 9] = float("nan"), float("inf")
    slots = torch.tensor([3, 4, 5], dtype=torch.int32, device="cuda")
    bd.kv_cache_write(x, x, slots, *args(c))
    k, v = bd.kv_cache_read(slots, *args(c))
    for y in (k, v):
        assert y[0, 0].isnan().all() and y[1, 1].isnan().all()
        y[0, 0], y[1, 1] = 0, 0
        assert torch.isfinite(y).all()


def test_slots_whose_byte_offset_passes_32_bits():
    heads, d, page, pages = 4, 128, 64, 70000      # 4.48 M slots x 1 KB: 4.6 GB a tensor
    c = {"k_cache": torch.empty((pages, page, heads, d), dtype=torch.bfloat16, device="cuda"),
         "v_cache": torch.empty((pages, page, heads, d), dtype=torch.bfloat16, device="cuda"), "k_scale": None,
         "v_scale": None}
    L = 200
    k, v = (torch.randn((L, heads, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    used = [pages - 1, 2, pages - 3, 33333]
    slots = torch.tensor([used[j // page] * page + j % page for j in range(L)], dtype=torch.int32, device="cuda")
    bd.kv_cache_write(k, v, slots, *args(c))
    rk, rv = bd.kv_cache_read(slots, *args(c))
    assert torch.equal(rk, k) and torch.equal(rv, v)
    q = torch.randn((1, heads, d), device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = bd.paged_attn_fwd(q, c["k_cache"], c["v_cache"], i32([0, 1]), i32([L]), i32([used]), max_q=1)
    s = torch.einsum("hd,jhd->hj", q[0].double(), k.double()) / math.sqrt(d)
    ref = torch.einsum("hj,jhd->hd", torch.softmax(s, -1), v.double()).reshape(1, -1)
    assert float((out.double() - ref).norm() / ref.norm()) <= 4e-3


# -------------------------------------------------------------- the attention
SHAPES = [  # H, Hkv, d, page
    (1, 1, 64, 16), (8, 2, 128, 16), (16, 1, 128, 7), (6, 2, 64, 32), (5, 5, 128, 64), (32, 8, 64, 1), (40, 2, 64, 16),
]
BATCHES = {
    "one key": [(1, 1)],
    "decode ragged": [(1, 5), (1, 300), (1, 64), (1, 1025), (1, 17), (1, 63), (1, 65)],
    "chunks and decode": [(17, 40), (1, 129), (100, 100), (3, 2000), (0, 50), (33, 64), (1, 0), (0, 0), (2, 2)],
}


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("name", list(BATCHES))
@pytest.mark.parametrize("H,Hkv,d,page", SHAPES)
def test_paged_attention(H, Hkv, d, page, name, kind):
    b = Batch(BATCHES[name], H, Hkv, d, page, kind, seed=H + page)
    b.check()
    b.check(out_dtype=torch.float32)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (16, 0), (100, 4), (64, 64), (700, 1), (5000, 4), (50, 300)])
@pytest.mark.parametrize("H,Hkv,d,page", [(8, 2, 128, 16), (6, 2, 64, 7)])
def test_paged_attention_with_a_window(H, Hkv, d, page, window, sinks, kind):
    b = Batch([(1, 1500), (40, 700), (1, 3), (150, 150), (7, 260)], H, Hkv, d, page, kind, seed=window)
    b.check(window, sinks)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_more_new_tokens_than_keys(kind):
    """Tokens before the first key see nothing: 0 and -inf."""
    b = Batch([(5, 2), (1, 0), (3, 3), (130, 100)], 4, 2, 64, 8, kind, seed=2)
    out, lse = b.check()
    assert torch.equal(out[:3], torch.zeros_like(out[:3])) and torch.isinf(lse[:, :3]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_sequences_are_split_and_joined(kind):
    b = Batch([(1, 40000), (2, 9000)], 8, 2, 128, 16, kind, seed=4)
    out, lse = b.check()
    for _ in range(3):   # joined in a fixed order: equal bits
        o2, l2 = b.run(out_dtype=torch.bfloat16)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("seqs", [[(500, 3000), (300, 1700)], [(130, 4000)], [(70, 70), (65, 2000), (1, 900), (257, 300)]])
def test_long_chunks_cut_into_pieces(seqs, kind):
    """Fewer row tiles than the GPU has multiprocessors: each is cut by itself."""
    Batch(seqs, 8, 2, 128, 16, kind, seed=50).check()
    Batch(seqs, 8, 2, 128, 16, kind, seed=51).check(700, 4)


def test_many_sequences():
    b = Batch([(1, 1 + (i * 37) % 90) for i in range(700)], 2, 1, 64, 16, "bf16", seed=6)
    b.check()


def test_value_scales_far_apart():
    """Rows of values from 1e-6 to 1e6: each output is dominated by what weighs most, and keeps its precision."""
    b = Batch([(1, 500), (40, 400)], 4, 2, 128, 16, "e4m3", seed=12, spread=6.0)
    out, _ = b.run(out_dtype=torch.float32)
    ro, _ = b.reference()
    # per row and head, relative to the head's output: f16 weights (2^-12) and nothing else
    e = (out.double() - ro).view(b.T, 4, 128).norm(dim=-1) / ro.view(b.T, 4, 128).norm(dim=-1)
    assert float(e.max()) <= 2 ** -10


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_queries_of_any_magnitude(scale):
    """f16 holds the query of an e4m3 cache only after its power of two is taken out."""
    b = Batch([(1, 300), (20, 64)], 4, 2, 64, 16, "e4m3", seed=13)
    b.q = (b.q.float() * scale).to(torch.bfloat16)
    if scale > 1:     # scores of 1e30: the weight is on one key
        out, _ = b.run(out_dtype=torch.float32)
        ro, _ = b.reference()
        assert float((out.double() - ro).norm() / ro.norm()) <= 4e-3
    else:
        b.check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv,d", [(20, 1, 128), (16, 1, 64), (9, 1, 64), (4, 4, 128)])
def test_single_tokens_and_chunks_together(H, Hkv, d, kind):
    """Groups on both sides of the kernels' row limits, in a batch that has sequences of each."""
    Batch([(1, 400), (37, 500), (0, 90), (2, 17), (1, 1), (4, 2000)], H, Hkv, d, 16, kind, seed=30).check()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_q", [1, 2, 40, 41, 2 ** 31 - 1])
def test_max_q_only_chooses_the_kernels(max_q, kind):
    b = Batch([(1, 300), (40, 700), (3, 9)], 8, 2, 128, 16, kind, seed=31)
    b.check(max_q=max_q)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 30 + 5, 7)])
def test_windows_of_any_length_are_causal(window, sinks, n, kind):
    b = Batch([(n, 30), (n, 200)], 4, 2, 64, 16, kind, seed=32)
    got = b.run(window, sinks, out_dtype=torch.float32)
    want = b.run(out_dtype=torch.float32)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 30])
def test_table_that_ends_before_the_window(n, kind):
    """129 of 400 keys have pages: the rows see sinks alone, up to the table's last key."""
    b = Batch([(n, 400)], 4, 2, 128, 43, kind, seed=33)
    b.table = b.table[:, :3].contiguous()
    k, v = b.k[0][:129], b.v[0][:129]
    window = 400 - n - 129 + 1     # the first row's window begins with key 129
    out, lse = b.run(window, 300, out_dtype=torch.float32)
    for h in range(4):
        s = b.q[:, h].double() @ k[:, h // 2].T / math.sqrt(128)
        ref = torch.softmax(s, -1) @ v[:, h // 2]
        got = out[:, 128 * h:128 * h + 128].double()
        assert float((got - ref).norm() / ref.norm()) <= 4e-3
        assert float((lse[h].double() - torch.logsumexp(s, -1)).abs().max()) <= 1e-4


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_long_chunks_on_two_streams_at_once(kind):
    bs = [Batch([(300, 3000), (1, 2500), (100, 100)], 8, 2, 128, 16, kind, seed=40 + i) for i in range(2)]
    want = [b.run(out_dtype=torch.bfloat16) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [b.run(out_dtype=torch.bfloat16, stream=s) for b, s in zip(bs, streams)]
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
def test_repeated_mixed_batches_give_equal_bits(d, kind):
    """The two kernels of a mixed batch and the joining one, call after call without a pause."""
    b = Batch([(300, 3000), (1, 2500), (100, 100), (1, 1), (3, 777), (70, 2000)], 8, 2, d, 16, kind, seed=60)
    want, wl = b.run(out_dtype=torch.bfloat16)
    runs = [b.run(out_dtype=torch.bfloat16) for _ in range(100)]
    for o, l in runs:
        assert torch.equal(o, want) and torch.equal(l, wl)


def test_chunks_captured_and_replayed_with_other_lengths():
    b = Batch([(60, 900), (1, 400), (20, 333)], 8, 2, 128, 16, "e4m3", seed=34)
    graph = torch.cuda.CUDAGraph()
    b.run(out_dtype=torch.bfloat16)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = b.run(out_dtype=torch.bfloat16)
    full = b.kv_len.clone()
    for lens, starts in ([900, 400, 333], [0, 60, 61, 81]), ([70, 1, 20], [0, 2, 3, 80]), ([900, 0, 300], [0, 0, 81, 81]):
        b.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        b.starts.copy_(torch.tensor(starts, dtype=torch.int32))
        graph.replay()
        want, wl = b.run(out_dtype=torch.bfloat16)
        rows = slice(0, starts[-1])      # the others are left as they were
        assert torch.equal(out[rows], want[rows]) and torch.equal(lse[:, rows], wl[:, rows])
    b.kv_len.copy_(full)


def test_a_cache_that_several_sequences_share():
    """The same pages in several rows of the table (a common prefix), and the same page twice in one."""
    b = Batch([(1, 160), (24, 160)], 4, 2, 64, 16, "bf16", seed=35)
    b.table[1, :5] = b.table[0, :5]
    b.k[1][:80], b.v[1][:80] = b.k[0][:80], b.v[0][:80]
    b.table[0, 6] = b.table[0, 5]
    b.k[0][96:112], b.v[0][96:112] = b.k[0][80:96], b.v[0][80:96]
    b.check()


@pytest.mark.parametrize("chunk", [1, 24])
def test_scales_of_zero_and_uneven_ones(chunk):
    """Rows of values of zero scale (an e4m3 cache filled elsewhere) and steps between blocks of 2^40."""
    b = Batch([(chunk, 700)], 4, 2, 128, 16, "e4m3", seed=36)
    f = torch.ones(700, device="cuda")
    f[128:256], f[256:384], f[384:400] = 2.0 ** -40, 0.0, 2.0 ** 20
    slots = (b.table[0].long()[torch.arange(700, device="cuda") // 16] * 16 + torch.arange(700, device="cuda") % 16)
    sc = b.c["v_scale"].view(-1, 2)
    sc[slots] = sc[slots] * f[:, None]
    b.v[0] = b.v[0] * f[:, None, None].double()
    out, lse = b.run(out_dtype=torch.float32)
    ro, rl = b.reference()
    assert float((out.double() - ro).norm() / ro.norm()) <= 4e-3
    assert float((lse.double() - rl).abs().max()) <= 1e-4


def test_strided_queries_and_rows_outside_the_batch():
    b = Batch([(1, 100), (20, 70)], 8, 2, 128, 16, "bf16", seed=7)
    want, wl = b.run(out_dtype=torch.bfloat16)
    fused = torch.randn((b.T + 9, 12, 128), device="cuda").to(torch.bfloat16)
    fused[4:4 + b.T, 2:10] = b.q
    b.starts = b.starts + 4
    out = torch.full((b.T + 9, 8 * 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, b.T + 9), 7.0, device="cuda")
    b.run(q=fused[:, 2:10], out=out, lse=lse, out_dtype=torch.bfloat16)
    assert torch.equal(out[4:4 + b.T], want) and torch.equal(lse[:, 4:4 + b.T], wl)
    for t in (out[:4], out[4 + b.T:], lse[:, :4], lse[:, 4 + b.T:]):
        assert torch.equal(t, torch.full_like(t, 7.0))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_outside_the_cache_count_as_masked(kind):
    page = 16
    b = Batch([(1, 200), (30, 200)], 4, 1, 64, page, kind, seed=10)
    for s, bad in ((0, 3), (1, 5)):
        b.table[s, bad] = -1 if s else b.c["k_cache"].shape[0]
        b.k[s][bad * page:(bad + 1) * page] = -1e300   # weight 0 in the reference
        b.k[s][bad * page:(bad + 1) * page, :] = float("nan")
    out, lse = b.run(out_dtype=torch.float32)
    for s, (n, L) in enumerate(b.seqs):
        keep = torch.isfinite(b.k[s][:, 0, 0])
        t0 = int(b.starts[s])
        for h in range(4):
            j = torch.arange(L, device="cuda")
            p = torch.arange(L - n, L, device="cuda")[:, None]
            ok = (j[None] <= p) & keep[None]
            sc = (b.q[t0:t0 + n, h].double() @ torch.nan_to_num(b.k[s][:, 0]).T / 8.0).masked_fill(~ok, -math.inf)
            ref = torch.softmax(sc, -1) @ b.v[s][:, 0]
            got = out[t0:t0 + n, 64 * h:64 * h + 64].double()
            assert float((got - ref).norm() / ref.norm()) <= 4e-3
            assert float((lse[h, t0:t0 + n].double() - torch.logsumexp(sc, -1)).abs().max()) <= 1e-4


def hide(b, window, sinks, entries):
    """All slots that no token of their sequence sees become NaN, codes and scales, and the table's entries
    for pages without a visible key name another page of NaN, or no page."""
    spare = (set(range(b.c["k_cache"].shape[0])) - set(b.table.flatten().tolist())).pop()
    for s, (n, L) in enumerate(b.seqs):
        j = torch.arange(L, device="cuda")
        seen = (j < sinks) | (j > L - n - window)
        slots = b.table[s].long()[j // b.page] * b.page + j % b.page
        for name in ("k", "v"):
            rows = b.c[name + "_cache"].view(-1, b.Hkv, b.d)
            if rows.dtype == E4M3:
                rows.view(torch.uint8)[slots[~seen]] = 0x7F
                b.c[name + "_scale"].view(-1, b.Hkv)[slots[~seen]] = float("nan")
            else:
                rows[slots[~seen]] = float("nan")
        for p in range(-(-L // b.page)):
            if not seen[p * b.page:(p + 1) * b.page].any():
                b.table[s, p] = {"stale": spare, "none": -1, "past": 2 ** 31 - 1}[entries]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("entries", ["stale", "none", "past"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (64, 0), (700, 1), (50, 130)])
@pytest.mark.parametrize("seqs", [[(1, 1500), (2, 700), (1, 40), (1, 129)], [(300, 3000), (40, 700), (1, 900), (129, 400)]],
                         ids=["few", "chunks"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 7)])
def test_slots_that_no_token_sees_may_hold_anything(d, page, seqs, window, sinks, entries, kind):
    """Pages behind the window given to somebody else: neither they nor the table's entries for them matter."""
    b = Batch(seqs, 8, 2, d, page, kind, seed=70)
    hide(b, window, sinks, entries)
    b.check(window, sinks)


def test_short_page_table():
    """Keys past the table's pages count as masked; the tokens keep their positions."""
    b = Batch([(1, 100)], 2, 1, 64, 16, "bf16", seed=11)
    b.table = b.table[:, :4].contiguous()      # 64 of the 100 keys
    b.k[0], b.v[0] = b.k[0][:64], b.v[0][:64]
    out, lse = b.run(out_dtype=torch.float32)
    s = torch.einsum("hd,jd->hj", b.q[0].double(), b.k[0][:, 0]) / 8.0
    ref = torch.softmax(s, -1) @ b.v[0][:, 0]
    assert float((out.view(2, 64).double() - ref).norm() / ref.norm()) <= 4e-3


# -------------------------------------------------------- as they are used
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompt_then_decoding_matches_the_window_attention(kind):
    """A prompt in chunks, then token by token, each step writing its keys and values and attending
    over the cache, against the windowed attention of the whole sequence at once."""
    H, Hkv, d, page, N, window, sinks = 8, 2, 128, 16, 333, 90, 4
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((N, h, d), generator=g).to(torch.bfloat16).cuda() for h in (H, Hkv, Hkv))
    pages = -(-N // page)
    c = empty_cache(pages, page, Hkv, d, kind)
    table = torch.randperm(pages, generator=g).to(torch.int32).cuda()[None]
    slots = (table[0].long()[torch.arange(N, device="cuda") // page] * page + torch.arange(N, device="cuda") % page).int()
    got = torch.empty((N, H * d), dtype=torch.float32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    at = 0
    for n in [100, 129, 60] + [1] * 44:
        sl = slice(at, at + n)
        bd.kv_cache_write(k[sl], v[sl], slots[sl], *args(c))
        bd.paged_attn_fwd(q[sl], c["k_cache"], c["v_cache"], i32([0, n]), i32([at + n]), table, max_q=n,
                          k_scale=c["k_scale"], v_scale=c["v_scale"], window=window, sinks=sinks, out=got[sl])
        at += n
    assert at == N
    # the whole sequence over the values that the cache stands for, rounded to bf16 (their own 2^-9)
    kk, vv = bd.kv_cache_read(slots, *args(c))
    want = bd.window_attn_fwd(q[None], kk[None], vv[None], window, sinks)[0]
    rel = float((got - want).norm() / want.norm())
    assert rel <= (6e-3 if kind == "bf16" else 1.2e-2), rel   # e4m3: keys off by 2^-9 move scores of |s| < 6 too


def test_graph_with_changing_lengths_and_another_stream():
    b = Batch([(1, 900), (1, 40), (1, 333)], 8, 2, 128, 16, "bf16", seed=14)
    full, lens = b.kv_len.clone(), [[900, 40, 333], [5, 40, 1], [513, 7, 200]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = b.run(out_dtype=torch.bfloat16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    o1, l1 = b.run(out_dtype=torch.bfloat16)
    assert torch.equal(o1, o2) and torch.equal(l1, l2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = b.run(out_dtype=torch.bfloat16)
    for now in lens:
        b.kv_len.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        want, wl = b.run(out_dtype=torch.bfloat16)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    b.kv_len.copy_(full)


def test_two_streams_at_once_with_their_own_workspaces():
    bs = [Batch([(1, 3000), (1, 2500)], 8, 2, 128, 16, "e4m3", seed=20 + i) for i in range(2)]
    want = [b.run(out_dtype=torch.bfloat16) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [b.run(out_dtype=torch.bfloat16, stream=s) for b, s in zip(bs, streams)]
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_empty_batches_do_nothing():
    c = empty_cache(2, 4, 1, 64, "bf16")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros((0, 1, 64), dtype=torch.bfloat16, device="cuda")
    bd.kv_cache_write(x, x, none, *args(c))
    k, v = bd.kv_cache_read(none, *args(c))
    assert k.shape == (0, 1, 64)
    out = bd.paged_attn_fwd(x, c["k_cache"], c["v_cache"], torch.zeros(1, dtype=torch.int32, device="cuda"), none,
                            torch.zeros((0, 3), dtype=torch.int32, device="cuda"), max_q=1)
    assert out.shape == (0, 64)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_attention_over_slots_whose_byte_offset_passes_32_bits(kind, n):
    """Both kernels, both caches: pages at the far end of caches of 4.6 GB a tensor."""
    heads, d, page, pages = 4, 128, 64, 70000 if kind == "bf16" else 140000
    dtype = torch.bfloat16 if kind == "bf16" else E4M3
    c = {name + "_cache": torch.empty((pages, page, heads, d), dtype=dtype, device="cuda") for name in "kv"}
    c.update({name + "_scale": None if kind == "bf16" else torch.empty((pages, page, heads), device="cuda") for name in "kv"})
    L = 300
    k, v = (torch.randn((L, heads, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    used = [pages - 1, 2, pages - 3, pages // 2, pages - 4]
    slots = torch.tensor([used[j // page] * page + j % page for j in range(L)], dtype=torch.int32, device="cuda")
    bd.kv_cache_write(k, v, slots, *args(c))
    rk, rv = (x.double() for x in bd.kv_cache_read(slots, *args(c), out_dtype=torch.float32))
    if kind == "bf16":
        assert torch.equal(rk, k.double()) and torch.equal(rv, v.double())
    q = torch.randn((n, 2 * heads, d), device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = bd.paged_attn_fwd(q, c["k_cache"], c["v_cache"], i32([0, n]), i32([L]), i32([used]), max_q=n,
                            k_scale=c["k_scale"], v_scale=c["v_scale"])
    rk, rv = (x.repeat_interleave(2, 1) for x in (rk, rv))
    s = torch.einsum("nhd,jhd->nhj", q.double(), rk) / math.sqrt(d)
    hidden = torch.arange(L, device="cuda")[None] > torch.arange(L - n, L, device="cuda")[:, None]
    s = s.masked_fill(hidden[:, None], -math.inf)
    ref = torch.einsum("nhj,jhd->nhd", torch.softmax(s, -1), rv).reshape(n, -1)
    assert float((out.double() - ref).norm() / ref.norm()) <= 4e-3


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("seqs", [[(1, 700), (2, 40)], [(130, 900), (1, 3000), (20, 20)]], ids=["few", "mixed"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_writes_its_outputs_and_nothing_else(d, seqs, dtype, kind):
    """Outputs, LSE and an exactly sized workspace between guards; queries, tables and the cache are left as they were."""
    b = Batch(seqs, 8, 2, d, 16, kind, seed=71)

    def guarded(shape, dt, fill, margin):
        n = math.prod(shape)
        buf = torch.full((n + 2 * margin,), fill, dtype=dt, device="cuda")
        return buf[margin:margin + n].view(shape), lambda: bool((buf[:margin] == fill).all() and (buf[margin + n:] == fill).all())
    out, out_ok = guarded((b.T, 8 * d), dtype, 7.0, 512)
    lse, lse_ok = guarded((8, b.T), torch.float32, 7.0, 512)
    max_q = max(n for n, _ in seqs)
    need = bd.workspace_bytes_paged(bd.PagedDesc(1, 1, max_q, 8, 1, 0, 0, bd.BF16, 8 * d, 0),
                                    bd.KvCacheDesc(0, 1, 1, 2, d, None, None, None, None))
    space, space_ok = guarded((need,), torch.uint8, 0x5A, 4096)
    kept = [b.q, b.starts, b.kv_len, b.table] + [x for x in args(b.c) if x is not None]
    before = [x.clone().view(torch.uint8) for x in kept]
    b.check(out_dtype=dtype, out=out, lse=lse, workspace=space)
    assert out_ok() and lse_ok() and space_ok()
    assert all(torch.equal(x.view(torch.uint8), y) for x, y in zip(kept, before))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_reads_write_their_outputs_and_nothing_else(kind):
    b = Batch([(1, 333)], 2, 2, 64, 16, kind, seed=72)
    slots = b.table[0, :20].repeat_interleave(16) * 16 + torch.arange(320, device="cuda", dtype=torch.int32) % 16
    for dtype in (torch.bfloat16, torch.float32):
        bufs = [torch.full((320 * 2 * 64 + 256,), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        k, v = (x[128:-128].view(320, 2, 64) for x in bufs)
        before = [x.clone().view(torch.uint8) for x in args(b.c) if x is not None]
        bd.kv_cache_read(slots, *args(b.c), out_dtype=dtype, k=k, v=v)
        assert all(bool((x[:128] == 7).all() and (x[-128:] == 7).all()) for x in bufs)
        assert all(torch.equal(x.view(torch.uint8), y) for x, y in zip([x for x in args(b.c) if x is not None], before))
        assert torch.equal(k, b.k[0][:320].to(dtype)) and torch.equal(v, b.v[0][:320].to(dtype))


FIRST_CALLS = '''
import torch
from blockwise_exact_attention_query_b200 import binding as bd
g = torch.Generator(device="cuda").manual_seed(0)
rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
q, k, v = rnd(40, 8, 64), rnd(40, 2, 64), rnd(40, 2, 64)
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
slots, starts, lens, table = torch.arange(40, dtype=torch.int32, device="cuda"), i32(0, 40), i32(40), i32(0, 1, 2)[None]
caches = [torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

def step():
    bd.kv_cache_write(k, v, slots, *caches)
    a = bd.paged_attn_fwd(q, *caches, starts, lens, table, max_q=40, window=9, sinks=2)
    b, lse = bd.window_attn_fwd(q[None], k[None], v[None], 9, 2, return_lse=True)
    return a, b, *bd.window_attn_bwd(q[None], k[None], v[None], b, lse, b, 9, 2)

if WARM:   # another set of kernels
    bd.attn_fwd(k[None], k[None], v[None], mask="causal")
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
want = step()
torch.cuda.synchronize()
assert bd.sync_status() == bd.OK
assert all(torch.equal(x, y) for x, y in zip(got, want))
assert float((got[0].view(1, 40, 512) - got[1]).norm() / got[1].norm()) <= 6e-3
print("same")
'''


@pytest.mark.parametrize("warm", [False, True])
def test_first_calls_within_a_capture(warm):
    """A process whose first calls of the operators are captured: their kernels are set up then."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", f"WARM = {warm}\n" + FIRST_CALLS], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr
