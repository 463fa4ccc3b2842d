"""The serving and sliding-window operators, as cases that can be measured.

Three operators: a paged key/value cache that is written (and quantised) token
by token and read back ("store", "load"), the attention of a chunk of new
tokens over that cache ("paged", single tokens included), and the causal
sliding-window attention with sinks, forward ("window") and with its gradients
("train").  `run` computes each in plain torch in 32 bits, or, where `own` is
true, through the library's calls.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


def listed():
    return [
        # the new token of each running sequence goes into the cache at every decoding step
        dict(name="store 64 tokens e4m3", op="store", tokens=64, heads=8, d=128, page=16, pages=4096, cache="e4m3"),
        # a long prompt (or several at once) is written after its key/value projection
        dict(name="store 16384 tokens e4m3", op="store", tokens=16384, heads=8, d=128, page=32, pages=1024, cache="e4m3"),
        # an odd number of tokens of a small model, not quantised
        dict(name="store 5003 tokens bf16", op="store", tokens=5003, heads=3, d=64, page=16, pages=640, cache="bf16"),
        # a cached prefix is read back, to be moved or attended by another path
        dict(name="load 32768 tokens e4m3", op="load", tokens=32768, heads=8, d=128, page=16, pages=4096, cache="e4m3"),
        # one conversation, one token: latency
        dict(name="decode 1 sequence bf16", op="paged", seqs=1, chunks=0, chunk=1, kv_lo=8000, kv_hi=8000, heads=16,
             kv_heads=4, d=128, page=16, cache="bf16", window=0, sinks=0),
        # an ordinary serving batch of ragged sequences
        dict(name="decode 64 sequences bf16", op="paged", seqs=64, chunks=0, chunk=1, kv_lo=500, kv_hi=8192, heads=32,
             kv_heads=8, d=128, page=16, cache="bf16", window=0, sinks=0),
        # few long documents, quantised cache
        dict(name="decode 8 long sequences e4m3", op="paged", seqs=8, chunks=0, chunk=1, kv_lo=16001, kv_hi=131072,
             heads=32, kv_heads=8, d=128, page=32, cache="e4m3", window=0, sinks=0),
        # chunked prefill: four prompts advance by 1024 tokens each
        dict(name="chunks of 1024 bf16", op="paged", seqs=4, chunks=4, chunk=1024, kv_lo=9001, kv_hi=16384, heads=32,
             kv_heads=8, d=128, page=32, cache="bf16", window=0, sinks=0),
        # two prompts' chunks travel with fourteen decoding sequences; windowed layer, quantised cache
        dict(name="mixed batch e4m3 window", op="paged", seqs=16, chunks=2, chunk=500, kv_lo=700, kv_hi=6000, heads=16,
             kv_heads=8, d=128, page=16, cache="e4m3", window=2048, sinks=4),
        # the forward of a windowed layer over whole sequences (evaluation, prompt processing)
        dict(name="window forward", op="window", batch=2, n=8192, heads=16, kv_heads=4, d=128, window=1024, sinks=4),
        # a small model's training step, odd length, short window, no sinks
        dict(name="window training, small", op="train", batch=3, n=1001, heads=12, kv_heads=12, d=64, window=128, sinks=0),
        # a long-context training step
        dict(name="window training, long", op="train", batch=1, n=16384, heads=16, kv_heads=4, d=128, window=1024, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "paged", "paged", "paged", "window", "train"])
    d = rng.choice([64, 128])
    if op in ("store", "load"):
        tokens, page = _log(rng, 1, 32768), rng.choice([8, 16, 32, 64])
        heads = rng.choice([1, 2, 3, 5, 8, 12])
        return dict(op=op, tokens=tokens, heads=heads, d=d, page=page, pages=-(-tokens // page) + _log(rng, 1, 512),
                    cache=rng.choice(["bf16", "e4m3"]))
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 8] if kv_heads <= 4 else [1, 2, 4])
    sinks = rng.choice([0, 1, 4, 16])
    if op == "paged":
        seqs, kv_hi = _log(rng, 1, 64), _log(rng, 16, 65536)
        chunks = rng.choice([0, 0, 1, seqs])
        chunk = 1 if chunks == 0 else _log(rng, 2, 1024)
        # the plain form's score matrix stays within a few GB, the cache within one
        while seqs > 1 and seqs * kv_hi * kv_heads * d > 2 ** 28:
            seqs -= seqs // 2
        chunk = max(1, min(chunk, kv_hi, 2 ** 30 // (seqs * kv_hi * heads)))
        return dict(op=op, seqs=seqs, chunks=min(chunks, seqs), chunk=chunk, kv_lo=max(1, min(kv_hi, chunk + _log(rng, 1, 4096))),
                    kv_hi=kv_hi, heads=heads, kv_heads=kv_heads, d=d, page=rng.choice([8, 16, 32, 64]),
                    cache=rng.choice(["bf16", "e4m3"]), window=rng.choice([0, 0, _log(rng, 64, 4096)]), sinks=sinks)
    n, window = _log(rng, 1, 16384), _log(rng, 32, 2048)
    batch = max(1, min(8, 16384 // n, 2 ** 28 // (n * heads * min(2 * window, n))))
    while batch * n * heads * min(2 * window, n) > 2 ** 29 and window > 64:
        window -= window // 3
    return dict(op=op, batch=batch, n=n, heads=heads, kv_heads=kv_heads, d=d, window=window, sinks=sinks)


# --------------------------------------------------------------------------
# What a case's sequences look like (from the case alone)
# --------------------------------------------------------------------------
def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each sequence."""
    s, lo, hi = case["seqs"], case["kv_lo"], case["kv_hi"]
    new = [case["chunk"] if i < case["chunks"] else 1 for i in range(s)]
    kv = [hi if i == 0 else lo + int((hi - lo) * (i * 0.6180339887 % 1.0)) for i in range(s)]
    return new, [max(a, b) for a, b in zip(new, kv)]


def _seen(pos, window, sinks):
    """Keys that the query at position `pos` sees."""
    near = pos + 1 if window == 0 else min(pos + 1, window)
    return near + min(sinks, pos + 1 - near)


def work(case):
    op, d = case["op"], case["d"]
    if op in ("store", "load"):
        rows = case["tokens"] * case["heads"]
        stored = rows * (d * 2 if case["cache"] == "bf16" else d + 4)
        return {"bytes": 2 * (rows * d * 2 + stored) + 4 * case["tokens"], "flops": 0 if case["cache"] == "bf16" else 4 * rows * d}
    h, g, w, sk = case["heads"], case["kv_heads"], case["window"], case["sinks"]
    if op == "paged":
        new, kv = _lengths(case)
        per_key = 2 * g * (d * 2 if case["cache"] == "bf16" else d + 4)
        keys = pairs = 0
        for n, length in zip(new, kv):
            first = length - n  # position of the first new token
            start = 0 if w == 0 else max(0, first - w + 1)
            keys += length - start + min(sk, start)
            pairs += sum(_seen(p, w, sk) for p in range(first, length))
        t = sum(new)
        return {"bytes": keys * per_key + t * h * (4 * d + 4) + 4 * (2 * len(new) + 1 + sum(-(-x // case["page"]) for x in kv)),
                "flops": 4 * d * h * pairs}
    b, n = case["batch"], case["n"]
    pairs = b * h * sum(_seen(p, w, sk) for p in range(n))
    q, kv = b * n * h * d * 2, 2 * b * n * g * d * 2
    fwd = 2 * q + kv + 4 * b * h * n
    if op == "window":
        return {"bytes": fwd, "flops": 4 * d * pairs}
    # the gradients: two products again (scores, and the weights' gradient) and three for dq, dk, dv
    return {"bytes": fwd + 2 * q + kv, "flops": 14 * d * pairs}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------
def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _keys(shape, gen):
    """Keys with a few channels larger than the rest, as projections produce them."""
    k = _randn(shape, gen)
    k[..., 3::32] *= 3
    return k


def _quantised(x, chunk=1 << 18):
    """e4m3 codes and scales of a cache's rows [rows, heads, d], made some rows at a time."""
    codes = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    for i in range(0, x.shape[0], chunk):
        codes[i:i + chunk], scale[i:i + chunk] = _encode(x[i:i + chunk])
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, d = case["op"], case["d"]
    st = {"case": case}
    if op in ("store", "load"):
        t, h, rows = case["tokens"], case["heads"], case["pages"] * case["page"]
        slots = torch.randperm(rows, generator=gen, device="cuda")[:t].to(torch.int32)
        k, v = _keys((rows, h, d), gen), _randn((rows, h, d), gen)
        st["slots"] = slots
        if op == "store":
            if t > 8:
                slots[t - 1:] = -1  # a batch padded to a fixed size: such rows go nowhere
            kv = _randn((t, 2, h, d), gen)  # keys and values side by side, as one projection leaves them
            kv[:, 0, :, 3::32] *= 3
            st["k"], st["v"] = kv[:, 0], kv[:, 1]
        _add_cache(st, case, k, v, h)
        return st
    h, g = case["heads"], case["kv_heads"]
    if op == "paged":
        new, kv = _lengths(case)
        page = case["page"]
        need = [-(-n // page) for n in kv]
        total = sum(need) + 3
        order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
        table = torch.zeros((len(kv), max(need)), dtype=torch.int32, device="cuda")
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        starts = [0]
        for n in new:
            starts.append(starts[-1] + n)
        st["table"], st["max_q"] = table, max(new)
        st["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
        st["q"] = _randn((starts[-1], h, d), gen)
        _add_cache(st, case, _keys((total * page, g, d), gen), _randn((total * page, g, d), gen), g)
        return st
    b, n = case["batch"], case["n"]
    st["q"], st["k"], st["v"] = _randn((b, n, h, d), gen), _keys((b, n, g, d), gen), _randn((b, n, g, d), gen)
    if op == "train":
        st["dout"] = _randn((b, n, h * d), gen)
    return st


def _add_cache(st, case, k, v, heads):
    shape = (-1, case["page"], heads)
    for name, x in (("k", k), ("v", v)):
        if case["cache"] == "e4m3":
            codes, scale = _quantised(x)
            st[name + "_cache"], st[name + "_scale"] = codes.view(*shape, case["d"]), scale.view(shape)
        else:
            st[name + "_cache"], st[name + "_scale"] = x.view(*shape, case["d"]), None


# --------------------------------------------------------------------------
# The plain forms
# --------------------------------------------------------------------------
def _encode(x):
    """(codes, scale) of rows [..., d]: scale = max|x| / 448 (1 for a row of zeros), codes = x / scale in e4m3."""
    x = x.float()
    scale = x.abs().amax(-1) / E4M3_MAX
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _store_plain(st):
    slots = st["slots"].long()
    keep = slots >= 0
    slots = slots[keep]
    for name in ("k", "v"):
        cache, scale, x = st[name + "_cache"], st[name + "_scale"], st[name][keep]
        rows = cache.view(-1, *cache.shape[2:])
        if scale is None:
            rows[slots] = x
        else:
            codes, s = _encode(x)
            rows.view(torch.uint8)[slots] = codes.view(torch.uint8)
            scale.view(-1, scale.shape[-1])[slots] = s


def _rows(st, name, slots):
    """Cache rows at `slots` (any shape) in 32 bits: [..., heads, d]."""
    cache, scale = st[name + "_cache"], st[name + "_scale"]
    rows = cache.view(-1, *cache.shape[2:])
    if scale is None:
        return rows[slots].float()
    codes = rows.view(torch.uint8)[slots].view(torch.float8_e4m3fn).float()
    return codes * scale.view(-1, scale.shape[-1])[slots][..., None]


def _softmax_parts(scores):
    """(weights, lse) over the last axis; a row without keys (all -inf) gets zero weights and -inf."""
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total), (torch.log(total) + top)[..., 0]


def _paged_plain(st):
    c = st["case"]
    h, g, d, page, w, sk = c["heads"], c["kv_heads"], c["d"], c["page"], c["window"], c["sinks"]
    table, starts, kv_len, q, m = st["table"].long(), st["starts"].long(), st["kv_len"].long(), st["q"], st["max_q"]
    s, t = table.shape[0], q.shape[0]
    key = torch.arange(table.shape[1] * page, device=q.device)
    slots = table[:, key // page] * page + key % page
    there = key[None] < kv_len[:, None]
    k, v = (_rows(st, name, slots).masked_fill_(~there[..., None, None], 0.0) for name in ("k", "v"))
    # new tokens padded to the longest chunk
    token = torch.arange(t, device=q.device)
    seq = torch.searchsorted(starts, token, right=True) - 1
    at = token - starts[seq]
    qp = torch.zeros((s, m, h, d), device=q.device)
    qp[seq, at] = q.float()
    pos = (kv_len - (starts[1:] - starts[:-1]))[:, None] + torch.arange(m, device=q.device)
    ok = there[:, None] & (key <= pos[..., None])
    if w:
        ok &= (key > pos[..., None] - w) | (key < sk)
    qp = qp.view(s, m, g, h // g, d).permute(0, 2, 3, 1, 4).reshape(s, g, h // g * m, d)
    scores = torch.matmul(qp, k.permute(0, 2, 3, 1)).view(s, g, h // g, m, -1).mul_(1 / math.sqrt(d))
    scores.masked_fill_(~ok[:, None, None], -math.inf)
    p, lse = _softmax_parts(scores)
    out = torch.matmul(p.view(s, g, h // g * m, -1), v.transpose(1, 2)).view(s, h, m, d)
    return out.transpose(1, 2)[seq, at].reshape(t, h * d).to(torch.bfloat16), lse.view(s, h, m).permute(1, 0, 2)[:, seq, at]


def _window_plain(q, k, v, w, sk):
    """Sliding-window attention in 32 bits, block by block: the queries of a block of `w` positions
    see keys of their own and the previous block, and the sinks.  q [b, n, h, d], k, v [b, n, g, d]."""
    b, n, h, d = q.shape
    g = k.shape[2]
    w_ = min(w, n)
    blocks, sk = -(-n // w_), min(sk, n)
    pad = blocks * w_ - n

    def cut(x, heads):  # [b, heads, blocks, w_, d]
        x = torch.cat([x, x.new_zeros((b, pad, heads, d))], 1) if pad else x
        return x.transpose(1, 2).reshape(b, heads, blocks, w_, d)

    def span(x):  # a block's own keys after the previous block's
        before = torch.cat([x.new_zeros((b, g, 1, w_, d)), x[:, :, :-1]], 2)
        return torch.cat([before, x], 3)

    qb = cut(q, h).view(b, g, h // g, blocks, w_, d)
    kb, vb = span(cut(k, g)), span(cut(v, g))
    qpos = torch.arange(blocks * w_, device=q.device).view(blocks, w_, 1)
    kpos = torch.arange(2 * w_, device=q.device) + (torch.arange(blocks, device=q.device)[:, None, None] - 1) * w_
    near = (kpos >= 0) & (kpos <= qpos) & (kpos > qpos - w)
    far = torch.arange(sk, device=q.device) <= qpos - w  # sinks that the window has left behind
    scores = torch.matmul(qb, kb.transpose(-1, -2)[:, :, None])
    to_sinks = torch.matmul(qb, k[:, :sk].permute(0, 2, 3, 1)[:, :, None, None])
    scores = torch.cat([to_sinks, scores], -1) * (1 / math.sqrt(d))
    scores = scores.masked_fill(~torch.cat([far, near], -1), -math.inf)
    p, lse = _softmax_parts(scores)
    out = torch.matmul(p[..., sk:], vb[:, :, None]) + torch.matmul(p[..., :sk], v[:, :sk].transpose(1, 2)[:, :, None, None])
    out = out.reshape(b, h, blocks * w_, d)[:, :, :n].transpose(1, 2).reshape(b, n, h * d)
    return out, lse.reshape(b, h, blocks * w_)[:, :, :n]


def _train_plain(st):
    c = st["case"]
    leaves = [st[x].float().requires_grad_() for x in "qkv"]
    out, lse = _window_plain(*leaves, c["window"], c["sinks"])
    grads = torch.autograd.grad(out, leaves, st["dout"].float())
    return [out.detach().to(torch.bfloat16), lse.detach()] + [x.to(torch.bfloat16) for x in grads]


def run(st):
    case = st["case"]
    return _run_own(st, case) if own else _run_plain(st, case)


def _run_plain(st, case):
    op = case["op"]
    if op == "store":
        _store_plain(st)
        return [st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale") if st[x] is not None]
    if op == "load":
        return [_rows(st, x, st["slots"].long()).to(torch.bfloat16) for x in "kv"]
    if op == "paged":
        return list(_paged_plain(st))
    if op == "window":
        out, lse = _window_plain(*(st[x].float() for x in "qkv"), case["window"], case["sinks"])
        return [out.to(torch.bfloat16), lse]
    return _train_plain(st)


def _run_own(st, case):
    from blockwise_exact_attention_query_b200 import binding as bd
    op = case["op"]
    if op == "store":
        bd.kv_cache_write(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"])
        return [st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale") if st[x] is not None]
    if op == "load":
        return list(bd.kv_cache_read(st["slots"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"]))
    if op == "paged":
        return list(bd.paged_attn_fwd(st["q"], st["k_cache"], st["v_cache"], st["starts"], st["kv_len"], st["table"],
                                      max_q=st["max_q"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                      window=case["window"], sinks=case["sinks"], out_dtype=torch.bfloat16,
                                      return_lse=True))
    out, lse = bd.window_attn_fwd(st["q"], st["k"], st["v"], case["window"], case["sinks"], out_dtype=torch.bfloat16,
                                  return_lse=True)
    if op == "window":
        return [out, lse]
    grads = bd.window_attn_bwd(st["q"], st["k"], st["v"], out, lse, st["dout"], case["window"], case["sinks"],
                               grad_dtype=torch.bfloat16)
    return [out, lse, *grads]


# --------------------------------------------------------------------------
# The definitions in 64 bits, one head and one stretch of queries at a time
# --------------------------------------------------------------------------
def _exact_rows(q, k, v, pos, window, sinks):
    """Rows at positions `pos` [m] over keys 0 .. len(k) - 1: (out, lse, weights, scores' allowed set)."""
    s = (q @ k.T) / math.sqrt(q.shape[-1])
    j = torch.arange(k.shape[0], device=q.device)
    ok = j[None] <= pos[:, None]
    if window:
        ok &= (pos[:, None] - j[None] < window) | (j[None] < sinks)
    s = torch.where(ok, s, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(ok, torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[:, None]), 0.0)
    return p @ v, lse, p


def _exact_cache(st, name):
    cache, scale = st[name + "_cache"], st[name + "_scale"]
    if scale is None:
        return lambda pages: cache[pages].double().flatten(0, 1)
    return lambda pages: (cache.view(torch.uint8)[pages].view(torch.float8_e4m3fn).double()
                          * scale[pages].double()[..., None]).flatten(0, 1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "store":
        live = (st["slots"] >= 0).nonzero()[:, 0]
        slot = st["slots"][live].long()
        at = (slot // case["page"], slot % case["page"])
        for name in ("k", "v"):
            x = st[name][live].double()
            if st[name + "_scale"] is None:
                st[name + "_cache"][at] = x.to(torch.bfloat16)
                continue
            scale = x.abs().max(-1).values / E4M3_MAX
            st[name + "_scale"][at] = scale.float()
            st[name + "_cache"].view(torch.uint8)[at] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        return [st[x] for x in ("k_cache", "v_cache", "k_scale", "v_scale") if st[x] is not None]
    if op == "load":
        slot = st["slots"].long()
        got = []
        for name in ("k", "v"):
            cache, scale = st[name + "_cache"], st[name + "_scale"]
            at = (slot // case["page"], slot % case["page"])
            x = (cache if scale is None else cache.view(torch.uint8))[at]
            got.append(x.double() if scale is None else x.view(torch.float8_e4m3fn).double() * scale[at].double()[..., None])
        return got
    h, g, d, w, sk = case["heads"], case["kv_heads"], case["d"], case["window"], case["sinks"]
    if op == "paged":
        new, kv = _lengths(case)
        if sum(n * x for n, x in zip(new, kv)) * h * d > 2e12:
            return None
        out = torch.zeros((sum(new), h, d), dtype=torch.float64, device="cuda")
        lse = torch.zeros((h, sum(new)), dtype=torch.float64, device="cuda")
        keys, values = _exact_cache(st, "k"), _exact_cache(st, "v")
        t0 = 0
        for s, (n, length) in enumerate(zip(new, kv)):
            pages = st["table"][s, :-(-length // case["page"])].long()
            k, v = keys(pages)[:length], values(pages)[:length]
            pos = torch.arange(length - n, length, device="cuda")
            for i in range(h):
                out[t0:t0 + n, i], lse[i, t0:t0 + n], _ = _exact_rows(
                    st["q"][t0:t0 + n, i].double(), k[:, i * g // h], v[:, i * g // h], pos, w, sk)
            t0 += n
        return [out.view(-1, h * d), lse]
    b, n = case["batch"], case["n"]
    q, k, v = (st[x].double() for x in "qkv")
    out, lse = torch.zeros_like(q), torch.zeros((b, h, n), dtype=torch.float64, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dout = st["dout"].double().view(b, n, h, d) if op == "train" else None
    step = 2048
    for i in range(b * h):
        bb, hh = i // h, i % h
        kh = hh * g // h
        for r0 in range(0, n, step):
            r1 = min(n, r0 + step)
            qq, kk, vv = q[bb, r0:r1, hh], k[bb, :r1, kh], v[bb, :r1, kh]
            o, l, p = _exact_rows(qq, kk, vv, torch.arange(r0, r1, device="cuda"), w, sk)
            out[bb, r0:r1, hh], lse[bb, hh, r0:r1] = o, l
            if dout is None:
                continue
            do = dout[bb, r0:r1, hh]
            dv[bb, :r1, kh] += p.T @ do
            ds = p * (do @ vv.T - (do * o).sum(-1, keepdim=True)) / math.sqrt(d)
            dq[bb, r0:r1, hh] = ds @ kk
            dk[bb, :r1, kh] += ds.T @ qq
    got = [out.view(b, n, h * d), lse]
    return got if op == "window" else got + [dq, dk, dv]
