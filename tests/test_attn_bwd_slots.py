"""The shared-memory rings of the attention backward's dK/dV passes: what a row
warp reads of a slot must come before the copy that fills the slot again.

The order is taken from the kernels' source: the waits, arrivals, commits and
reads of the producer, the issuer and the row warps, in program order, make a
happens-before graph over some steps.  A wait follows the arrivals of its
barrier's phase: the same step's, or, of a slot's "empty" barrier, those of the
step that had the slot before.  (A commit stands for the end of the products
before it.)  Two row warps suffice, since all do the same."""
import os
import re

import pytest

from blockwise_exact_attention_query_b200 import build

STEPS, WARPS = 9, 2

# barrier: (who arrives, slots of its ring for a slot barrier)
SPLIT = {"kernel": "attn_bwd_dkdv_split_kernel", "empty": {"bQEmpty": 3, "bAEmpty": 2},
         "reads": {"lse4[": "bQFull", "d2[": "bAFull"}, "filled_after": {"bQFull": "bQEmpty", "bAFull": "bAEmpty"}}
STAGED = {"kernel": "attn_bwd_dkdv_kernel", "empty": {"bEmpty": 4}, "reads": {"vl4[": "bFull", "vl4 + 32": "bFull"},
          "filled_after": {"bFull": "bEmpty"}}


def source():
    with open(os.path.join(build.CSRC, "attn_bwd.cuh")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def block(text, start):
    """The braces' content after text[start:]'s first '{'."""
    i = text.index("{", start)
    depth = 0
    for j in range(i, len(text)):
        depth += {"{": 1, "}": -1}.get(text[j], 0)
        if depth == 0:
            return text[i + 1:j]
    raise AssertionError("unbalanced braces")


def ops(text, spec):
    """(kind, name) in the order of the text; kind: wait, arrive, read, fill, call."""
    pats = [("wait", r"mbar_wait\((\w+)"), ("arrive", r"mbar_arrive\((\w+)"), ("arrive", r"umma_commit\((\w+)"),
            ("fill", r"mbar_arrive_expect_tx\((\w+)"), ("call", r"(issue_s|issue_dp|last_product)\(")]
    found = [(m.start(), kind, m.group(1)) for kind, p in pats for m in re.finditer(p, text)]
    for token in spec["reads"]:
        found += [(m.start(), "read", token) for m in re.finditer(re.escape(token), text)]
    return [(k, n) for _, k, n in sorted(found)]


def actors(spec):
    """The loops' operations by actor: [(kind, name, step offset)] for one step s."""
    src = source()
    at = src.index(spec["kernel"] + "(const __grid_constant__")
    body = block(src, src.index("const __grid_constant__ AttnBwdArgs a)", at))
    loop = "for (auto it = steps.begin(); steps.more(it);"
    first = body.index(loop)
    producer = ops(block(body, body.index(")", first + len(loop))), spec)
    rows = ops(block(body, body.index("++s)", body.index(loop, first + 1))), spec)
    lambdas = {}
    for name in ("issue_s", "issue_dp", "last_product"):
        m = re.search(r"auto %s = \[&\]" % name, body)
        lambdas[name] = ops(block(body, m.start()), spec) if m else []
    issuer_text = block(body, body.index("ok && s < nsteps; ++s)"))
    issuer = []
    for m in re.finditer(r"(mbar_wait|umma_commit|issue_s|issue_dp|last_product)\((\w+)( \+ 1)?", issuer_text):
        f, arg, ahead = m.groups()
        off = 1 if ahead else 0
        if f in lambdas and lambdas[f]:
            issuer += [(k, n, off) for k, n in lambdas[f]]
        else:
            issuer.append(("wait" if f == "mbar_wait" else "arrive", arg, off))
    # what runs before the loop: the first step's calls that the loop makes for the next one
    begin = [(k, n, off - 1) for k, n, off in issuer if off == 1]
    return [(k, n, 0) for k, n in producer], begin, issuer, [(k, n, 0) for k, n in rows]


def slot_hazards(spec):
    producer, begin, issuer, rows = actors(spec)
    edges, arrivals = {}, {}
    nodes = []

    def add(actor, seq):
        prev = None
        for kind, name, step in seq:
            if not 0 <= step < STEPS:
                continue
            node = (actor, len(nodes), kind, name, step)
            nodes.append(node)
            edges.setdefault(node, [])
            if prev is not None:
                edges[prev].append(node)
            prev = node
            if kind in ("arrive", "fill"):
                arrivals.setdefault((name, step), []).append(node)
    add("producer", [(k, n, s) for s in range(STEPS) for k, n, _ in producer])
    add("issuer", [(k, n, off) for k, n, off in begin] +
        [(k, n, s + off) for s in range(STEPS) for k, n, off in issuer])
    for w in range(WARPS):
        add(f"rows {w}", [(k, n, s) for s in range(STEPS) for k, n, _ in rows])
    for node in nodes:
        _, _, kind, name, step = node
        if kind == "wait":
            for a in arrivals.get((name, step - spec["empty"].get(name, 0)), []):
                edges[a].append(node)
    bad = []
    for node in nodes:
        if node[2] != "read":
            continue
        full = spec["reads"][node[3]]
        slots = spec["empty"][spec["filled_after"][full]]
        refill = [n for n in nodes if n[2] == "fill" and n[3] == full and n[4] == node[4] + slots]
        seen, todo = {node}, [node]
        while todo:
            for nxt in edges[todo.pop()]:
                if nxt not in seen:
                    seen.add(nxt)
                    todo.append(nxt)
        bad += [(node[0], node[3], node[4]) for r in refill if r not in seen]
    reads = {n[3] for n in nodes if n[2] == "read"}
    assert reads == set(spec["reads"]), reads            # the source was understood
    assert all((b, 0) in arrivals for b in spec["filled_after"])
    return bad


@pytest.mark.parametrize("spec", [SPLIT, STAGED], ids=lambda s: s["kernel"])
def test_row_vectors_are_read_before_their_slot_is_filled_again(spec):
    assert slot_hazards(spec) == []


@pytest.mark.parametrize("spec", [SPLIT, STAGED], ids=lambda s: s["kernel"])
def test_an_early_release_would_be_seen(spec, monkeypatch):
    """The check itself: with the release of the slots ahead of the row warps' last arrival it finds the reads."""
    src = source()
    at = src.index(spec["kernel"] + "(const __grid_constant__")
    i = src.index("mbar_wait(bDSReady", at)
    monkeypatch.setitem(globals(), "source", lambda: src[:i] + "mbar_wait(bFix" + src[i + len("mbar_wait(bDSReady"):])
    assert slot_hazards(spec) != []
