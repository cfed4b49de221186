"""GPU: trees of different sizes in one batch (spec_build_tree_batch with
n_valid) through window attention and acceptance from given numbers, with
whatever a caller may leave in the absent nodes' entries."""
import numpy as np
import pytest
import torch

from _util import dev, host, i32, zeros_i32
from oracle import accept as ACC
from test_gpu_window import Case, R
from test_gpu_verify_probs import probs
from tree_speculative_decoding_attn_gb300 import specverify as sv
from tree_speculative_decoding_attn_gb300 import synth

pytestmark = pytest.mark.gpu

SIZES = [12, 1, 5, 9]


def built(N, prefix, stale):
    """Device tree arrays of SIZES' random trees in N entries each; `stale`
    fills the absent entries of parents[]."""
    shapes = [R(60 + i, n, (4, 3, 2)) if n > 3 else synth.chain(n) for i, n in enumerate(SIZES)]
    par = np.full((len(SIZES), N), stale, np.int32)
    for b, s in enumerate(shapes):
        par[b, :s.n] = s.parents
    o = [zeros_i32(len(SIZES), N) for _ in range(4)]
    anc, st = torch.zeros((len(SIZES), N, 1), dtype=torch.int64, device="cuda"), zeros_i32(1)
    sv.spec_build_tree_batch(i32(par), i32(prefix), o[0], o[1], anc, o[2], o[3], n_valid=i32(SIZES), dev_status=st)
    assert int(st.item()) == 0
    return par, o[0], anc, o[2], o[3]


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("stale", [-1, 0, 3, 11, 1 << 20])
def test_acceptance_looks_at_no_absent_node(draft, stale):
    """Absent nodes' probabilities are NaN, their tokens and numbers arbitrary."""
    g = np.random.default_rng(7)
    B, N, V = len(SIZES), 12, 300
    par, _, _, fc, ns = built(N, [0] * B, stale)
    p = probs(g, (B, N, V), 3.0, torch.float32)
    q = probs(g, (B, N, V), 3.0, torch.float32) if draft else None
    tok = np.argsort(-p, -1)[:, :, 0].astype(np.int32)          # each node's own best token ...
    tok = np.take_along_axis(tok, np.clip(par, 0, N - 1), 1)   # ... of its parent
    u, ub = g.random((B, N)).astype(np.float32), g.random(B).astype(np.float32)
    want = ACC.accept_probs(p, q, tok, host(fc), host(ns), u, ub, N)
    for b, n in enumerate(SIZES):
        p[b, n:], u[b, n:], tok[b, n:] = np.nan, np.nan, g.integers(-5, V + 5, N - n)
        if draft:
            q[b, n:] = np.nan
    o, st = [zeros_i32(B), zeros_i32(B, N), zeros_i32(B)], zeros_i32(1)
    sv.spec_verify_probs(dev(p), i32(tok), i32(par), fc, ns, dev(u), dev(ub), *o,
                         draft_probs=None if q is None else dev(q), dev_status=st)
    for x, y in zip(o, want):
        np.testing.assert_array_equal(host(x), y)
    assert int(st.item()) == 0


@pytest.mark.parametrize("dtype,hq,hkv,D,prefix,window,page", [
    ("bf16", 2, 1, 128, [300, 0, 131, 40], 100, 128),      # few rows
    ("f32", 2, 1, 64, [300, 0, 131, 40], 100, 0),
    ("f32", 2, 1, 64, [6000, 0, 131, 40], 5000, 128),      # tiles on CUDA cores
    ("bf16", 64, 2, 128, [2900, 0, 131, 40], 2800, 0),     # SM pairs
    ("bf16", 32, 1, 64, [2900, 0, 131, 40], 2, 128),       # ... a window shorter than the trees
])
def test_window_attention_with_absent_nodes(dtype, hq, hkv, D, prefix, window, page):
    """Absent nodes' queries and keys are NaN and their values huge (finite,
    as the header asks): nothing of it reaches another row."""
    N = 12
    c = Case(dtype, len(SIZES), hq, hkv, D, prefix, R(60, N, (4, 3, 2)), window, 4, page=page, seed=5)
    _, depth, anc, _, _ = built(N, prefix, -1)
    c.depth, words = host(depth), host(anc)[:, :, 0].astype(np.uint64)
    c.mask = ((words[:, :, None] >> np.arange(N, dtype=np.uint64)) & np.uint64(1)).astype(bool)
    t = c.tensors()
    t["depth"], t["anc"] = depth, anc
    for b, n in enumerate(SIZES):
        t["q"][b, n:], t["kt"][b, :, n:], t["vt"][b, :, n:] = float("nan"), float("nan"), 3e38
    c.call(t)
    assert int(t["status"].item()) == 0
    # the absent rows, which mean nothing, from a call without NaN; the others as they came
    clean = c.tensors()
    clean["depth"], clean["anc"] = depth, anc
    c.call(clean)
    for b, n in enumerate(SIZES):
        t["out"][b, n:] = clean["out"][b, n:]
    c.check(t)


@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("node,told", [(1, True), (2, True), (3, False), (4, False), (5, True), (6, False)])
def test_a_bad_probability_is_told_if_the_walk_tests_it(draft, node, told):
    """0 has the children 1, 2, 3, of which 2 is kept; 2 has the child 5; 1
    has the child 4, 3 the child 6.  A node's own entry of its parent's row
    is NaN where no sum reads it."""
    V = 64
    par = np.array([[-1, 0, 0, 0, 1, 2, 3]], np.int32)
    fc, ns = np.array([[1, 4, 5, 6, -1, -1, -1]], np.int32), np.array([[-1, 2, 3, -1, -1, -1, -1]], np.int32)
    tok = np.array([[0, 11, 12, 13, 14, 15, 16]], np.int32)
    p = np.full((1, 7, V), 1 / V, np.float32)
    u = np.array([[0, 0.999, 0, 0.5, 0.5, 0.999, 0.5]], np.float32)
    q = np.full((1, 7, V), 1 / V, np.float32) if draft else None
    if draft:
        q[0, 0, 11] = 0.9     # refused (u q >= p); what is left of 12 is then more than nothing
        q[0, 0, 12] = 1e-6
        q[0, 2, 15] = 0.9
    p[0, par[0, node], tok[0, node]] = np.nan
    o, st = [zeros_i32(1), zeros_i32(1, 7), zeros_i32(1)], zeros_i32(1)
    sv.spec_verify_probs(dev(p), i32(tok), i32(par), i32(fc), i32(ns), dev(u), dev(np.full(1, 0.5, np.float32)), *o,
                         draft_probs=None if q is None else dev(q), dev_status=st)
    if node != 2:             # (2's NaN counts as 0: refused)
        assert host(o[1])[0, :2].tolist() == [0, 2]
    if draft and node == 3:   # row 0 is summed after 1's refusal, 13's entry with it
        told = True
    assert int(st.item()) == (sv.DEV_BAD_PROB if told else 0)
