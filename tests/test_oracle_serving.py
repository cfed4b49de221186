"""Oracle pins of the serving operators: window attention, acceptance from
given numbers, pages (no GPU)."""
import numpy as np
import pytest

from oracle import accept as ACC
from oracle import attention as A
from oracle import pages as PG
from oracle import tree as T
from tree_speculative_decoding_attn_gb300 import synth


def _inputs(seed, B, N, hq, hkv, D, S):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    return n(B, N, hq, D), n(B, hkv, S, D), n(B, hkv, S, D), n(B, hkv, N, D), n(B, hkv, N, D)


def test_a_window_over_everything_is_tree_attention():
    shape = synth.random_tree(3, 12, (4, 3, 2))
    depth, mask = T.depth_and_mask(shape.parents)
    q, kc, vc, kt, vt = _inputs(1, 2, 12, 4, 2, 8, 40)
    prefix = [33, 7]
    o, _, _ = A.tree_attention_window(q, kc, vc, kt, vt, prefix, np.stack([depth] * 2), np.stack([mask] * 2), 1000, 0)
    np.testing.assert_allclose(o, A.tree_attention(q, kc, vc, kt, vt, prefix, mask), atol=1e-12)
    # sinks over everything make any window whole
    o, _, _ = A.tree_attention_window(q, kc, vc, kt, vt, prefix, np.stack([depth] * 2), np.stack([mask] * 2), 1, 1000)
    np.testing.assert_allclose(o, A.tree_attention(q, kc, vc, kt, vt, prefix, mask), atol=1e-12)


def test_a_chain_in_a_window_is_banded_causal_attention():
    """A chain after a prefix equals rows of one sequence whose row x sees
    the columns x - window < y <= x and y < sinks."""
    N, P, W, S = 7, 20, 6, 2
    depth, mask = np.arange(N), np.tril(np.ones((N, N), bool))
    q, kc, vc, kt, vt = _inputs(2, 1, N, 1, 1, 8, P)
    o, _, _ = A.tree_attention_window(q, kc, vc, kt, vt, [P], depth[None], mask[None], W, S)
    k, v = np.concatenate([kc[0, 0], kt[0, 0]]), np.concatenate([vc[0, 0], vt[0, 0]])
    x, y = np.arange(P, P + N)[:, None], np.arange(P + N)[None]
    s = np.where((y <= x) & ((x - y < W) | (y < S)), q[0, :, 0] @ k.T / np.sqrt(8), -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    np.testing.assert_allclose(o[0, :, 0], p / p.sum(1, keepdims=True) @ v, atol=1e-12)


def test_a_node_that_sees_nothing_gets_zeros():
    q, kc, vc, kt, vt = _inputs(3, 1, 2, 1, 1, 8, 4)
    mask = np.array([[[True, False], [False, False]]])
    o, a, e = A.tree_attention_window(q, kc, vc, kt, vt, [0], np.zeros((1, 2), int), mask, 5, 0)
    assert (o[0, 1] == 0).all() and (a[0, 1] == 0).all() and np.allclose(o[0, 0, 0], vt[0, 0, 0])


@pytest.mark.parametrize("stochastic", [False, True])
def test_the_first_token_follows_the_target(stochastic):
    """One node with two drafted children: whatever the drafts, the step's
    first token (the accepted child's, or the bonus) has the target's
    distribution.  20000 draws per setting; a count's standard deviation is
    at most sqrt(n / 4) = 71, five of them 354."""
    g = np.random.default_rng(5)
    n, V = 20000, 5
    p = np.array([0.4, 0.3, 0.15, 0.1, 0.05])
    q = np.array([0.1, 0.5, 0.2, 0.1, 0.1])
    fc, ns = np.array([[1, -1, -1]]), np.array([[-1, 2, -1]])
    probs, drafts = np.tile(p, (1, 3, 1)), np.tile(q, (1, 3, 1))
    count = np.zeros(V)
    for _ in range(n):
        tok = np.array([[0, *(g.choice(V, 2, p=q) if stochastic else (1, 2))]])
        length, path, bonus = ACC.accept_probs(probs, drafts if stochastic else None, tok, fc, ns, g.random((1, 3)),
                                               g.random(1), 2)
        count[tok[0, path[0, 1]] if length[0] else bonus[0]] += 1
    assert (np.abs(count - n * p) < 354).all(), (count, n * p)


def test_probs_rule_equals_the_enumerated_one_for_a_point_mass_drafter():
    """A drafter whose row is a point mass rejects like a deterministic
    draft: the same paths and bonuses from the same numbers."""
    g = np.random.default_rng(6)
    fc, ns = np.array([[1, -1]]), np.array([[-1, -1]])
    for _ in range(200):
        p = g.dirichlet(np.ones(6), (1, 2))
        t = int(g.integers(6))
        q = np.zeros((1, 2, 6))
        q[..., t] = 1
        args = (np.array([[0, t]]), fc, ns, g.random((1, 2)), g.random(1), 2)
        for x, y in zip(ACC.accept_probs(p, None, *args), ACC.accept_probs(p, q, *args)):
            np.testing.assert_array_equal(x, y)


def test_pages_life():
    """Two requests, one forked; their shared page is copied once and kept
    once; the window's leavers go; compaction leaves rows where their table says."""
    bs, nb = 4, 12
    g = np.random.default_rng(7)
    pools = [g.standard_normal((2, nb, 3, bs, 2)) for _ in range(2)]
    table = np.array([[7, 2, -1, -1], [9, -1, -1, -1]], np.int32)
    prefix = np.array([6, 4], np.int32)
    ref = np.bincount(table[table >= 0], minlength=nb).astype(np.int32)
    rows = lambda t, pl, b, n: [pl[0][:, t[b, x // bs], :, x % bs] for x in range(n)]  # noqa: E731
    before = rows(table, pools, 0, 6)
    t, lens, ref = PG.fork(table, prefix, np.array([0, 0, -1]), ref)
    assert lens.tolist() == [6, 6, 0] and ref[7] == ref[2] == 2 and ref[9] == 0
    pools, t, ref, fits = PG.reserve(pools, t, lens, np.array([3, 3, 0]), ref, bs)
    # sequence 0 copies page 1 (block 0) and gets page 2 (block 1); sequence 1 keeps block 2 and gets block 3
    assert fits and t[0].tolist() == [7, 0, 1, -1] and t[1].tolist() == [7, 2, 3, -1] and ref[2] == 1
    for b in (0, 1):
        np.testing.assert_array_equal(rows(t, pools, b, 6), before)
    pools, t, ref, used, remap = PG.compact(pools, t, ref)
    assert used == 5 and sorted(set(t[t >= 0])) == [0, 1, 2, 3, 4] and remap[7] == 4
    np.testing.assert_array_equal(rows(t, pools, 1, 6), before)
    t, ref = PG.free(t, np.array([10, 6, 0]), ref, bs, window=3, sinks=0)
    # positions 8, 9 of sequence 0 and 4, 5 of sequence 1 are still seen
    assert t[0].tolist() == [-1, -1, 1, -1] and t[1].tolist() == [-1, 2, -1, -1] and ref.sum() == 2
