"""Pins of the latent oracle: against direct sums, and its two forms against each other."""
import math

import numpy as np

from oracle import latent as LO


def test_tree_attention_is_the_sum_over_visible_rows():
    g = np.random.default_rng(1)
    q, cache, tree = g.standard_normal((1, 2, 1, 6)), g.standard_normal((1, 4, 6)), g.standard_normal((1, 2, 6))
    mask = np.array([[[True, False], [True, True]]])
    out, size = LO.tree_attention(q, cache, tree, [3], mask, 4, 0.5)
    for i in range(2):
        rows = [cache[0, 0], cache[0, 1], cache[0, 2], tree[0, 0]] + ([tree[0, 1]] if i else [])
        w = [math.exp(0.5 * float(q[0, i, 0] @ r)) for r in rows]
        want = sum(a * r[:4] for a, r in zip(w, rows)) / sum(w)
        np.testing.assert_allclose(out[0, i, 0], want, rtol=1e-12)
        np.testing.assert_allclose(size[0, i, 0], sum(a * abs(r[:4]) for a, r in zip(w, rows)) / sum(w), rtol=1e-12)


def test_nothing_visible_gives_zeros():
    out, _ = LO.tree_attention(np.ones((1, 1, 1, 3)), np.ones((1, 2, 3)), np.ones((1, 1, 3)), [0], np.zeros((1, 1, 1), bool), 2, 1.0)
    assert (out == 0).all()
    out, _ = LO.prompt_attention(np.ones((3, 1, 4)), np.ones((1, 1, 2)), np.ones((1, 2)), np.ones((1, 1, 5)), [0, 3], [0, 1], 1.0)
    assert (out[:2] == 0).all() and (out[2] == 1).all()


def test_absorbed_equals_expanded():
    """x = (W_uk^T q) . c + q_r . k_r and out = W_uv (sum p c), whichever product comes first."""
    g = np.random.default_rng(2)
    H, lat, dk, R, dv, P, n = 3, 8, 5, 2, 4, 7, 3
    wk, wv = g.standard_normal((H, dk, lat)), g.standard_normal((H, lat, dv))
    rows, q, qr = g.standard_normal((P + n, lat + R)), g.standard_normal((n, H, dk)), g.standard_normal((n, H, R))
    ql = np.concatenate([np.einsum("nhd,hdl->nhl", q, wk), qr], -1)
    a, _ = LO.tree_attention(ql[None], rows[None], rows[None, P:], [P], np.tril(np.ones((n, n), bool))[None], lat, 0.3)
    k, v = np.einsum("hdl,tl->thd", wk, rows[:, :lat]), np.einsum("tl,hld->thd", rows[:, :lat], wv)
    b, _ = LO.prompt_attention(np.concatenate([q, qr], -1), k, rows[:, lat:], v, [0, n], [0, P + n], 0.3)
    np.testing.assert_allclose(np.einsum("nhl,hld->nhd", a[0], wv), b, rtol=1e-9)


def test_slots_worked_example():
    table = np.array([[5, 2], [7, -1]])
    off, slots, pos, err = LO.slots(table, [3, 0], [3, 2], 7, 4, 8)
    assert off.tolist() == [0, 3, 5] and not err
    assert slots.tolist() == [23, 8, 9, 28, 29, -1, -1] and pos.tolist() == [3, 4, 5, 0, 1, -1, -1]
