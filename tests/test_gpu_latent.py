"""GPU parity: tree attention over latent rows against float64."""
import numpy as np
import pytest
import torch

from _util import dev, i32, zeros_i32
from oracle import latent as LO
from oracle import tree as T
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
BF, F32 = torch.bfloat16, torch.float32


def trees(g, B, N):
    """Random parents of each sequence, and their masks [B, N, N]."""
    mask = np.zeros((B, N, N), bool)
    for b in range(B):
        par = [-1] + [int(g.integers(max(0, i - 9), i)) for i in range(1, N)]
        mask[b] = T.depth_and_mask(np.asarray(par))[1]
    return mask


def words(mask):
    return dev(np.stack([T.mask_words_multi(m) for m in mask]).view(np.int64))


def bound(q, rows, size, ref, latent, dtype, n_keys):
    """What the arithmetic may be off by, element by element.

    Scores are float32 sums of D products, each addition off by at most 2^-23
    of the sum of sizes; e^x then by twice that in relative terms (weight and
    normaliser).  A probability is rounded to bf16 (half a step, 2^-8) for the
    product, which sums n_keys of them in float32; the output is rounded once
    more.  float32 has no rounding of P and 2^-24 for the output."""
    D = rows.shape[-1]
    x = max(float((np.abs(a.reshape(-1, D)) @ np.abs(r).T).max()) for a, r in zip(q, rows))
    rel = 2 * (D + 8) * 2.0 ** -23 * x * SCALE + (n_keys + 8) * 2.0 ** -23
    if dtype is BF:
        return size * (rel + 2.0 ** -8) * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8 + 1e-30
    return size * rel + np.abs(ref) * 2.0 ** -24 + 1e-30


def make(seed, B, N, H, lat, prefix, dtype, page, spread=1.0):
    g = np.random.default_rng(seed)
    D, S = lat + 64, max(max(prefix), 1) + 5
    t = lambda *s: torch.from_numpy(g.standard_normal(s, np.float32) * spread).to(dtype)  # noqa: E731
    q, cache, tree, mask = t(B, N, H, D), t(B, S, D), t(B, N, D), trees(g, B, N)
    c = dict(B=B, N=N, H=H, lat=lat, prefix=list(prefix), dtype=dtype, page=page, q=q, cache=cache, tree=tree, mask=mask)
    if page:
        pages = [-(-p // page) for p in prefix]
        nb = sum(pages) + 2
        ids, k = g.permutation(nb), 0
        table = np.full((B, max(1, max(pages))), -1, np.int32)
        pool = torch.full((nb, page, D), float("nan"), dtype=dtype)     # what no sequence holds is not read for the result
        for b, n in enumerate(pages):
            table[b, :n] = ids[k:k + n]
            for j in range(n):
                rows = cache[b, j * page:min((j + 1) * page, prefix[b])]
                pool[ids[k + j], :len(rows)] = rows
            k += n
        c.update(table=table, pool=pool)
    else:
        for b, p in enumerate(prefix):
            cache[b, p:] = float("nan")
    return c


def call(c, max_prefix=None, out=None, st=None, workspace=None, prefix=None):
    B, N, H, lat = c["B"], c["N"], c["H"], c["lat"]
    out = torch.full((B, N, H, lat), 7.0, dtype=c["dtype"], device="cuda") if out is None else out
    st = zeros_i32(1) if st is None else st
    mp = max(c["prefix"]) if max_prefix is None else max_prefix
    more = dict(workspace=workspace, dev_status=st)
    p = i32(c["prefix"]) if prefix is None else prefix
    if c["page"]:
        sv.tree_attn_verify_latent_paged(c["q"].cuda(), c["pool"].cuda(), i32(c["table"]), c["tree"].cuda(), p,
                                         words(c["mask"]), out, mp, SCALE, **more)
    else:
        sv.tree_attn_verify_latent(c["q"].cuda(), c["cache"].cuda(), c["tree"].cuda(), p, words(c["mask"]), out, mp, SCALE,
                                   **more)
    return out, st


def check(c, out, st, skip=()):
    q, cache, tree = (c[k].double().numpy() for k in ("q", "cache", "tree"))
    assert int(st.item()) == 0
    ref, size = LO.tree_attention(q, cache, tree, c["prefix"], c["mask"], c["lat"], SCALE)
    rows = [np.concatenate([cache[b, :c["prefix"][b]], tree[b]]) for b in range(c["B"])]
    got = out.double().cpu().numpy()
    for b in range(c["B"]):
        if b in skip:
            continue
        tol = bound(q[b:b + 1], rows[b][None], size[b], ref[b], c["lat"], c["dtype"], len(rows[b]))
        err = np.abs(got[b] - ref[b])
        assert bool(np.isfinite(got[b]).all())
        worst = float((err / tol).max())
        assert worst <= 1.0, (b, worst)


SHAPES = [
    # B, N, H, latent, prefixes, page
    (1, 1, 16, 512, [0], 0), (1, 1, 1, 512, [1], 0), (1, 1, 16, 512, [5000], 128), (2, 5, 4, 256, [129, 1], 0),
    (3, 2, 3, 512, [63, 64, 65], 128), (4, 7, 20, 512, [127, 128, 129, 0], 256), (2, 64, 2, 512, [300, 77], 0),
    (2, 65, 1, 256, [300, 512], 128), (1, 128, 3, 512, [200], 128), (2, 129, 2, 512, [1, 640], 0), (1, 256, 5, 512, [333], 128),
    (1, 256, 1, 256, [0], 0), (2, 33, 128, 512, [1000, 257], 128), (5, 3, 40, 256, [900, 0, 1, 128, 511], 128),
    (40, 1, 16, 512, [(37 * i) % 700 for i in range(40)], 128), (2, 60, 32, 512, [2000, 513], 128), (1, 4, 128, 256, [9000], 0),
]


@pytest.mark.parametrize("B,N,H,lat,prefix,page", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_matches_float64(lib, B, N, H, lat, prefix, page, dtype):
    c = make(B * 100 + N, B, N, H, lat, prefix, dtype, page)
    check(c, *call(c))
