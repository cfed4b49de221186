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


def test_rows_of_nothing_are_zeros(lib):
    """Empty masks with an empty prefix, on all three kernels (rows, few rows, float32)."""
    for N, H, dtype in ((65, 3, BF), (5, 2, BF), (5, 2, F32)):
        c = make(3, 2, N, H, 512, [0, 130], dtype, 0)
        c["mask"][:, 1::2] = False
        out, st = call(c)
        check(c, out, st)
        assert float(out[0, 1::2].abs().max()) == 0.0


@pytest.mark.parametrize("N,H,dtype", [(33, 4, BF), (4, 3, BF), (4, 3, F32)])
def test_not_a_number(lib, N, H, dtype):
    """A NaN query makes its row NaN, a NaN key the rows that see it; no others."""
    c = make(7, 2, N, H, 512, [300, 200], dtype, 128)
    c["q"][0, 1, 2, 5] = float("nan")
    out, _ = call(c)
    bad = out.isnan().any(-1).cpu()
    want = torch.zeros(2, N, H, dtype=torch.bool)
    want[0, 1, 2] = True
    assert torch.equal(bad, want)
    c = make(7, 2, N, H, 512, [300, 200], dtype, 128)
    c["tree"][1, 2, 560] = float("nan")           # a rotary element of node 2: only scores take it
    out, _ = call(c)
    want = torch.from_numpy(c["mask"][1][:, 2])
    assert torch.equal(out[1].isnan().any(-1).all(-1).cpu(), want) and not out[0].isnan().any()
    assert torch.equal(out[1].isnan().any(-1).any(-1).cpu(), want)


@pytest.mark.parametrize("N,H,dtype", [(33, 4, BF), (4, 3, BF), (4, 3, F32)])
@pytest.mark.parametrize("lat", [256, 512])
def test_scores_that_jump(lib, N, H, dtype, lat):
    """Each later tile's scores far above the ones before (the running maximum
    moves, sums and outputs are scaled down), then far below."""
    c = make(11, 1, N, H, lat, [900], dtype, 0, spread=0.5)
    up = torch.arange(900) // 64
    up = torch.where(up < 8, up, 15 - up).float()
    c["q"][..., lat] = 16.0
    c["cache"][0, :900, lat] = (up * 8).to(dtype)    # 128 a step times the scale: 9.2 in the exponent, 13.3 in powers of 2
    check(c, *call(c))


@pytest.mark.parametrize("N,H", [(40, 4), (2, 3)])
def test_refused_lengths_leave_their_rows(lib, N, H):
    c = make(5, 3, N, H, 512, [200, 100, 300], BF, 0)
    for bad in (-1, 301, 2 ** 31 - 1):
        p = i32([200, bad, 300])
        out, st = call(c, prefix=p)
        assert int(st.item()) == sv.DEV_CAPACITY and bool((out[1] == 7.0).all())
        st.zero_()
        check(c, out, st, skip=(1,))


@pytest.mark.parametrize("N,H,dtype", [(40, 4, BF), (2, 3, BF), (2, 3, F32)])
def test_bad_blocks_read_as_zeros(lib, N, H, dtype):
    c = make(6, 2, N, H, 512, [500, 260], dtype, 128)
    good = make(6, 2, N, H, 512, [500, 260], dtype, 128)
    for bad in (-3, 10 ** 6):
        c["table"] = good["table"].copy()
        c["table"][0, 1] = bad
        out, st = call(c)
        assert int(st.item()) == sv.DEV_BAD_BLOCK
        c["cache"] = good["cache"].clone()
        c["cache"][0, 128:256] = 0
        st.zero_()
        check(c, out, st)


@pytest.mark.parametrize("N,H,P", [(1, 16, 20000), (3, 40, 9000), (1, 16, 40), (200, 2, 10)])
def test_loose_bounds_and_one_sequence_in_many_parts(lib, N, H, P):
    """A long sequence over all parts of the GPU, and a max_prefix far above the lengths."""
    c = make(8, 1, N, H, 512, [P], BF, 128)
    wide = np.full((1, 400), -1, np.int32)
    wide[:, :c["table"].shape[1]] = c["table"]
    c["table"] = wide
    check(c, *call(c, max_prefix=400 * 128))
    check(c, *call(c))


def test_many_sequences_and_refused_ones_among_them(lib):
    prefix = [(i * 53) % 400 for i in range(150)]
    for N, H in ((1, 7), (3, 33)):
        c = make(9, 150, N, H, 256, prefix, BF, 128)
        bad = [i for i in range(150) if i % 7 == 3 or 40 < i < 80]
        p = list(prefix)
        for i in bad:
            p[i] = 401
        out, st = call(c, prefix=i32(p), max_prefix=400)
        assert int(st.item()) == sv.DEV_CAPACITY and bool((out[bad] == 7.0).all())
        st.zero_()
        check(c, out, st, skip=bad)


@pytest.mark.parametrize("N,H", [(20, 8), (1, 16)])
def test_a_pool_whose_offsets_pass_32_bits(lib, N, H):
    """Rows past 2^31 elements and past 2^32 bytes of the pool."""
    D, page, nb = 576, 128, 33000
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.empty(nb, page, D, dtype=BF, device="cuda")
    used = [nb - 1, 3, 29300, nb - 2]
    for b in used:
        pool[b] = torch.randn(page, D, generator=g, device="cuda").to(BF)
    c = make(10, 1, N, H, 512, [470], BF, 0)
    c["cache"] = torch.cat([pool[b] for b in used])[None].cpu()
    out = torch.empty(1, N, H, 512, dtype=BF, device="cuda")
    st = zeros_i32(1)
    sv.tree_attn_verify_latent_paged(c["q"].cuda(), pool, i32([used]), c["tree"].cuda(), i32([470]), words(c["mask"]), out,
                                     470, SCALE, dev_status=st)
    check(c, out, st)


@pytest.mark.parametrize("N,H,dtype", [(20, 8, BF), (1, 16, BF), (3, 4, F32)])
def test_captured_replayed_on_other_lengths_and_repeatable(lib, N, H, dtype):
    c = make(12, 4, N, H, 512, [700, 20, 0, 333], dtype, 128)
    size = sv.tree_attn_latent_workspace_bytes(dtype, 4, N, H, 512, 64, 700)
    ws = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    q, pool, tab, tree, mask = c["q"].cuda(), c["pool"].cuda(), i32(c["table"]), c["tree"].cuda(), words(c["mask"])
    p, out, st = i32(c["prefix"]), torch.empty(4, N, H, 512, dtype=dtype, device="cuda"), zeros_i32(1)
    run = lambda: sv.tree_attn_verify_latent_paged(q, pool, tab, tree, p, mask, out, 700, SCALE, workspace=ws, dev_status=st)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run()
    side.synchronize()
    check(c, out, st)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lengths in ([700, 20, 0, 333], [1, 0, 0, 300], [650, 20, 0, 7], [700, 20, 0, 333]):
        p.copy_(i32(lengths))
        out.fill_(9.0)
        ws.fill_(255)                       # nothing in it needs to start at any value
        graph.replay()
        torch.cuda.synchronize()
        check(dict(c, prefix=lengths), out, st)
    assert torch.equal(out, first)


def test_two_calls_at_once(lib):
    """Two streams, their own workspaces, both large enough to fill the GPU."""
    cs = [make(20 + i, 6, 16, 16, 512, [1500 - 100 * j for j in range(6)], BF, 128) for i in range(2)]
    alone = [call(c)[0] for c in cs]
    torch.cuda.synchronize()
    args = [(c["q"].cuda(), c["pool"].cuda(), i32(c["table"]), c["tree"].cuda(), i32(c["prefix"]), words(c["mask"]))
            for c in cs]
    size = sv.tree_attn_latent_workspace_bytes(BF, 6, 16, 16, 512, 64, 1500)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in cs]
    outs, sts = [torch.empty_like(a) for a in alone], [zeros_i32(1) for _ in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for a, w, o, t, s in zip(args, ws, outs, sts, streams):
            with torch.cuda.stream(s):
                sv.tree_attn_verify_latent_paged(*a, o, 1500, SCALE, workspace=w, dev_status=t)
    torch.cuda.synchronize()
    for a, o, t in zip(alone, outs, sts):
        assert int(t.item()) == 0 and torch.equal(a, o)


def test_views_at_sixteen_byte_offsets(lib):
    """Tensors that begin anywhere on a 16-byte boundary of their storage."""
    for N, H, dtype in ((20, 8, BF), (2, 5, BF), (2, 5, F32)):
        c = make(13, 2, N, H, 256, [200, 300], dtype, 0)
        step = 16 // c["q"].element_size()

        def moved(x):
            flat = torch.empty(x.numel() + step, dtype=x.dtype, device="cuda")
            flat[step:] = x.flatten().cuda()
            return flat[step:].view(x.shape)
        out, st = moved(torch.zeros(2, N, H, 256, dtype=dtype)), zeros_i32(1)
        sv.tree_attn_verify_latent(moved(c["q"]), moved(c["cache"]), moved(c["tree"]), i32(c["prefix"]), words(c["mask"]), out,
                                   300, SCALE, dev_status=st)
        check(c, out, st)


def test_wrapper_refuses(lib):
    B, N, H, D = 2, 3, 4, 576
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    good = dict(q=z(B, N, H, D), cache=z(B, 100, D), tree=z(B, N, D), prefix_len=zeros_i32(B), anc_mask=z(B, N, dt=torch.int64),
                out=z(B, N, H, 512), max_prefix=90, scale=SCALE)
    sv.tree_attn_verify_latent(**good)
    for kw in (dict(q=z(B, N, H, D, dt=torch.float16)), dict(cache=z(B, 100, 512)), dict(cache=z(B + 1, 100, D)),
               dict(cache=z(B, 100, D, dt=F32)), dict(tree=z(B, N + 1, D)), dict(out=z(B, N, H, D)), dict(max_prefix=101),
               dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(prefix_len=zeros_i32(B + 1)),
               dict(anc_mask=z(B, N + 1, dt=torch.int64)), dict(q=z(B, N, H, D).cpu()), dict(tree=z(B, D, N).transpose(1, 2)),
               dict(workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), dict(q=z(B, N, H, 192), tree=z(B, N, 192),
                                                                                      cache=z(B, 100, 192), out=z(B, N, H, 128))):
        with pytest.raises((ValueError, TypeError, KeyError, sv.SpecError)):
            sv.tree_attn_verify_latent(**{**good, **kw})
    paged = dict(good, pages=z(4, 128, D), block_table=torch.zeros(B, 2, dtype=torch.int32, device="cuda"))
    del paged["cache"]
    sv.tree_attn_verify_latent_paged(**paged)
    for kw in (dict(pages=z(4, 64, D)), dict(pages=z(4, 192, D)), dict(block_table=z(B, 2)), dict(max_prefix=257),
               dict(block_table=torch.zeros(B + 1, 2, dtype=torch.int32, device="cuda"))):
        with pytest.raises((ValueError, TypeError, sv.SpecError)):
            sv.tree_attn_verify_latent_paged(**{**paged, **kw})


@pytest.mark.parametrize("B,N,H,lat,lo,hi", [(70, 1, 64, 256, 300, 340), (66, 1, 33, 256, 700, 700), (30, 6, 64, 256, 128, 140),
                                             (45, 2, 100, 512, 0, 60), (140, 1, 16, 256, 200, 256), (33, 1, 16, 512, 0, 130)])
def test_units_that_are_not_cut(lib, B, N, H, lat, lo, hi):
    """Whole units a part, one or several, with sequences that are refused among them."""
    prefix = [lo + (31 * i) % (hi - lo + 1) for i in range(B)]
    c = make(21, B, N, H, lat, prefix, BF, 128)
    out, st = call(c)
    check(c, out, st)
    refused = [b for b in (0, 31, 32, B - 1) if b < B]
    other = list(prefix)
    for b in refused:
        other[b] = -1 if b % 2 else max(prefix) + 1
    again, st = call(c, prefix=i32(other))
    assert int(st.item()) == sv.DEV_CAPACITY
    check(c, again, zeros_i32(1), skip=refused)
    for b in refused:
        assert bool((again[b] == 7.0).all())


def test_parts_in_halves_of_a_unit(lib):
    """Six units over more rows than L2 holds: 75 parts instead of 76."""
    c = make(22, 2, 3, 90, 256, [82000, 82000], BF, 0)
    check(c, *call(c))


@pytest.mark.parametrize("H,lat,P", [(4, 512, 3200), (9, 256, 9001), (16, 512, 2047)])
def test_float32_in_many_ranges(lib, H, lat, P):
    c = make(23, 1, 1, H, lat, [P], F32, 0)
    check(c, *call(c))
