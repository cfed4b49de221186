"""GPU parity: tree attention in a sliding window with sinks, contiguous and
paged, against the 64-bit oracle.

Tolerance, from the arithmetic (A = sum p |v| of the row, E = the largest
scale * sum |q||k| of it, J keys):
- a product sum of D terms in float32 is off by at most D 2^-23 of sum |q||k|,
  which moves a probability by twice that relative (numerator and
  denominator): 2 D 2^-23 E;
- the sums over keys, sequential at worst: 2 J 2^-24; exp2, the scale's
  rounding and the division: 2^-20;
- bf16: each probability is rounded to bf16 for the second product, half a
  step 2^-8, and so is the output: 2^-8 |o| (float32: 2^-24 |o|).
"""
import numpy as np
import pytest
import torch

from _util import dev, host, i32, zeros_i32
from oracle import attention as A
from oracle import tree as T
from tree_speculative_decoding_attn_gb300 import specverify as sv
from tree_speculative_decoding_attn_gb300 import synth

pytestmark = pytest.mark.gpu


def tolerance(ref, mag, big, dtype, D, J):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24
    p = half if dtype == torch.bfloat16 else 0.0
    return half * np.abs(ref) + mag * (p + 2 * D * 2.0 ** -23 * big + 2 * J * 2.0 ** -24 + 2.0 ** -20) * (1 + half)


class Case:
    """Inputs of one call; ``page`` 0 is a contiguous cache, otherwise the
    blocks outside the window are not even in the table."""

    def __init__(self, dtype, B, hq, hkv, D, prefix, shapes, window, sinks, page=0, q_scale=1.0, seed=0, fill=None):
        g = np.random.default_rng(seed)
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        self.B, self.hq, self.hkv, self.D, self.page = B, hq, hkv, D, page
        self.window, self.sinks, self.prefix = window, sinks, np.asarray(prefix, np.int32)
        shapes = shapes if isinstance(shapes, list) else [shapes] * B
        self.N = N = shapes[0].n
        dm = [T.depth_and_mask(s.parents) for s in shapes]
        self.depth, self.mask = np.stack([x[0] for x in dm]), np.stack([x[1] for x in dm])
        rnd = lambda *s: (lambda x: synth.round_bf16(x) if dtype == "bf16" else x)(  # noqa: E731
            g.standard_normal(s).astype(np.float32))
        self.mp = int(self.prefix.max())
        S = -(-(self.mp + 5) // page) * page if page else self.mp + 5
        self.q, self.kt, self.vt = rnd(B, N, hq, D) * q_scale, rnd(B, hkv, N, D), rnd(B, hkv, N, D)
        self.kc, self.vc = rnd(B, hkv, S, D), rnd(B, hkv, S, D)
        if fill is not None:             # what no node may see
            for b, P in enumerate(self.prefix):
                dead = [x for x in range(S) if x >= P or (x >= sinks and P - x >= window)]
                self.kc[b, :, dead], self.vc[b, :, dead] = fill
        if page:
            ids = g.permutation(B * (S // page) + 2)
            self.table = np.full((B, S // page), -1, np.int32)
            self.kp = np.full((len(ids), hkv, page, D), np.nan, np.float32)
            self.vp = self.kp.copy()
            for b, P in enumerate(self.prefix):
                for j in range(-(-int(P) // page)):
                    at = np.arange(j * page, (j + 1) * page)
                    if not ((at < P) & ((at < sinks) | (P - at < window))).any():
                        continue
                    self.table[b, j] = ids[b * (S // page) + j]
                    self.kp[self.table[b, j]] = self.kc[b, :, at].swapaxes(0, 1)
                    self.vp[self.table[b, j]] = self.vc[b, :, at].swapaxes(0, 1)

    def tensors(self):
        words = np.stack([T.mask_words_multi(m) for m in self.mask])
        t = dict(q=dev(self.q, self.dt), kt=dev(self.kt, self.dt), vt=dev(self.vt, self.dt), prefix=i32(self.prefix),
                 depth=i32(self.depth), anc=dev(words.view(np.int64)), status=zeros_i32(1),
                 out=torch.full(self.q.shape, float("nan"), dtype=self.dt, device="cuda"))
        if self.page:
            t.update(k=dev(self.kp, self.dt), v=dev(self.vp, self.dt), table=i32(self.table))
        else:
            t.update(k=dev(self.kc, self.dt), v=dev(self.vc, self.dt))
        size = sv.tree_attn_window_workspace_bytes(self.dt, self.B, self.N, self.hq, self.hkv, self.D, self.mp,
                                                   self.window, self.sinks)
        t["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        return t

    def call(self, t, mp=None):
        more = dict(sinks=self.sinks, workspace=t["ws"], dev_status=t["status"])
        mp = self.mp if mp is None else mp
        if self.page:
            sv.tree_attn_verify_window_paged(t["q"], t["k"], t["v"], t["table"], t["kt"], t["vt"], t["prefix"],
                                             t["depth"], t["anc"], t["out"], mp, self.window, **more)
        else:
            sv.tree_attn_verify_window(t["q"], t["k"], t["v"], t["kt"], t["vt"], t["prefix"], t["depth"], t["anc"],
                                       t["out"], mp, self.window, **more)

    def check(self, t, rows=slice(None)):
        got = host(t["out"])
        finite = [np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) for x in (self.kc, self.vc)]
        ref, mag, big = A.tree_attention_window(self.q, *finite, self.kt, self.vt, self.prefix, self.depth, self.mask,
                                                self.window, self.sinks)
        J = min(self.mp, self.window) + min(self.sinks, self.mp) + self.N
        excess = np.abs(got - ref) - tolerance(ref, mag, big, self.dt, self.D, J)
        assert np.isfinite(got[rows]).all()
        assert (excess[rows] <= 0).all(), float(excess[rows].max())


R = synth.random_tree
CASES = [
    # dtype, B, hq, hkv, D, prefix, tree(s), window, sinks, page
    ("f32", 1, 4, 4, 64, [131], R(1, 5, (2, 2)), 50, 4, 0),
    ("f32", 2, 6, 2, 128, [300, 0], R(2, 20, (4, 3, 2)), 128, 0, 128),
    ("f32", 2, 4, 1, 64, [90, 257], R(3, 70, (6, 5, 4)), 3, 1, 0),          # a window shorter than the tree is deep
    ("bf16", 2, 8, 2, 64, [500, 33], R(4, 12, (3, 3)), 100, 70, 0),
    ("bf16", 3, 24, 4, 64, [900, 4, 2000], R(18, 100, (6, 5, 3)), 700, 130, 128),  # head_dim 64, two mask words, ranges
    ("bf16", 1, 4, 4, 64, [5000], R(19, 200, (8, 6, 4, 3)), 3000, 30, 0),   # ... parts, two tree tiles
    ("bf16", 9, 32, 8, 64, [(211 * i) % 1500 for i in range(9)], synth.chain(1), 300, 4, 128),
    ("bf16", 1, 32, 8, 128, [2000], synth.chain(1), 1024, 4, 0),            # one token
    ("bf16", 3, 8, 8, 128, [1, 0, 700], synth.chain(1), 256, 0, 128),
    ("bf16", 4, 32, 8, 128, [900, 128, 4, 1500], R(5, 60, (10, 4, 3, 2, 2)), 512, 4, 128),
    ("bf16", 2, 64, 8, 128, [1300, 1111], R(6, 32, (4, 3, 2)), 300, 130, 0),
    ("bf16", 2, 14, 2, 128, [400, 1000], R(7, 9, (3, 3)), 200, 5, 0),       # seven heads a KV head
    ("bf16", 2, 12, 4, 128, [640, 130], R(8, 33, (6, 4, 2)), 129, 128, 256),  # three
    ("bf16", 2, 16, 8, 128, [700, 260], R(9, 256, (8, 6, 4, 3)), 64, 4, 0),  # two tree tiles
    ("bf16", 1, 16, 2, 128, [385], R(10, 100, (6, 5, 3)), 2, 3, 128),       # almost nothing but sinks
    ("bf16", 2, 8, 2, 128, [260, 5], R(11, 16, (4, 3)), 1, 0, 0),           # itself only
    ("bf16", 2, 8, 1, 128, [77, 1024], R(12, 64, (8, 4, 3, 2, 2)), 100000, 9, 0),  # a window over everything
    ("bf16", 1, 8, 1, 128, [9000], R(13, 32, (4, 3, 2)), 8000, 16, 0),      # one row group across every SM
    ("bf16", 3, 16, 2, 128, [3000, 40, 900], R(15, 40, (6, 4, 2)), 2500, 200, 128),  # many parts, few, one
    ("bf16", 2, 8, 2, 128, [4000, 1], R(16, 200, (8, 6, 4, 3)), 3000, 7, 0),  # parts of four row groups a KV head
    ("bf16", 5, 64, 8, 128, [6000, 5000, 0, 300, 6100], R(17, 24, (4, 3, 2)), 5000, 4, 128),  # equal ranges
    ("bf16", 70, 4, 2, 128, [(37 * i) % 300 for i in range(70)], R(14, 8, (3, 2)), 90, 4, 0),
    # few rows and keys, joined by a cluster: sixteen CTAs, short prefixes that leave CTAs idle, one CTA, two rounds
    ("f32", 1, 4, 4, 64, [1001], R(20, 5, (2, 2)), 333, 4, 0),
    ("f32", 2, 6, 3, 128, [470, 3], R(21, 16, (5, 3)), 450, 7, 128),
    ("f32", 1, 8, 1, 128, [0], R(22, 7, (3, 2)), 9, 2, 0),
    ("f32", 1, 2, 2, 64, [2000], R(23, 40, (5, 3, 2)), 400, 33, 0),
    # ... groups of heads too wide for the tensor cores
    ("bf16", 1, 160, 1, 64, [800], synth.chain(1), 300, 4, 0),
    ("bf16", 2, 130, 1, 128, [500, 90], synth.chain(3), 2000, 4, 128),
    ("bf16", 1, 32, 8, 128, [5000], synth.chain(1), 4000, 4, 128),          # 251 keys a CTA
    ("bf16", 40, 16, 8, 128, [(97 * i) % 700 for i in range(40)], synth.chain(1), 256, 4, 0),  # clusters of one
    ("f32", 1, 8, 2, 128, [1500], R(25, 100, (6, 5, 3)), 900, 30, 128),     # row groups, two mask words
    # past what a cluster takes: tiles on CUDA cores and a merge; one token over a long window
    ("f32", 1, 2, 1, 64, [9000], R(26, 30, (5, 3, 2)), 5000, 4, 0),
    ("bf16", 8, 32, 8, 128, [3000, 1, 2950, 0, 130, 2000, 2999, 257], synth.chain(1), 2900, 4, 128),
    ("f32", 2, 4, 2, 128, [6000, 0], R(32, 70, (6, 5, 4)), 5000, 40, 128),
    # enough rows for the SM-pair kernel: windows shorter than the tree, itself only, everything
    ("bf16", 8, 32, 8, 128, [385, 0, 5, 1000, 128, 700, 1, 64], R(27, 60, (10, 4, 3, 2, 2)), 2, 3, 128),
    ("bf16", 8, 32, 8, 128, [260, 5, 0, 999, 128, 700, 1, 64], R(28, 60, (10, 4, 3, 2, 2)), 1, 0, 0),
    ("bf16", 8, 56, 8, 128, [260, 5, 0, 999, 128, 700, 1, 64], R(29, 64, (8, 4, 3, 2, 2)), 100000, 9, 128),
    ("bf16", 8, 24, 8, 64, [260, 5, 0, 999, 128, 700, 1, 64], R(30, 150, (8, 6, 4, 3)), 200, 70, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_window_matches_the_oracle(case):
    c = Case(*CASES[case], seed=case)
    t = c.tensors()
    c.call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    c.check(t)


@pytest.mark.parametrize("case", [3, 4, 5, 9, 10, 11, 13, 14])
def test_peaky_scores(case):
    c = Case(*CASES[case], q_scale=4.0, seed=100 + case)
    t = c.tensors()
    c.call(t)
    c.check(t)


@pytest.mark.parametrize("case", [0, 3, 4, 6, 7, 10, 11, 12, 14])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -3e38])
def test_rows_nobody_sees_may_hold_anything(case, fill):
    c = Case(*CASES[case], seed=200 + case, fill=(fill, fill))
    t = c.tensors()
    c.call(t)
    c.check(t)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
def test_empty_masks_give_zeros(dtype, D):
    c = Case(dtype, 2, 8, 2, D, [0, 500], R(3, 10, (3, 3)), 40, 0, seed=3)
    c.mask[:, 4] = False
    t = c.tensors()
    c.call(t)
    c.check(t)
    assert (host(t["out"])[0, 4] == 0).all() and (host(t["out"])[1, 4] != 0).any()


def test_scores_that_jump_from_tile_to_tile():
    """Keys scaled by 1.5 per 128: every tile's scores exceed the running max."""
    c = Case("bf16", 2, 16, 4, 128, [1200, 900], R(5, 64, (4, 4, 4)), 1000, 4, seed=23)
    c.kc = synth.round_bf16(c.kc * (1.5 ** (np.arange(c.kc.shape[2]) // 128)).astype(np.float32)[None, None, :, None])
    t = c.tensors()
    c.call(t)
    c.check(t)


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
def test_a_prefix_beyond_its_bound_is_reported(dtype, D):
    c = Case(dtype, 3, 8, 2, D, [300, 900, 2000], R(2, 8, (3, 2)), 100, 4, seed=1)
    t = c.tensors()
    c.call(t, mp=1000)
    assert int(t["status"].item()) == sv.DEV_CAPACITY
    c.check(t, rows=slice(0, 2))
    assert np.isnan(host(t["out"])[2]).all()


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
def test_a_bad_block_is_reported_where_it_is_read(dtype, D):
    c = Case(dtype, 2, 8, 2, D, [600, 600], R(2, 8, (3, 2)), 100, 0, page=128, seed=1)
    t = c.tensors()
    t["table"][0, 0] = 1 << 20            # outside the window: not read
    c.call(t)
    assert int(t["status"].item()) == 0
    c.check(t)
    t["table"][1, 4] = 1 << 20
    c.call(t)
    assert int(t["status"].item()) == sv.DEV_BAD_BLOCK
    c.check(t, rows=slice(0, 1))


def test_depths_out_of_range_count_as_the_nearest():
    c = Case("bf16", 1, 8, 2, 128, [500], R(2, 8, (3, 2)), 100, 4, seed=1)
    c.depth[0, 3], c.depth[0, 5] = -1000000, 1 << 30
    t = c.tensors()
    c.call(t)
    c.depth[0, 3], c.depth[0, 5] = 0, 7
    c.check(t)


def test_two_streams_and_a_captured_graph():
    """Two calls that overlap, each with a workspace of its own, and one
    captured and replayed on new inputs."""
    a, b = (Case("bf16", 2, 32, 8, 128, [3000, 700], R(s, 32, (4, 3, 2)), 600, 4, page=128, seed=s) for s in (1, 2))
    ta, tb = a.tensors(), b.tensors()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.call(ta)
        with torch.cuda.stream(s2):
            b.call(tb)
    torch.cuda.synchronize()
    a.check(ta)
    b.check(tb)
    want = ta["out"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call(ta)
    ta["out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ta["out"], want)
    for k in ("q", "k", "v", "kt", "vt", "prefix", "table", "depth", "anc"):
        if ta[k].shape == tb[k].shape:
            ta[k].copy_(tb[k])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ta["out"], tb["out"])


def many(page=0, seed=1, **more):
    """Enough rows for the SM-pair kernel, with an empty prefix among them."""
    return Case("bf16", 8, 32, 8, 128, [900, 0, 33, 500, 256, 1000, 700, 64], R(31, 60, (10, 4, 3, 2, 2)), 300, 4,
                page=page, seed=seed, **more)


@pytest.mark.parametrize("fill", [float("nan"), float("-inf")])
@pytest.mark.parametrize("page", [0, 128])
def test_many_rows_nobody_sees_may_hold_anything(page, fill):
    c = many(page, fill=(fill, fill))
    t = c.tensors()
    c.call(t)
    c.check(t)


def test_many_rows_with_empty_masks_and_depths_out_of_range():
    c = many()
    c.mask[:, 4] = False
    c.depth[:, 7], c.depth[:, 9] = -5, 1 << 30
    t = c.tensors()
    c.call(t)
    c.depth[:, 7], c.depth[:, 9] = 0, c.N - 1
    c.check(t)
    assert (host(t["out"])[1, 4] == 0).all()


def test_many_rows_report_a_bound_and_a_block():
    c = many(128)
    t = c.tensors()
    c.call(t, mp=950)
    assert int(t["status"].item()) == sv.DEV_CAPACITY
    good = [0, 1, 2, 3, 4, 6, 7]
    c.check(t, rows=good)
    assert np.isnan(host(t["out"])[5]).all()
    t = c.tensors()
    t["table"][5, 2] = 1 << 20            # outside the window: not read
    c.call(t)
    assert int(t["status"].item()) == 0
    c.check(t)
    t["table"][5, 6] = 1 << 20
    c.call(t)
    assert int(t["status"].item()) == sv.DEV_BAD_BLOCK
    c.check(t, rows=good)


def test_many_rows_on_two_streams_and_in_a_graph():
    a, b = many(128, seed=1), many(128, seed=2)
    ta, tb = a.tensors(), b.tensors()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.call(ta)
        with torch.cuda.stream(s2):
            b.call(tb)
    torch.cuda.synchronize()
    a.check(ta)
    b.check(tb)
    want = ta["out"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.call(ta)
    ta["out"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(ta["out"], want)


def test_a_long_window_in_float32():
    """More keys than a cluster takes: rows nobody sees, an empty mask, a
    prefix beyond its bound, a bad block."""
    c = Case("f32", 3, 4, 2, 64, [5200, 0, 7000], R(33, 20, (4, 3, 2)), 4500, 5, page=128, seed=4,
             fill=(float("nan"), float("nan")))
    c.mask[1, 4] = False
    t = c.tensors()
    c.call(t)
    assert int(t["status"].item()) == 0
    c.check(t)
    assert (host(t["out"])[1, 4] == 0).all()
    t = c.tensors()
    c.call(t, mp=6000)
    assert int(t["status"].item()) == sv.DEV_CAPACITY
    c.check(t, rows=slice(0, 2))
    assert np.isnan(host(t["out"])[2]).all()
    t = c.tensors()
    t["table"][2, 40] = 1 << 20
    c.call(t)
    assert int(t["status"].item()) == sv.DEV_BAD_BLOCK
    c.check(t, rows=slice(0, 2))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 4, 5, 16, 17, 70])
def test_few_rows_of_every_count(dtype, D, n):
    """Row counts around the groups of 4 and 16, prefixes around the blocks
    of 16 keys and the CTAs' shares."""
    c = Case(dtype, 6, 2, 1, D, [0, 1, 15, 16, 129, 777], synth.chain(n), 131, 3, page=128, seed=n)
    t = c.tensors()
    c.call(t)
    assert int(t["status"].item()) == 0
    c.check(t)


def test_paged_equals_contiguous_where_the_tiles_agree():
    """A window over everything: the same tiles in the same order."""
    c = Case("bf16", 2, 32, 8, 128, [700, 300], R(4, 24, (4, 3, 2)), 100000, 0, page=128, seed=9)
    t = c.tensors()
    c.call(t)
    paged = t["out"].clone()
    c.page = 0
    t.update(k=dev(c.kc, c.dt), v=dev(c.vc, c.dt))
    c.call(t)
    assert torch.equal(paged, t["out"])


def test_a_long_cache_whose_offsets_pass_32_bits():
    """One KV head of 2^24.6 rows x 128 in bf16 (about 6.5 GB a side): the
    window lies past element 2^31 and byte 2^32."""
    P = 25_000_000
    c = Case("bf16", 1, 4, 1, 128, [700], R(4, 8, (3, 2)), 300, 4, seed=9)
    t = c.tensors()
    k = torch.empty((1, 1, P + 8, 128), dtype=c.dt, device="cuda")
    v = torch.empty_like(k)
    for big, small in ((k, t["k"]), (v, t["v"])):
        big[0, 0, :4] = small[0, 0, :4]
        big[0, 0, P - 300:P] = small[0, 0, 400:700]
    t.update(k=k, v=v, prefix=i32([P]))
    c.call(t, mp=P)
    assert int(t["status"].item()) == 0
    c.check(t)


def test_wrapper_refuses_what_the_kernel_could_not_check():
    c = Case("bf16", 2, 8, 2, 128, [60, 50], R(2, 8, (3, 2)), 20, 4, seed=1)
    t = c.tensors()
    for key, bad in (("depth", t["depth"][:, :4].contiguous()), ("kt", t["kt"][:1]), ("v", t["v"].float()),
                     ("prefix", t["prefix"].long()), ("anc", t["anc"][:1]), ("out", t["out"][..., :64]),
                     ("q", t["q"].cpu()), ("prefix", t["prefix"].cpu())):
        with pytest.raises((ValueError, TypeError)):
            c.call(dict(t, **{key: bad}))
    with pytest.raises(sv.SpecError):
        c.call(dict(t, **{k: t[k].half() for k in ("q", "k", "v", "kt", "vt", "out")}))
    for w, s in ((0, 0), (5, -1)):
        c.window, c.sinks = w, s
        with pytest.raises(sv.SpecError):
            c.call(t)
