"""GPU parity: acceptance from given probabilities and given uniform numbers.

Every output is an integer and has to equal the 64-bit oracle's.  The two
disagree only where a number falls within about 2^-45 of a border (sums of
float64 there, of 2^-58 units here), which these seeded inputs do not hold.
"""
import numpy as np
import pytest
import torch

from _util import dev, host, i32, zeros_i32
from oracle import accept as ACC
from oracle import tree as T
from tree_speculative_decoding_attn_gb300 import specverify as sv
from tree_speculative_decoding_attn_gb300 import synth

pytestmark = pytest.mark.gpu


def probs(g, shape, std, dtype):
    z = g.standard_normal(shape) * std
    e = np.exp(z - z.max(-1, keepdims=True))
    p = (e / e.sum(-1, keepdims=True)).astype(np.float32)
    return synth.round_bf16(p) if dtype == torch.bfloat16 else p


class Case:
    def __init__(self, B, V, shapes, draft, dtype=torch.float32, seed=0, std=2.0):
        g = np.random.default_rng(seed)
        self.B, self.V, self.dtype = B, V, dtype
        shapes = shapes if isinstance(shapes, list) else [shapes] * B
        self.N = N = shapes[0].n
        self.par = np.stack([s.parents for s in shapes]).astype(np.int32)
        links = [T.child_links(s.parents) for s in shapes]
        self.fc, self.ns = (np.stack([x[k] for x in links]).astype(np.int32) for k in (0, 1))
        self.cap = max(int(T.depth_and_mask(s.parents)[0].max()) for s in shapes) + 1
        self.p = probs(g, (B, N, V), std, dtype)
        self.q = probs(g, (B, N, V), std, dtype) if draft else None
        self.tok = np.zeros((B, N), np.int32)
        for b in range(B):
            best = np.argsort(-self.p[b], axis=-1)
            for i in range(1, N):
                v = self.par[b, i]
                if draft:                     # a draw of the drafter
                    c = np.cumsum(self.q[b, v].astype(np.float64))
                    self.tok[b, i] = min(V - 1, np.searchsorted(c, g.random() * c[-1], side="right"))
                else:                         # one of the target's better tokens, now and then a repeated one
                    self.tok[b, i] = best[v, int(g.integers(0, min(V, 12)))]
        self.u, self.ub = g.random((B, N)).astype(np.float32), g.random(B).astype(np.float32)

    def run(self, cap=None, p=None):
        cap = self.cap if cap is None else cap
        o = [zeros_i32(self.B), zeros_i32(self.B, cap), zeros_i32(self.B)]
        st = zeros_i32(1)
        sv.spec_verify_probs(dev(self.p, self.dtype) if p is None else p, i32(self.tok), i32(self.par), i32(self.fc),
                             i32(self.ns), dev(self.u), dev(self.ub), *o,
                             draft_probs=None if self.q is None else dev(self.q, self.dtype), dev_status=st)
        return [host(x) for x in o] + [int(st.item())]

    def check(self):
        *got, status = self.run()
        ref = ACC.accept_probs(self.p, self.q, self.tok, self.fc, self.ns, self.u, self.ub, self.cap)
        assert status == 0
        for x, y in zip(got, ref):
            np.testing.assert_array_equal(x, y)
        return got


R = synth.random_tree
CASES = [
    (3, 1, synth.chain(1)),
    (4, 7, synth.chain(4)),
    (16, 1000, R(1, 20, (4, 3, 2))),
    (5, 32001, R(2, 60, (10, 4, 3, 2, 2))),
    (2, 50257, R(3, 64, (8, 4, 3, 2, 2))),
    (2, 1003, synth.chain(256)),
    (70, 333, R(4, 32, (4, 3, 2))),
    (3, 2048, R(5, 256, (16, 6, 4))),
    (1, 128256, R(6, 17, (16,))),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_the_oracle(case, draft, dtype):
    B, V, shape = CASES[case]
    for s, std in ((0, 1.0), (1, 4.0), (2, 12.0)):   # flat rows, and rows of a few likely tokens
        Case(B, V, shape, draft, dtype, seed=31 * case + s, std=std).check()


def test_many_small_draws_with_drafts_near_the_target():
    """Siblings are rejected now and then, up to several in a row."""
    hit = 0
    for seed in range(10):
        c = Case(64, 50, R(7, 30, (6, 4)), True, seed=seed, std=1.0)
        g = np.random.default_rng(seed + 1000)
        c.q = (c.p * (0.7 + 0.6 * g.random(c.p.shape))).astype(np.float32)
        c.q /= c.q.sum(-1, keepdims=True)
        hit += c.check()[0].sum()
    assert hit > 100


def test_many_siblings_of_a_drafter_that_is_far_off():
    """The target never has what the drafter draws: every sibling is refused
    and the residual's weight on the drafter grows by about one each time."""
    for n, seed in ((18, 0), (60, 1), (255, 2)):
        c = Case(4, 40, R(seed, n + 1, (n,)), True, seed=seed)
        c.q[:] = 0
        c.q[:, :, 3], c.q[:, :, 5] = 0.75, 0.25
        c.p[:] = 0
        c.p[:, :, 3], c.p[:, :, 5], c.p[:, :, 9], c.p[:, :, 11] = 1e-3, 2e-3, 0.497, 0.5
        c.tok[:, 1:] = np.where(np.random.default_rng(seed).random((4, n)) < 0.75, 3, 5)
        c.u[:] = 0.999
        *got, status = c.run()
        ref = ACC.accept_probs(c.p, c.q, c.tok, c.fc, c.ns, c.u, c.ub, c.cap)
        assert status == 0 and (got[0] == 0).all()
        for x, y in zip(got, ref):
            np.testing.assert_array_equal(x, y)


def test_numbers_at_the_ends():
    for u, ub in ((0.0, 0.0), (0.0, 1.0), (1.0, 0.0), (1.0, 1.0), (np.nan, np.nan), (-1.0, 2.0)):
        for draft in (False, True):
            c = Case(4, 99, R(7, 30, (6, 4)), draft, seed=3)
            c.u[:], c.ub[:] = u, ub
            *got, status = c.run()
            clean = lambda x: np.where(np.nan_to_num(x, nan=-1) <= 0, 0, np.minimum(x, 1 - 2.0 ** -24)).astype(np.float32)  # noqa: E731
            ref = ACC.accept_probs(c.p, c.q, c.tok, c.fc, c.ns, clean(c.u), clean(c.ub), c.cap)
            assert status == 0
            for x, y in zip(got, ref):
                np.testing.assert_array_equal(x, y)


def test_a_residual_of_nothing_gives_way_to_the_target():
    c = Case(3, 64, synth.chain(2), True, seed=1)
    c.q = c.p.copy()                          # p = q: nothing is left after a rejection
    c.u[:] = 1.0                              # and only u q < p keeps a draft ...
    c.p[:, 0, c.tok[:, 1]] *= 0.5             # ... which this one is not
    c.check()
    d = Case(3, 4, R(1, 5, (4,)), False, seed=1)
    d.tok[:, 1:] = np.arange(4)               # every token drafted, every draft refused
    d.p[:] = 0.25
    d.u[:] = 1.0
    d.p[:, 0] = [0.25, 0.25, 0.25, 0.1]
    d.check()


def test_zeros_repeats_and_one_hot_rows():
    c = Case(8, 40, R(7, 30, (6, 4)), False, seed=3)
    c.tok[:, 2] = c.tok[:, 1]                 # siblings or not: a repeated token
    c.p[:, ::3] = 0
    c.p[:, ::3, 7] = 1
    c.check()
    d = Case(8, 40, R(7, 30, (6, 4)), True, seed=3)
    d.q[:, ::2] = 0
    d.q[:, ::2, 11] = 1
    d.tok[:, 1:] = 11
    d.check()


@pytest.mark.parametrize("draft", [False, True])
def test_device_errors(draft):
    bad_token = Case(2, 100, R(7, 30, (6, 4)), draft, seed=3)
    bad_token.tok[0, bad_token.fc[0, 0]] = 100
    *got, status = bad_token.run()
    assert status == sv.DEV_BAD_TOKEN and got[1][0, 1] != bad_token.fc[0, 0]
    loop = Case(2, 100, R(7, 30, (6, 4)), draft, seed=3)
    loop.u[:] = 1.0
    loop.ns[0, loop.fc[0, 0]] = loop.fc[0, 0]
    *got, status = loop.run()
    assert status == sv.DEV_BAD_PARENTS and got[0][0] == 0
    stray = Case(2, 100, R(7, 30, (6, 4)), draft, seed=3)
    stray.par[0, 1:] = [1 << 30, -5] * 14 + [3]
    assert stray.run()[3] == sv.DEV_BAD_PARENTS
    short = Case(2, 100, synth.chain(6), draft, seed=3)
    short.u[:] = 0.0
    *got, status = short.run(cap=3)
    assert status == sv.DEV_CAPACITY and (got[0] == 2).all() and (got[1] == [0, 1, 2]).all()
    for value in (np.nan, -0.5, 1.5, np.inf):
        prob = Case(2, 100, R(7, 30, (6, 4)), draft, seed=3)
        prob.p[0, :, 50] = value
        *got, status = prob.run()
        assert status == sv.DEV_BAD_PROB
        prob.p[0, :, 50] = 0
        ref = ACC.accept_probs(prob.p, prob.q, prob.tok, prob.fc, prob.ns, prob.u, prob.ub, prob.cap)
        for x, y in zip(got, ref):
            np.testing.assert_array_equal(x, y)
    for V, value in ((100, 1.0), (70001, 0.5), (128256, 1.0)):        # no distribution: sums far past 1
        flood = Case(2, V, synth.chain(2), draft, seed=3)
        flood.p[0] = value
        flood.u[0] = 1.0
        flood.tok[0, 1] = 0
        flood.p[0, :, 0] = 0
        *got, status = flood.run()
        assert status == sv.DEV_BAD_PROB and got[0][0] == 0 and got[2][0] == 0
    empty = Case(2, 100, R(7, 30, (6, 4)), draft, seed=3)
    empty.p[0] = 0
    *got, status = empty.run()
    assert status == sv.DEV_BAD_PROB and got[0][0] == 0 and got[2][0] == 0


def test_rows_whose_offsets_pass_32_bits():
    """2 x 64 x 35 000 000 bf16 probabilities of which the last node's row decides."""
    V, N = 35_000_000, 64
    c = Case(1, 8, synth.chain(N), False, seed=3)
    p = torch.zeros((1, N, V), dtype=torch.bfloat16, device="cuda")
    c.tok[0] = V - 1 - np.arange(N)
    for i in range(N - 1):
        p[0, i, int(c.tok[0, i + 1])] = 1
    p[0, N - 1, V - 3], p[0, N - 1, 5] = 0.5, 0.5
    c.V, c.u[:] = V, 0.5
    for ub, want in ((0.25, 5), (0.75, V - 3)):
        c.ub[:] = ub
        *got, status = c.run(p=p)
        assert status == 0 and got[0][0] == N - 1 and got[2][0] == want


def test_on_another_stream_and_captured():
    c = Case(8, 5000, R(7, 30, (6, 4)), True, seed=5)
    want = c.check()
    t = [dev(c.p), i32(c.tok), i32(c.par), i32(c.fc), i32(c.ns), dev(c.u), dev(c.ub)]
    o, q = [zeros_i32(8), zeros_i32(8, c.cap), zeros_i32(8)], dev(c.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.spec_verify_probs(*t, *o, draft_probs=q)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(o, want):
        np.testing.assert_array_equal(host(x), y)
        x.zero_()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        sv.spec_verify_probs(*t, *o, draft_probs=q)
    s.synchronize()
    for x, y in zip(o, want):
        np.testing.assert_array_equal(host(x), y)


def test_wrapper_refuses():
    c = Case(2, 64, synth.chain(3), True, seed=3)
    p, q = dev(c.p), dev(c.q)
    t = dict(tok=i32(c.tok), par=i32(c.par), fc=i32(c.fc), ns=i32(c.ns), u=dev(c.u), ub=dev(c.ub), n=zeros_i32(2),
             path=zeros_i32(2, 4), bonus=zeros_i32(2))
    call = lambda p=p, q=q, **kw: sv.spec_verify_probs(p, *dict(t, **kw).values(), draft_probs=q)  # noqa: E731
    call()
    for kw in (dict(q=q.bfloat16()), dict(q=q[:1]), dict(u=t["u"].double()), dict(ub=t["ub"][:1]), dict(tok=t["tok"][:, :2]),
               dict(n=t["n"].long()), dict(path=t["path"][:1]), dict(p=p.cpu())):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    with pytest.raises(sv.SpecError):
        call(p=p.half(), q=q.half())
