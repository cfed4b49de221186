"""GPU parity: window tree attention whose bound on the prefix lengths
(max_prefix) is far above them, as a serving loop passes that sizes its calls
by its cache.  Launch plans follow from the bound, the work from the lengths:
parts of which none, some or all are cut, row groups whole, equal ranges, the
few-row kernels, tiles on CUDA cores."""
import numpy as np
import pytest
import torch

from test_gpu_window import Case, R
from tree_speculative_decoding_attn_gb300 import specverify as sv
from tree_speculative_decoding_attn_gb300 import synth

pytestmark = pytest.mark.gpu

BOUND = 8192


class Loose(Case):
    """A case whose cache holds BOUND positions, NaN past the lengths."""

    def __init__(self, *args, **more):
        super().__init__(*args, **more)
        pad = BOUND - self.kc.shape[2]
        self.kc, self.vc = (np.pad(x, ((0, 0), (0, 0), (0, pad), (0, 0)), constant_values=np.nan)
                            for x in (self.kc, self.vc))
        if self.page:
            self.table = np.pad(self.table, ((0, 0), (0, BOUND // self.page - self.table.shape[1])), constant_values=-1)

    def tensors(self):
        t = super().tensors()
        size = sv.tree_attn_window_workspace_bytes(self.dt, self.B, self.N, self.hq, self.hkv, self.D, BOUND,
                                                   self.window, self.sinks)
        t["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
        return t

    def call(self, t):
        super().call(t, mp=BOUND)


CASES = [
    # dtype, B, hq, hkv, D, prefix, tree, window, sinks, page
    ("bf16", 4, 32, 8, 128, [300, 0, 1, 130], R(40, 64, (10, 4, 3, 2, 2)), 4096, 4, 128),  # parts, none cut
    ("bf16", 1, 32, 8, 128, [300], R(41, 60, (10, 4, 3, 2, 2)), 4096, 4, 0),
    ("bf16", 2, 16, 2, 64, [40, 300], R(42, 100, (6, 5, 3)), 5000, 4, 0),
    ("bf16", 4, 32, 8, 128, [300, 0, 2900, 1300], R(43, 64, (10, 4, 3, 2, 2)), 4096, 130, 128),  # ... some cut
    ("bf16", 9, 64, 8, 128, [(97 * i) % 400 for i in range(9)], R(44, 32, (4, 3, 2)), 300, 4, 0),  # whole
    ("bf16", 10, 64, 8, 128, [(97 * i) % 400 for i in range(10)], R(45, 32, (4, 3, 2)), 6000, 4, 128),  # ranges
    ("bf16", 3, 32, 8, 128, [130, 0, 300], synth.chain(1), 1024, 4, 128),  # few rows
    ("f32", 2, 4, 2, 128, [300, 0], R(46, 16, (5, 3)), 500, 4, 0),
    ("f32", 2, 4, 2, 64, [300, 1], R(47, 20, (4, 3, 2)), 6000, 40, 128),   # tiles on CUDA cores
]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_what_follows_the_call_comes_after_all_of_its_work(case, captured):
    """The output is read by a copy queued right behind the call, and the
    workspace is overwritten behind that."""
    c = Loose(*CASES[case], seed=300 + case)
    t = c.tensors()
    copy = torch.zeros_like(t["out"])

    def step():
        c.call(t)
        copy.copy_(t["out"])
        t["ws"].zero_()
    step()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        step = graph.replay
    for _ in range(3):
        t["out"].fill_(float("nan"))
        step()
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    assert torch.equal(copy, t["out"])
    c.check(t)


TOP = 2 ** 31 - 1
SHAPES = [("bf16", 1, 8, 2, 128, 3), ("bf16", 6, 32, 4, 128, 60), ("bf16", 2, 24, 2, 64, 100), ("bf16", 1, 16, 2, 128, 60),
          ("f32", 2, 4, 2, 64, 9)]


@pytest.mark.parametrize("window,sinks", [(TOP, 0), (TOP, TOP), (1, TOP), (1, 0), (TOP - 1, 1), (40, 1 << 25)])
@pytest.mark.parametrize("longest", [0, 1, 700, 4500])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_the_ends_of_the_arguments(shape, longest, window, sinks):
    """The largest and smallest windows and sinks, empty caches, and a scale
    of the caller's."""
    dtype, B, hq, hkv, D, n = SHAPES[shape]
    prefix = [longest * (B - i) // B for i in range(B)]
    tree = synth.chain(n) if n < 6 else R(70 + shape, n, (10, 4, 3, 2, 2) if n > 9 else (4, 3, 2))
    for page in (0, 128):
        c = Case(dtype, B, hq, hkv, D, prefix, tree, min(window, 10 ** 6), min(sinks, 10 ** 6), page, seed=500 + shape)
        c.window, c.sinks = window, sinks
        t = c.tensors()
        c.call(t)
        assert int(t["status"].item()) == 0
        c.check(t)
        # twice the scale on half the queries: the same products, bit for bit
        want, t["q"] = t["out"].clone(), t["q"] * 0.5
        f = sv.tree_attn_verify_window_paged if page else sv.tree_attn_verify_window
        f(t["q"], t["k"], t["v"], *([t["table"]] if page else []), t["kt"], t["vt"], t["prefix"], t["depth"], t["anc"],
          t["out"], c.mp, window, sinks=sinks, scale=2 * float(np.float32(1) / np.sqrt(np.float32(D))), workspace=t["ws"])
        assert torch.equal(t["out"], want)
