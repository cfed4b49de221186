"""GPU: the pair kernel's hand-offs between two SMs under load.  Calls repeat,
alone, beside copies and products on another stream, and beside one another,
and every result has the same bits."""
import numpy as np
import pytest
import torch

import test_gpu_latent as base
from _latent_plan import plan
from _util import i32, zeros_i32
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def prepared(seed, lengths, nodes, heads, latent):
    assert plan(lengths, nodes, heads, latent).kernel == "pairs"
    g, B, D = torch.Generator(device="cuda").manual_seed(seed), len(lengths), latent + 64
    t = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=BF)  # noqa: E731
    words = base.words(base.trees(np.random.default_rng(seed), B, nodes))
    size = sv.tree_attn_latent_workspace_bytes(BF, B, nodes, heads, latent, 64, max(lengths))
    args = [t(B, nodes, heads, D), t(B, max(lengths), D), t(B, nodes, D), i32(lengths), words]
    out, st, ws = t(B, nodes, heads, latent), zeros_i32(1), torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(into):
        sv.tree_attn_verify_latent(*args, into, max(lengths), base.SCALE, workspace=ws, dev_status=st)
        return into
    return run, out, st


# (ends inside a tile, so that rows are cleared; lengths that cut units, and whole units)
CASES = [([900 + 61 * i for i in range(12)], 32, 16, 512), ([3001] * 5, 6, 64, 512), ([1777, 40, 2500], 40, 21, 256),
         ([700] * 64, 1, 64, 512)]


@pytest.mark.parametrize("lengths,nodes,heads,latent", CASES)
def test_repeats_under_load(lib, lengths, nodes, heads, latent):
    run, like, st = prepared(3, lengths, nodes, heads, latent)
    first = run(torch.empty_like(like)).clone()
    torch.cuda.synchronize()
    side, a = torch.cuda.Stream(), torch.randn(2048, 2048, device="cuda", dtype=BF)
    big = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for load in range(3):
        for _ in range(60):
            if load:
                with torch.cuda.stream(side):
                    big.fill_(1) if load == 1 else torch.mm(a, a)
            out = run(torch.full_like(like, 7.0))
            wrong += (out.view(torch.int16) != first.view(torch.int16)).sum()
    torch.cuda.synchronize()
    assert int(wrong) == 0 and int(st.item()) == 0


def test_two_calls_beside_one_another_repeat(lib):
    calls = [prepared(5 + i, *CASES[i]) for i in (0, 1)]
    first = [run(torch.empty_like(like)).clone() for run, like, _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    outs = [torch.empty_like(f) for f in first]
    wrong = [torch.zeros((), dtype=torch.int64, device="cuda") for _ in calls]
    torch.cuda.synchronize()
    for _ in range(60):
        for (run, _, _), o, f, w, s in zip(calls, outs, first, wrong, streams):
            with torch.cuda.stream(s):
                run(o.fill_(7.0))
                w += (o.view(torch.int16) != f.view(torch.int16)).sum()
    torch.cuda.synchronize()
    assert all(int(w) == 0 for w in wrong) and all(int(st.item()) == 0 for _, _, st in calls)
