"""GPU: what window tree attention makes of NaN that a row does see, in every
kernel behind the two entry points: the row is NaN, as softmax has it, and no
other row is touched."""
import numpy as np
import pytest
import torch

from _util import host
from test_gpu_window import Case, R
from tree_speculative_decoding_attn_gb300 import synth

pytestmark = pytest.mark.gpu

CASES = [
    # dtype, B, hq, hkv, D, prefix, tree, window, sinks, page
    ("bf16", 2, 8, 2, 128, [700, 20], synth.chain(2), 300, 4, 128),              # few rows, streamed
    ("f32", 2, 4, 2, 64, [700, 20], R(50, 9, (3, 3)), 300, 4, 0),               # few rows
    ("f32", 2, 4, 2, 64, [6500, 20], R(51, 9, (3, 3)), 6000, 40, 128),          # tiles on CUDA cores, merged
    ("bf16", 40, 8, 2, 128, [500 + i for i in range(40)], R(52, 60, (10, 4, 3, 2, 2)), 300, 4, 0),  # SM pairs, whole
    ("bf16", 2, 16, 2, 128, [4000, 300], R(53, 60, (10, 4, 3, 2, 2)), 3500, 4, 128),  # ... parts
    ("bf16", 5, 64, 8, 128, [6000, 5000, 0, 300, 6100], R(17, 24, (4, 3, 2)), 5000, 4, 128),  # ... ranges
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_query_that_is_nan_gives_nan_in_its_row_alone(case):
    c = Case(*CASES[case], seed=400 + case)
    at = [(0, 0, 0), (1, c.N - 1, c.hq - 1), (c.B - 1, c.N // 2, 1)]
    t = c.tensors()
    for b, i, h in at:
        t["q"][b, i, h, c.D - 1] = float("nan")
    c.call(t)
    got = host(t["out"])
    for b, i, h in at:
        assert np.isnan(got[b, i, h]).all()
        t["q"][b, i, h, c.D - 1] = float(c.q[b, i, h, c.D - 1])
    nan = np.isnan(got).any(-1)
    assert nan.sum() == len(set(at))
    # the other rows, against the oracle: the three rows computed again without NaN
    out = t["out"].clone()
    c.call(t)
    for b, i, h in at:
        out[b, i, h] = t["out"][b, i, h]
    t["out"] = out
    c.check(t)


@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_key_that_is_nan_gives_nan_in_the_rows_that_see_it(case):
    """The first sink (seen by every node) of sequence 0's first KV head."""
    c = Case(*CASES[case], seed=420 + case)
    t = c.tensors()
    block = c.table[0, 0] if c.page else 0
    t["k"][block, 0, 0, 3] = float("nan")
    c.call(t)
    nan = np.isnan(host(t["out"]))
    G = c.hq // c.hkv
    assert nan[0, :, :G].all()
    nan[0, :, :G] = False
    assert not nan.any()
