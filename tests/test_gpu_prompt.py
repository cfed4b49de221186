"""GPU parity: causal attention of packed prompt tokens against float64."""
import numpy as np
import pytest
import torch

from _util import i32, zeros_i32
from oracle import latent as LO
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
BF = torch.bfloat16


def bound(q, k, k_rope, q_off, kv_off, size, ref):
    """Scores: float32 sums of 192 products, each addition off by at most
    2^-23 of the sum of sizes, which e^x doubles (weight and normaliser); sums
    over the keys the same; P and the output are rounded to bf16 (2^-8 each)."""
    x = 0.0
    for b in range(len(q_off) - 1):
        kk, rr = np.abs(k[kv_off[b]:kv_off[b + 1]]), np.abs(k_rope[kv_off[b]:kv_off[b + 1]])
        qq = np.abs(q[q_off[b]:q_off[b + 1]])
        if qq.size and kk.size:
            x = max(x, max(float((qq[:, h, :128] @ kk[:, h].T + qq[:, h, 128:] @ rr.T).max()) for h in range(q.shape[1])))
    n = max(np.diff(kv_off), default=0)
    rel = 2 * 200 * 2.0 ** -23 * x * SCALE + (n + 8) * 2.0 ** -23
    return size * (rel + 2.0 ** -8) * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8 + 1e-30


def make(seed, H, new, total, spare=0, layout="projection"):
    """Packed inputs; rows behind the last sequence hold NaN."""
    g = torch.Generator().manual_seed(seed)
    q_off, kv_off = np.cumsum([0] + list(new)), np.cumsum([0] + list(total))
    Tq, Tk = int(q_off[-1]) + spare, int(kv_off[-1]) + spare
    t = lambda *s: torch.randn(*s, generator=g).to(BF)  # noqa: E731
    q, rows = t(max(Tq, 1), H, 192), t(max(Tk, 1), 576)
    if layout == "projection":      # the halves of one projection's output
        kv = t(max(Tk, 1), H, 256)
        k, v = kv[:, :, :128], kv[:, :, 128:]
    elif layout == "heads first":
        kv = t(2, H, max(Tk, 1), 128)
        k, v = kv[0].transpose(0, 1), kv[1].transpose(0, 1)
    else:
        k, v = t(max(Tk, 1), H, 128), t(max(Tk, 1), H, 128)
    if spare:
        for x, n in ((q, q_off[-1]), (rows, kv_off[-1]), (k, kv_off[-1]), (v, kv_off[-1])):
            x[int(n):] = float("nan")
    return dict(q=q, k=k, v=v, rope=rows[:, 512:], q_off=q_off, kv_off=kv_off, max_q=max(new))


def like(x):
    """To the GPU with the strides that it has here."""
    base = x._base if x._base is not None else x
    return torch.as_strided(base.cuda(), x.size(), x.stride(), x.storage_offset())


def call(c, out=None, st=None, **kw):
    out = torch.full(c["q"].shape[:2] + (128,), 7.0, dtype=BF, device="cuda") if out is None else out
    st = zeros_i32(1) if st is None else st
    sv.prompt_attn_latent(c["q"].cuda(), like(c["k"]), like(c["rope"]), like(c["v"]), i32(c["q_off"]), i32(c["kv_off"]), out,
                          kw.get("max_q", c["max_q"]), SCALE, dev_status=st)
    return out, st


def check(c, out, st):
    assert int(st.item()) == 0
    n, m = int(c["q_off"][-1]), int(c["kv_off"][-1])
    q, k, r, v = (c[x].double().numpy() for x in ("q", "k", "rope", "v"))
    ref, size = LO.prompt_attention(q[:n], k[:m], r[:m], v[:m], c["q_off"], c["kv_off"], SCALE)
    got = out.double().cpu().numpy()
    assert (got[n:] == 7.0).all()                 # rows of no sequence
    assert np.isfinite(got[:n]).all()
    err = np.abs(got[:n] - ref)
    worst = float((err / bound(q[:n], k[:m], r[:m], c["q_off"], c["kv_off"], size, ref)).max(initial=0.0))
    assert worst <= 1.0, worst


CASES = [
    # heads, new tokens, all tokens
    (1, [1], [1]), (3, [5], [5]), (2, [127, 128, 129], [127, 128, 129]), (2, [255, 256, 257, 1], [255, 256, 257, 1]),
    (16, [300, 17, 0, 64], [300, 17, 0, 64]), (2, [1000], [1000]), (4, [1, 3, 130], [4000, 3, 1500]),
    (2, [200, 7], [513, 640]), (1, [0, 0, 9], [5, 0, 9]), (5, [70, 300], [20, 299]), (1, [600], [128]), (1, [3], [0]),
]


@pytest.mark.parametrize("H,new,total", CASES)
def test_matches_float64(lib, H, new, total):
    c = make(H + sum(total), H, new, total, spare=9)
    check(c, *call(c))


@pytest.mark.parametrize("layout", ["projection", "heads first", "dense"])
def test_layouts_of_keys_and_values(lib, layout):
    c = make(5, 3, [140, 1, 33], [200, 77, 33], layout=layout)
    check(c, *call(c))
