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


def test_few_units_are_cut_into_parts(lib):
    """One head and few queries behind many keys: keys in parts, some of which
    show some queries nothing."""
    for new, total, H in (([5], [9000], 1), ([300], [5000], 3), ([256, 1], [700, 6000], 2), ([2000], [2000], 1),
                          ([400], [390], 1), ([3, 0], [4000, 4000], 2)):
        assert sv.prompt_attn_latent_workspace_bytes(len(new), H, 128, 64, sum(new), sum(total), max(new)) > 0 \
            or sum(total) < 1024
        c = make(len(new) + H, H, new, total, spare=70)
        check(c, *call(c))


def test_scores_that_jump(lib):
    for H, n in ((2, 700), (40, 300)):
        c = make(4, H, [n], [n])
        step = torch.arange(n) // 64
        step = torch.where(step < 6, step, 11 - step).float()
        c["q"][..., 128] = 16.0
        c["rope"][:, 0] = (step * 8).to(BF)
        check(c, *call(c))


def test_not_a_number_and_what_is_not_read(lib):
    """A NaN query makes its row NaN alone; another sequence's rows may be NaN."""
    c = make(5, 2, [200, 40, 60], [260, 40, 90])
    c["q"][17, 1, 150] = float("nan")
    out, _ = call(c)
    bad = out.isnan().any(-1).cpu()
    assert int(bad.sum()) == 1 and bool(bad[17, 1])
    c = make(5, 2, [200, 40, 60], [260, 40, 90])
    for x in ("k", "v", "rope"):
        c[x][260:300] = float("nan")
    c["q"][200:240] = float("nan")
    out, st = call(c)
    assert bool(out[200:240].isnan().all()) and not out[:200].isnan().any() and not out[240:].isnan().any()


def test_refused_offsets_leave_their_rows(lib):
    for H in (2, 30):
        c = make(6, H, [100, 50, 30], [200, 60, 30])
        good, _ = call(c)
        for q_off, kv_off, bad in (([0, 100, 90, 180], [0, 200, 260, 290], (1,)), ([0, 100, 150, 9999], [0, 200, 260, 290], (2,)),
                                   ([0, 100, 150, 180], [0, 200, 260, 291], (2,)), ([-5, 100, 150, 180], [0, 200, 260, 290], (0,)),
                                   ([0, 100, 150, 180], [0, 200, 100, 290], (1, 2)),
                                   ([0, 100, 150, 180], [0, -2 ** 31, 260, 290], (0, 1))):
            out, st = call(dict(c, q_off=q_off, kv_off=kv_off))
            assert int(st.item()) == sv.DEV_CAPACITY
            for b, (lo, hi) in enumerate(((0, 100), (100, 150), (150, 180))):
                if b not in bad and (b != 2 or q_off[2] == 150) and kv_off[b:b + 2] == c["kv_off"].tolist()[b:b + 2]:
                    assert torch.equal(out[lo:hi], good[lo:hi])
            if bad == (2,):
                assert bool((out[150:] == 7.0).all())
        out, st = call(c, max_q=60)
        assert int(st.item()) == sv.DEV_CAPACITY and bool((out[:100] == 7.0).all()) and torch.equal(out[100:], good[100:])
        out, st = call(c, max_q=10 ** 6)
        assert int(st.item()) == 0 and torch.equal(out, good)
        out, st = call(c, max_q=0)
        assert bool((out == 7.0).all())


@pytest.mark.parametrize("H,new,total", [(2, [300, 40], [2000, 90]), (40, [300, 40], [700, 90])])
def test_captured_on_another_stream_and_two_at_once(lib, H, new, total):
    cs = [make(30 + i, H, new, total) for i in range(2)]
    alone = [call(c)[0] for c in cs]
    args = [(c["q"].cuda(), like(c["k"]), like(c["rope"]), like(c["v"]), i32(c["q_off"]), i32(c["kv_off"])) for c in cs]
    size = sv.prompt_attn_latent_workspace_bytes(2, H, 128, 64, sum(new), sum(total), max(new))
    ws = [torch.empty(max(16, size), dtype=torch.uint8, device="cuda") for _ in cs]
    outs, sts = [torch.empty_like(a) for a in alone], [zeros_i32(1) for _ in cs]
    graphs, streams = [], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for a, w, o, t in zip(args, ws, outs, sts):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.prompt_attn_latent(*a, o, max(new), SCALE, workspace=w, dev_status=t)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.fill_(3.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, o, t in zip(alone, outs, sts):
            assert int(t.item()) == 0 and torch.equal(a, o)


def test_wrapper_refuses(lib):
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    good = dict(q=z(5, 2, 192), k=z(9, 2, 128), k_rope=z(9, 64), v=z(9, 2, 128), q_offsets=i32([0, 5]), kv_offsets=i32([0, 9]),
                out=z(5, 2, 128), max_q=5, scale=SCALE)
    sv.prompt_attn_latent(**good)
    sv.prompt_attn_latent(**dict(good, v=z(9, 2, 264)[:, :, 8:136]))
    for kw in (dict(q=z(5, 2, 128)), dict(k=z(9, 3, 128)), dict(k_rope=z(8, 64)), dict(v=z(9, 2, 64)), dict(out=z(5, 2, 192)),
               dict(kv_offsets=i32([0, 9, 9])), dict(q=z(5, 2, 192, dt=torch.float32)), dict(scale=-1.0), dict(max_q=-1),
               dict(v=z(9, 2, 132)[:, :, 4:]), dict(v=z(9, 2, 130)[:, :, :128]), dict(k=z(9, 128, 2).transpose(1, 2)),
               dict(k_rope=z(9, 68)[:, 4:]), dict(v=z(1, 2, 128).expand(9, 2, 128)), dict(q=good["q"].cpu())):
        with pytest.raises((ValueError, TypeError, sv.SpecError)):
            sv.prompt_attn_latent(**{**good, **kw})


def test_more_queries_than_none_are_reported(lib):
    c = make(12, 2, [0, 40, 0], [10, 90, 0])
    out, st = call(c, max_q=0)
    assert int(st.item()) == sv.DEV_CAPACITY and bool((out == 7.0).all())
    out, st = call(make(13, 2, [0, 0], [2000, 7], spare=5), max_q=0)
    assert int(st.item()) == 0 and bool((out == 7.0).all())


@pytest.mark.parametrize("H,new,total", [(24, [1500, 700], [3000, 700]), (2, [200, 129], [9000, 4000])])
def test_runs_agree_with_one_another(lib, H, new, total):
    c = make(14, H, new, total)
    first, st = call(c)
    check(c, first, st)
    for _ in range(20):
        out, st = call(c)
        assert int(st.item()) == 0 and torch.equal(out, first)
