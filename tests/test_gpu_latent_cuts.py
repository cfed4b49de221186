"""GPU: latent tree calls whose units are cut between parts and joined, in every
form of the join, with results that are counts (test_latent_schedule.py checks
on the CPU that each case is shared out as it says, and that a lost or doubled
group of keys shows)."""
import numpy as np
import pytest
import torch

import test_gpu_latent as base
from _latent_counts import CASES, expected, group_column, odd, tolerance, tree_column
from _latent_plan import plan
from _util import i32, zeros_i32
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

BF, F32, SCALE = torch.bfloat16, torch.float32, base.SCALE


def rows_of(length, latent, dtype):
    at = np.arange(length)
    x = torch.zeros(length, latent + 64, dtype=dtype, device="cuda")
    x[torch.arange(length), torch.from_numpy(group_column(at, latent))] = 1.0
    x[:, latent] = torch.from_numpy(odd(at).astype(np.float32)).to(dtype).cuda()
    return x


def make(lengths, nodes, heads, latent, page, dtype):
    g = np.random.default_rng(nodes * heads)
    B, D, top = len(lengths), latent + 64, max(x or 0 for x in lengths)
    q = torch.zeros(B, nodes * heads, D, dtype=dtype, device="cuda")
    q[:, 1::2, latent] = -30000.0            # times the scale: -2165, whose exponential is 0 in float32
    tree = torch.zeros(B, nodes, D, dtype=dtype, device="cuda")
    tree[:, torch.arange(nodes), torch.from_numpy(tree_column(np.arange(nodes), latent))] = 1.0
    mask = base.trees(g, B, nodes)
    c = dict(q=q.view(B, nodes, heads, D), tree=tree, mask=mask, top=top)
    prefix = [top + 1 if x is None else x for x in lengths]          # more than max_prefix: refused
    nan = float("nan")
    if page:
        pages = [-(-(x or 0) // page) for x in lengths]
        ids, k = g.permutation(sum(pages) + 3), 0
        table = np.full((B, max(1, max(pages))), -1, np.int32)
        pool = torch.full((len(ids), page, D), nan, dtype=dtype, device="cuda")
        for b, n in enumerate(pages):
            table[b, :n] = ids[k:k + n]
            rows = rows_of(lengths[b] or 0, latent, dtype)
            for j in range(n):
                piece = rows[j * page:(j + 1) * page]
                pool[int(ids[k + j]), :len(piece)] = piece
            k += n
        c.update(pool=pool, table=i32(table))
    else:
        cache = torch.full((B, top + 9, D), nan, dtype=dtype, device="cuda")
        for b, x in enumerate(lengths):
            cache[b, :x or 0] = rows_of(x or 0, latent, dtype)
        c.update(cache=cache)
    c.update(prefix=i32(prefix), words=base.words(mask))
    return c


def call(c, out, st, **kw):
    if "pool" in c:
        sv.tree_attn_verify_latent_paged(c["q"], c["pool"], c["table"], c["tree"], c["prefix"], c["words"], out, c["top"], SCALE,
                                         dev_status=st, **kw)
    else:
        sv.tree_attn_verify_latent(c["q"], c["cache"], c["tree"], c["prefix"], c["words"], out, c["top"], SCALE, dev_status=st,
                                   **kw)


def check(lengths, nodes, heads, latent, c, out, st, half_step):
    assert int(st.item()) == (sv.DEV_CAPACITY if None in lengths else 0)
    for b, x in enumerate(lengths):
        if x is None:
            assert bool((out[b] == 7.0).all())
            continue
        ref = torch.from_numpy(expected(x, nodes, heads, latent, c["mask"][b])).cuda()
        err, tol = (out[b].double() - ref).abs(), tolerance(ref, half_step)
        bad = ~(err <= tol)                     # (a NaN is bad too)
        assert not bool(bad.any()), (b, x, bad.nonzero()[:3].tolist(), int(bad.sum()))


@pytest.mark.parametrize("name", CASES)
def test_every_group_counts_once(lib, name):
    lengths, nodes, heads, latent, page, kernel, mode, form = CASES[name]
    p = plan(lengths, nodes, heads, latent)
    assert (p.kernel, p.mode, p.form) == (kernel, mode, form)
    c, st = make(lengths, nodes, heads, latent, page, BF), zeros_i32(1)
    out = torch.full((len(lengths), nodes, heads, latent), 7.0, dtype=BF, device="cuda")
    size = sv.tree_attn_latent_workspace_bytes(BF, len(lengths), nodes, heads, latent, 64, c["top"])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")          # NaN wherever a float is not written
    call(c, out, st, workspace=ws)
    check(lengths, nodes, heads, latent, c, out, st, 2.0 ** -8)
    # the cuts that the kernel found, which it leaves at the workspace's beginning
    found = ws[:16 * p.parts].view(torch.int32).view(-1, 4).cpu().tolist()
    assert {i: tuple(d[:3]) for i, d in enumerate(found) if d[3]} == p.cuts


@pytest.mark.parametrize("name", ["pairs 512, more units than parts", "pairs 256, more units than parts", "few 512, more units than parts",
                                  "few 256, more units than parts"])
def test_cut_units_match_float64(lib, name):
    """The same shares of work with random values, bf16 against float64."""
    lengths, nodes, heads, latent, page, *_ = CASES[name]
    some = [b for b in range(len(lengths)) if lengths[b] < 1500][::4]       # (what is compared; all run)
    c = base.make(41, len(lengths), nodes, heads, latent, lengths, BF, page)
    out, st = base.call(c)
    base.check(c, out, st, skip=[b for b in range(len(lengths)) if b not in some])


@pytest.mark.parametrize("lengths,nodes,heads,latent", [([5000, 70], 3, 7, 512), ([20000], 1, 3, 256), ([900] * 9, 4, 9, 512),
                                                        ([3000, 1, 0, 2999], 2, 16, 256)])
def test_float32_ranges_count_once(lib, lengths, nodes, heads, latent):
    c, st = make(lengths, nodes, heads, latent, 0, F32), zeros_i32(1)
    out = torch.full((len(lengths), nodes, heads, latent), 7.0, dtype=F32, device="cuda")
    call(c, out, st)
    check(lengths, nodes, heads, latent, c, out, st, 2.0 ** -24)
