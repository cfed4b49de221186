"""GPU parity of the latent kernel on SM pairs at sizes that the kernel of few
rows would take: the cache (or the block table) is so wide, and max_prefix as
large, that the call may have many tiles."""
import numpy as np
import pytest
import torch

import test_gpu_latent as base
from _util import i32, zeros_i32
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

BF, SCALE = base.BF, base.SCALE
plain_call = base.call


def wide(c):
    """c with room for more than 1064 tiles of 16 rows x 64 keys, and that room."""
    units = c["B"] * -(-c["N"] * c["H"] // 16)
    room = 128 * -(-64 * (1070 // units + 1) // 128)
    assert c["N"] * c["H"] > 16 and units * (room // 64) > 1064
    c = dict(c)
    if c["page"]:
        room = -(-room // c["page"]) * c["page"]
        table = np.full((c["B"], max(room // c["page"], c["table"].shape[1])), -1, np.int32)
        table[:, :c["table"].shape[1]] = c["table"]
        c["table"] = table
        room = table.shape[1] * c["page"]
    else:
        room = max(room, c["cache"].shape[1])
        cache = torch.full((c["B"], room, c["cache"].shape[2]), float("nan"), dtype=c["dtype"])
        cache[:, :c["cache"].shape[1]] = c["cache"]
        c["cache"] = cache
    return c, room


def wide_call(c, max_prefix=None, **kw):
    c, room = wide(c)
    return plain_call(c, max_prefix=room, **kw)


@pytest.mark.parametrize("B,N,H,lat,prefix,page", [s for s in base.SHAPES if s[1] * s[2] > 16])
def test_matches_float64(lib, B, N, H, lat, prefix, page):
    c = base.make(B * 100 + N, B, N, H, lat, prefix, BF, page)
    base.check(c, *wide_call(c))


def test_rows_of_nothing_are_zeros(lib):
    c = base.make(3, 2, 65, 3, 512, [0, 130], BF, 0)
    c["mask"][:, 1::2] = False
    out, st = wide_call(c)
    base.check(c, out, st)
    assert float(out[0, 1::2].abs().max()) == 0.0


def test_not_a_number(lib, monkeypatch):
    monkeypatch.setattr(base, "call", wide_call)
    base.test_not_a_number(lib, 33, 4, BF)


@pytest.mark.parametrize("lat", [256, 512])
def test_scores_that_jump(lib, monkeypatch, lat):
    monkeypatch.setattr(base, "call", wide_call)
    base.test_scores_that_jump(lib, 33, 4, BF, lat)


def test_bad_blocks_read_as_zeros(lib, monkeypatch):
    monkeypatch.setattr(base, "call", wide_call)
    base.test_bad_blocks_read_as_zeros(lib, 40, 4, BF)


def test_refused_lengths_leave_their_rows(lib):
    c, room = wide(base.make(5, 3, 40, 4, 512, [200, 100, 300], BF, 0))
    for bad in (-1, room + 1, 2 ** 31 - 1):
        out, st = plain_call(c, max_prefix=room, prefix=i32([200, bad, 300]))
        assert int(st.item()) == sv.DEV_CAPACITY and bool((out[1] == 7.0).all())
        base.check(c, out, zeros_i32(1), skip=(1,))


def test_a_pool_whose_offsets_pass_32_bits(lib):
    D, page, nb = 576, 128, 33000
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.empty(nb, page, D, dtype=BF, device="cuda")
    used = [nb - 1, 3, 29300, nb - 2]
    for b in used:
        pool[b] = torch.randn(page, D, generator=g, device="cuda").to(BF)
    c = base.make(10, 1, 20, 8, 512, [470], BF, 0)
    c["cache"] = torch.cat([pool[b] for b in used])[None].cpu()
    out = torch.empty(1, 20, 8, 512, dtype=BF, device="cuda")
    st = zeros_i32(1)
    table = np.full((1, 400), -1, np.int32)
    table[0, :4] = used
    sv.tree_attn_verify_latent_paged(c["q"].cuda(), pool, i32(table), c["tree"].cuda(), i32([470]), base.words(c["mask"]), out,
                                     400 * 128, SCALE, dev_status=st)
    base.check(c, out, st)


def test_captured_replayed_on_other_lengths_and_repeatable(lib):
    base.test_captured_replayed_on_other_lengths_and_repeatable(lib, 60, 8, BF)


def test_narrow_and_wide_calls(lib):
    """The same inputs by either kernel."""
    c = base.make(31, 3, 5, 13, 512, [100, 0, 700], BF, 128)
    for run in (plain_call, wide_call):
        out, st = run(c)
        base.check(c, out, st)
