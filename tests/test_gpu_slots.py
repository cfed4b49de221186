"""GPU parity: the rows of packed tokens in a paged cache, and their copies."""
import numpy as np
import pytest
import torch

from _util import host, i32, zeros_i32
from oracle import latent as LO
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu


def tables(g, prefix, new, page, spare=4, wide=0):
    pages = [-(-max(0, int(p + max(0, n))) // page) for p, n in zip(prefix, new)]
    nb = sum(pages) + spare
    ids, k = g.permutation(nb), 0
    table = np.full((len(pages), max(1, max(pages)) + wide), -1, np.int32)
    for i, n in enumerate(pages):
        table[i, :n] = ids[k:k + n]
        k += n
    return table, nb


def run(table, prefix, new, room, page, nb, positions=True):
    B = len(prefix)
    off, slots, pos, st = i32([9] * (B + 1)), i32([9] * room), i32([9] * room), zeros_i32(1)
    sv.kv_pages_slots(i32(table), i32(prefix), i32(new), off, slots, page, nb, positions=pos if positions else None,
                      dev_status=st)
    return host(off), host(slots), host(pos), int(st.item())


@pytest.mark.parametrize("B,top,page,spare", [(1, 1, 128, 0), (1, 1000, 1, 3), (3, 5, 16, 1), (64, 1, 128, 0), (64, 3000, 128, 50),
                                              (255, 40, 64, 0), (256, 9, 3, 7), (257, 9, 256, 1), (4096, 7, 5, 2), (1000, 300, 7, 0)])
def test_slots_match(lib, B, top, page, spare):
    g = np.random.default_rng(B + top)
    new, prefix = g.integers(-1, top + 1, B), g.integers(0, 3 * page + 1, B)
    new[0] = max(1, new[0])
    table, nb = tables(g, prefix, new, page)
    room = int(np.maximum(new, 0).sum()) + spare
    got = run(table, prefix, new, room, page, nb)
    want = LO.slots(table, prefix, new, room, page, nb)
    for a, b in zip(got[:3], want[:3]):
        np.testing.assert_array_equal(a, b)
    assert got[3] == 0 and not want[3]


def test_what_has_no_place_is_reported(lib):
    table = np.array([[3, -1], [1, 99], [0, 2]], np.int32)
    # a missing block, one outside the pool, and a sequence that passes its table
    for new, code in (([5, 0, 0], sv.DEV_BAD_BLOCK), ([0, 6, 0], sv.DEV_BAD_BLOCK), ([0, 0, 9], sv.DEV_CAPACITY)):
        off, slots, pos, st = run(table, [0, 0, 0], new, 12, 4, 4)
        w_off, w_slots, w_pos, err = LO.slots(table, [0, 0, 0], new, 12, 4, 4)
        np.testing.assert_array_equal(off, w_off)
        np.testing.assert_array_equal(slots, w_slots)
        np.testing.assert_array_equal(pos, w_pos)
        assert st == code and err
    off, slots, pos, st = run(table, [-1, 0, 0], [1, 2, 0], 4, 4, 4)
    assert st == sv.DEV_CAPACITY and slots.tolist() == [-1, 4, 5, -1] and pos.tolist() == [-1, 0, 1, -1]
    # more tokens than room, far more than 32 bits hold among them
    off, slots, pos, st = run(table, [0, 0, 0], [3, 2, 3], 4, 4, 4)
    assert st == sv.DEV_CAPACITY and off.tolist() == [0, 3, 4, 4] and slots.tolist() == [12, 13, 14, 4]
    off, slots, pos, st = run(table, [0, 0, 0], [1, 2 ** 31 - 1, 2 ** 31 - 1], 3, 4, 4)
    assert st == sv.DEV_CAPACITY and off.tolist() == [0, 1, 3, 3] and slots.tolist() == [12, 4, 5]


@pytest.mark.parametrize("T,hkv,D,page,dtype", [(1, 1, 576, 128, torch.bfloat16), (1000, 1, 576, 128, torch.bfloat16),
                                                (77, 3, 64, 16, torch.float32), (5, 8, 128, 1, torch.bfloat16),
                                                (513, 2, 8, 64, torch.bfloat16), (30000, 1, 320, 256, torch.float32)])
def test_rows_go_in_and_come_out(lib, T, hkv, D, page, dtype):
    g = np.random.default_rng(T)
    nb = -(-T // page) + 3
    slots = g.permutation(nb * page)[:T].astype(np.int32)
    slots[::5] = -1 - slots[::5] % 3
    pages = torch.randn(nb, hkv, page, D).to(dtype)
    rows = torch.randn(T, hkv, D).to(dtype)
    d_pages, d_rows, st = pages.cuda(), rows.cuda(), zeros_i32(1)
    sv.kv_slots_write(d_pages, i32(slots), d_rows, dev_status=st)
    want = pages.clone()
    live = torch.from_numpy(slots >= 0)
    at = torch.from_numpy(slots)[live].long()
    want[at // page, :, at % page] = rows[live]
    assert torch.equal(d_pages.cpu(), want)
    back = torch.full_like(d_rows, 3.0)
    sv.kv_slots_read(d_pages, i32(slots), back, dev_status=st)
    assert torch.equal(back.cpu(), torch.where(live[:, None, None], rows, torch.zeros_like(rows)))
    assert int(st.item()) == 0


def test_slots_past_the_pool_are_reported(lib):
    pages, rows, st = torch.zeros(2, 1, 4, 8, device="cuda"), torch.ones(3, 1, 8, device="cuda"), zeros_i32(1)
    sv.kv_slots_write(pages, i32([8, 3, 2 ** 31 - 1]), rows, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_BLOCK and float(pages.sum()) == 8.0 and float(pages[0, 0, 3].sum()) == 8.0
    st.zero_()
    sv.kv_slots_read(pages, i32([8, 3, 2 ** 31 - 1]), rows, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_BLOCK and rows.sum(-1).flatten().tolist() == [0.0, 8.0, 0.0]
