"""GPU: the page operators at the ends of their arguments' ranges: lengths,
demands, parents and counts that are any int, windows and spares up to the
largest.  Bit for bit against the oracle, which is given the sequences that
the header says take part."""
import numpy as np
import pytest
import torch

from _util import host, i32, zeros_i32
from oracle import pages as PG
from test_gpu_pages import counts, filled, pool
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

TOP, LOW = 2 ** 31 - 1, -2 ** 31
WILD = [LOW, LOW + 1, -1, 0, 1, TOP - 1, TOP]


@pytest.mark.parametrize("B,mb,nb,bs", [(14, 6, 70, 4), (2000, 9, 30011, 3)])
@pytest.mark.parametrize("window,sinks,spare", [(0, 0, 0), (TOP, 0, 0), (1, TOP, 0), (1, 0, TOP), (TOP, TOP, TOP), (3, 1, 2)])
def test_free(B, mb, nb, bs, window, sinks, spare):
    g = np.random.default_rng(B)
    table, prefix, ref = filled(g, B, mb, nb, bs)
    prefix[::2] = np.resize(np.asarray(WILD, np.int32), len(prefix[::2]))
    want = PG.free(table, prefix, ref, bs, window, sinks, spare)
    d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
    sv.kv_pages_free(d_table, i32(prefix), d_ref, d_table, d_ref, bs, window, sinks, spare, dev_status=st)
    assert int(st.item()) == 0
    for x, y in zip((d_table, d_ref), want):
        np.testing.assert_array_equal(host(x), y)


@pytest.mark.parametrize("B,mb,nb", [(14, 6, 70), (2000, 9, 30011)])
def test_fork(B, mb, nb):
    g = np.random.default_rng(B)
    table, prefix, ref = filled(g, B, mb, nb, 4)
    parent = g.integers(0, B, B).astype(np.int32)
    parent[::2] = np.resize(np.asarray([*WILD, B, B - 1], np.int64), len(parent[::2])).astype(np.int32)
    want = PG.fork(table, prefix, np.where((parent < 0) | (parent >= B), -1, parent), ref)
    o, st = [zeros_i32(B, mb), zeros_i32(B), zeros_i32(nb)], zeros_i32(1)
    sv.kv_pages_fork(i32(table), i32(prefix), i32(parent), i32(ref), *o, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_PARENTS
    for x, y in zip(o, want):
        np.testing.assert_array_equal(host(x), y)


@pytest.mark.parametrize("B,mb,nb,bs", [(14, 6, 200, 4), (1100, 3, 9000, 3)])
def test_reserve(B, mb, nb, bs):
    """A demand that no sequence can have, a length that none has: left out."""
    g = np.random.default_rng(B)
    table, prefix, ref = filled(g, B, mb, nb, bs, share=0.5)
    need = g.integers(0, bs + 2, B).astype(np.int32)
    need = np.where(prefix + need > mb * bs, 0, need).astype(np.int32)
    need[::3] = np.resize(np.asarray(WILD, np.int32), len(need[::3]))
    prefix[1::3] = np.resize(np.asarray(WILD, np.int32), len(prefix[1::3]))
    end = prefix.astype(np.int64) + need
    takes = (need > 0) & (prefix >= 0) & (end <= mb * bs)
    k, v = pool(1, 1, nb, 1, bs, 8, torch.bfloat16)
    want, t, r, fits = PG.reserve([host(k), host(v)], table, np.where(takes, prefix, 0), np.where(takes, need, 0), ref, bs)
    assert fits
    d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
    sv.kv_pages_reserve(k, v, d_table, i32(prefix), i32(need), d_ref, d_table, d_ref, dev_status=st)
    assert int(st.item()) == sv.DEV_CAPACITY
    for x, y in zip((d_table, d_ref, k, v), (t, r, *want)):
        np.testing.assert_array_equal(host(x), y)


@pytest.mark.parametrize("nb", [70, 9000])
def test_counts_of_any_size(nb):
    """Compaction moves a block whose count is the largest int, and takes one
    below zero for free; a shared block with such a count is copied."""
    g = np.random.default_rng(nb)
    table, _, _ = filled(g, 14, 6, nb, 4, share=0)
    ref = counts(table, nb)
    ref[ref > 0] = np.resize(np.asarray([1, TOP, 2], np.int32), int((ref > 0).sum()))
    ref[ref == 0] = np.resize(np.asarray([0, -1, LOW], np.int32), int((ref == 0).sum()))
    k, v = pool(1, 1, nb, 1, 4, 8, torch.bfloat16)
    want, t, r, used, remap = PG.compact([host(k), host(v)], table, ref)
    d_table, d_ref, st, d_used, d_map = i32(table), i32(ref), zeros_i32(1), zeros_i32(1), zeros_i32(nb)
    sv.kv_pages_compact(k, v, d_table, d_ref, d_table, d_ref, d_used, remap=d_map, dev_status=st)
    assert int(st.item()) == 0 and int(d_used.item()) == used
    for x, y in zip((d_table, d_ref, k, v, d_map), (t, r, *want, remap)):
        np.testing.assert_array_equal(host(x), y)
    prefix, need = np.full(14, 2, np.int32), np.full(14, 1, np.int32)
    want, t2, r2, fits = PG.reserve(want, t, prefix, need, r, 4)
    assert fits
    sv.kv_pages_reserve(k, v, d_table, i32(prefix), i32(need), d_ref, d_table, d_ref, dev_status=st)
    assert int(st.item()) == 0
    for x, y in zip((d_table, d_ref, k, v), (t2, r2, *want)):
        np.testing.assert_array_equal(host(x), y)
