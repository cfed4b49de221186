"""GPU parity: forking, reserving, freeing and compacting a paged cache's
blocks, bit for bit against the oracle, and a serving run over them."""
import numpy as np
import pytest
import torch

from _util import dev, host, i32, zeros_i32
from oracle import pages as PG
from tree_speculative_decoding_attn_gb300 import specverify as sv
from tree_speculative_decoding_attn_gb300 import synth

pytestmark = pytest.mark.gpu


def counts(table, nb):
    return np.bincount(table[(table >= 0) & (table < nb)], minlength=nb).astype(np.int32)


def filled(g, B, mb, nb, bs, share=0.3):
    """A table of random lengths with some shared beginnings, its lengths and counts."""
    ids, k = g.permutation(nb), 0
    table, prefix = np.full((B, mb), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        if b and g.random() < share:
            prefix[b], table[b] = prefix[b - 1], table[b - 1]
            continue
        n = int(g.integers(0, mb * bs))
        pages = -(-n // bs)
        if k + pages > nb - 1:
            continue
        table[b, :pages], prefix[b] = ids[k:k + pages], n
        k += pages
    return table, prefix, counts(table, nb)


SHAPES = [(1, 1, 1, 1), (5, 7, 40, 16), (64, 33, 1500, 128), (300, 5, 9001, 4), (4096, 2, 5000, 2), (2000, 9, 30011, 3)]


@pytest.mark.parametrize("B,mb,nb,bs", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork_matches_the_oracle(B, mb, nb, bs, in_place):
    g = np.random.default_rng(B + mb)
    table, prefix, ref = filled(g, B, mb, nb, bs)
    ref[::7] += 1                                            # pinned by someone else
    for out in (B, max(1, B // 2), min(4096, 2 * B + 1)):
        parent = g.integers(-1, B, out).astype(np.int32)
        d_ref = i32(ref)
        o = [torch.full((out, mb), 77, dtype=torch.int32, device="cuda"), zeros_i32(out),
             d_ref if in_place else zeros_i32(nb)]
        st = zeros_i32(1)
        sv.kv_pages_fork(i32(table), i32(prefix), i32(parent), d_ref, *o, dev_status=st)
        assert int(st.item()) == 0
        for x, y in zip(o, PG.fork(table, prefix, parent, ref)):
            np.testing.assert_array_equal(host(x), y)


@pytest.mark.parametrize("B,mb,nb,bs", SHAPES)
@pytest.mark.parametrize("window,sinks,spare", [(0, 0, 0), (1, 0, 0), (5, 3, 1), (130, 4, 40), (1 << 30, 0, 0)])
def test_free_matches_the_oracle(B, mb, nb, bs, window, sinks, spare):
    g = np.random.default_rng(B + mb)
    table, prefix, ref = filled(g, min(B, 300), mb, nb, bs)
    prefix = np.maximum(0, prefix - g.integers(0, 2 * bs + 1, len(prefix))).astype(np.int32)
    want = PG.free(table, prefix, ref, bs, window, sinks, spare)
    for in_place in (False, True):
        d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
        o = [d_table, d_ref] if in_place else [torch.full_like(d_table, 77), torch.full_like(d_ref, 77)]
        sv.kv_pages_free(d_table, i32(prefix), d_ref, *o, bs, window, sinks, spare, dev_status=st)
        assert int(st.item()) == 0
        for x, y in zip(o, want):
            np.testing.assert_array_equal(host(x), y)


@pytest.mark.parametrize("nb", [1024, 1025, 8192, 8193, 70001])
@pytest.mark.parametrize("fill", [0.0, 0.5, 0.999, 1.0])
@pytest.mark.parametrize("in_place", [False, True])
def test_plans_over_pools_of_every_size(nb, fill, in_place):
    """Pools around the sizes at which a plan takes another scan or another
    CTA, from empty to full, with the free blocks bunched at either end."""
    g = np.random.default_rng(nb)
    mb, bs = 8, 4
    ref = (g.random(nb) < fill).astype(np.int32)
    ref[: nb // 3] = (np.arange(nb // 3) % 97 != 5) if fill > 0.4 else 0
    held = np.flatnonzero(ref)
    B = 40
    table = np.full((B, mb), -1, np.int32)
    if len(held):
        table[:, :4] = g.choice(held, (B, 4))
        ref = np.maximum(ref, counts(table, nb))
    prefix, need = np.full(B, 14, np.int32), g.integers(0, 17, B).astype(np.int32)
    k, v = pool(1, 1, nb, 1, bs, 8, torch.bfloat16)
    pools = [host(k), host(v)]
    for op in ("reserve", "compact"):
        d_table, d_ref, st, used = i32(table), i32(ref), zeros_i32(1), zeros_i32(1)
        o = [d_table, d_ref] if in_place else [torch.full_like(d_table, 77), torch.full_like(d_ref, 77)]
        if op == "reserve":
            want, t, r, fits = PG.reserve(pools, table, prefix, need, ref, bs)
            sv.kv_pages_reserve(k, v, d_table, i32(prefix), i32(need), d_ref, *o, dev_status=st)
            assert int(st.item()) == (0 if fits else sv.DEV_CAPACITY)
        else:
            want, t, r, n, _ = PG.compact(pools, table, ref)
            sv.kv_pages_compact(k, v, d_table, d_ref, *o, used, dev_status=st)
            assert int(st.item()) == 0 and int(used.item()) == n
        for x, y in zip([*o, k, v], [t, r, *want]):
            np.testing.assert_array_equal(host(x), y)
        table, ref, pools = t, r, want


POOLS = [  # layers, hkv, block size, head_dim, dtype
    (1, 1, 4, 8, torch.bfloat16), (3, 2, 16, 64, torch.float32), (2, 8, 128, 128, torch.bfloat16), (1, 3, 5, 4, torch.float32),
]


def pool(seed, L, nb, hkv, bs, D, dtype):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((L, nb, hkv, bs, D), generator=gen, device="cuda").to(dtype) for _ in range(2)]


@pytest.mark.parametrize("L,hkv,bs,D,dtype", POOLS)
@pytest.mark.parametrize("B,mb,nb", [(1, 2, 3), (6, 5, 50), (64, 6, 700), (1500, 3, 4000)])
@pytest.mark.parametrize("in_place", [False, True])
def test_reserve_matches_the_oracle(L, hkv, bs, D, dtype, B, mb, nb, in_place):
    if B > 64 and bs > 16:
        pytest.skip("covered at smaller pages")
    g = np.random.default_rng(B + bs)
    table, prefix, ref = filled(g, B, mb, nb, bs, share=0.5)
    for least in (1, 0):
        need = g.integers(least - 1, 2 * bs + 2, B).astype(np.int32)
        if least:                                            # room for everybody
            need = np.where(prefix + need > mb * bs, 0, need).astype(np.int32)
        # a smaller demand until it fits, so that most settings do something
        need[(np.cumsum(-(-np.maximum(need, 0) // bs) + 1) > (ref <= 0).sum())] = 0
        k, v = pool(B, L, nb, hkv, bs, D, dtype)
        pools = [host(k), host(v)]
        want_pools, want_table, want_ref, fits = PG.reserve(pools, table, prefix, need, ref, bs)
        over = bool(((need > 0) & (prefix + need > mb * bs)).any())
        d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
        o = [d_table, d_ref] if in_place else [torch.full_like(d_table, 77), torch.full_like(d_ref, 77)]
        sv.kv_pages_reserve(k, v, d_table, i32(prefix), i32(need), d_ref, *o, dev_status=st)
        assert int(st.item()) == (0 if fits and not over else sv.DEV_CAPACITY)
        for x, y in zip([*o, k, v], [want_table, want_ref, *want_pools]):
            np.testing.assert_array_equal(host(x), y)


@pytest.mark.parametrize("in_place", [False, True])
def test_reserve_without_room_changes_nothing(in_place):
    g = np.random.default_rng(2)
    table, prefix, ref = filled(g, 8, 6, 30, 16, share=0.5)
    ref[ref == 0] = 1                                        # nothing is free
    ref[5] = 0                                               # but one
    need = np.full(8, 16, np.int32)
    k, v = pool(1, 2, 30, 2, 16, 64, torch.bfloat16)
    before = [k.clone(), v.clone()]
    d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
    o = [d_table, d_ref] if in_place else [torch.full_like(d_table, 77), torch.full_like(d_ref, 77)]
    sv.kv_pages_reserve(k, v, d_table, i32(prefix), i32(need), d_ref, *o, dev_status=st)
    assert int(st.item()) == sv.DEV_CAPACITY
    np.testing.assert_array_equal(host(o[0]), table)
    np.testing.assert_array_equal(host(o[1]), ref)
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])


@pytest.mark.parametrize("L,hkv,bs,D,dtype", POOLS)
@pytest.mark.parametrize("B,mb,nb", [(1, 1, 1), (6, 5, 50), (64, 6, 700), (30, 9, 5003)])
@pytest.mark.parametrize("in_place", [False, True])
def test_compact_matches_the_oracle(L, hkv, bs, D, dtype, B, mb, nb, in_place):
    if nb > 700 and bs > 16:
        pytest.skip("covered at smaller pages")
    g = np.random.default_rng(B + bs)
    table, prefix, ref = filled(g, B, mb, nb, bs)
    ref[g.integers(0, nb, 1 + nb // 9)] += 1                 # pinned blocks outside the table
    k, v = pool(B, L, nb, hkv, bs, D, dtype)
    want_pools, want_table, want_ref, used, remap = PG.compact([host(k), host(v)], table, ref)
    d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
    o = [d_table, d_ref] if in_place else [torch.full_like(d_table, 77), torch.full_like(d_ref, 77)]
    d_used, d_map = zeros_i32(1), zeros_i32(nb)
    sv.kv_pages_compact(k, v, d_table, d_ref, *o, d_used, remap=d_map, dev_status=st)
    assert int(st.item()) == 0 and int(d_used.item()) == used
    for x, y in zip([*o, k, v, d_map], [want_table, want_ref, *want_pools, remap]):
        np.testing.assert_array_equal(host(x), y)


def test_bad_entries_are_reported_and_dropped():
    nb, bs = 20, 4
    table = np.array([[3, 1 << 30, -7], [4, 5, nb]], np.int32)
    ref = counts(table, nb)
    prefix = np.array([12, 12], np.int32)
    st = zeros_i32(1)
    o = [zeros_i32(2, 3), zeros_i32(2), zeros_i32(nb)]
    sv.kv_pages_fork(i32(table), i32(prefix), i32([1, 2]), i32(ref), *o, dev_status=st)
    assert int(st.item()) in (sv.DEV_BAD_BLOCK, sv.DEV_BAD_PARENTS)
    assert host(o[0]).tolist() == [[4, 5, -1], [-1, -1, -1]] and host(o[1]).tolist() == [12, 0]
    st.zero_()
    sv.kv_pages_free(i32(table), i32(prefix), i32(ref), o[0], o[2], bs, dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_BLOCK and host(o[0]).tolist() == [[3, -1, -1], [4, 5, -1]]
    np.testing.assert_array_equal(host(o[2]), ref)
    st.zero_()
    k, v = pool(1, 1, nb, 1, bs, 8, torch.bfloat16)
    table[0, 2], ref[5] = 9, 0                               # names of blocks nobody counts
    sv.kv_pages_compact(k, v, i32(table), i32(ref), o[0], o[2], zeros_i32(1), dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_BLOCK and host(o[0]).tolist() == [[0, -1, -1], [1, -1, -1]]
    st.zero_()
    sv.kv_pages_reserve(k, v, i32([[nb + 3]]), i32([1]), i32([2]), i32(ref), zeros_i32(1, 1), o[2], dev_status=st)
    assert int(st.item()) == sv.DEV_BAD_BLOCK


def test_a_pool_whose_offsets_pass_32_bits():
    """9 GB a side: blocks at both ends of the pool, copied and moved."""
    L, nb, hkv, bs, D = 2, 9000, 4, 128, 512
    k = torch.zeros((L, nb, hkv, bs, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    table = np.array([[nb - 1, -1], [nb - 1, -1]], np.int32)
    ref = counts(table, nb)
    k[:, nb - 1], v[:, nb - 1] = 3, 4
    d_table, d_ref, st = i32(table), i32(ref), zeros_i32(1)
    sv.kv_pages_reserve(k, v, d_table, i32([100, 100]), i32([1, 1]), d_ref, d_table, d_ref, dev_status=st)
    assert host(d_table).tolist() == [[0, -1], [nb - 1, -1]] and int(st.item()) == 0
    assert (k[:, 0, :, :100] == 3).all() and (v[:, 0, :, :100] == 4).all() and (k[:, 0, :, 100:] == 0).all()
    sv.kv_pages_compact(k, v, d_table, d_ref, d_table, d_ref, zeros_i32(1), dev_status=st)
    assert host(d_table).tolist() == [[0, -1], [1, -1]] and int(st.item()) == 0
    assert (k[:, 1] == 3).all() and (v[:, 1] == 4).all()


def test_calls_in_a_row_captured_and_replayed():
    """fork, reserve, free and compact as one graph, replayed from a fresh state."""
    g = np.random.default_rng(4)
    nb, bs, B, mb = 300, 16, 12, 9
    table, prefix, ref = filled(g, B, mb - 3, nb, bs, share=0.5)
    table = np.pad(table, ((0, 0), (0, 3)), constant_values=-1)
    parent = g.integers(-1, B, B).astype(np.int32)
    k0, v0 = pool(3, 2, nb, 2, bs, 64, torch.bfloat16)
    pools = [host(k0), host(v0)]
    t1, lens, r1 = PG.fork(table, prefix, parent, ref)
    need = np.full(B, 20, np.int32)
    pools, t2, r2, fits = PG.reserve(pools, t1, lens, need, r1, bs)
    assert fits
    t3, r3 = PG.free(t2, lens, r2, bs, 40, 4, 20)
    pools, t4, r4, used, _ = PG.compact(pools, t3, r3)
    a, b, n = i32(table), torch.empty_like(i32(table)), zeros_i32(B)
    r, p, par, nd, used_d, st = i32(ref), i32(prefix), i32(parent), i32(need), zeros_i32(1), zeros_i32(1)
    k, v = k0.clone(), v0.clone()
    ws = torch.empty(sv.kv_pages_workspace_bytes(B, mb, nb), dtype=torch.uint8, device="cuda")

    def steps():
        sv.kv_pages_fork(a, p, par, r, b, n, r, dev_status=st)
        sv.kv_pages_reserve(k, v, b, n, nd, r, b, r, workspace=ws, dev_status=st)
        sv.kv_pages_free(b, n, r, b, r, bs, 40, 4, 20, dev_status=st)
        sv.kv_pages_compact(k, v, b, r, b, r, used_d, workspace=ws, dev_status=st)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(2):
        k.copy_(k0), v.copy_(v0), r.copy_(i32(ref))
        graph.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(used_d.item()) == used
        for x, y in zip((b, n, r, k, v), (t4, lens, r4, *pools)):
            np.testing.assert_array_equal(host(x), y)


def test_wrapper_refuses():
    k, v = pool(1, 1, 8, 1, 4, 8, torch.bfloat16)
    t, p, r = i32([[0, 1], [2, -1]]), i32([8, 4]), i32([1, 1, 1, 0, 0, 0, 0, 0])
    t2, r2, n = torch.empty_like(t), torch.empty_like(r), zeros_i32(1)
    bad = [
        lambda: sv.kv_pages_fork(t, p, i32([0, 1]), r, t, p, r2),                 # not in place
        lambda: sv.kv_pages_fork(t, p, i32([0, 1]), r, t2[:1], torch.empty_like(p), r2),
        lambda: sv.kv_pages_free(t.long(), p, r, t2, r2, 4),
        lambda: sv.kv_pages_free(t, p[:1], r, t2, r2, 4),
        lambda: sv.kv_pages_free(t, None, r, t2, r2, 4),
        lambda: sv.kv_pages_free(t.cpu(), p, r, t2, r2, 4),
        lambda: sv.kv_pages_free(t, p, r, t2, r2, 0),
        lambda: sv.kv_pages_free(t, p, r, t2, r2, 4, window=-1),
        lambda: sv.kv_pages_reserve(k, v[:, :4], t, p, p, r, t2, r2),
        lambda: sv.kv_pages_reserve(k, v.float(), t, p, p, r, t2, r2),
        lambda: sv.kv_pages_reserve(k, v, t, p, p, r[:4], t2, r2),
        lambda: sv.kv_pages_reserve(k, v, t, p, p, r, t2, r2, workspace=n.view(torch.uint8)),
        lambda: sv.kv_pages_reserve(k.double(), v.double(), t, p, p, r, t2, r2),
        lambda: sv.kv_pages_compact(k, v, t, r, t2, r2, n.long()),
        lambda: sv.kv_pages_compact(k, v, t, r, t2, r2, n, remap=zeros_i32(4)),
        lambda: sv.kv_pages_compact(k[..., :4].contiguous(), v[..., :4].contiguous(), t, r, t2, r2, n),
    ]
    for call in bad:
        with pytest.raises((ValueError, TypeError, sv.SpecError)):
            call()
    both = torch.zeros(12, dtype=torch.int32, device="cuda")                      # counts that lie across each other
    with pytest.raises(sv.SpecError):
        sv.kv_pages_free(t, p, both[:8], t2, both[4:], 4)


def test_serving_steps_over_one_pool():
    """Two requests, each sampled three times, decode eight tree steps over one
    pool: reserve, window attention, acceptance from given numbers, commit,
    free, now and then a compaction and a fork.  The rows the table names,
    the lengths and the tokens equal those of a plain program that keeps every
    sequence's rows in a list of its own."""
    from oracle import accept as ACC
    from oracle import attention as A
    from oracle import tree as T
    g = np.random.default_rng(8)
    B, N, hq, hkv, D, bs, nb, mb, V, W, S = 6, 7, 8, 2, 128, 128, 40, 8, 500, 150, 4
    shape = synth.random_tree(2, N, (3, 2))
    depth, mask = T.depth_and_mask(shape.parents)
    fc, ns = T.child_links(shape.parents)
    rnd = lambda *s: synth.round_bf16(g.standard_normal(s).astype(np.float32))  # noqa: E731
    bf = torch.bfloat16
    # two prompts in slots 0 and 1; the plain program's rows: per sequence K and V [rows, hkv, D]
    prefix = np.array([300, 129, 0, 0, 0, 0], np.int32)
    rows = [[rnd(int(p), hkv, D), rnd(int(p), hkv, D)] for p in prefix]
    table = np.full((B, mb), -1, np.int32)
    table[0, :3], table[1, :2] = [11, 30, 5], [17, 2]
    kp, vp = (np.full((1, nb, hkv, bs, D), np.nan, np.float32) for _ in range(2))
    for b in (0, 1):
        for x in range(prefix[b]):
            kp[0, table[b, x // bs], :, x % bs], vp[0, table[b, x // bs], :, x % bs] = rows[b][0][x], rows[b][1][x]
    k, v, st = dev(kp, bf), dev(vp, bf), zeros_i32(1)
    t, t2, p, p2, r = i32(table), zeros_i32(B, mb), i32(prefix), zeros_i32(B), i32(counts(table, nb))
    ws = torch.empty(sv.kv_pages_workspace_bytes(B, mb, nb), dtype=torch.uint8, device="cuda")
    used = zeros_i32(1)

    def fork(parent):
        nonlocal t, t2, p, p2, rows
        sv.kv_pages_fork(t, p, i32(parent), r, t2, p2, r, dev_status=st)
        t, t2, p, p2 = t2, t, p2, p
        rows = [[x.copy() for x in rows[i]] if i >= 0 else [rnd(0, hkv, D)] * 2 for i in parent]

    fork([0, 0, 0, 1, 1, 1])
    anc = dev(np.broadcast_to(T.mask_words_multi(mask), (B, N, 1)).copy().view(np.int64))
    par, fcd, nsd, dep = (i32(np.broadcast_to(x, (B, N))) for x in (shape.parents, fc, ns, depth))
    for step in range(8):
        if step == 5:
            fork([4, 0, 1, -1, 4, 5])
        lens = [len(x[0]) for x in rows]
        assert host(p).tolist() == lens
        sv.kv_pages_reserve(k, v, t, p, i32([N if n else 0 for n in lens]), r, t, r, workspace=ws, dev_status=st)
        if step in (2, 6):
            sv.kv_pages_compact(k, v, t, r, t, r, used, workspace=ws, dev_status=st)
            assert int(used.item()) == int((r > 0).sum().item()) and int((r[int(used.item()):]).sum().item()) == 0
        q, kt, vt = rnd(B, N, hq, D), rnd(B, hkv, N, D), rnd(B, hkv, N, D)
        out = torch.zeros((B, N, hq, D), dtype=bf, device="cuda")
        sv.tree_attn_verify_window_paged(dev(q, bf), k[0], v[0], t, dev(kt, bf), dev(vt, bf), p, dep, anc, out, mb * bs, W,
                                         sinks=S, dev_status=st)
        probs = g.dirichlet(np.full(V, 0.02), (B, N)).astype(np.float32)
        tok = np.zeros((B, N), np.int32)
        best = np.argsort(-probs, -1)
        rank = shape.rank
        for i in range(1, N):
            tok[:, i] = best[:, shape.parents[i], rank[i]]
        u, ub = g.random((B, N)).astype(np.float32), g.random(B).astype(np.float32)
        n_acc, path, bonus = zeros_i32(B), zeros_i32(B, 4), zeros_i32(B)
        sv.spec_verify_probs(dev(probs), i32(tok), par, fcd, nsd, dev(u), dev(ub), n_acc, path, bonus, dev_status=st)
        n_acc[torch.tensor([n == 0 for n in lens], device="cuda")] = -1           # an empty slot commits nothing ...
        st_commit = zeros_i32(1)                                                  # ... and is reported for it
        sv.kv_commit_paged(k[0], v[0], t, dev(kt, bf), dev(vt, bf), n_acc, path, p, p, dev_status=st_commit)
        assert int(st_commit.item()) == (sv.DEV_CAPACITY if 0 in lens else 0)
        sv.kv_pages_free(t, p, r, t, r, bs, W, S, dev_status=st)
        assert int(st.item()) == 0
        # the plain program
        live = [b for b in range(B) if lens[b]]
        ref_len, ref_path, ref_bonus = ACC.accept_probs(probs, None, tok, np.broadcast_to(fc, (B, N)),
                                                        np.broadcast_to(ns, (B, N)), u, ub, 4)
        np.testing.assert_array_equal(host(n_acc)[live], ref_len[live])
        np.testing.assert_array_equal(host(bonus)[live], ref_bonus[live])
        got = host(out)
        for b in live:
            kc, vc = (x.swapaxes(0, 1)[None] for x in rows[b])
            ref, mag, _ = A.tree_attention_window(q[b:b + 1], kc, vc, kt[b:b + 1], vt[b:b + 1], [lens[b]], depth[None],
                                                  mask[None], W, S)
            # probabilities and outputs in bf16 (2^-8 each), the rest below 2^-10 at scores of a few units
            assert (np.abs(got[b] - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + (2.0 ** -8 + 2.0 ** -10) * mag[0]).all()
            new = [int(x) for x in ref_path[b, :ref_len[b] + 1]]
            rows[b] = [np.concatenate([rows[b][0], kt[b][:, new].swapaxes(0, 1)]),
                       np.concatenate([rows[b][1], vt[b][:, new].swapaxes(0, 1)])]
        # every row a later step can see is where the table says
        tab, kk, vv = host(t), host(k), host(v)
        for b in live:
            P = len(rows[b][0])
            for x in range(P):
                if x < S or P - x < W:
                    np.testing.assert_array_equal(kk[0, tab[b, x // bs], :, x % bs], rows[b][0][x])
                    np.testing.assert_array_equal(vv[0, tab[b, x // bs], :, x % bs], rows[b][1][x])
                elif x // bs * bs >= S and P - (x // bs + 1) * bs + 1 >= W:
                    assert tab[b, x // bs] == -1
        np.testing.assert_array_equal(host(r), counts(tab, nb))
