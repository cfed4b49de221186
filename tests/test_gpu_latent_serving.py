"""Caches of one pool in the commit and the page calls, and a run of all
operators of a latent cache together."""
import numpy as np
import pytest
import torch

from _util import dev, host, i32, zeros_i32
from oracle import latent as LO
from oracle import tree as T
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def rnd(g, *s, dtype=BF):
    return torch.from_numpy(g.standard_normal(s).astype(np.float32)).to(dtype).cuda()


@pytest.mark.parametrize("L,D,dtype", [(1, 576, BF), (3, 320, torch.float32)])
def test_one_pool_commits_as_the_first_of_two(lib, L, D, dtype):
    g = np.random.default_rng(3)
    B, N, S, page, nb = 4, 9, 80, 16, 30
    tree = rnd(g, L, B, 1, N, D, dtype=dtype)
    n_acc, prefix = i32([0, 3, 2, 5]), i32([0, 17, 40, 74])
    path = i32([[0, 1, 4, 6, 7, 8]] * B)
    cache = rnd(g, L, B, 1, S, D, dtype=dtype)
    both, alone = [cache.clone(), cache.clone()], cache.clone()
    p2, p1, st = zeros_i32(B), zeros_i32(B), zeros_i32(1)
    sv.kv_commit(*both, tree, tree, n_acc, path, prefix, p2, st)
    sv.kv_commit(alone, None, tree, None, n_acc, path, prefix, p1, st)
    assert torch.equal(alone, both[0]) and torch.equal(p1, p2) and int(st.item()) == 0
    table = i32(g.permutation(nb)[:B * 6].reshape(B, 6))
    pages = rnd(g, L, nb, 1, page, D, dtype=dtype)
    both, alone = [pages.clone(), pages.clone()], pages.clone()
    sv.kv_commit_paged(*both, table, tree, tree, n_acc, path, prefix, p2, st)
    sv.kv_commit_paged(alone, None, table, tree, None, n_acc, path, prefix, p1, st)
    assert torch.equal(alone, both[0]) and not torch.equal(alone, pages) and torch.equal(p1, p2) and int(st.item()) == 0
    with pytest.raises(sv.SpecError):
        sv.kv_commit(alone, None, tree, tree, n_acc, path, prefix)
    with pytest.raises(sv.SpecError):
        sv.kv_commit_paged(alone, alone.clone(), table, tree, None, n_acc, path, prefix)


def test_one_pool_in_the_fused_commit(lib):
    g = np.random.default_rng(4)
    B, N, V, S, D = 5, 7, 300, 64, 576
    par = np.array([-1, 0, 0, 1, 1, 2, 3])
    fc, ns = T.child_links(par)
    logits = g.standard_normal((B, N, V)).astype(np.float32)
    tok = np.zeros((B, N), np.int32)
    for i in range(1, N):
        tok[:, i] = logits[:, par[i]].argmax(-1) if i in (1, 3, 6) else 5
    args = [dev(logits)] + [i32(np.broadcast_to(x, (B, N)).copy()) for x in (tok, par, fc, ns)]
    tree, cache, prefix = rnd(g, 2, B, 1, N, D), rnd(g, 2, B, 1, S, D), i32([0, 10, 3, 60, 7])
    both, alone = [cache.clone(), cache.clone()], cache.clone()
    o = [[zeros_i32(B), zeros_i32(B, 4), zeros_i32(B)] for _ in range(2)]
    p = [zeros_i32(B), zeros_i32(B)]
    sv.spec_accept_commit(sv.GREEDY, *args, *o[0], *both, tree, tree, prefix, p[0])
    sv.spec_accept_commit(sv.GREEDY, *args, *o[1], alone, None, tree, None, prefix, p[1])
    assert torch.equal(alone, both[0]) and not torch.equal(alone, cache) and torch.equal(*p)
    for a, b in zip(*o):
        assert torch.equal(a, b)


@pytest.mark.parametrize("L,D,bs", [(1, 576, 128), (2, 64, 16)])
def test_one_pool_grows_and_is_packed_as_the_first_of_two(lib, L, D, bs):
    g = np.random.default_rng(5)
    B, mb, nb = 6, 5, 40
    ids = g.permutation(nb)
    table = np.full((B, mb), -1, np.int32)
    table[:3, :2], table[3:, :2] = ids[:2], ids[2:4]                # shared beginnings
    ref = np.bincount(table[table >= 0], minlength=nb).astype(np.int32)
    prefix, need = i32([2 * bs - 3] * B), i32([5, bs, 0, 1, 2 * bs, 4])
    pool = rnd(g, L, nb, 1, bs, D)
    res = []
    for two in (True, False):
        k, v = pool.clone(), pool.clone() if two else None
        t, r, n, st = i32(table), i32(ref), zeros_i32(1), zeros_i32(1)
        sv.kv_pages_reserve(k, v, t, prefix, need, r, t, r, dev_status=st)
        grown = (k.clone(), t.clone(), r.clone())
        sv.kv_pages_compact(k, v, t, r, t, r, n, dev_status=st)
        assert int(st.item()) == 0
        res.append(grown + (k, t, r, n))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert not torch.equal(res[0][0], pool) and not torch.equal(res[0][3], res[0][0])


def near(got, ref, size, keys, scores):
    """bf16 results: P and the output are rounded (2^-8 each); scores are
    float32 sums (of at most 584 products, 2^-23 of their sizes' sum each),
    which the exponential doubles."""
    rel = 2 * 584 * 2.0 ** -23 * scores + (keys + 8) * 2.0 ** -23 + 2.0 ** -8
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = size * rel * (1 + 2.0 ** -8) + np.abs(ref) * 2.0 ** -8 + 1e-30
    assert (err <= tol).all(), float((err / tol).max())


def test_prompts_then_tree_steps_over_one_latent_pool(lib):
    """Three requests: their prompts arrive in two chunks, the rows go to
    reserved pages by the slot map, the expanded form attends; then three tree
    steps in the absorbed form, each committing a path."""
    g = np.random.default_rng(6)
    B, H, lat, D, bs, nb, mb, N, scale = 3, 5, 512, 576, 128, 30, 8, 6, 192 ** -0.5
    chunks = [np.array([150, 1, 260]), np.array([40, 300, 0])]
    room = 500                                                       # more than any chunk: a padded batch
    par = np.array([-1, 0, 0, 1, 2, 3])
    mask = T.depth_and_mask(par)[1]
    pool = torch.full((nb, 1, bs, D), float("nan"), dtype=BF, device="cuda")
    table, ref, prefix, st = torch.full((B, mb), -1, dtype=torch.int32, device="cuda"), zeros_i32(nb), zeros_i32(B), zeros_i32(1)
    ws = torch.empty(sv.kv_pages_workspace_bytes(B, mb, nb), dtype=torch.uint8, device="cuda")
    offsets, slots, pos = zeros_i32(B + 1), zeros_i32(room), zeros_i32(room)
    all_off, all_slots = zeros_i32(B + 1), zeros_i32(1200)
    w = rnd(g, lat, H * 256) * 0.05
    rows = [np.zeros((0, D), np.float32) for _ in range(B)]          # the plain program's

    for new in chunks:
        need = i32(new)
        sv.kv_pages_reserve(pool, None, table, prefix, need, ref, table, ref, workspace=ws, dev_status=st)
        sv.kv_pages_slots(table, prefix, need, offsets, slots, bs, nb, positions=pos, dev_status=st)
        fresh = rnd(g, room, 1, D)
        sv.kv_slots_write(pool, slots, fresh, dev_status=st)
        # everything kept so far and the chunk itself, in order, to be expanded
        sv.kv_pages_slots(table, zeros_i32(B), prefix + need, all_off, all_slots, bs, nb, dev_status=st)
        kept = torch.full((1200, 1, D), 3.0, dtype=BF, device="cuda")
        sv.kv_slots_read(pool, all_slots, kept, dev_status=st)
        kv = (kept[:, 0, :lat] @ w).view(-1, H, 256)
        q = rnd(g, room, H, 192)
        out = torch.full((room, H, 128), 7.0, dtype=BF, device="cuda")
        sv.prompt_attn_latent(q, kv[:, :, :128], kept[:, 0, lat:], kv[:, :, 128:], offsets, all_off, out, int(new.max()), scale,
                              dev_status=st)
        assert int(st.item()) == 0
        off = np.cumsum([0] + new.tolist())
        for b in range(B):
            rows[b] = np.concatenate([rows[b], host(fresh[off[b]:off[b + 1], 0])])
        total = np.cumsum([0] + [len(r) for r in rows])
        assert host(offsets).tolist() == off.tolist() and host(all_off).tolist() == total.tolist()
        np.testing.assert_array_equal(host(kept[:total[-1], 0]), np.concatenate(rows))
        assert float(kept[total[-1]:].abs().max()) == 0.0 and bool((slots[off[-1]:] == -1).all())
        want = np.concatenate([np.arange(len(r) - n, len(r)) for r, n in zip(rows, new)])
        np.testing.assert_array_equal(host(pos)[:off[-1]], want)
        x = [t[:n].double().cpu().numpy() for t, n in ((q, off[-1]), (kv[:, :, :128], total[-1]), (kept[:, 0, lat:], total[-1]),
                                                        (kv[:, :, 128:], total[-1]))]
        ref_o, size = LO.prompt_attention(*x, off, total, scale)
        top = max(float(np.abs(a).max()) for a in x[:3])
        near(out[:off[-1]], ref_o, size, 500, min(40.0, 192 * top * top * scale))
        assert bool((out[off[-1]:] == 7.0).all())
        prefix += need

    size_ws = sv.tree_attn_latent_workspace_bytes(BF, B, N, H, lat, 64, mb * bs)
    scratch = torch.empty(max(16, size_ws), dtype=torch.uint8, device="cuda")
    anc = dev(np.broadcast_to(T.mask_words_multi(mask), (B, N, 1)).copy().view(np.int64))
    for step in range(3):
        sv.kv_pages_reserve(pool, None, table, prefix, i32([N] * B), ref, table, ref, workspace=ws, dev_status=st)
        q, tree = rnd(g, B, N, H, D), rnd(g, B, N, D)
        out = torch.empty(B, N, H, lat, dtype=BF, device="cuda")
        sv.tree_attn_verify_latent_paged(q, pool[:, 0], table, tree, prefix, anc, out, mb * bs, scale, workspace=scratch,
                                         dev_status=st)
        n_acc, path = i32([step, 3, 0]), i32([[0, 1, 3, 5]] * B)
        sv.kv_commit_paged(pool, None, table, tree[:, None], None, n_acc, path, prefix, prefix, dev_status=st)
        assert int(st.item()) == 0
        for b in range(B):
            cache = rows[b][None]
            ref_o, size = LO.tree_attention(q[b:b + 1].double().cpu().numpy(), cache, tree[b:b + 1].double().cpu().numpy(),
                                            [len(rows[b])], mask[None], lat, scale)
            x = float((np.abs(host(q[b])).reshape(-1, D) @ np.abs(np.concatenate([rows[b], host(tree[b])])).T).max()) * scale
            near(out[b], ref_o[0], size[0], len(rows[b]) + N, x)
            rows[b] = np.concatenate([rows[b], host(tree[b])[[0, 1, 3, 5][:int(n_acc[b]) + 1]]])
        assert host(prefix).tolist() == [len(r) for r in rows]
    tab, kept = host(table), host(pool)
    for b in range(B):
        for i in range(len(rows[b])):
            np.testing.assert_array_equal(kept[tab[b, i // bs], 0, i % bs], rows[b][i])


def test_absorbed_and_expanded_forms_agree(lib):
    """The last tokens of a prompt by both forms, in exact numbers the same
    function: q W_uk against the latents, then W_uv, and k = W_uk c, v = W_uv c."""
    g = np.random.default_rng(7)
    H, lat, P, N, scale = 4, 512, 700, 4, 192 ** -0.5
    wk, wv = rnd(g, H, 128, lat) * 0.04, rnd(g, H, lat, 128) * 0.04
    rows, qn, qr = rnd(g, P + N, 576), rnd(g, N, H, 128), rnd(g, N, H, 64)
    q = torch.cat([torch.einsum("nhd,hdl->nhl", qn.float(), wk.float()).to(BF), qr], -1)
    mask = np.tril(np.ones((N, N), bool))                            # a chain
    out = torch.empty(1, N, H, lat, dtype=BF, device="cuda")
    sv.tree_attn_verify_latent(q[None].contiguous(), rows[None, :P].contiguous(), rows[None, P:].contiguous(), i32([P]),
                               dev(T.mask_words_multi(mask)[None].view(np.int64)), out, P, scale)
    absorbed = torch.einsum("nhl,hld->nhd", out[0].float(), wv.float())
    c = rows[:, :lat].float()
    k, v = (torch.einsum("hdl,tl->thd", wk.float(), c).to(BF), torch.einsum("tl,hld->thd", c, wv.float()).to(BF))
    got = torch.empty(N, H, 128, dtype=BF, device="cuda")
    sv.prompt_attn_latent(torch.cat([qn, qr], -1), k, rows[:, lat:], v, i32([0, N]), i32([0, P + N]), got, N, scale)
    # both round q or k, the values and the results to bf16: a few 2^-8 of values of size 0.3
    assert float((absorbed - got.float()).abs().max()) < 8 * 2.0 ** -8 * float(v.float().abs().max())
