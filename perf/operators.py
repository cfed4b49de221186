"""The serving operators around the tree-verification step, as cases to measure.

Three groups, used together by a serving loop over a paged cache:

- ``window``: attention of a tree of drafted tokens (or of one token) over the
  last ``window`` positions and the first ``sinks`` ones, contiguous or paged;
- ``verify``: acceptance of drafted tokens from given probabilities and given
  uniform numbers, with the bonus token from the residual;
- ``fork`` / ``reserve`` / ``compact``: the life of the cache's pages.

``run`` computes a case in plain torch, or through the library where ``own``
is true.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"


def listed():
    return [
        # one token of one sequence past its window: a chat at batch 1, where launches count
        dict(name="window_decode_b1", op="window", dtype=BF16, batch=1, hq=32, hkv=8, dim=128, nodes=1, pmin=5000,
             pmax=5000, window=1024, sinks=4, page=128),
        # the small exact shape in float32: odd prefix, window inside it
        dict(name="window_tiny_f32", op="window", dtype=F32, batch=1, hq=4, hkv=4, dim=64, nodes=5, pmin=1001,
             pmax=1001, window=333, sinks=4, page=0),
        # ragged prefixes, some shorter than the window, a 60-node dynamic tree over a paged cache
        dict(name="window_ragged_paged_b8", op="window", dtype=BF16, batch=8, hq=32, hkv=8, dim=128, nodes=60, pmin=512,
             pmax=8192, window=1024, sinks=4, page=128),
        # long contexts: a wide window, sinks filling a tile and a bit
        dict(name="window_long_b4", op="window", dtype=BF16, batch=4, hq=32, hkv=8, dim=128, nodes=64, pmin=32768,
             pmax=32768, window=4096, sinks=130, page=0),
        # batched serving with 64 query heads, paged
        dict(name="window_serving_b64", op="window", dtype=BF16, batch=64, hq=64, hkv=8, dim=128, nodes=32, pmin=4096,
             pmax=4096, window=2048, sinks=4, page=128),
        # a short chain of deterministic drafts for one sequence
        dict(name="verify_chain_b1", op="verify", dtype=F32, batch=1, nodes=6, width=1, vocab=32000, draft=False),
        # a dynamic tree whose siblings are draws of the drafter
        dict(name="verify_tree_b8", op="verify", dtype=F32, batch=8, nodes=60, width=4, vocab=128256, draft=True),
        # batched serving, deterministic siblings
        dict(name="verify_serving_b64", op="verify", dtype=BF16, batch=64, nodes=32, width=4, vocab=128256, draft=False),
        # tables and counts only: 64 slots rearranged (beams, finished requests), then what left the window is let go
        dict(name="pages_fork_free_b64", op="fork", batch=64, blocks=5000, pages=64, page=128, window=2048, sinks=4),
        # one sequence grows by a tree's path: nothing shared, latency only
        dict(name="pages_reserve_b1", op="reserve", dtype=BF16, batch=1, fan=1, layers=1, hkv=8, dim=128, blocks=64,
             pages=32, page=128, need=8),
        # sixteen requests, four samples each, write into their shared last page
        dict(name="pages_reserve_fork_b64", op="reserve", dtype=BF16, batch=64, fan=4, layers=4, hkv=8, dim=128,
             blocks=512, pages=20, page=128, need=8),
        # a pool with holes is packed to its low end
        dict(name="pages_compact", op="compact", dtype=BF16, batch=32, layers=4, hkv=8, dim=128, blocks=768, pages=16,
             page=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "verify", "fork", "reserve", "compact"])
    if op == "window":
        while True:
            f32 = rng.random() < 0.2
            hkv = rng.choice([1, 2, 4, 8])
            group = rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
            nodes = _log(rng, 1, 256)
            pmax = _log(rng, 1, 20000)
            page = rng.choice([0, 128, 256])
            c = dict(op=op, dtype=F32 if f32 else BF16, batch=_log(rng, 1, 4 if f32 else 64), hq=hkv * group, hkv=hkv,
                     dim=64 if f32 else 128, nodes=min(nodes, 24) if f32 else nodes, pmin=rng.randint(0, pmax),
                     pmax=pmax, window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 64, 130]), page=page)
            rows = c["nodes"] * group
            w = work(c)
            top = work(listed()[4])
            if rows <= (512 if c["nodes"] <= 64 else 2048) and w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"] \
                    and c["batch"] * hkv * pmax <= 64 * 8 * 4096 and (not f32 or w["flops"] < 2e9):
                return c
    if op == "verify":
        nodes = _log(rng, 1, 128)
        vocab = _log(rng, 1000, 130000)
        most = 64 * 32 * 128256 // (nodes * vocab)
        dft = rng.random() < 0.5
        return dict(op=op, dtype=rng.choice([F32, F32, BF16]), batch=_log(rng, 1, max(1, min(64, most // (2 if dft else 1)))),
                    nodes=nodes, width=rng.randint(1, 6), vocab=vocab, draft=dft)
    page = rng.choice([128, 256, 16, 64])
    if op == "fork":
        batch, pages = _log(rng, 1, 64), _log(rng, 1, 64)
        return dict(op=op, batch=batch, blocks=batch * pages + rng.randint(1, 900), pages=pages, page=page,
                    window=rng.choice([0, 1, 100, 1000, 4096]), sinks=rng.choice([0, 4, 130]))
    layers, hkv, dim = rng.randint(1, 4), rng.choice([1, 2, 3, 8]), rng.choice([64, 128])
    dtype = rng.choice([BF16, F32])
    if op == "reserve":
        batch, fan, pages = _log(rng, 1, 64), rng.randint(1, 5), _log(rng, 1, 20)
        need = rng.randint(1, 40)
        blocks = -(-batch // fan) * pages + batch * (2 + need // page) + rng.randint(0, 30)
        while blocks * page * layers > 512 * 128 * 4 // (2 if dtype == F32 else 1) and layers > 1:
            layers -= 1
        return dict(op=op, dtype=dtype, batch=batch, fan=fan, layers=layers, hkv=hkv, dim=dim, blocks=blocks,
                    pages=pages, page=page, need=need)
    batch, pages = _log(rng, 1, 32), _log(rng, 1, 16)
    return dict(op=op, dtype=dtype, batch=batch, layers=layers if dtype == BF16 else 1, hkv=hkv, dim=dim,
                blocks=batch * pages + rng.randint(1, 200), pages=pages, page=page)


# ------------------------------------------------------------------ inputs


def _torch_type(c):
    return torch.float32 if c["dtype"] == F32 else torch.bfloat16


def _size(c):
    return 4 if c["dtype"] == F32 else 2


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _prefixes(c):
    """Prefix lengths spread over [pmin, pmax], the longest first."""
    b = c["batch"]
    return [c["pmax"] - (c["pmax"] - c["pmin"]) * i // max(1, b - 1) for i in range(b)]


def _tree(rng, nodes, width, depth=6):
    """A random tree in node order, children of a node ascending: parents, depth, links, sibling rank."""
    parents, level, kids = [-1], [0], [0]
    for i in range(1, nodes):
        open_ = [j for j in range(i) if kids[j] < width and level[j] < depth]
        j = open_[int(rng.integers(len(open_)))] if open_ else i - 1
        kids[j] += 1
        parents.append(j)
        level.append(level[j] + 1)
        kids.append(0)
    order = sorted(range(1, nodes), key=lambda i: level[i])
    new = {0: 0}
    for k, i in enumerate(order):
        new[i] = k + 1
    par = [-1] + [new[parents[i]] for i in order]
    dep = [0] + [level[i] for i in order]
    first, nxt, last, rank = [-1] * nodes, [-1] * nodes, [-1] * nodes, [0] * nodes
    for i in range(1, nodes):
        p = par[i]
        if first[p] < 0:
            first[p] = i
        else:
            nxt[last[p]] = i
            rank[i] = rank[last[p]] + 1
        last[p] = i
    return par, dep, first, nxt, rank


def _mask_words(par):
    n = len(par)
    seen, words = [], (n + 63) // 64
    out = np.zeros((n, words), np.uint64)
    for i, p in enumerate(par):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        for w in range(words):
            out[i, w] = (seen[i] >> (64 * w)) & 0xFFFFFFFFFFFFFFFF
    return out.view(np.int64)


def _held_pages(c, p, slack):
    """Pages of a sequence that a window over prefix p still needs (or that the next rows go to)."""
    page, lo = c["page"], p - c["window"] + 1
    return [j for j in range(-(-(p + slack) // page)) if j * page < c["sinks"] or (j + 1) * page > lo]


def _prepare_window(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    t, b, n, d, hkv = _torch_type(c), c["batch"], c["nodes"], c["dim"], c["hkv"]
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=t)  # noqa: E731
    prefix = _prefixes(c)
    trees = [_tree(rng, n, 6, 8) for _ in range(b)]
    s = dict(case=c, prefix=_i32(prefix), max_prefix=max(prefix), q=normal(b, n, c["hq"], d), kt=normal(b, hkv, n, d),
             vt=normal(b, hkv, n, d), depth=_i32([x[1] for x in trees]),
             anc=torch.from_numpy(np.stack([_mask_words(x[0]) for x in trees])).cuda())
    if c["page"]:
        held = [_held_pages(c, p, 16) for p in prefix]
        blocks = sum(len(h) for h in held) + 3
        ids = rng.permutation(blocks)
        table = np.full((b, max(1, max(h[-1] for h in held) + 1)), -1, np.int32)
        k = 0
        for i, h in enumerate(held):
            table[i, h] = ids[k:k + len(h)]
            k += len(h)
        s.update(table=_i32(table), k=normal(blocks, hkv, c["page"], d), v=normal(blocks, hkv, c["page"], d))
    else:
        s.update(k=normal(b, hkv, max(prefix) + 64, d), v=normal(b, hkv, max(prefix) + 64, d))
    if own:
        from tree_speculative_decoding_attn_gb300 import specverify as sv
        size = sv.tree_attn_window_workspace_bytes(t, b, n, c["hq"], hkv, d, s["max_prefix"], c["window"], c["sinks"])
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    s.update(out=torch.empty_like(s["q"]), status=_i32([0]))
    return s


def _prepare_verify(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, n, v = c["batch"], c["nodes"], c["vocab"]
    trees = [_tree(rng, n, c["width"], n if c["width"] == 1 else 6) for _ in range(b)]
    par, first, nxt, rank = (np.array([x[k] for x in trees]) for k in (0, 2, 3, 4))
    logits = torch.randn((b, n, v), generator=g, device="cuda") * 2.5
    drafted = logits + 0.5 * torch.randn((b, n, v), generator=g, device="cuda")
    kids = int(rank.max()) + 1
    if c["draft"]:
        q = torch.softmax(drafted, -1)
        picks = torch.multinomial(q.view(b * n, v), kids, replacement=True, generator=g).view(b, n, kids)
        q = q.to(_torch_type(c))
    else:
        q = None
        # a sibling of rank r is the drafter's r-th best token, made likely for the target as often as good drafts are
        picks = drafted.topk(kids, dim=-1).indices
        lift = torch.rand((b, n, 1), generator=g, device="cuda") < 0.7
        at = picks[:, :, :1]
        logits.scatter_(2, at, torch.where(lift, logits.amax(-1, keepdim=True) + 6.0, logits.gather(2, at)))
    p = torch.softmax(logits, -1).to(_torch_type(c))
    del logits, drafted
    pt, rt = torch.from_numpy(np.maximum(par, 0)).cuda(), torch.from_numpy(rank).cuda()
    rows = torch.arange(b, device="cuda")[:, None]
    s = dict(case=c, p=p, q=q, tok=picks[rows, pt, rt].int().contiguous(), parents=_i32(par), first=_i32(first), next=_i32(nxt),
             u=torch.rand((b, n), generator=g, device="cuda"), ub=torch.rand((b,), generator=g, device="cuda"),
             cap=n if c["width"] == 1 else min(n, 8), kids=kids, status=_i32([0]))
    s.update(acc_len=_i32([0] * b), path=_i32([[0] * s["cap"]] * b), bonus=_i32([0] * b))
    return s


def _pool(c, g):
    shape = (c["layers"], c["blocks"], c["hkv"], c["page"], c["dim"])
    return [torch.randn(shape, generator=g, device="cuda", dtype=_torch_type(c)) for _ in range(2)]


def _counts(table, blocks):
    return np.bincount(table[table >= 0].ravel(), minlength=blocks).astype(np.int32)


def _prepare_fork(c, seed):
    rng = np.random.default_rng(seed)
    b, mb, page = c["batch"], c["pages"], c["page"]
    prefix = rng.integers(0, mb * page, b)
    ids, k = rng.permutation(c["blocks"]), 0
    table = np.full((b, mb), -1, np.int32)
    for i, p in enumerate(prefix):
        n = -(-int(p) // page)
        table[i, :n] = ids[k:k + n]
        k += n
    parent = rng.integers(0, b, b)              # samples continue from some sequence
    parent[rng.random(b) < 0.5] = -2
    parent = np.where(parent == -2, np.arange(b), parent)
    parent[rng.random(b) < 0.1] = -1            # a finished slot
    ref = _counts(table, c["blocks"])
    z = np.zeros((b, mb), np.int32)
    return dict(case=c, table=_i32(table), prefix=_i32(prefix), parent=_i32(parent), ref=_i32(ref), forked=_i32(z),
                forked_prefix=_i32(prefix * 0), forked_ref=_i32(ref), table_out=_i32(z), ref_out=_i32(ref), status=_i32([0]))


def _prepare_reserve(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, fan, mb, page = c["batch"], c["fan"], c["pages"], c["page"]
    wide = mb + c["need"] // page + 2
    ids, k = rng.permutation(c["blocks"]), 0
    table, prefix = np.full((b, wide), -1, np.int32), np.zeros(b, np.int32)
    for i in range(0, b, fan):
        p = (mb - 1) * page + _mid_rows(c, i // fan)
        n = -(-p // page)
        table[i:i + fan, :n] = ids[k:k + n]
        prefix[i:i + fan] = p
        k += n
    k_pages, v_pages = _pool(c, g)
    ref = _counts(table, c["blocks"])
    s = dict(case=c, k=k_pages, v=v_pages, table=_i32(table), prefix=_i32(prefix), need=_i32([c["need"]] * b),
             ref=_i32(ref), table_out=_i32(table), ref_out=_i32(ref), status=_i32([0]))
    if own:
        from tree_speculative_decoding_attn_gb300 import specverify as sv
        size = sv.kv_pages_workspace_bytes(b, wide, c["blocks"])
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


def _mid_rows(c, i):
    """Rows in use of the last page of request i (spread over the page, deterministic)."""
    return 1 + (i * 37 + c["page"] // 2) % c["page"]


def _prepare_compact(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    b, mb = c["batch"], c["pages"]
    table = rng.permutation(c["blocks"])[:b * mb].reshape(b, mb).astype(np.int32)
    if b > 1:
        table[b - 1, :mb // 2] = table[0, :mb // 2]       # a shared beginning
    table[b // 2, mb // 2:] = -1
    k_pages, v_pages = _pool(c, g)
    ref = _counts(table, c["blocks"])
    s = dict(case=c, k=k_pages, v=v_pages, table=_i32(table), ref=_i32(ref), table_out=_i32(table), ref_out=_i32(ref),
             used=_i32([0]), status=_i32([0]))
    if own:
        from tree_speculative_decoding_attn_gb300 import specverify as sv
        size = sv.kv_pages_workspace_bytes(b, mb, c["blocks"])
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return {"window": _prepare_window, "verify": _prepare_verify, "fork": _prepare_fork, "reserve": _prepare_reserve,
            "compact": _prepare_compact}[case["op"]](case, seed)


# ------------------------------------------------------------------ plain forms


def _plain_window(s):
    c = s["case"]
    b, n, hq, d = s["q"].shape
    hkv, w, sinks = c["hkv"], c["window"], c["sinks"]
    dev = s["q"].device
    p = s["prefix"].long()[:, None]
    span = min(w - 1, s["max_prefix"])
    head = min(sinks, s["max_prefix"])
    # the positions any row can see: the sinks, then the window of the root
    near = p - span + torch.arange(span, device=dev)[None]
    first = torch.arange(head, device=dev)[None].expand(b, -1)
    at = torch.cat([first, near], 1)
    there = torch.cat([first < p, near >= sinks], 1) & (at >= 0)
    safe = torch.where(there, at, 0)
    if c["page"]:
        blk = s["table"].long().gather(1, safe // c["page"]).clamp(min=0)
        k = s["k"][blk, :, safe % c["page"]].permute(0, 2, 1, 3)
        v = s["v"][blk, :, safe % c["page"]].permute(0, 2, 1, 3)
    else:
        seq = torch.arange(b, device=dev)[:, None]
        k = s["k"][seq, :, safe].permute(0, 2, 1, 3)
        v = s["v"][seq, :, safe].permute(0, 2, 1, 3)
    k = torch.cat([k, s["kt"]], 2).float()
    v = torch.cat([v, s["vt"]], 2).float()
    depth = s["depth"].long()
    pos = p + depth
    see = there[:, None] & ((at[:, None] < sinks) | (at[:, None] > pos[:, :, None] - w))
    node = torch.arange(n, device=dev)
    anc = ((s["anc"][:, :, node // 64] >> (node % 64)) & 1).bool()
    anc = anc & ((pos[:, None] < sinks) | (pos[:, None] > pos[:, :, None] - w))
    see = torch.cat([see, anc], 2)
    see = see[:, None, :, None].expand(b, hkv, n, hq // hkv, see.shape[-1]).reshape(b, hkv, n * (hq // hkv), -1)
    q = s["q"].float().view(b, n, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    x = (q @ k.transpose(2, 3)) * d ** -0.5
    x = torch.where(see, x, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True))
    o = (e @ v) / e.sum(-1, keepdim=True)
    return o.view(b, hkv, n, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, n, hq, d).to(s["q"].dtype)


def _plain_verify(s):
    b, n, v = s["p"].shape
    dev = s["p"].device
    seq = torch.arange(b, device=dev)
    node = torch.zeros(b, dtype=torch.long, device=dev)
    going = torch.ones(b, dtype=torch.bool, device=dev)
    length = torch.zeros(b, dtype=torch.int32, device=dev)
    path = torch.full((b, s["cap"]), -1, dtype=torch.int32, device=dev)
    path[:, 0] = 0
    left = None
    for step in range(s["cap"]):
        p = s["p"][seq, node].double()
        q = s["q"][seq, node].double() if s["q"] is not None else None
        w, mass = p.clone(), torch.ones(b, dtype=torch.float64, device=dev)
        child = torch.where(going, s["first"][seq, node].long(), -1)
        took = torch.full_like(child, -1)
        for _ in range(s["kids"]):
            live = (child >= 0) & (took < 0)
            c = child.clamp(min=0)
            t = s["tok"][seq, c].long()
            wt = w[seq, t]
            bar = s["u"][seq, c].double() * mass
            if q is not None:
                bar = bar * q[seq, t]
            ok = live & (bar < wt)
            took = torch.where(ok, child, took)
            no = live & ~ok
            if q is None:
                w[seq, t] = torch.where(no, 0.0, wt)
                mass = torch.where(no, (mass - wt).clamp(min=0), mass)
            else:
                rest = torch.where(mass[:, None] > 0, w / mass[:, None] - q, 0.0).clamp(min=0)
                w = torch.where(no[:, None], rest, w)
                mass = torch.where(no, w.sum(-1), mass)
            child = torch.where(no, s["next"][seq, c].long(), child)
            child = torch.where(live, child, -1)
        # what the bonus is drawn from, for the sequences that stop here
        w = torch.where((w.sum(-1) > 0)[:, None], w, p)
        left = w if left is None else torch.where(going[:, None], w, left)
        going = going & (took >= 0)
        if step + 1 < s["cap"]:
            path[:, step + 1] = torch.where(going, took.int(), path[:, step + 1])
        length += going.int()
        node = torch.where(going, took, node)
    cum = left.cumsum(-1)
    bonus = (cum <= s["ub"].double()[:, None] * cum[:, -1:]).sum(-1).clamp(max=v - 1).int()
    return length, path, bonus


def _add_refs(ref, table, sign):
    held = table >= 0
    return ref.scatter_add(0, table.clamp(min=0).long().flatten(), (sign * held).int().flatten())


def _plain_fork(s):
    c, table, parent = s["case"], s["table"], s["parent"].long()
    live = parent >= 0
    forked = torch.where(live[:, None], table[parent.clamp(min=0)], -1)
    prefix = torch.where(live, s["prefix"][parent.clamp(min=0)], 0)
    ref = _add_refs(_add_refs(s["ref"], table, -1), forked, 1)
    j = torch.arange(table.shape[1], device=table.device) * c["page"]
    p = prefix[:, None]
    keep = j < p
    if c["window"] > 0:
        keep = keep & ((j < c["sinks"]) | (j + c["page"] > p - c["window"] + 1))
    gone = torch.where(keep, -1, forked)
    return forked, prefix, ref, torch.where(keep, forked, -1), _add_refs(ref, gone, -1)


def _plain_reserve(s):
    c, table, ref = s["case"], s["table"], s["ref"]
    b, wide = table.shape
    page, blocks = c["page"], c["blocks"]
    p, need = s["prefix"][:, None], s["need"][:, None]
    j = torch.arange(wide, device=table.device, dtype=torch.int32)[None]
    write = (need > 0) & (j >= p // page) & (j <= (p + need - 1) // page) & (p + need <= wide * page)
    at = table.clamp(min=0).long()
    held, count = table >= 0, ref[at]
    shared = write & held & (count > 1)
    order = torch.arange(b * wide, device=table.device).view(b, wide)
    zero = torch.zeros(blocks, dtype=torch.long, device=table.device)
    writers = zero.scatter_add(0, at.flatten(), shared.long().flatten())
    last = (zero - 1).scatter_reduce(0, at.flatten(), torch.where(shared, order, -1).flatten(), "amax")
    copy = shared & ~((writers[at] >= count) & (last[at] == order))
    fresh = write & (~held | copy)
    free = torch.argsort((ref > 0).int(), stable=True)
    rank = (fresh.flatten().cumsum(0) - 1).view(b, wide).clamp(min=0)
    fits = fresh.sum() <= (ref <= 0).sum()
    copy, fresh = copy & fits, fresh & fits
    out = torch.where(fresh, free[rank.clamp(max=blocks - 1)].int(), table)
    ref_out = ref.scatter_add(0, at.flatten(), -copy.int().flatten())
    ref_out[out[fresh].long()] = 1
    part = copy & (j == p // page) & (p % page > 0)
    old, new = table[part].long(), out[part].long()
    rows = (p % page).expand(b, wide)[part]
    valid = (torch.arange(page, device=table.device)[None] < rows[:, None])[None, :, None, :, None]
    for pool in (s["k"], s["v"]):
        pool[:, new] = torch.where(valid, pool[:, old], pool[:, new])
    return out, ref_out, s["k"], s["v"]


def _plain_compact(s):
    table, ref = s["table"], s["ref"]
    ids = torch.arange(ref.numel(), device=ref.device)
    used = ref > 0
    n = used.sum()
    src, dst = ids[used & (ids >= n)], ids[~used & (ids < n)]
    to = torch.where(used, ids, -1)
    to[src] = dst
    for pool in (s["k"], s["v"]):
        pool[:, dst] = pool[:, src]
    ref_out = ref.clone()
    ref_out[dst] = ref[src]
    ref_out[src] = 0
    out = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), -1)
    return out, torch.where(ids < n, ref_out, 0), n.int().view(1), s["k"], s["v"]


# ------------------------------------------------------------------ the library's calls


def _own(s):
    from tree_speculative_decoding_attn_gb300 import specverify as sv
    c = s["case"]
    if c["op"] == "window":
        more = dict(sinks=c["sinks"], workspace=s["workspace"], dev_status=s["status"])
        if c["page"]:
            sv.tree_attn_verify_window_paged(s["q"], s["k"], s["v"], s["table"], s["kt"], s["vt"], s["prefix"], s["depth"],
                                             s["anc"], s["out"], s["max_prefix"], c["window"], **more)
        else:
            sv.tree_attn_verify_window(s["q"], s["k"], s["v"], s["kt"], s["vt"], s["prefix"], s["depth"], s["anc"],
                                       s["out"], s["max_prefix"], c["window"], **more)
        return s["out"]
    if c["op"] == "verify":
        sv.spec_verify_probs(s["p"], s["tok"], s["parents"], s["first"], s["next"], s["u"], s["ub"], s["acc_len"],
                             s["path"], s["bonus"], draft_probs=s["q"], dev_status=s["status"])
        return s["acc_len"], s["path"], s["bonus"]
    if c["op"] == "fork":
        sv.kv_pages_fork(s["table"], s["prefix"], s["parent"], s["ref"], s["forked"], s["forked_prefix"],
                         s["forked_ref"], dev_status=s["status"])
        sv.kv_pages_free(s["forked"], s["forked_prefix"], s["forked_ref"], s["table_out"], s["ref_out"], c["page"],
                         window=c["window"], sinks=c["sinks"], dev_status=s["status"])
        return s["forked"], s["forked_prefix"], s["forked_ref"], s["table_out"], s["ref_out"]
    if c["op"] == "reserve":
        sv.kv_pages_reserve(s["k"], s["v"], s["table"], s["prefix"], s["need"], s["ref"], s["table_out"], s["ref_out"],
                            workspace=s["workspace"], dev_status=s["status"])
        return s["table_out"], s["ref_out"], s["k"], s["v"]
    sv.kv_pages_compact(s["k"], s["v"], s["table"], s["ref"], s["table_out"], s["ref_out"], s["used"],
                        workspace=s["workspace"], dev_status=s["status"])
    return s["table_out"], s["ref_out"], s["used"], s["k"], s["v"]


def run(state):
    if own:
        return _own(state)
    return {"window": _plain_window, "verify": _plain_verify, "fork": _plain_fork, "reserve": _plain_reserve,
            "compact": _plain_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and exact values


def work(case):
    c = case
    if c["op"] == "window":
        keys = [min(p, c["window"] - 1) + min(c["sinks"], max(0, p - c["window"] + 1)) for p in _prefixes(c)]
        rows = c["nodes"] * c["hq"] // c["hkv"]
        row = c["dim"] * _size(c)
        total = sum(keys) + c["batch"] * c["nodes"]
        return {"bytes": 2 * c["hkv"] * total * row + 2 * c["batch"] * c["nodes"] * c["hq"] * row
                + c["batch"] * c["nodes"] * (4 + 8 * ((c["nodes"] + 63) // 64)),
                "flops": 4 * c["hkv"] * rows * c["dim"] * total}
    if c["op"] == "verify":
        # the row the bonus is drawn from, and per node its links, number and one probability (two with a drafter's)
        rows = 2 if c["draft"] else 1
        b, e = c["batch"], _size(c)
        return {"bytes": b * (rows * c["vocab"] * e + c["nodes"] * (20 + rows * e)), "flops": b * rows * c["vocab"]}
    if c["op"] == "fork":
        n = c["batch"] * c["pages"]
        return {"bytes": 4 * (4 * n + 4 * c["blocks"] + 4 * c["batch"]), "flops": 4 * n}
    row = c["hkv"] * c["dim"] * _size(c) * c["layers"] * 2
    if c["op"] == "reserve":
        rows = sum((min(c["fan"], c["batch"] - i) - 1) * (_mid_rows(c, i // c["fan"]) % c["page"])
                   for i in range(0, c["batch"], c["fan"]))
        wide = c["pages"] + c["need"] // c["page"] + 2
        return {"bytes": 2 * rows * row + 8 * (c["batch"] * (wide + 1) + c["blocks"]), "flops": c["blocks"]}
    # used pages lie anywhere in the pool: those past the used count move
    held = c["batch"] * c["pages"] - (c["pages"] - c["pages"] // 2) - (c["pages"] // 2 if c["batch"] > 1 else 0)
    moved = held * (c["blocks"] - held) / c["blocks"]
    return {"bytes": 2 * moved * c["page"] * row + 8 * (c["batch"] * c["pages"] + c["blocks"]), "flops": c["blocks"]}


def _exact_window(c, s):
    """Every prefix position of a sequence in turn, masked by its position, in 64 bits."""
    b, n, hq, d = s["q"].shape
    group = hq // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    prefix, anc = s["prefix"].tolist(), s["anc"].cpu().numpy().view(np.uint64)
    depth = s["depth"].cpu().numpy()
    for i in range(b):
        p = prefix[i]
        if c["page"]:
            tab = [max(0, x) for x in s["table"][i].tolist()][:-(-p // c["page"])]
            k, v = ([x[t] for t in tab] for x in (s["k"], s["v"]))
            k, v = (torch.cat(x, 1)[:, :p] if x else s["kt"][i][:, :0] for x in (k, v))
        else:
            k, v = s["k"][i, :, :p], s["v"][i, :, :p]
        k, v = torch.cat([k, s["kt"][i]], 1).double(), torch.cat([v, s["vt"][i]], 1).double()
        where = np.concatenate([np.arange(p), p + depth[i]])
        mine = (p + depth[i])[:, None]
        ok = np.ones((n, p + n), bool)
        for t in range(n):
            ok[:, p + t] = (anc[i, :, t // 64] >> np.uint64(t % 64)) & np.uint64(1)
        ok &= (where[None] < c["sinks"]) | (mine - where[None] < c["window"])
        ok = torch.from_numpy(ok).cuda()
        for h in range(c["hkv"]):
            q = s["q"][i, :, h * group:(h + 1) * group].double()
            x = torch.einsum("ngd,jd->ngj", q, k[h]) / math.sqrt(d)
            x = x.masked_fill(~ok[:, None], -math.inf)
            x = x - x.max(-1, keepdim=True).values
            e = x.exp()
            e = e / e.sum(-1, keepdim=True)
            out[i, :, h * group:(h + 1) * group] = torch.einsum("ngj,jd->ngd", e, v[h])
    return out


def _exact_verify(c, s):
    """One sequence after another on the host."""
    b, cap = c["batch"], s["cap"]
    tok, first, nxt = (s[k].cpu().numpy() for k in ("tok", "first", "next"))
    u, ub = s["u"].cpu().numpy().astype(np.float64), s["ub"].cpu().numpy().astype(np.float64)
    lens, paths, bonus = np.zeros(b, np.int32), np.full((b, cap), -1, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        at, path = 0, [0]
        while True:
            p = s["p"][i, at].double().cpu().numpy()
            q = s["q"][i, at].double().cpu().numpy() if c["draft"] else None
            r, child, hit = p.copy(), int(first[i, at]), -1
            while child >= 0:
                t = int(tok[i, child])
                if u[i, child] * (q[t] if c["draft"] else max(0.0, r_left(p, r))) < r[t]:
                    hit = child
                    break
                if c["draft"]:
                    r = np.maximum(r - q, 0.0)
                    r = r / r.sum() if r.sum() > 0 else r
                else:
                    r[t] = 0.0
                child = int(nxt[i, child])
            if hit < 0:
                break
            at = hit
            path.append(hit)
        r = r if r.sum() > 0 else p
        run_ = np.cumsum(r)
        lens[i], bonus[i] = len(path) - 1, min(c["vocab"] - 1, int(np.searchsorted(run_, ub[i] * run_[-1], side="right")))
        paths[i, :len(path)] = path
    return tuple(torch.from_numpy(x) for x in (lens, paths, bonus))


def r_left(p, r):
    """What removals have left of a row that sums to one."""
    return 1.0 - p[r != p].sum()


def exact(case, seed):
    if case["op"] == "window":
        return _exact_window(case, prepare(case, seed))
    if case["op"] == "verify":
        return _exact_verify(case, prepare(case, seed))
    return None
