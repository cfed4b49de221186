"""The operators of a latent cache and of packed prompts, as cases to measure.

Three groups, the life of a cache that holds one latent vector a token:

- ``latent``: attention of a tree of drafted tokens (or of one token) over
  latent rows, the queries and outputs in the latent space (absorbed form),
  contiguous or paged;
- ``prompt``: causal attention of packed prompt tokens over keys and values
  expanded from the latents, with one rotary key for all heads;
- ``slots``: where the packed tokens of requests lie in a paged cache, from
  the requests' lengths and block tables, and the rows' way in or out.

``run`` computes a case in plain torch, or through the library where ``own``
is true.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = "bf16", "f32"
ROPE = 64           # rotary dims of a latent row and of an expanded query
HEAD = 128          # expanded dims of a key (without the rotary ones) and of a value


def listed():
    return [
        # one token of one chat: launches and the split of one long row of keys
        dict(name="latent_decode_b1", op="latent", dtype=BF16, batch=1, hq=16, latent=512, nodes=1, pmin=5000, pmax=5000,
             page=128),
        # the small exact shape in float32
        dict(name="latent_tiny_f32", op="latent", dtype=F32, batch=1, hq=4, latent=256, nodes=5, pmin=129, pmax=129, page=0),
        # dynamic trees of 60 nodes over ragged prefixes in pages
        dict(name="latent_ragged_b8", op="latent", dtype=BF16, batch=8, hq=32, latent=512, nodes=60, pmin=512, pmax=8192,
             page=128),
        # batched decoding without drafts
        dict(name="latent_decode_b64", op="latent", dtype=BF16, batch=64, hq=64, latent=512, nodes=1, pmin=4096, pmax=4096,
             page=128),
        # batched serving, trees of 32 nodes
        dict(name="latent_serving_b32", op="latent", dtype=BF16, batch=32, hq=64, latent=512, nodes=32, pmin=4096,
             pmax=4096, page=128),
        # long contexts, a short chain of drafts, all heads of a large model
        dict(name="latent_long_b4", op="latent", dtype=BF16, batch=4, hq=128, latent=512, nodes=4, pmin=32768, pmax=32768,
             page=0),
        # short prompts that arrived together
        dict(name="prompt_short_b8", op="prompt", batch=8, hq=16, qmin=17, qmax=300, kept=0),
        # one long prompt
        dict(name="prompt_long", op="prompt", batch=1, hq=32, qmin=8192, qmax=8192, kept=0),
        # chunks of prompts whose beginnings are in the cache
        dict(name="prompt_chunks_b4", op="prompt", batch=4, hq=32, qmin=384, qmax=512, kept=6000),
        # the rows of one decoding step: latency only
        dict(name="slots_step_b64", op="slots", dtype=BF16, write=True, batch=64, nmin=1, nmax=1, kept=4000, hkv=1, dim=576,
             page=128, spare=0),
        # prompts of sixteen requests go into their pages, in a buffer with room behind the last one
        dict(name="slots_prompts_b16", op="slots", dtype=BF16, write=True, batch=16, nmin=100, nmax=4096, kept=0, hkv=1,
             dim=576, page=128, spare=1000),
        # the latents of cached beginnings come out, to be expanded for the next chunk
        dict(name="slots_fetch_b4", op="slots", dtype=BF16, write=False, batch=4, nmin=6000, nmax=8192, kept=0, hkv=1,
             dim=576, page=128, spare=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["latent", "latent", "prompt", "slots"])
    if op == "latent":
        top = work(listed()[4])
        while True:
            f32 = rng.random() < 0.2
            pmax = _log(rng, 1, 32768)
            c = dict(op=op, dtype=F32 if f32 else BF16, batch=_log(rng, 1, 4 if f32 else 64),
                     hq=rng.choice([1, 2, 3, 5, 8, 12, 16, 20, 32, 40, 64, 96, 128]), latent=rng.choice([256, 512, 512]),
                     nodes=_log(rng, 1, 24 if f32 else 256), pmin=rng.randint(0, pmax), pmax=pmax,
                     page=rng.choice([0, 128, 256]))
            w = work(c)
            if w["bytes"] <= 2 * top["bytes"] and w["flops"] <= top["flops"] and c["batch"] * pmax <= 64 * 8192 \
                    and (not f32 or w["flops"] < 1e9):
                return c
    if op == "prompt":
        top = work(listed()[7])
        while True:
            qmax = _log(rng, 1, 4096)
            c = dict(op=op, batch=_log(rng, 1, 16), hq=rng.choice([1, 2, 3, 5, 8, 16, 32, 64]), qmin=rng.randint(0, qmax),
                     qmax=qmax, kept=rng.choice([0, 0, _log(rng, 1, 16384)]))
            w = work(c)
            if w["bytes"] <= 2 * top["bytes"] and w["flops"] <= top["flops"]:
                return c
    while True:
        nmax = _log(rng, 1, 8192)
        hkv, dim, dtype = rng.choice([(1, 576), (1, 320), (2, 128), (8, 128), (3, 64)]) + (rng.choice([BF16, BF16, F32]),)
        c = dict(op=op, dtype=dtype, write=rng.random() < 0.6, batch=_log(rng, 1, 256), nmin=rng.randint(0, nmax), nmax=nmax,
                 kept=rng.choice([0, _log(rng, 1, 5000)]), hkv=hkv, dim=dim, page=rng.choice([16, 64, 128, 256]),
                 spare=rng.choice([0, 1, 77, 2000]))
        if work(c)["bytes"] <= 2 * work(listed()[10])["bytes"]:
            return c


# ------------------------------------------------------------------ inputs


def _torch_type(c):
    return torch.float32 if c.get("dtype") == F32 else torch.bfloat16


def _size(c):
    return 4 if c.get("dtype") == F32 else 2


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(x, np.int32))).cuda()


def _spread(lo, hi, n):
    """n lengths spread over [lo, hi], the longest first."""
    return [hi - (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _tree(rng, nodes):
    """Parents of a random tree in level order."""
    par, depth = [-1], [0]
    for i in range(1, nodes):
        j = int(rng.integers(max(0, i - 12), i))
        par.append(j)
        depth.append(depth[j] + 1)
    order = sorted(range(nodes), key=lambda i: depth[i])
    new = {old: k for k, old in enumerate(order)}
    return [-1 if par[i] < 0 else new[par[i]] for i in order]


def _mask_words(par):
    n = len(par)
    seen, out = [], np.zeros((n, (n + 63) // 64), np.uint64)
    for i, p in enumerate(par):
        seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        for w in range(out.shape[1]):
            out[i, w] = (seen[i] >> (64 * w)) & 0xFFFFFFFFFFFFFFFF
    return out.view(np.int64)


def _tables(rng, lengths, page, spare):
    """Block tables for sequences of the given lengths, blocks in any order; the pool's blocks."""
    pages = [-(-n // page) for n in lengths]
    blocks = sum(pages) + spare
    ids, k = rng.permutation(blocks), 0
    table = np.full((len(lengths), max(1, max(pages))), -1, np.int32)
    for i, n in enumerate(pages):
        table[i, :n] = ids[k:k + n]
        k += n
    return table, blocks


def _prepare_latent(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    t, b, n, d = _torch_type(c), c["batch"], c["nodes"], c["latent"] + ROPE
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=t)  # noqa: E731
    prefix = _spread(c["pmin"], c["pmax"], b)
    s = dict(case=c, lengths=prefix, prefix=_i32(prefix), max_prefix=max(prefix), scale=(HEAD + ROPE) ** -0.5,
             q=normal(b, n, c["hq"], d), tree=normal(b, n, d),
             anc=torch.from_numpy(np.stack([_mask_words(_tree(rng, n)) for _ in range(b)])).cuda())
    if c["page"]:
        table, blocks = _tables(rng, prefix, c["page"], 3)
        s.update(table=_i32(table), cache=normal(blocks, c["page"], d))
    else:
        s.update(cache=normal(b, max(prefix) + 64, d))
    if own:
        from tree_speculative_decoding_attn_gb300 import specverify as sv
        size = sv.tree_attn_latent_workspace_bytes(t, b, n, c["hq"], c["latent"], ROPE, s["max_prefix"])
        s["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    s.update(out=torch.empty(b, n, c["hq"], c["latent"], dtype=t, device="cuda"), status=_i32([0]))
    return s


def _prompt_lengths(c):
    new = _spread(c["qmin"], c["qmax"], c["batch"])
    return new, [n + k for n, k in zip(new, _spread(c["kept"] // 2, c["kept"], c["batch"]))]


def _prepare_prompt(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    new, all_ = _prompt_lengths(c)
    h = c["hq"]
    kv = normal(max(1, sum(all_)), h, 2 * HEAD)         # one projection of the latents gives keys and values
    rows = normal(max(1, sum(all_)), 512 + ROPE)        # the cache's rows: latents, then the rotary key
    q = normal(max(1, sum(new)), h, HEAD + ROPE)
    return dict(case=c, new=new, all=all_, q=q, k=kv[:, :, :HEAD], v=kv[:, :, HEAD:], k_rope=rows[:, 512:],
                q_off=_i32(np.cumsum([0] + new)), kv_off=_i32(np.cumsum([0] + all_)), max_q=max(new),
                scale=(HEAD + ROPE) ** -0.5, out=torch.zeros(q.shape[0], h, HEAD, dtype=torch.bfloat16, device="cuda"),
                status=_i32([0]))


def _prepare_slots(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    t, new = _torch_type(c), _spread(c["nmin"], c["nmax"], c["batch"])
    kept = [(c["kept"] + 37 * i) % (c["kept"] + 1) for i in range(c["batch"])]
    table, blocks = _tables(rng, [n + k for n, k in zip(new, kept)], c["page"], 5)
    room = sum(new) + c["spare"]
    normal = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=t)  # noqa: E731
    return dict(case=c, table=_i32(table), prefix=_i32(kept), new=_i32(new), pages=normal(blocks, c["hkv"], c["page"], c["dim"]),
                rows=normal(max(1, room), c["hkv"], c["dim"]), offsets=_i32([0] * (c["batch"] + 1)),
                slots=_i32([0] * max(1, room)), pos=_i32([0] * max(1, room)), status=_i32([0]))


def prepare(case, seed):
    return {"latent": _prepare_latent, "prompt": _prepare_prompt, "slots": _prepare_slots}[case["op"]](case, seed)


# ------------------------------------------------------------------ plain forms


def _plain_latent(s):
    c = s["case"]
    b, n, hq, d = s["q"].shape
    lat, dev = c["latent"], s["q"].device
    node = torch.arange(n, device=dev)
    anc = ((s["anc"][:, :, node // 64] >> (node % 64)) & 1).bool()
    out = torch.empty_like(s["out"])
    for i in range(b):
        p = s["lengths"][i]
        if c["page"]:
            at = torch.arange(p, device=dev)
            rows = s["cache"][s["table"][i].long()[at // c["page"]], at % c["page"]]
        else:
            rows = s["cache"][i, :p]
        k = torch.cat([rows, s["tree"][i]]).float()
        x = (s["q"][i].float().view(n * hq, d) @ k.t()) * s["scale"]
        x = x.view(n, hq, p + n)
        x[:, :, p:] = torch.where(anc[i][:, None], x[:, :, p:], -math.inf)
        e = torch.exp(x - x.amax(-1, keepdim=True))
        o = (e.view(n * hq, p + n) @ k[:, :lat]) / e.sum(-1).view(-1, 1)
        out[i] = o.view(n, hq, lat).to(out.dtype)
    return out


def _plain_prompt(s):
    out = torch.zeros_like(s["out"])
    q0 = k0 = 0
    for nq, nk in zip(s["new"], s["all"]):
        if nq:
            q = s["q"][q0:q0 + nq].float().transpose(0, 1)
            k = torch.cat([s["k"][k0:k0 + nk], s["k_rope"][k0:k0 + nk, None].expand(-1, q.shape[0], -1)], -1).float()
            x = (q @ k.permute(1, 2, 0)) * s["scale"]
            pos = torch.arange(nq, device=x.device)[:, None] + (nk - nq)
            x = torch.where(torch.arange(nk, device=x.device)[None] <= pos, x, -math.inf)
            e = torch.exp(x - x.amax(-1, keepdim=True))
            o = (e @ s["v"][k0:k0 + nk].float().transpose(0, 1)) / e.sum(-1, keepdim=True)
            out[q0:q0 + nq] = o.transpose(0, 1).to(out.dtype)
        q0, k0 = q0 + nq, k0 + nk
    return out


def _plain_slots(s):
    c = s["case"]
    new, page = s["new"].long(), c["page"]
    off = torch.cat([new.new_zeros(1), new.cumsum(0)])
    t = torch.arange(s["slots"].shape[0], device=new.device)
    seq = torch.searchsorted(off[1:].contiguous(), t, right=True)
    there = seq < new.shape[0]
    seq = torch.where(there, seq, 0)
    pos = s["prefix"].long()[seq] + t - off[seq]
    at = torch.where(there, pos // page, 0)
    blk = s["table"].long()[seq, at]
    slots = torch.where(there, blk * page + pos % page, -1)
    pos = torch.where(there, pos, -1)
    offsets, slots32, pos = off.int(), slots.int(), pos.int()
    if c["write"]:
        live = slots >= 0
        to = slots[live]
        s["pages"][to // page, :, to % page] = s["rows"][live]
        return offsets, slots32, pos, s["pages"]
    got = s["pages"][slots.clamp(min=0) // page, :, slots.clamp(min=0) % page]
    return offsets, slots32, pos, torch.where((slots >= 0)[:, None, None], got, 0)


# ------------------------------------------------------------------ the library's calls


def _own(s):
    from tree_speculative_decoding_attn_gb300 import specverify as sv
    c = s["case"]
    if c["op"] == "latent":
        more = dict(workspace=s["workspace"], dev_status=s["status"])
        if c["page"]:
            sv.tree_attn_verify_latent_paged(s["q"], s["cache"], s["table"], s["tree"], s["prefix"], s["anc"], s["out"],
                                             s["max_prefix"], s["scale"], **more)
        else:
            sv.tree_attn_verify_latent(s["q"], s["cache"], s["tree"], s["prefix"], s["anc"], s["out"], s["max_prefix"],
                                       s["scale"], **more)
        return s["out"]
    if c["op"] == "prompt":
        sv.prompt_attn_latent(s["q"], s["k"], s["k_rope"], s["v"], s["q_off"], s["kv_off"], s["out"], s["max_q"],
                              s["scale"], dev_status=s["status"])
        return s["out"]
    sv.kv_pages_slots(s["table"], s["prefix"], s["new"], s["offsets"], s["slots"], c["page"], s["pages"].shape[0],
                      positions=s["pos"], dev_status=s["status"])
    if c["write"]:
        sv.kv_slots_write(s["pages"], s["slots"], s["rows"], dev_status=s["status"])
        return s["offsets"], s["slots"], s["pos"], s["pages"]
    sv.kv_slots_read(s["pages"], s["slots"], s["rows"], dev_status=s["status"])
    return s["offsets"], s["slots"], s["pos"], s["rows"]


def run(state):
    if own:
        return _own(state)
    return {"latent": _plain_latent, "prompt": _plain_prompt, "slots": _plain_slots}[state["case"]["op"]](state)


# ------------------------------------------------------------------ work and exact values


def work(case):
    c = case
    if c["op"] == "latent":
        keys = sum(_spread(c["pmin"], c["pmax"], c["batch"])) + c["batch"] * c["nodes"]
        d, rows = c["latent"] + ROPE, c["nodes"] * c["hq"]
        return {"bytes": _size(c) * (keys * d + c["batch"] * rows * (d + c["latent"]))
                + 8 * c["batch"] * c["nodes"] * ((c["nodes"] + 63) // 64),
                "flops": 2 * rows * keys * (d + c["latent"])}
    if c["op"] == "prompt":
        new, all_ = _prompt_lengths(c)
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(new, all_))
        used = sum(m for n, m in zip(new, all_) if n)
        return {"bytes": 2 * (sum(new) * c["hq"] * (2 * HEAD + ROPE) + used * (c["hq"] * 2 * HEAD + ROPE)),
                "flops": 2 * pairs * c["hq"] * (2 * HEAD + ROPE)}
    total = sum(_spread(c["nmin"], c["nmax"], c["batch"]))
    pages = sum(-(-n // c["page"]) for n in _spread(c["nmin"], c["nmax"], c["batch"]))
    return {"bytes": 2 * total * c["hkv"] * c["dim"] * _size(c) + 8 * (total + c["spare"]) + 4 * pages + 12 * c["batch"],
            "flops": 4 * total}


def _exact_latent(c, s):
    """Every row of every sequence against all keys in 64 bits, a head at a time."""
    lat, out = c["latent"], torch.empty(s["out"].shape, dtype=torch.float64, device="cuda")
    words = s["anc"].cpu().numpy().view(np.uint64)
    for i, p in enumerate(s["lengths"]):
        if c["page"]:
            blocks = s["table"][i].tolist()[:-(-p // c["page"])]
            rows = torch.cat([s["cache"][x] for x in blocks])[:p] if p else s["tree"][i][:0]
        else:
            rows = s["cache"][i][:p]
        k = torch.cat([rows, s["tree"][i]]).double()
        ok = np.ones((c["nodes"], k.shape[0]), bool)
        for t in range(c["nodes"]):
            ok[:, p + t] = (words[i, :, t // 64] >> np.uint64(t % 64)) & np.uint64(1)
        hide = torch.from_numpy(~ok).cuda()
        for h in range(c["hq"]):
            x = torch.einsum("nd,jd->nj", s["q"][i, :, h].double(), k) * s["scale"]
            out[i, :, h] = torch.softmax(x.masked_fill(hide, -math.inf), -1) @ k[:, :lat]
    return out


def _exact_prompt(c, s):
    """One head of one sequence after another in 64 bits, the queries in pieces."""
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for nq, nk in zip(s["new"], s["all"]):
        for h in range(c["hq"]):
            kn, kr = s["k"][k0:k0 + nk, h].double(), s["k_rope"][k0:k0 + nk].double()
            v = s["v"][k0:k0 + nk, h].double()
            for lo in range(0, nq, 2048):
                hi = min(nq, lo + 2048)
                q = s["q"][q0 + lo:q0 + hi, h].double()
                end = nk - nq + hi                   # keys past the piece's last query are seen by none of it
                x = (q[:, :HEAD] @ kn[:end].T + q[:, HEAD:] @ kr[:end].T) * s["scale"]
                x.masked_fill_(torch.ones_like(x, dtype=torch.bool).triu_(nk - nq + lo + 1), -math.inf)
                out[q0 + lo:q0 + hi, h] = torch.softmax(x, -1) @ v[:end]
        q0, k0 = q0 + nq, k0 + nk
    return out


def exact(case, seed):
    if case["op"] == "slots":
        return None
    if work(case)["flops"] > 8e11:
        return None
    s = prepare(case, seed)
    return _exact_latent(case, s) if case["op"] == "latent" else _exact_prompt(case, s)
