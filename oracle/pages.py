"""The life of a paged cache's blocks (oracle; test infrastructure only).

"5.3 Medusa、EAGLE 与 MTP" (infra-guide), section 8, closing remarks: a serving
engine keeps the KV cache in blocks addressed by block tables.  One entry at a
time, in order, with plain Python lists; tables hold -1 for "no block".
"""
from __future__ import annotations

import numpy as np


def fork(table, prefix_len, parent, ref):
    """Sequence i continues parent[i] (< 0: empty slot): new table, lengths, counts."""
    out = np.full((len(parent), table.shape[1]), -1, np.int32)
    lens, ref = np.zeros(len(parent), np.int32), ref.copy()
    for i, p in enumerate(parent):
        if p >= 0:
            out[i], lens[i] = table[p], prefix_len[p]
    for sign, t in ((-1, table), (1, out)):
        for blk in t.ravel():
            if blk >= 0:
                ref[blk] += sign
    return out, lens, ref


def free(table, prefix_len, ref, block_size, window=0, sinks=0, spare=0):
    """Drops the entries of pages without a position that is still needed."""
    out, ref = table.copy(), ref.copy()
    for b in range(table.shape[0]):
        P = int(prefix_len[b])
        for j in range(table.shape[1]):
            at = range(j * block_size, (j + 1) * block_size)
            # a page begun below P + spare, with a sink or a position that a node at P sees or that comes after it
            needed = at[0] < P + spare and (window <= 0 or any(x < sinks or P - x < window for x in at))
            if table[b, j] >= 0 and not needed:
                ref[table[b, j]] -= 1
                out[b, j] = -1
    return out, ref


def reserve(pools, table, prefix_len, need, ref, block_size):
    """Blocks for positions prefix_len .. + need - 1; a block that another
    entry still holds is replaced by a copy of its rows below prefix_len.
    Returns (pools, table, ref, fits); nothing changes where it does not fit."""
    out, cnt, new = table.copy(), ref.copy(), [p.copy() for p in pools]
    free_ids = [i for i in range(len(ref)) if ref[i] <= 0]
    for b in range(table.shape[0]):
        P, n = int(prefix_len[b]), int(need[b])
        if n <= 0 or P + n > table.shape[1] * block_size:
            continue
        for j in range(P // block_size, (P + n - 1) // block_size + 1):
            old = out[b, j]
            if old >= 0 and cnt[old] <= 1:
                continue
            if not free_ids:
                return [p.copy() for p in pools], table.copy(), ref.copy(), False
            blk = free_ids.pop(0)
            out[b, j] = blk
            cnt[blk] = 1
            if old >= 0:
                cnt[old] -= 1
                rows = max(0, min(block_size, P - j * block_size))
                for p in new:
                    p[:, blk, :, :rows] = p[:, old, :, :rows]
    return new, out, cnt, True


def compact(pools, table, ref):
    """Used blocks at or past their number go to the free ones below it, in order."""
    used = int((ref > 0).sum())
    src = [i for i in range(len(ref)) if ref[i] > 0 and i >= used]
    dst = [i for i in range(len(ref)) if ref[i] <= 0 and i < used]
    remap = np.where(ref > 0, np.arange(len(ref)), -1).astype(np.int32)
    new, cnt = [p.copy() for p in pools], np.maximum(ref, 0)
    for s, d in zip(src, dst):
        remap[s] = d
        cnt[d], cnt[s] = ref[s], 0
        for p in new:
            p[:, d] = p[:, s]
    out = np.where(table >= 0, remap[np.maximum(table, 0)], -1).astype(np.int32)
    return new, out, cnt, used, remap
