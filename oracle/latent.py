"""Attention over latent rows and the places of packed tokens, plain numpy in float64."""
import numpy as np


def softmax_rows(x):
    """Softmax of the last axis; a row of -inf alone gives zeros."""
    m = x.max(-1, keepdims=True) if x.shape[-1] else np.zeros(x.shape[:-1] + (1,))
    m = np.where(np.isneginf(m), 0.0, m)
    e = np.exp(x - m)
    s = e.sum(-1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s != 0)


def tree_attention(q, cache, tree, prefix, mask, latent, scale):
    """q [B, N, H, D], cache [B, S, D] (rows past a prefix are not read), tree
    [B, N, D], mask [B, N, N]: out [B, N, H, latent] and, of the same shape,
    the mean size of what was summed (sum of p |c|) for error bounds."""
    B, N, H, _ = q.shape
    out, size = np.zeros((B, N, H, latent)), np.zeros((B, N, H, latent))
    for b in range(B):
        p = int(prefix[b])
        k = np.concatenate([cache[b, :p], tree[b]]).astype(np.float64)
        see = np.concatenate([np.ones((N, p), bool), mask[b]], 1)
        for h in range(H):
            x = np.where(see, q[b, :, h].astype(np.float64) @ k.T * scale, -np.inf)
            w = softmax_rows(x)
            out[b, :, h], size[b, :, h] = w @ k[:, :latent], w @ np.abs(k[:, :latent])
    return out, size


def prompt_attention(q, k, k_rope, v, q_off, kv_off, scale):
    """Packed causal attention: out [Tq, H, Dv] and the mean size of what was summed."""
    Tq, H, _ = q.shape
    D = k.shape[-1]
    out, size = np.zeros((Tq, H, v.shape[-1])), np.zeros((Tq, H, v.shape[-1]))
    for b in range(len(q_off) - 1):
        q0, q1, k0, k1 = q_off[b], q_off[b + 1], kv_off[b], kv_off[b + 1]
        n, m = q1 - q0, k1 - k0
        see = np.arange(m)[None] <= np.arange(n)[:, None] + (m - n)
        for h in range(H):
            qq = q[q0:q1, h].astype(np.float64)
            x = (qq[:, :D] @ k[k0:k1, h].astype(np.float64).T + qq[:, D:] @ k_rope[k0:k1].astype(np.float64).T) * scale
            w = softmax_rows(np.where(see, x, -np.inf))
            vv = v[k0:k1, h].astype(np.float64)
            out[q0:q1, h], size[q0:q1, h] = w @ vv, w @ np.abs(vv)
    return out, size


def slots(table, prefix, new, room, block_size, num_blocks):
    """offsets, slots, positions (int32) and the set of device errors."""
    B, mb = table.shape
    off, errors = [0], set()
    out, pos = np.full(room, -1, np.int32), np.full(room, -1, np.int32)
    t = 0
    for b in range(B):
        for i in range(max(0, int(new[b]))):
            if t >= room:
                errors.add("capacity")
                break
            p = int(prefix[b]) + i
            if prefix[b] < 0 or p >= mb * block_size:
                errors.add("capacity")
            else:
                pos[t] = p
                blk = int(table[b, p // block_size])
                if 0 <= blk < num_blocks:
                    out[t] = blk * block_size + p % block_size
                else:
                    errors.add("block")
            t += 1
        off.append(t)
    return np.asarray(off, np.int32), out, pos, errors
