"""Python binding of libspecverify (the C ABI in ``include/specverify.h``).

Argument marshalling only: every function takes torch CUDA tensors (caller
owned), checks their dtype/device/contiguity, passes raw device pointers
and sizes to the C entry point of the same name on the current torch
stream, and raises ``SpecError`` on a non-zero status.  No step of the
method runs here.  There is no fallback: if the library is missing or a
tensor is not on a CUDA device, the call fails loudly.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libspecverify.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CAPACITY, ERR_CUDA = range(5)
(DEV_OK, DEV_BAD_PARENTS, DEV_CAPACITY, DEV_BAD_PATH, DEV_BAD_POOL, DEV_BAD_TOKEN, DEV_TIMEOUT, DEV_INTERNAL,
 DEV_BAD_BLOCK, DEV_BAD_PROB) = range(10)
F32, BF16 = 0, 1
GREEDY, TYPICAL, REJECT, REJECT_STOCHASTIC = 0, 1, 2, 3
MAX_NODES = 256
PAGES_MAX_BATCH = 4096


def mask_words(n_nodes):
    """uint64 words of one node's ancestor mask."""
    return (n_nodes + 63) // 64

_lib = None

_vp, _i, _f, _u64, _i64, _sz = C.c_void_p, C.c_int, C.c_float, C.c_uint64, C.c_int64, C.c_size_t
_SIGS = {
    "spec_status_string": ([_i], C.c_char_p),
    "spec_abi_version": ([], _i),
    "spec_medusa_heads_workspace_bytes": ([_i, _i, _i, _i], _sz),
    "spec_medusa_heads": ([_vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _sz, _vp, _vp], _i),
    "spec_topk": ([_vp, _i, _i, _i, _i, _i, _vp, _vp, _vp], _i),
    "spec_build_tree": ([_vp, _vp, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i),
    "spec_build_tree_dynamic": ([_vp, _vp, _vp, _i, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _vp], _i),
    "spec_build_tree_batch": ([_vp, _vp, _vp, _vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp], _i),
    "spec_tree_expand": ([_vp, _i, _i, _i, _i, _vp, _i, _f, _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp], _i),
    "spec_eagle_round_workspace_bytes": ([_i] * 10, _sz),
    "spec_eagle_round": ([_vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _f,
                          _vp, _vp, _vp, _vp, _vp, _i, _vp, _i, _vp, _vp, _sz, _vp, _vp], _i),
    "tree_attn_workspace_bytes": ([_i, _i, _i, _i, _i, _i, _i, _i], _sz),
    "tree_attn_plan_splits": ([_i, _i, _i, _i, _i, _i, _vp], _i),
    "tree_attn_verify": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f, _i,
                          _vp, _sz, _vp, _vp], _i),
    "tree_attn_verify_paged": ([_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                _i, _f, _i, _vp, _sz, _vp, _vp], _i),
    "tree_attn_window_workspace_bytes": ([_i] * 9, _sz),
    "tree_attn_verify_window": ([_vp] * 9 + [_i] * 10 + [_f, _vp, _sz, _vp, _vp], _i),
    "tree_attn_verify_window_paged": ([_vp] * 4 + [_i] * 3 + [_vp] * 6 + [_i] * 9 + [_f, _vp, _sz, _vp, _vp], _i),
    "tree_attn_verify_noalloc": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _i, _f,
                                  _i, _vp, _vp], _i),
    "spec_lm_head_workspace_bytes": ([_i, _i, _i], _sz),
    "spec_lm_head": ([_vp, _vp, _i, _i, _i, _vp, _vp, _sz, _vp, _vp], _i),
    "spec_lm_head_accept_workspace_bytes": ([_i, _i, _i, _i], _sz),
    "spec_lm_head_accept": ([_i, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _f, _f, _f, _i, _vp, _vp, _vp, _vp, _sz,
                             _vp, _vp], _i),
    "spec_accept": ([_i, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _f, _f, _f, _u64, _u64, _i, _vp, _vp,
                     _vp, _vp, _vp], _i),
    "spec_verify_probs": ([_vp, _vp] + [_i] * 4 + [_vp] * 6 + [_i] + [_vp] * 5, _i),
    "kv_pages_workspace_bytes": ([_i, _i, _i], _sz),
    "kv_pages_fork": ([_vp] * 3 + [_i] * 4 + [_vp] * 6, _i),
    "kv_pages_free": ([_vp] * 2 + [_i] * 7 + [_vp] * 5, _i),
    "kv_pages_reserve": ([_vp, _vp] + [_i] * 6 + [_vp, _i, _i] + [_vp] * 6 + [_sz, _vp, _vp], _i),
    "kv_pages_compact": ([_vp, _vp] + [_i] * 6 + [_vp, _i, _i] + [_vp] * 6 + [_sz, _vp, _vp], _i),
    "kv_commit_paged": ([_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _vp,
                         _vp], _i),
    "kv_commit": ([_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp, _vp, _vp], _i),
    "spec_accept_commit": ([_i, _vp, _vp, _i, _i, _i, _i, _vp, _vp, _vp, _vp, _f, _f, _f, _u64, _u64, _i, _vp, _vp,
                            _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp], _i),
    "tree_attn_latent_workspace_bytes": ([_i] * 7, _sz),
    "tree_attn_verify_latent": ([_vp] * 6 + [_i] * 8 + [_f, _vp, _sz, _vp, _vp], _i),
    "tree_attn_verify_latent_paged": ([_vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp] + [_i] * 7 +
                                      [_f, _vp, _sz, _vp, _vp], _i),
    "prompt_attn_latent_workspace_bytes": ([_i] * 7, _sz),
    "prompt_attn_latent": ([_vp, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp] + [_i] * 7 +
                           [_f, _vp, _sz, _vp, _vp], _i),
    "kv_pages_slots": ([_vp, _vp, _vp] + [_i] * 5 + [_vp] * 5, _i),
    "kv_slots_write": ([_vp, _vp, _vp] + [_i] * 6 + [_vp, _vp], _i),
    "kv_slots_read": ([_vp, _vp, _vp] + [_i] * 6 + [_vp, _vp], _i),
}


class SpecError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn}: status {code} ({spec_status_string(code)})")
        self.code = code


def load(path: str | None = None):
    """Load the shared library once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or os.environ.get("SPECVERIFY_LIB", LIB_PATH)
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = C.CDLL(p)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes, fn.restype = args, res
    _lib = lib
    return lib


def exported_symbols():
    return sorted(_SIGS)


# ---------------------------------------------------------------- helpers

_DT = {torch.float32: F32, torch.bfloat16: BF16}


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


def _device(t):
    """(index, stream) of a call by its first tensor: its device, which has to
    be the current one, and that device's current stream."""
    index = t.get_device()
    if index < 0 or index != torch._C._cuda_getDevice():
        raise ValueError(f"a tensor on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return index, torch._C._cuda_getCurrentRawStream(index)


def _ptr(t, index, dtype, shape):
    """Device pointer of a tensor once it is checked: on the call's device,
    contiguous, and of the dtype and shape the C entry point takes it for."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        raise ValueError(f"expected a CUDA tensor, not {type(t).__name__}") from None
    raise _refusal(t, index, dtype, shape)


def _sized(t, index, dtype, numel=None):
    """As _ptr, for a tensor of any shape (of numel elements, if given)."""
    if t.get_device() == index and t.is_contiguous() and t.dtype is dtype and numel in (None, t.numel()):
        return t.data_ptr()
    raise _refusal(t, index, dtype, (numel,))


def _word(t, index):
    """The optional device status word."""
    return None if t is None else _sized(t, index, torch.int32)


def _refusal(t, index, dtype, shape):
    if t.get_device() != index:
        return ValueError(f"expected a tensor on cuda:{index}, not {t.device}")
    if t.dtype is not dtype:
        return TypeError(f"dtype {t.dtype}, expected {dtype}")
    return ValueError(f"expected a contiguous tensor of shape {tuple(shape)}, not {tuple(t.shape)}")


def _want(t, *dtypes):
    if t is not None and t.dtype not in dtypes:
        raise TypeError(f"dtype {t.dtype} not in {dtypes}")
    return t


def _stream():
    # (torch.cuda.current_stream() builds a Stream object: 3 us a call)
    return C.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))


def _check(fn, code):
    if code != OK:
        raise SpecError(fn, code)


def spec_status_string(code: int) -> str:
    return load().spec_status_string(int(code)).decode()


def spec_abi_version() -> int:
    return int(load().spec_abi_version())


# ---------------------------------------------------------------- entry points


def spec_medusa_heads_workspace_bytes(batch, n_heads, hidden, vocab):
    return int(load().spec_medusa_heads_workspace_bytes(batch, n_heads, hidden, vocab))


def _scratch(nbytes, like):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=like.device)


def spec_medusa_heads(h, w1, b1, w2, z, logits, workspace=None, dev_status=None):
    """z (bf16) and logits (float32) of every head; ``workspace`` (uint8,
    at least spec_medusa_heads_workspace_bytes) is allocated per call when
    not given."""
    B, d = h.shape
    K, V = w2.shape[0], w2.shape[1]
    for t in (h, w1, w2, z):
        _want(t, torch.bfloat16)
    _want(b1, torch.bfloat16)
    _want(logits, torch.float32)
    if workspace is None:
        workspace = _scratch(spec_medusa_heads_workspace_bytes(B, K, d, V), h)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("spec_medusa_heads", load().spec_medusa_heads(_p(h), _p(w1), _p(b1), _p(w2), B, K, d, V, _p(z),
                                                         _p(logits), _p(workspace), ws_bytes, _p(dev_status),
                                                         _stream()))


def spec_topk(rows, s, idx_out, val_out=None, row_len=None):
    _want(rows, torch.float32, torch.bfloat16)
    _want(idx_out, torch.int32); _want(val_out, torch.float32)
    n_rows, stride = rows.reshape(-1, rows.shape[-1]).shape
    _check("spec_topk", load().spec_topk(_p(rows), _DT[rows.dtype], n_rows, row_len or stride, stride, s,
                                         _p(idx_out), _p(val_out), _stream()))


def spec_build_tree(parents, rank, cand_tok, root_tok, prefix_len, tok, depth, pos_ids, anc_mask,
                    first_child, next_sibling, dev_status=None):
    B, N = depth.shape
    levels = cand_tok.shape[1] if cand_tok is not None else 0
    s = cand_tok.shape[2] if cand_tok is not None else 0
    for t in (parents, rank, cand_tok, root_tok, prefix_len, tok, depth, pos_ids, first_child, next_sibling,
              dev_status):
        _want(t, torch.int32)
    _want(anc_mask, torch.int64)
    _check("spec_build_tree", load().spec_build_tree(
        _p(parents), _p(rank), _p(cand_tok), levels, s, _p(root_tok), _p(prefix_len), B, N, _p(tok),
        _p(depth), _p(pos_ids), _p(anc_mask), _p(first_child), _p(next_sibling), _p(dev_status), _stream()))


def spec_build_tree_batch(parents, prefix_len, depth, pos_ids, anc_mask, first_child, next_sibling, n_valid=None,
                          tok_in=None, tok=None, dev_status=None):
    """One tree per sequence: parents [B, N] (first n_valid[b] entries
    valid), tokens copied from tok_in when given."""
    B, N = parents.shape
    for t in (parents, n_valid, tok_in, tok, prefix_len, depth, pos_ids, first_child, next_sibling, dev_status):
        _want(t, torch.int32)
    _want(anc_mask, torch.int64)
    _check("spec_build_tree_batch", load().spec_build_tree_batch(
        _p(parents), _p(n_valid), _p(tok_in), _p(prefix_len), B, N, _p(tok), _p(depth), _p(pos_ids), _p(anc_mask),
        _p(first_child), _p(next_sibling), _p(dev_status), _stream()))


def spec_build_tree_dynamic(pool_parent, pool_tok, pool_conf, prefix_len, tok, parents_out, depth, pos_ids,
                            anc_mask, first_child, next_sibling, pool_index=None, val=None, dev_status=None):
    B, M = pool_parent.shape
    N = tok.shape[1]
    _want(pool_conf, torch.float32); _want(val, torch.float32); _want(anc_mask, torch.int64)
    _check("spec_build_tree_dynamic", load().spec_build_tree_dynamic(
        _p(pool_parent), _p(pool_tok), _p(pool_conf), M, _p(prefix_len), B, N, _p(tok), _p(parents_out),
        _p(depth), _p(pos_ids), _p(anc_mask), _p(first_child), _p(next_sibling), _p(pool_index), _p(val),
        _p(dev_status), _stream()))


def spec_tree_expand(draft_logits, frontier, k, temperature, pool_parent, pool_tok, pool_conf, pool_val,
                     pool_count, next_frontier, dev_status=None):
    B, F, V = draft_logits.shape
    _check("spec_tree_expand", load().spec_tree_expand(
        _p(draft_logits), _DT[draft_logits.dtype], B, F, V, _p(frontier), k, float(temperature),
        _p(pool_parent), _p(pool_tok), _p(pool_conf), _p(pool_val), _p(pool_count), pool_parent.shape[1],
        _p(next_frontier), next_frontier.shape[1], _p(dev_status), _stream()))


EAGLE_WEIGHTS = ("fc", "ln1", "qkv", "o", "ln2", "gate_up", "down", "lnf", "lm", "emb")


class _EagleWeights(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in EAGLE_WEIGHTS]


def spec_eagle_round_workspace_bytes(batch, n_front, hidden, hq, hkv, head_dim, ffn, vocab, s_max, max_prefix):
    return int(load().spec_eagle_round_workspace_bytes(batch, n_front, hidden, hq, hkv, head_dim, ffn, vocab, s_max,
                                                       max_prefix))


def spec_eagle_round(weights, k_prefix, v_prefix, prefix_len, max_prefix, k_nodes, v_nodes, feat, frontier, depth, k,
                     temperature, pool_parent, pool_tok, pool_conf, pool_val, pool_count, next_frontier,
                     draft_logits=None, workspace=None, dev_status=None):
    """One EAGLE drafting round; ``weights`` maps the names in EAGLE_WEIGHTS
    to bf16 tensors (layouts in the C header)."""
    B, _, d = feat.shape
    hkv, S, D = k_prefix.shape[1], k_prefix.shape[2], k_prefix.shape[3]
    hq = weights["o"].shape[1] // D
    ffn = weights["down"].shape[1]
    V = weights["lm"].shape[0]
    F = frontier.shape[1]
    for n in EAGLE_WEIGHTS:
        _want(weights[n], torch.bfloat16)
    for t in (k_prefix, v_prefix, k_nodes, v_nodes, feat):
        _want(t, torch.bfloat16)
    _want(draft_logits, torch.float32)
    w = _EagleWeights(*[_p(weights[n]).value for n in EAGLE_WEIGHTS])
    if workspace is None:
        workspace = _scratch(spec_eagle_round_workspace_bytes(B, F, d, hq, hkv, D, ffn, V, S, int(max_prefix)), feat)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("spec_eagle_round", load().spec_eagle_round(
        C.c_void_p(C.addressof(w)), B, d, hq, hkv, D, ffn, V, _p(k_prefix), _p(v_prefix), S, _p(prefix_len),
        int(max_prefix), _p(k_nodes), _p(v_nodes), _p(feat), _p(frontier), F, int(depth), int(k), float(temperature),
        _p(pool_parent), _p(pool_tok), _p(pool_conf), _p(pool_val), _p(pool_count), pool_parent.shape[1],
        _p(next_frontier), next_frontier.shape[1], _p(draft_logits), _p(workspace), ws_bytes, _p(dev_status),
        _stream()))


def tree_attn_workspace_bytes(dtype, batch, n_nodes, hq, hkv, head_dim, max_prefix, num_splits=0):
    code = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load().tree_attn_workspace_bytes(code, batch, n_nodes, hq, hkv, head_dim, max_prefix, num_splits))


def tree_attn_plan_splits(dtype, batch, n_nodes, hq, hkv, head_dim, host_prefix_len):
    """Split count for a batch whose prefix lengths the host knows (a
    sequence of ints); pass it as num_splits."""
    import numpy as np
    code = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    arr = np.ascontiguousarray(np.asarray(host_prefix_len, dtype=np.int32))
    n = int(load().tree_attn_plan_splits(code, batch, n_nodes, hq, hkv, head_dim,
                                         arr.ctypes.data_as(C.c_void_p)))
    if n <= 0:
        raise SpecError("tree_attn_plan_splits", ERR_INVALID_ARG)
    return n


def tree_attn_verify(q, k_cache, v_cache, k_tree, v_tree, prefix_len, anc_mask, out, max_prefix,
                     scale=0.0, num_splits=0, workspace=None, dev_status=None):
    B, N, Hq, D = q.shape
    Hkv, S = k_cache.shape[1], k_cache.shape[2]
    _want(q, torch.float32, torch.bfloat16)
    for t in (k_cache, v_cache, k_tree, v_tree, out):
        if t.dtype != q.dtype:
            raise TypeError("q, caches, tree K/V and out must share one dtype")
    _want(anc_mask, torch.int64); _want(prefix_len, torch.int32)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tree_attn_verify", load().tree_attn_verify(
        _p(q), _p(k_cache), _p(v_cache), _p(k_tree), _p(v_tree), _p(prefix_len), _p(anc_mask), _p(out),
        _DT[q.dtype], B, N, Hq, Hkv, D, S, int(max_prefix), float(scale), int(num_splits), _p(workspace),
        ws_bytes, _p(dev_status), _stream()))


def tree_attn_verify_paged(q, k_pages, v_pages, block_table, k_tree, v_tree, prefix_len, anc_mask, out, max_prefix,
                           scale=0.0, num_splits=0, workspace=None, dev_status=None):
    """tree_attn_verify over a paged prefix cache: k_pages/v_pages
    [num_blocks, Hkv, block_size, D], block_table [B, max_blocks] int32."""
    B, N, Hq, D = q.shape
    nb, Hkv, bs = k_pages.shape[0], k_pages.shape[1], k_pages.shape[2]
    _want(q, torch.float32, torch.bfloat16)
    for t in (k_pages, v_pages, k_tree, v_tree, out):
        if t.dtype != q.dtype:
            raise TypeError("q, pages, tree K/V and out must share one dtype")
    _want(anc_mask, torch.int64); _want(prefix_len, torch.int32); _want(block_table, torch.int32)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("tree_attn_verify_paged", load().tree_attn_verify_paged(
        _p(q), _p(k_pages), _p(v_pages), _p(block_table), bs, nb, block_table.shape[1], _p(k_tree), _p(v_tree),
        _p(prefix_len), _p(anc_mask), _p(out), _DT[q.dtype], B, N, Hq, Hkv, D, int(max_prefix), float(scale),
        int(num_splits), _p(workspace), ws_bytes, _p(dev_status), _stream()))


def tree_attn_window_workspace_bytes(dtype, batch, n_nodes, hq, hkv, head_dim, max_prefix, window, sinks=0):
    code = _DT[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load().tree_attn_window_workspace_bytes(code, batch, n_nodes, hq, hkv, head_dim, int(max_prefix),
                                                       int(window), int(sinks)))


def tree_attn_verify_window(q, k_cache, v_cache, k_tree, v_tree, prefix_len, depth, anc_mask, out, max_prefix, window,
                            sinks=0, scale=0.0, workspace=None, dev_status=None):
    """tree_attn_verify over the last ``window`` positions and the first
    ``sinks`` ones; depth [B, N] int32 gives the nodes' positions.
    ``workspace`` (uint8, tree_attn_window_workspace_bytes) is allocated per
    call when not given."""
    B, N, Hq, D = q.shape
    _, Hkv, S, _ = k_cache.shape
    code = _DT.get(q.dtype, -1)
    if workspace is None:
        workspace = _scratch(tree_attn_window_workspace_bytes(code, B, N, Hq, Hkv, D, max_prefix, window, sinks), q)
    i, stream = _device(q)
    dt, i32, kv, tree = q.dtype, torch.int32, (B, Hkv, S, D), (B, Hkv, N, D)
    args = (_ptr(q, i, dt, q.shape), _ptr(k_cache, i, dt, kv), _ptr(v_cache, i, dt, kv), _ptr(k_tree, i, dt, tree),
            _ptr(v_tree, i, dt, tree), _ptr(prefix_len, i, i32, (B,)), _ptr(depth, i, i32, (B, N)),
            _sized(anc_mask, i, torch.int64, B * N * mask_words(N)), _ptr(out, i, dt, q.shape))
    _check("tree_attn_verify_window", load().tree_attn_verify_window(
        *args, code, B, N, Hq, Hkv, D, S, int(max_prefix), int(window), int(sinks), float(scale),
        _sized(workspace, i, torch.uint8), workspace.numel(), _word(dev_status, i), stream))


def tree_attn_verify_window_paged(q, k_pages, v_pages, block_table, k_tree, v_tree, prefix_len, depth, anc_mask, out,
                                  max_prefix, window, sinks=0, scale=0.0, workspace=None, dev_status=None):
    """tree_attn_verify_window over a paged prefix cache: k_pages/v_pages
    [num_blocks, Hkv, block_size, D], block_table [B, max_blocks] int32."""
    B, N, Hq, D = q.shape
    nb, Hkv, bs, _ = k_pages.shape
    mb = block_table.shape[1]
    code = _DT.get(q.dtype, -1)
    if workspace is None:
        workspace = _scratch(tree_attn_window_workspace_bytes(code, B, N, Hq, Hkv, D, max_prefix, window, sinks), q)
    i, stream = _device(q)
    dt, i32, kv, tree = q.dtype, torch.int32, (nb, Hkv, bs, D), (B, Hkv, N, D)
    args = (_ptr(q, i, dt, q.shape), _ptr(k_pages, i, dt, kv), _ptr(v_pages, i, dt, kv),
            _ptr(block_table, i, i32, (B, mb)), bs, nb, mb, _ptr(k_tree, i, dt, tree), _ptr(v_tree, i, dt, tree),
            _ptr(prefix_len, i, i32, (B,)), _ptr(depth, i, i32, (B, N)),
            _sized(anc_mask, i, torch.int64, B * N * mask_words(N)), _ptr(out, i, dt, q.shape))
    _check("tree_attn_verify_window_paged", load().tree_attn_verify_window_paged(
        *args, code, B, N, Hq, Hkv, D, int(max_prefix), int(window), int(sinks), float(scale),
        _sized(workspace, i, torch.uint8), workspace.numel(), _word(dev_status, i), stream))


NOALLOC_SCRATCH_BYTES = 32 << 20


def tree_attn_verify_noalloc(q, k_cache, v_cache, k_tree, v_tree, prefix_len, anc_mask, out, max_prefix,
                             scale=0.0, num_splits=0, dev_status=None):
    """tree_attn_verify for callers that cannot allocate: the split-KV
    partials live in the library's own fixed device array (32 MiB, shared by
    every call; calls that overlap on the GPU race on it)."""
    B, N, Hq, D = q.shape
    Hkv, S = k_cache.shape[1], k_cache.shape[2]
    _want(q, torch.float32, torch.bfloat16)
    for t in (k_cache, v_cache, k_tree, v_tree, out):
        if t.dtype != q.dtype:
            raise TypeError("q, caches, tree K/V and out must share one dtype")
    _want(anc_mask, torch.int64); _want(prefix_len, torch.int32)
    _check("tree_attn_verify_noalloc", load().tree_attn_verify_noalloc(
        _p(q), _p(k_cache), _p(v_cache), _p(k_tree), _p(v_tree), _p(prefix_len), _p(anc_mask), _p(out),
        _DT[q.dtype], B, N, Hq, Hkv, D, S, int(max_prefix), float(scale), int(num_splits), _p(dev_status),
        _stream()))


def spec_lm_head_workspace_bytes(rows, hidden, vocab):
    return int(load().spec_lm_head_workspace_bytes(rows, hidden, vocab))


def spec_lm_head(hid, w, logits, dev_status=None, workspace=None):
    R, d = hid.shape
    V = w.shape[0]
    _want(hid, torch.bfloat16); _want(w, torch.bfloat16); _want(logits, torch.float32)
    if workspace is None:
        workspace = _scratch(spec_lm_head_workspace_bytes(R, d, V), hid)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("spec_lm_head", load().spec_lm_head(_p(hid), _p(w), R, d, V, _p(logits), _p(workspace), ws_bytes,
                                               _p(dev_status), _stream()))


def spec_lm_head_accept_workspace_bytes(batch, n_nodes, hidden, vocab):
    return int(load().spec_lm_head_accept_workspace_bytes(batch, n_nodes, hidden, vocab))


def spec_lm_head_accept(mode, hid, w, tok, parents, first_child, next_sibling, acc_len, acc_path, bonus,
                        temperature=1.0, eps=0.0, delta=0.0, dev_status=None, workspace=None):
    """LM head fused with greedy / typical acceptance.  hid [B, N, hidden]
    bf16, w [V, hidden] bf16; outputs as spec_accept."""
    B, N, d = hid.shape
    V = w.shape[0]
    _want(hid, torch.bfloat16); _want(w, torch.bfloat16)
    if workspace is None:
        workspace = _scratch(spec_lm_head_accept_workspace_bytes(B, N, d, V), hid)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("spec_lm_head_accept", load().spec_lm_head_accept(
        int(mode), _p(hid), _p(w), B, N, d, V, _p(tok), _p(parents), _p(first_child), _p(next_sibling),
        float(temperature), float(eps), float(delta), acc_path.shape[1], _p(acc_len), _p(acc_path), _p(bonus),
        _p(workspace), ws_bytes, _p(dev_status), _stream()))


def spec_accept(mode, logits, tok, parents, first_child, next_sibling, acc_len, acc_path, bonus,
                temperature=1.0, eps=0.0, delta=0.0, seed=0, step=0, dev_status=None, draft_logits=None):
    B, N, V = logits.shape
    _want(logits, torch.float32, torch.bfloat16)
    if draft_logits is not None and (draft_logits.dtype != logits.dtype or draft_logits.shape != logits.shape):
        raise TypeError("draft_logits must match logits in dtype and shape")
    _check("spec_accept", load().spec_accept(
        int(mode), _p(logits), _p(draft_logits), _DT[logits.dtype], B, N, V, _p(tok), _p(parents), _p(first_child),
        _p(next_sibling), float(temperature), float(eps), float(delta), int(seed), int(step),
        acc_path.shape[1], _p(acc_len), _p(acc_path), _p(bonus), _p(dev_status), _stream()))


def spec_accept_commit(mode, logits, tok, parents, first_child, next_sibling, acc_len, acc_path, bonus, k_cache,
                       v_cache, k_tree, v_tree, prefix_len, prefix_len_out=None, temperature=1.0, eps=0.0,
                       delta=0.0, seed=0, step=0, dev_status=None, draft_logits=None):
    """spec_accept and kv_commit (contiguous cache) in one launch."""
    B, N, V = logits.shape
    _want(logits, torch.float32, torch.bfloat16)
    if draft_logits is not None and (draft_logits.dtype != logits.dtype or draft_logits.shape != logits.shape):
        raise TypeError("draft_logits must match logits in dtype and shape")
    if k_cache.dim() == 4:
        L, (_, Hkv, S, D) = 1, k_cache.shape
    else:
        L, _, Hkv, S, D = k_cache.shape
    _check("spec_accept_commit", load().spec_accept_commit(
        int(mode), _p(logits), _p(draft_logits), _DT[logits.dtype], B, N, V, _p(tok), _p(parents), _p(first_child),
        _p(next_sibling), float(temperature), float(eps), float(delta), int(seed), int(step), acc_path.shape[1],
        _p(acc_len), _p(acc_path), _p(bonus), _p(k_cache), _p(v_cache), _p(k_tree), _p(v_tree),
        k_cache.element_size(), L, Hkv, S, D, _p(prefix_len), _p(prefix_len_out), _p(dev_status), _stream()))


def kv_commit(k_cache, v_cache, k_tree, v_tree, acc_len, acc_path, prefix_len, prefix_len_out=None,
              dev_status=None):
    if k_cache.dim() == 4:
        L, (B, Hkv, S, D) = 1, k_cache.shape
    else:
        L, B, Hkv, S, D = k_cache.shape
    N = k_tree.shape[-2]
    _check("kv_commit", load().kv_commit(
        _p(k_cache), _p(v_cache), _p(k_tree), _p(v_tree), k_cache.element_size(), L, B, Hkv, S, N, D,
        _p(acc_len), _p(acc_path), acc_path.shape[1], _p(prefix_len), _p(prefix_len_out), _p(dev_status),
        _stream()))


def kv_commit_paged(k_pages, v_pages, block_table, k_tree, v_tree, acc_len, acc_path, prefix_len,
                    prefix_len_out=None, dev_status=None):
    """kv_commit into a paged cache [L, num_blocks, Hkv, block_size, D] (or
    without the layer axis) addressed by block_table [B, max_blocks]."""
    if k_pages.dim() == 4:
        L, (nb, Hkv, bs, D) = 1, k_pages.shape
    else:
        L, nb, Hkv, bs, D = k_pages.shape
    B, N = block_table.shape[0], k_tree.shape[-2]
    _want(block_table, torch.int32)
    _check("kv_commit_paged", load().kv_commit_paged(
        _p(k_pages), _p(v_pages), _p(block_table), bs, nb, block_table.shape[1], _p(k_tree), _p(v_tree),
        k_pages.element_size(), L, B, Hkv, N, D, _p(acc_len), _p(acc_path), acc_path.shape[1], _p(prefix_len),
        _p(prefix_len_out), _p(dev_status), _stream()))


def spec_verify_probs(target_probs, tok, parents, first_child, next_sibling, u_accept, u_bonus, acc_len, acc_path,
                      bonus, draft_probs=None, dev_status=None):
    """Acceptance from given probabilities [B, N, V] (float32 or bf16) and
    given uniform numbers u_accept [B, N], u_bonus [B] (float32); draft_probs
    where siblings are draws of the drafter.  Outputs as spec_accept."""
    B, N, V = target_probs.shape
    dt, i32, f32 = target_probs.dtype, torch.int32, torch.float32
    i, stream = _device(target_probs)
    node, cap = (B, N), acc_path.shape[1]
    _check("spec_verify_probs", load().spec_verify_probs(
        _ptr(target_probs, i, dt, (B, N, V)), None if draft_probs is None else _ptr(draft_probs, i, dt, (B, N, V)),
        _DT.get(dt, -1), B, N, V, _ptr(tok, i, i32, node), _ptr(parents, i, i32, node), _ptr(first_child, i, i32, node),
        _ptr(next_sibling, i, i32, node), _ptr(u_accept, i, f32, node), _ptr(u_bonus, i, f32, (B,)), cap,
        _ptr(acc_len, i, i32, (B,)), _ptr(acc_path, i, i32, (B, cap)), _ptr(bonus, i, i32, (B,)),
        _word(dev_status, i), stream))


def kv_pages_workspace_bytes(batch, max_blocks, num_blocks):
    return int(load().kv_pages_workspace_bytes(batch, max_blocks, num_blocks))


def kv_pages_fork(block_table, prefix_len, parent, ref_count, table_out, prefix_len_out, ref_out, dev_status=None):
    """Sequence i of the new batch continues sequence parent[i] (< 0: empty)."""
    B, mb = block_table.shape
    out, nb, i32 = parent.shape[0], ref_count.shape[0], torch.int32
    i, stream = _device(block_table)
    _check("kv_pages_fork", load().kv_pages_fork(
        _ptr(block_table, i, i32, (B, mb)), _ptr(prefix_len, i, i32, (B,)), _ptr(parent, i, i32, (out,)), B, out,
        mb, nb, _ptr(ref_count, i, i32, (nb,)), _ptr(table_out, i, i32, (out, mb)),
        _ptr(prefix_len_out, i, i32, (out,)), _ptr(ref_out, i, i32, (nb,)), _word(dev_status, i), stream))


def kv_pages_free(block_table, prefix_len, ref_count, table_out, ref_out, block_size, window=0, sinks=0, spare=0,
                  dev_status=None):
    """Drops the entries whose pages no later step needs (window 0: none has left)."""
    B, mb = block_table.shape
    nb, i32 = ref_count.shape[0], torch.int32
    i, stream = _device(block_table)
    _check("kv_pages_free", load().kv_pages_free(
        _ptr(block_table, i, i32, (B, mb)), _ptr(prefix_len, i, i32, (B,)), B, mb, int(block_size), nb, int(window),
        int(sinks), int(spare), _ptr(ref_count, i, i32, (nb,)), _ptr(table_out, i, i32, (B, mb)),
        _ptr(ref_out, i, i32, (nb,)), _word(dev_status, i), stream))


def _pool(i, k_pages, v_pages):
    """(K, V, element bytes, layers, KV heads, head_dim, block size, blocks)
    of a pool with or without the layer axis."""
    L, (nb, Hkv, bs, D) = (1, k_pages.shape) if k_pages.dim() == 4 else (k_pages.shape[0], k_pages.shape[1:])
    dt, shape = k_pages.dtype, k_pages.shape
    v = None if v_pages is None else _ptr(v_pages, i, dt, shape)    # None: a cache of one pool
    return _ptr(k_pages, i, dt, shape), v, k_pages.element_size(), L, Hkv, D, bs, nb


def kv_pages_reserve(k_pages, v_pages, block_table, prefix_len, need, ref_count, table_out, ref_out, workspace=None,
                     dev_status=None):
    """Makes the next need[b] rows of every sequence writable (new blocks,
    copies of shared ones).  ``workspace`` (uint8, kv_pages_workspace_bytes)
    is allocated per call when not given."""
    B, mb = block_table.shape
    i32 = torch.int32
    i, stream = _device(block_table)
    pool = _pool(i, k_pages, v_pages)
    nb = pool[-1]
    if workspace is None:
        workspace = _scratch(kv_pages_workspace_bytes(B, mb, nb), block_table)
    _check("kv_pages_reserve", load().kv_pages_reserve(
        *pool, _ptr(block_table, i, i32, (B, mb)), B, mb, _ptr(prefix_len, i, i32, (B,)), _ptr(need, i, i32, (B,)),
        _ptr(ref_count, i, i32, (nb,)), _ptr(table_out, i, i32, (B, mb)), _ptr(ref_out, i, i32, (nb,)),
        _sized(workspace, i, torch.uint8), workspace.numel(), _word(dev_status, i), stream))


def kv_pages_compact(k_pages, v_pages, block_table, ref_count, table_out, ref_out, n_used, remap=None, workspace=None,
                     dev_status=None):
    """Packs the used blocks into the pool's low end; n_used [1] int32 and
    remap [num_blocks] int32 (optional) are outputs."""
    B, mb = block_table.shape
    i32 = torch.int32
    i, stream = _device(block_table)
    pool = _pool(i, k_pages, v_pages)
    nb = pool[-1]
    if workspace is None:
        workspace = _scratch(kv_pages_workspace_bytes(B, mb, nb), block_table)
    _check("kv_pages_compact", load().kv_pages_compact(
        *pool, _ptr(block_table, i, i32, (B, mb)), B, mb, _ptr(ref_count, i, i32, (nb,)),
        _ptr(table_out, i, i32, (B, mb)), _ptr(ref_out, i, i32, (nb,)), _ptr(n_used, i, i32, (1,)),
        None if remap is None else _ptr(remap, i, i32, (nb,)),
        _sized(workspace, i, torch.uint8), workspace.numel(), _word(dev_status, i), stream))


def kv_pages_slots(block_table, prefix_len, new_len, offsets, slots, block_size, num_blocks, positions=None,
                   dev_status=None):
    """Rows of the pool where the next new_len[b] tokens of every sequence,
    packed one sequence behind the other, lie: offsets [B + 1], slots [room]
    and positions [room] (optional), all int32; -1 behind the last token."""
    B, mb = block_table.shape
    i32, room, each = torch.int32, slots.numel(), (B,)
    i, stream = _device(block_table)
    code = load().kv_pages_slots(
        _ptr(block_table, i, i32, (B, mb)), _ptr(prefix_len, i, i32, each), _ptr(new_len, i, i32, each), B, mb, block_size,
        num_blocks, room, _ptr(offsets, i, i32, (B + 1,)), _ptr(slots, i, i32, (room,)),
        None if positions is None else _ptr(positions, i, i32, (room,)), _word(dev_status, i), stream)
    if code != OK:
        raise SpecError("kv_pages_slots", code)


def _slot_rows(name, call, pages, slots, rows, dev_status):
    shape, T, dt = pages.shape, slots.numel(), pages.dtype
    nb, Hkv, bs, D = shape
    i, stream = _device(pages)
    code = call(_ptr(pages, i, dt, shape), _ptr(slots, i, torch.int32, (T,)), _ptr(rows, i, dt, (T, Hkv, D)),
                pages.element_size(), T, Hkv, D, bs, nb, _word(dev_status, i), stream)
    if code != OK:
        raise SpecError(name, code)


def kv_slots_write(pages, slots, rows, dev_status=None):
    """rows [T, Hkv, D] into their slots of one pool [num_blocks, Hkv,
    block_size, D]; negative slots are left out."""
    _slot_rows("kv_slots_write", load().kv_slots_write, pages, slots, rows, dev_status)


def kv_slots_read(pages, slots, rows, dev_status=None):
    """rows [T, Hkv, D] out of their slots; zeros where a slot is negative."""
    _slot_rows("kv_slots_read", load().kv_slots_read, pages, slots, rows, dev_status)


ROPE_DIM = 64    # rotary elements at the end of a latent row


def tree_attn_latent_workspace_bytes(dtype, batch, n_nodes, hq, latent_dim, rope_dim, max_prefix):
    code = _DT.get(dtype, -1) if isinstance(dtype, torch.dtype) else int(dtype)     # (0 bytes for other types, as in C)
    return int(load().tree_attn_latent_workspace_bytes(code, batch, n_nodes, hq, latent_dim, rope_dim, max_prefix))


def tree_attn_verify_latent(q, cache, tree, prefix_len, anc_mask, out, max_prefix, scale, workspace=None,
                            dev_status=None):
    """Tree attention over a cache of latent rows: q [B, N, Hq, latent + 64],
    cache [B, s_max, latent + 64], tree [B, N, latent + 64], out [B, N, Hq,
    latent] (float32 or bf16, latent 256 or 512).  ``workspace`` (uint8,
    tree_attn_latent_workspace_bytes) is allocated per call when not given."""
    (B, N, Hq, D), (_, S, _) = q.shape, cache.shape
    dt, i32, lat = q.dtype, torch.int32, D - ROPE_DIM
    i, stream = _device(q)
    if workspace is None:
        workspace = _scratch(tree_attn_latent_workspace_bytes(dt, B, N, Hq, lat, ROPE_DIM, max_prefix), q)
    code = load().tree_attn_verify_latent(
        _ptr(q, i, dt, (B, N, Hq, D)), _ptr(cache, i, dt, (B, S, D)), _ptr(tree, i, dt, (B, N, D)),
        _ptr(prefix_len, i, i32, (B,)), _sized(anc_mask, i, torch.int64, B * N * ((N + 63) // 64)),
        _ptr(out, i, dt, (B, N, Hq, lat)), _DT.get(dt, -1), B, N, Hq, lat, ROPE_DIM, S, max_prefix, scale,
        _sized(workspace, i, torch.uint8), workspace.numel(), _word(dev_status, i), stream)
    if code != OK:
        raise SpecError("tree_attn_verify_latent", code)


def tree_attn_verify_latent_paged(q, pages, block_table, tree, prefix_len, anc_mask, out, max_prefix, scale,
                                  workspace=None, dev_status=None):
    """tree_attn_verify_latent over pages [num_blocks, block_size, latent + 64]
    addressed by block_table [B, max_blocks]."""
    (B, N, Hq, D), (nb, bs, _), (_, mb) = q.shape, pages.shape, block_table.shape
    dt, i32, lat = q.dtype, torch.int32, D - ROPE_DIM
    i, stream = _device(q)
    if workspace is None:
        workspace = _scratch(tree_attn_latent_workspace_bytes(dt, B, N, Hq, lat, ROPE_DIM, max_prefix), q)
    code = load().tree_attn_verify_latent_paged(
        _ptr(q, i, dt, (B, N, Hq, D)), _ptr(pages, i, dt, (nb, bs, D)), _ptr(block_table, i, i32, (B, mb)), bs, nb, mb,
        _ptr(tree, i, dt, (B, N, D)), _ptr(prefix_len, i, i32, (B,)),
        _sized(anc_mask, i, torch.int64, B * N * ((N + 63) // 64)), _ptr(out, i, dt, (B, N, Hq, lat)), _DT.get(dt, -1),
        B, N, Hq, lat, ROPE_DIM, max_prefix, scale, _sized(workspace, i, torch.uint8), workspace.numel(),
        _word(dev_status, i), stream)
    if code != OK:
        raise SpecError("tree_attn_verify_latent_paged", code)


def _strided(t, index, dtype, shape):
    """Pointer of a tensor whose last dim alone has to be contiguous (a column range of a wider one)."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and (t.stride(-1) == 1 or t.shape[-1] == 1):
        return t.data_ptr()
    raise _refusal(t, index, dtype, shape)


def _step(t, d, least):
    """Elements between neighbours along dim d (any number where there is one)."""
    return t.stride(d) if t.shape[d] > 1 else least


def prompt_attn_latent_workspace_bytes(batch, hq, head_dim, rope_dim, total_q, total_kv, max_q):
    return int(load().prompt_attn_latent_workspace_bytes(batch, hq, head_dim, rope_dim, total_q, total_kv, max_q))


def prompt_attn_latent(q, k, k_rope, v, q_offsets, kv_offsets, out, max_q, scale, workspace=None, dev_status=None):
    """Causal attention of packed prompt tokens: q [Tq, Hq, 192], k and v [Tk,
    Hq, 128], k_rope [Tk, 64] (bf16; k, v and k_rope may be column ranges of
    wider tensors), offsets [B + 1] int32, out [Tq, Hq, 128].  ``workspace``
    (uint8, prompt_attn_latent_workspace_bytes) is allocated per call when not
    given."""
    (Tq, Hq, _), (Tk, _, D) = q.shape, k.shape
    bf, i32, B = torch.bfloat16, torch.int32, q_offsets.shape[0] - 1
    i, stream = _device(q)
    kv = (Tk, Hq, D)
    args = (_ptr(q, i, bf, (Tq, Hq, D + ROPE_DIM)), _strided(k, i, bf, kv), _step(k, 0, Hq * D), _step(k, 1, D),
            _strided(k_rope, i, bf, (Tk, ROPE_DIM)), _step(k_rope, 0, ROPE_DIM), _strided(v, i, bf, kv),
            _step(v, 0, Hq * D), _step(v, 1, D), _ptr(q_offsets, i, i32, (B + 1,)), _ptr(kv_offsets, i, i32, (B + 1,)),
            _ptr(out, i, bf, (Tq, Hq, D)), B, Hq, D, ROPE_DIM, Tq, Tk, max_q, scale)
    status, call = _word(dev_status, i), load().prompt_attn_latent
    if workspace is not None:
        code = call(*args, _sized(workspace, i, torch.uint8), workspace.numel(), status, stream)
    else:
        # most calls need none: the size is asked for only where the call refuses to do without
        code = call(*args, None, 0, status, stream)
        if code == ERR_CAPACITY:
            workspace = _scratch(prompt_attn_latent_workspace_bytes(B, Hq, D, ROPE_DIM, Tq, Tk, max_q), q)
            code = call(*args, workspace.data_ptr(), workspace.numel(), status, stream)
    if code != OK:
        raise SpecError("prompt_attn_latent", code)
