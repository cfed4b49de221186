"""The serving operators refuse malformed arguments with a status before any
launch (host-side failure injection, no GPU; placeholder addresses are never
dereferenced, and the test is skipped where a GPU is visible)."""
import pytest
import torch

from tree_speculative_decoding_attn_gb300 import _build
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers only on a GPU-less host")

P, MIS, NULL = 0x100000, 0x100004, None
INV, UNS, CAP = sv.ERR_INVALID_ARG, sv.ERR_UNSUPPORTED, sv.ERR_CAPACITY


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load()


def _window(lib, q=P, k=P, depth=P, dtype=sv.F32, B=2, N=8, hq=16, hkv=2, D=128, s_max=1024, mp=512, w=100, s=4, ws=NULL,
            ws_bytes=0):
    return lib.tree_attn_verify_window(q, k, P, P, P, P, depth, P, P, dtype, B, N, hq, hkv, D, s_max, mp, w, s, 0.0, ws,
                                       ws_bytes, NULL, NULL)


def _paged(lib, table=P, bs=128, nb=64, mb=8, **kw):
    a = dict(dict(dtype=sv.F32, B=2, N=8, hq=16, hkv=2, D=128, mp=512, w=100, s=4), **kw)
    return lib.tree_attn_verify_window_paged(P, P, P, table, bs, nb, mb, P, P, P, P, P, P, a["dtype"], a["B"], a["N"],
                                             a["hq"], a["hkv"], a["D"], a["mp"], a["w"], a["s"], 0.0, NULL, 0, NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), INV), (dict(depth=NULL), INV), (dict(k=MIS), INV), (dict(w=0), INV), (dict(w=-5), INV), (dict(s=-1), INV),
    (dict(dtype=9), UNS), (dict(hq=15), INV), (dict(D=96), UNS), (dict(N=257), UNS), (dict(N=64, hq=128), UNS),
    (dict(N=65, hq=130, hkv=1), UNS), (dict(N=256, hq=1 << 24, hkv=1), UNS),
    (dict(B=0), INV), (dict(mp=2048), CAP), (dict(mp=-1), INV), (dict(B=1 << 15, hkv=4), UNS),
    (dict(B=1024, hkv=2, s_max=1 << 20), UNS),
    (dict(B=1, N=1, hq=2, mp=60000, s_max=60000, w=60000), CAP),         # splits need a workspace
    (dict(B=1, N=1, hq=2, mp=60000, s_max=60000, w=60000, ws=MIS, ws_bytes=1 << 30), CAP),
])
def test_window_refuses(lib, kw, code):
    assert _window(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(table=NULL), INV), (dict(bs=64), INV), (dict(bs=192), INV), (dict(nb=0), INV), (dict(mb=0), INV),
    (dict(mp=1025), CAP), (dict(nb=1 << 23), UNS), (dict(mb=1 << 24), UNS), (dict(w=0), INV), (dict(hkv=0), INV),
])
def test_paged_window_refuses(lib, kw, code):
    assert _paged(lib, **kw) == code


def test_window_workspace_is_zero_for_bad_shapes(lib):
    f = lib.tree_attn_window_workspace_bytes
    assert f(sv.F32, 2, 8, 15, 2, 128, 512, 100, 4) == 0 and f(sv.F32, 2, 8, 16, 2, 128, 512, 0, 4) == 0
    assert f(sv.F32, 1, 1, 2, 2, 128, 60000, 60000, 4) > 0


def test_short_window_calls_need_no_workspace(lib):
    f = lib.tree_attn_window_workspace_bytes
    assert f(sv.F32, 1, 5, 4, 4, 64, 1001, 333, 4) == 0
    assert f(sv.F32, 1, 5, 4, 4, 64, 60000, 5000, 4) > 0 and f(sv.BF16, 1, 1, 32, 8, 128, 60000, 1024, 4) == 0


def _verify(lib, p=P, q=NULL, dtype=sv.F32, B=2, N=8, V=100, u=P, cap=4):
    return lib.spec_verify_probs(p, q, dtype, B, N, V, P, P, P, P, u, P, cap, P, P, P, NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(p=NULL), INV), (dict(u=NULL), INV), (dict(p=MIS), INV), (dict(q=MIS), INV), (dict(dtype=3), UNS),
    (dict(B=0), INV), (dict(V=0), INV), (dict(cap=0), INV), (dict(N=257), UNS), (dict(cap=258), UNS), (dict(B=70000), UNS),
])
def test_verify_probs_refuses(lib, kw, code):
    assert _verify(lib, **kw) == code


FAR = 0x40000000


def test_pages_refuse(lib):
    fork = lambda table=P, B=2, out=2, mb=4, nb=16, ref=P + 4096, t2=FAR, p2=FAR + 4096, r2=FAR + 8192: lib.kv_pages_fork(  # noqa: E731
        table, P + 8192, P + 12288, B, out, mb, nb, ref, t2, p2, r2, NULL, NULL)
    for kw, code in ((dict(table=NULL), INV), (dict(B=0), INV), (dict(out=0), INV), (dict(mb=0), INV), (dict(nb=0), INV),
                     (dict(B=5000), UNS), (dict(out=5000), UNS), (dict(t2=P), INV), (dict(t2=P + 16), INV),
                     (dict(r2=P + 4100), INV), (dict(p2=P + 8192), INV), (dict(p2=P + 12288), INV)):
        assert fork(**kw) == code, kw
    free = lambda table=P, t2=FAR, bs=16, w=0, s=0, spare=0, r2=FAR + 8192, B=2: lib.kv_pages_free(  # noqa: E731
        table, P + 8192, B, 4, bs, 16, w, s, spare, P + 4096, t2, r2, NULL, NULL)
    for kw, code in ((dict(table=NULL), INV), (dict(bs=0), INV), (dict(w=-1), INV), (dict(s=-1), INV), (dict(spare=-1), INV),
                     (dict(t2=P + 4), INV), (dict(r2=P + 4092), INV), (dict(B=5000), UNS)):
        assert free(**kw) == code, kw
    size = lib.kv_pages_workspace_bytes(2, 4, 16)
    assert size > 0 and lib.kv_pages_workspace_bytes(0, 4, 16) == 0 and lib.kv_pages_workspace_bytes(5000, 4, 16) == 0

    def grow(k=P, v=P, e=2, L=1, hkv=2, D=64, bs=16, nb=16, B=2, mb=4, ws=P, n=size, t2=FAR, compact=False):
        if compact:
            return lib.kv_pages_compact(k, v, e, L, hkv, D, bs, nb, P, B, mb, P + 4096, t2, FAR + 8192, P, NULL, ws, n, NULL,
                                        NULL)
        return lib.kv_pages_reserve(k, v, e, L, hkv, D, bs, nb, P, B, mb, P + 8192, P, P + 4096, t2, FAR + 8192, ws, n, NULL,
                                    NULL)
    for compact in (False, True):
        for kw, code in ((dict(k=NULL), INV), (dict(v=MIS), INV), (dict(e=3), UNS), (dict(e=1), UNS), (dict(L=0), INV),
                         (dict(D=6), UNS), (dict(bs=0), INV), (dict(nb=0), INV), (dict(B=5000), UNS),
                         (dict(nb=1 << 26, bs=64), UNS), (dict(t2=P + 8), INV), (dict(ws=NULL), CAP), (dict(ws=MIS), CAP),
                         (dict(n=size - 1), CAP)):
            assert grow(compact=compact, **kw) == code, kw
