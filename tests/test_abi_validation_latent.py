"""The operators of a latent cache refuse malformed arguments with a status
before any launch (host-side failure injection, no GPU; placeholder addresses
are never dereferenced, and the test is skipped where a GPU is visible)."""
import math

import pytest
import torch

from tree_speculative_decoding_attn_gb300 import _build
from tree_speculative_decoding_attn_gb300 import specverify as sv

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers only on a GPU-less host")

P, MIS, NULL, FAR = 0x100000, 0x100004, None, 0x40000000
INV, UNS, CAP = sv.ERR_INVALID_ARG, sv.ERR_UNSUPPORTED, sv.ERR_CAPACITY


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load()


def _latent(lib, q=P, cache=P, tree=P, prefix=P, anc=P, out=P, dtype=sv.BF16, B=2, N=8, H=16, lat=512, rope=64, s_max=1024,
            mp=512, scale=0.1, ws=P, n=1 << 40):
    return lib.tree_attn_verify_latent(q, cache, tree, prefix, anc, out, dtype, B, N, H, lat, rope, s_max, mp, scale, ws, n,
                                       NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), INV), (dict(cache=NULL), INV), (dict(tree=NULL), INV), (dict(prefix=NULL), INV), (dict(anc=NULL), INV),
    (dict(out=NULL), INV), (dict(q=MIS), INV), (dict(cache=MIS), INV), (dict(tree=MIS), INV), (dict(out=MIS), INV),
    (dict(dtype=2), UNS), (dict(B=0), INV), (dict(N=0), INV), (dict(H=0), INV), (dict(mp=-1), INV), (dict(s_max=-1), INV),
    (dict(N=257), UNS), (dict(H=129), UNS), (dict(lat=128), UNS), (dict(lat=576), UNS), (dict(rope=32), UNS),
    (dict(B=65536), UNS), (dict(B=65535, N=256, H=128), UNS), (dict(B=2048, s_max=1 << 20), UNS), (dict(mp=1025), CAP),
    (dict(s_max=2 ** 31 - 1, mp=2 ** 31 - 1, B=1), UNS), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(ws=NULL), CAP), (dict(ws=MIS), CAP), (dict(n=1000), CAP),
    (dict(dtype=sv.F32, ws=NULL), CAP), (dict(N=1, ws=NULL), CAP),
])
def test_latent_refuses(lib, kw, code):
    assert _latent(lib, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(table=NULL), INV), (dict(bs=64), INV), (dict(bs=192), INV), (dict(bs=0), INV), (dict(nb=0), INV), (dict(mb=0), INV),
    (dict(mp=1025), CAP), (dict(nb=1 << 24), UNS), (dict(mb=1 << 24), UNS), (dict(nb=2 ** 31 - 1, bs=2 ** 31 - 128), UNS),
    (dict(lat=64), UNS), (dict(scale=0.0), INV),
])
def test_paged_latent_refuses(lib, kw, code):
    a = dict(dict(table=P, bs=128, nb=64, mb=8, mp=512, lat=512, scale=0.1), **kw)
    assert lib.tree_attn_verify_latent_paged(P, P, a["table"], a["bs"], a["nb"], a["mb"], P, P, P, P, sv.BF16, 2, 8, 16, a["lat"],
                                             64, a["mp"], a["scale"], P, 1 << 40, NULL, NULL) == code


def test_latent_workspace_sizes(lib):
    f = lib.tree_attn_latent_workspace_bytes
    for bad in ((3, 2, 8, 16, 512, 64, 100), (sv.BF16, 0, 8, 16, 512, 64, 100), (sv.BF16, 2, 257, 16, 512, 64, 100),
                (sv.BF16, 2, 8, 16, 500, 64, 100), (sv.BF16, 2, 8, 16, 512, 63, 100), (sv.BF16, 2, 8, 16, 512, 64, -1),
                (sv.BF16, 65535, 256, 128, 512, 64, 100), (sv.F32, 1 << 30, 256, 128, 512, 64, 2 ** 31 - 1)):
        assert f(*bad) == 0
    assert f(sv.BF16, 2, 8, 16, 512, 64, 100) > 0 and f(sv.BF16, 1, 1, 16, 512, 64, 5000) > 0
    assert f(sv.F32, 1, 1, 1, 256, 64, 10) == 0
    # bounded whatever the batch: parts of the GPU, not of the work
    assert f(sv.BF16, 65535, 1, 16, 512, 64, 1 << 20) == f(sv.BF16, 200, 1, 16, 512, 64, 1 << 20) < 1 << 25


def _prompt(lib, q=P, k=P, kt=256, kh=128, r=P, rt=576, v=P, vt=256, vh=128, qo=P, ko=P, out=P, B=2, H=4, D=128, R=64, tq=10,
            tk=20, mq=8, scale=0.1, ws=P, n=1 << 40):
    return lib.prompt_attn_latent(q, k, kt, kh, r, rt, v, vt, vh, qo, ko, out, B, H, D, R, tq, tk, mq, scale, ws, n, NULL, NULL)


@pytest.mark.parametrize("kw,code", [
    (dict(q=NULL), INV), (dict(k=NULL), INV), (dict(r=NULL), INV), (dict(v=NULL), INV), (dict(qo=NULL), INV), (dict(ko=NULL), INV),
    (dict(out=NULL), INV), (dict(q=MIS), INV), (dict(k=MIS), INV), (dict(r=MIS), INV), (dict(v=MIS), INV), (dict(out=MIS), INV),
    (dict(kt=120), INV), (dict(kt=0), INV), (dict(kt=-256), INV), (dict(kh=132), INV), (dict(rt=60), INV), (dict(rt=68), INV),
    (dict(vt=1 << 40), INV), (dict(vh=4), INV), (dict(B=0), INV), (dict(H=0), INV), (dict(tq=0), INV), (dict(tk=0), INV),
    (dict(mq=-1), INV), (dict(D=64), UNS), (dict(R=32), UNS), (dict(B=65536), UNS), (dict(H=65536), UNS),
    (dict(H=4, tq=1 << 29), UNS), (dict(tk=(1 << 30) + 1), UNS), (dict(H=1, tq=1 << 24, mq=1 << 24), UNS), (dict(scale=0.0), INV),
    (dict(scale=math.nan), INV), (dict(tk=5000, ws=NULL), CAP), (dict(tk=5000, ws=MIS), CAP), (dict(tk=5000, n=16), CAP),
])
def test_prompt_refuses(lib, kw, code):
    assert _prompt(lib, **kw) == code


def test_prompt_workspace_sizes(lib):
    f = lib.prompt_attn_latent_workspace_bytes
    assert f(1, 32, 128, 64, 8192, 8192, 8192) == 0 and f(8, 16, 128, 64, 1000, 1000, 300) == 0
    assert 0 < f(1, 16, 128, 64, 256, 16384, 256) < 1 << 25
    assert f(1, 16, 64, 64, 256, 16384, 256) == 0 and f(0, 16, 128, 64, 256, 16384, 256) == 0


def test_slots_refuse(lib):
    def slots(table=P, prefix=P + 4096, new=P + 8192, B=2, mb=4, bs=16, nb=16, room=100, off=FAR, out=FAR + 4096, pos=FAR + 8192):
        return lib.kv_pages_slots(table, prefix, new, B, mb, bs, nb, room, off, out, pos, NULL, NULL)
    for kw, code in ((dict(table=NULL), INV), (dict(prefix=NULL), INV), (dict(new=NULL), INV), (dict(off=NULL), INV),
                     (dict(out=NULL), INV), (dict(B=0), INV), (dict(mb=0), INV), (dict(bs=0), INV), (dict(nb=0), INV),
                     (dict(room=0), INV), (dict(B=5000), UNS), (dict(room=(1 << 30) + 1), UNS), (dict(nb=1 << 27, bs=1 << 10), UNS),
                     (dict(mb=1 << 20, bs=1 << 12), UNS), (dict(off=P), INV), (dict(out=P + 4), INV), (dict(out=P + 4092), INV),
                     (dict(pos=P + 8196), INV), (dict(out=FAR + 8), INV), (dict(pos=FAR + 4100), INV), (dict(pos=FAR + 8), INV)):
        assert slots(**kw) == code, kw

    for name in ("kv_slots_write", "kv_slots_read"):
        def rows(pages=P, s=P, r=P, e=2, n=5, hkv=1, D=576, bs=16, nb=16):
            return getattr(lib, name)(pages, s, r, e, n, hkv, D, bs, nb, NULL, NULL)
        for kw, code in ((dict(pages=NULL), INV), (dict(s=NULL), INV), (dict(r=NULL), INV), (dict(pages=MIS), INV),
                         (dict(r=MIS), INV), (dict(e=1), UNS), (dict(e=3), UNS), (dict(n=0), INV), (dict(hkv=0), INV),
                         (dict(D=0), INV), (dict(D=6), UNS), (dict(bs=0), INV), (dict(nb=0), INV), (dict(nb=1 << 27, bs=64), UNS),
                         (dict(n=1 << 30, hkv=2), UNS)):
            assert rows(**kw) == code, kw


def test_one_pool_wants_no_second_tree(lib):
    commit = lambda kc=P, vc=NULL, kt=P, vt=NULL: lib.kv_commit(kc, vc, kt, vt, 2, 1, 2, 1, 64, 16, 576, P, P, 8, NULL, NULL, NULL, NULL)  # noqa: E731
    assert commit(vc=P) == INV and commit(vt=P) == INV and commit(kt=NULL) == INV and commit() == INV   # (no prefix_len)
    paged = lambda v=NULL, vt=NULL, table=NULL: lib.kv_commit_paged(P, v, table, 128, 8, 4, P, vt, 2, 1, 2, 1, 16, 576, P, P, 8, P, NULL, NULL, NULL)  # noqa: E731
    assert paged(v=P, table=P) == INV and paged(vt=P, table=P) == INV and paged() == INV


def test_slots_refuse_rows_in_the_pool(lib):
    pool, rows, lst = 16 * 16 * 576 * 2, 5 * 576 * 2, 20
    base = 1 << 34
    for name, slots_at in (("kv_slots_write", ((base, INV), (base + pool - 4, INV))),
                           ("kv_slots_read", ((FAR, INV), (FAR + rows - 4, INV)))):
        def call(r=FAR, s=base - 4096, pages=base):
            return getattr(lib, name)(pages, s, r, 2, 5, 1, 576, 16, 16, NULL, NULL)
        for r in (base, base + pool - 16, base - rows + 16):
            assert call(r=r, s=FAR) == INV
        for s, code in slots_at:
            assert call(s=s) == code
