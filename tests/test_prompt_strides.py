"""Strides of prompt_attn_latent through the C entry point: which are refused, and
that one which nothing steps by is not looked at."""
import ctypes as C
import math

import pytest
import torch

from tree_speculative_decoding_attn_gb300 import _build
from tree_speculative_decoding_attn_gb300 import specverify as sv

P, NULL, INV = 0x100000, None, sv.ERR_INVALID_ARG
ANY = (8, 0, -64, 3, 1 << 60)      # none of them a stride that a call steps by


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers only on a GPU-less host")
def test_which_strides_are_refused():
    _build.build()
    lib = sv.load()

    def call(H=4, tk=20, kt=512, kh=128, rt=576, vt=512, vh=128):
        return lib.prompt_attn_latent(P, P, kt, kh, P, rt, P, vt, vh, P, P, P, 2, H, 128, 64, 10, tk, 8, 0.1, NULL, 0, NULL, NULL)
    for name in ("kt", "kh", "vt", "vh"):
        for bad in (0, 8, 120, 132, -128, 1 << 38):
            assert call(**{name: bad}) == INV, (name, bad)
    for bad in (0, 56, 68, -64, 1 << 38):
        assert call(rt=bad) == INV
    # nothing is refused but by the launch, which needs a GPU
    assert call() == sv.ERR_CUDA and call(kt=128, kh=(1 << 38) - 8) == sv.ERR_CUDA
    for x in ANY:
        assert call(H=1, kh=x, vh=x) == sv.ERR_CUDA and call(tk=1, kt=x, vt=x, rt=x) == sv.ERR_CUDA
        assert call(H=1, kt=x) == INV and call(tk=1, vh=x) == INV


@pytest.mark.gpu
@pytest.mark.parametrize("hq,total", [(1, 70), (3, 1), (1, 1)])
def test_strides_that_nothing_steps_by(lib, hq, total):
    g = torch.Generator().manual_seed(hq + total)
    t = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    n = min(total, 9)
    q, k, v, rope = t(n, hq, 192), t(total, hq, 128), t(total, hq, 128), t(total, 64)
    q_off, kv_off = (torch.tensor([0, x], dtype=torch.int32, device="cuda") for x in (n, total))
    want = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    sv.prompt_attn_latent(q, k, rope, v, q_off, kv_off, want, n, 192 ** -0.5)
    p = lambda x: C.c_void_p(x.data_ptr())  # noqa: E731
    for x in ANY:
        kh, kt, rt = (x if hq == 1 else 128), (x if total == 1 else hq * 128), (x if total == 1 else 64)
        out = torch.zeros_like(want)
        code = lib.prompt_attn_latent(p(q), p(k), kt, kh, p(rope), rt, p(v), kt, kh, p(q_off), p(kv_off), p(out), 1, hq, 128, 64,
                                      n, total, n, 192 ** -0.5, NULL, 0, NULL, torch.cuda.current_stream().cuda_stream)
        assert code == sv.OK
        torch.cuda.synchronize()
        assert torch.equal(out, want) and math.isfinite(float(out.float().sum()))
