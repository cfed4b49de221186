"""The size queries of the latent operators at the ends of their ranges and for
types that they do not take (no GPU)."""
import pytest
import torch

from tree_speculative_decoding_attn_gb300 import _build
from tree_speculative_decoding_attn_gb300 import specverify as sv


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load()


def float32_bytes(batch, nodes, heads, latent, max_prefix):
    """Ranges of 16 keys or multiples, as many as fill the SMs once and at most
    128; a range's partial is latent + 4 words a row."""
    ctas = batch * -(-nodes * heads // 8)
    tiles = -(-(max_prefix + nodes) // 16)
    n = max(1, min((152 if latent == 512 else 304) // ctas, tiles, 128))
    splits = -(-tiles // -(-tiles // n))
    return 0 if splits == 1 else batch * nodes * heads * splits * (latent + 4) * 4


@pytest.mark.parametrize("max_prefix", [0, 1, 15, 16, 100, 5000, (1 << 30) - 257, (1 << 30) - 16, 1 << 30])
def test_float32_workspace(lib, max_prefix):
    for batch in (1, 2, 10, 76, 77, 152, 200, 65535):
        for nodes, heads in ((1, 1), (1, 16), (5, 4), (60, 32), (256, 16)):
            for latent in (256, 512):
                got = lib.tree_attn_latent_workspace_bytes(sv.F32, batch, nodes, heads, latent, 64, max_prefix)
                assert got == float32_bytes(batch, nodes, heads, latent, max_prefix), (batch, nodes, heads, latent)


def test_types_that_the_calls_do_not_take_need_nothing(lib):
    """As in C: 0, so that a call without a workspace gets the call's own refusal."""
    size = sv.tree_attn_latent_workspace_bytes
    for dtype in (torch.float16, torch.float64, torch.int32, 2, -1):
        assert size(dtype, 2, 8, 16, 512, 64, 100) == 0
    assert size(torch.bfloat16, 2, 8, 16, 512, 64, 100) == size(sv.BF16, 2, 8, 16, 512, 64, 100) > 0


@pytest.mark.gpu
def test_other_types_are_refused_with_a_status(lib):
    z = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt, device="cuda")  # noqa: E731
    n, i32, words = z(2, dt=torch.int32), torch.int32, z(2, 3, dt=torch.int64)
    for workspace in (None, z(1 << 20, dt=torch.uint8)):
        with pytest.raises(sv.SpecError) as e:
            sv.tree_attn_verify_latent(z(2, 3, 4, 576), z(2, 100, 576), z(2, 3, 576), n, words, z(2, 3, 4, 512), 90, 0.1,
                                       workspace=workspace)
        assert e.value.code == sv.ERR_UNSUPPORTED
        with pytest.raises(sv.SpecError) as e:
            sv.tree_attn_verify_latent_paged(z(2, 3, 4, 576), z(4, 128, 576), z(2, 2, dt=i32), z(2, 3, 576), n, words,
                                             z(2, 3, 4, 512), 90, 0.1, workspace=workspace)
        assert e.value.code == sv.ERR_UNSUPPORTED
