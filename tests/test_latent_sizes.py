"""The size queries of the latent operators at the ends of their ranges and for
types that they do not take (no GPU)."""
import pytest

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
