"""Sizes whose products pass 32 or 64 bits: size queries answer any shape,
refused ones with 0, and calls refuse them; in a process of their own (no GPU)."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from tree_speculative_decoding_attn_gb300 import _build

HUGE = [(65536, 65536), (32768, 131072), (1 << 30, 4), (65536, 1)]


@pytest.mark.parametrize("query,tail", [("tree_attn_window_workspace_bytes", ", 60000, 60000, 4"),
                                        ("tree_attn_window_workspace_bytes", ", 2147483647, 2147483647, 0"),
                                        ("tree_attn_workspace_bytes", ", 60000, 0")])
def test_size_queries_survive_products_past_32_bits(query, tail):
    _build.build()
    calls = "; ".join(f"print(lib.{query}(sv.F32, {b}, 1, {h}, {h}, 128{tail}))" for b, h in HUGE)
    r = subprocess.run([sys.executable, "-c", f"from tree_speculative_decoding_attn_gb300 import specverify as sv; "
                        f"lib = sv.load(); {calls}"], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr)
    if "window" in query:  # more sequences and KV heads than the call takes
        assert r.stdout.split() == ["0"] * len(HUGE)


@pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder pointers only on a GPU-less host")
@pytest.mark.parametrize("num_blocks,hkv,block_size", [(1 << 30, 1 << 14, 1 << 20), (1 << 24, 1 << 15, 1 << 25),
                                                       (1 << 29, 1 << 8, 1 << 27), (1 << 20, 1 << 10, 1 << 10)])
def test_pools_of_too_many_rows_are_refused(num_blocks, hkv, block_size):
    """Products that wrap 64 bits to 0, and one past the limit (placeholder
    addresses, never dereferenced: every call is refused on the host)."""
    _build.build()
    code = f"""
from tree_speculative_decoding_attn_gb300 import specverify as sv
lib, P, n, h, bs = sv.load(), 0x100000, {num_blocks}, {hkv}, {block_size}
print(lib.tree_attn_verify_window_paged(P, P, P, P, bs, n, 1, P, P, P, P, P, P, 0, 1, 1, h, h, 128, 100, 50, 4, 0.0, P, 1 << 40,
                                        None, None),
      lib.tree_attn_verify_paged(P, P, P, P, bs, n, 1, P, P, P, P, P, 0, 1, 1, h, h, 128, 100, 0.0, 0, P, 1 << 40, None, None),
      lib.kv_commit_paged(P, P, P, bs, n, 1, P, P, 2, 1, 1, h, 1, 128, P, P, 2, P, P, None, None),
      lib.kv_pages_compact(P, P, 2, 1, h, 128, bs, n, P, 1, 1, P, P, P, P, None, P, 1 << 50, None, None))
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["2"] * 4    # SPEC_ERR_UNSUPPORTED
