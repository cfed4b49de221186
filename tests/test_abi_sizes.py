"""Size queries answer any shape, refused ones with 0: shapes whose products
pass 32 bits, asked in a process of their own (no GPU)."""
import subprocess
import sys

import pytest

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
