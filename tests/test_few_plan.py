"""The plan of the few-row window kernels on devices that run clusters of 16
CTAs and on ones that stop at 8, from a program of its own linked with the
library (host arithmetic, no GPU)."""
import os
import shutil
import subprocess

import pytest

from tree_speculative_decoding_attn_gb300 import _build

SRC = r"""
#include <cstdio>
#include "kernels.h"
int main() {
  const int batches[] = {1, 2, 7, 64}, nodes[] = {1, 5, 64, 200}, bounds[] = {0, 1, 333, 2112, 2120, 4224, 4230, 60000};
  for (int dtype = 0; dtype < 2; ++dtype)
    for (int b : batches)
      for (int n : nodes)
        for (int mp : bounds)
          for (int pairs = 0; pairs <= dtype; ++pairs)
            for (int most = 8; most <= 16; most += 8) {
              SvAttnShape s{dtype, b, n, 8, 2, 128, mp, mp};
              s.window = 1 << 20;
              SvAttnPlan p{};
              const bool few = sv_attn_few_plan(s, pairs, most, &p);
              printf("%d %d %d %d %d %d %d %d %d\n", dtype, b, n, mp, pairs, most, few, p.splits, p.chunk);
            }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    lib = _build.build()
    at = tmp_path_factory.mktemp("plan")
    src, exe = at / "plan.cpp", at / "plan"
    src.write_text(SRC)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc")))
    subprocess.run(["g++", "-std=c++17", "-I" + _build.CSRC, "-I" + _build.INCLUDE, "-I" + os.path.join(cuda, "include"),
                    str(src), lib, "-Wl,-rpath," + os.path.dirname(lib), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_no_plan_passes_the_largest_cluster(plans):
    assert len(plans) > 500
    for dtype, b, n, mp, pairs, most, few, splits, chunk in plans:
        if not few:
            continue
        assert splits in (1, 2, 4, 8, 16) and splits <= most
        if dtype == 0:  # float32: a CTA's shared memory holds up to 264 keys, and the CTAs hold all
            assert chunk <= 264 and splits * chunk >= mp + n


def test_every_call_has_a_plan_at_8_and_16_is_taken_where_it_may(plans):
    took = {k: any(p[7] == k for p in plans if p[5] == k and p[6]) for k in (8, 16)}
    assert took == {8: True, 16: True}
    for dtype, b, n, mp, pairs, most, few, splits, chunk in plans:
        if dtype == 1 and not pairs:  # no other kernel takes these: the streaming one has no bound on the keys
            assert few
        if dtype == 0:                # past what the cluster's shared memory holds: tiles with a workspace
            assert few == (mp + n <= most * 264)
