"""Sizes of the pieces that rows are moved in (csrc/row_vec.hpp): those whose last piece its parts make up compile, others
are refused. The host compiler's pass only, nothing is built."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_expert_layer_amd", "csrc")
SOURCE = """
#include "row_vec.hpp"
__global__ void move(const void* a, void* b, int left) {
  moe::RowVec<%s, %d> v;
  v.load(a, 0, left);
  v.store(b, 0, left);
}
"""


@pytest.mark.parametrize("bf16,n,taken", [("true", 4, True), ("true", 8, True), ("false", 4, True), ("false", 8, True),
                                          ("true", 16, False), ("false", 2, False)])
def test_pieces(tmp_path, bf16, n, taken):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    src = tmp_path / "move.hip"
    src.write_text(SOURCE % (bf16, n))
    r = subprocess.run([hipcc, "--cuda-host-only", "-fsyntax-only", "-std=c++17", "--offload-arch=gfx950", "-I", CSRC,
                        "-I", os.path.join(ROOT, "include"), str(src)], capture_output=True, text=True, timeout=300)
    assert (r.returncode == 0) == taken, r.stderr[-2000:]
    assert taken or "static assertion" in r.stderr or "static_assert" in r.stderr
