"""The device arithmetic of the linear cross entropy, as far as the compiler
alone can tell (csrc/ce.cuh)."""
import os
import shutil
import subprocess

import pytest

import tcgen05_tmem_gemm_b200 as dg

CSRC = os.path.join(os.path.dirname(os.path.abspath(dg.__file__)), "csrc")
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

KERNEL = """
#include "ce.cuh"
__global__ void kernel(const float *in, float *out) {
    float z[%d], m = -INFINITY, s = 0.f;
    for (int i = 0; i < %d; ++i) z[i] = in[i];
    dg::join_logits(m, s, z);
    out[0] = m, out[1] = s;
}
"""


def compiles(tmp_path, n):
    src = tmp_path / f"join{n}.cu"
    src.write_text(KERNEL % (n, n))
    r = subprocess.run([NVCC, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I" + CSRC,
                        "-I" + os.path.join(CSRC, "..", "..", "include"), "-c", str(src), "-o", str(tmp_path / "join.o")],
                       capture_output=True, text=True)
    return r.returncode == 0, r.stdout + r.stderr


@pytest.mark.skipif(not os.path.exists(NVCC), reason="no nvcc")
def test_logits_are_joined_four_or_more_at_a_time(tmp_path):
    """join_logits starts four chains with z[0] .. z[3]: for a shorter array that reads past its end, so it
    must not compile."""
    ok, log = compiles(tmp_path, 4)
    assert ok, log
    for n in (1, 3):
        ok, log = compiles(tmp_path, n)
        assert not ok and "four chains" in log, log
