"""dg_gemv_w4 where a block is a single warp: at most 16 columns and 128 k.
Tolerances are those of test_gpu_gemv_w4."""
import functools
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_gemv_w4 import run_case, weights

pytestmark = pytest.mark.gpu


big = functools.lru_cache(lambda: weights(4096, 16384, 128)[:2])


def leave_nan_in_shared_memory():
    """A call whose activations, all NaN, fill the shared memory of every SM."""
    codes, scales = big()
    x = torch.full((8, 4096), math.nan, device="cuda", dtype=torch.bfloat16)
    y = torch.empty(8, 16384, device="cuda")
    for _ in range(3):
        dg.gemv_w4(x, codes, scales, y)
    assert bool(y.isnan().all())


@pytest.mark.parametrize("N", [1, 8, 16])
@pytest.mark.parametrize("K", [1, 33, 64, 100, 128])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_warp_of_columns(N, K, group):
    for R in (1, 2, 3, 4, 8):
        leave_nan_in_shared_memory()
        run_case(R, K, N, group, "bf16", "f32", zeros=True, out="f32")
        leave_nan_in_shared_memory()
        run_case(R, K, N, group, "f16", "f16", out="f16")
