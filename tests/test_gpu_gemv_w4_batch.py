"""gemv_w4 of activations with several row dims.  Tolerances are those of test_gpu_gemv_w4."""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_gemv_w4 import check, dense, expected, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T", [(2, 3), (1, 8), (8, 1), (1, 1)])
def test_sequences_and_tokens(B, T):
    K, N = 256, 72
    codes, scales, zeros = weights(K, N, 64, zeros=True)
    W = dense(codes, scales, zeros, 64, K)
    longer = torch.randn(B, T + 2, K, device="cuda").bfloat16()
    for x in (longer[:, 1:T + 1], longer[:, 1:T + 1].contiguous()):
        y = torch.empty(B, T, N, device="cuda")
        dg.gemv_w4(x, codes, scales, y, zeros=zeros, group=64)
        want, tol = expected(x, W, y, 1.0, 0.0, None, "none")
        check(y, want, tol)


def test_more_than_eight_rows_are_refused():
    codes, scales, _ = weights(64, 8, 32)
    x, y = torch.zeros(3, 3, 64, device="cuda").bfloat16(), torch.zeros(3, 3, 8, device="cuda")
    with pytest.raises(dg.DgError) as e:
        dg.gemv_w4(x, codes, scales, y, group=32)
    assert e.value.status == dg.DG_ERR_UNSUPPORTED
