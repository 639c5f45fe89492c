"""dg_linear_ce and dg_linear_ce_grad with one and two rows against a [V x D] weight (dot products on the CUDA
cores), for logits that are not finite.  Tolerances are those of test_gpu_linear_ce."""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_linear_ce import check_forward, inputs, run_forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("V", [1, 3, 700, 5003])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_row_that_is_not_finite_stays_alone(V, bad, dtype):
    x, w, y, _ = inputs(2, 64, V, dtype, ignored=0.0)
    for row in (0, 1):
        x2 = x.clone()
        x2[row, 9] = bad
        loss, lse = run_forward(x2, w, y)
        # an infinity in x gives logits of +infinity and -infinity, in a vocabulary of one either
        if bad != bad or V > 3:
            assert bool(loss[row].isnan()) and bool(lse[row].isnan())
        check_forward(x[1 - row:2 - row], w, y[1 - row:2 - row], loss[1 - row:2 - row], lse[1 - row:2 - row])
        loss1, lse1 = run_forward(x2[row:row + 1], w, y[row:row + 1])
        assert torch.equal(loss1.isnan(), loss[row:row + 1].isnan())


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("V", [5, 700, 5003])
def test_logits_of_minus_infinity_do_not_count(T, V):
    # columns of W at -infinity under a positive x: their logits are -infinity
    x, w, y, _ = inputs(T, 64, V, "bf16", ignored=0.0)
    x = x.abs() + 0.25
    gone = torch.zeros(V, dtype=torch.bool)
    gone[torch.randperm(V, generator=torch.Generator().manual_seed(V))[:V // 2]] = True
    gone = gone.cuda()
    kept = (~gone).nonzero()[:, 0]
    y = kept[y % len(kept)]
    masked = w.clone()
    masked[:, gone] = -math.inf
    loss, lse = run_forward(x, masked.t().contiguous().t(), y)
    check_forward(x, w[:, kept], torch.searchsorted(kept, y), loss, lse)
    # every logit -infinity: the sum of exponentials is 0
    masked.fill_(-math.inf)
    _, lse = run_forward(x, masked.t().contiguous().t(), y)
    assert bool((lse == -math.inf).all())


@pytest.mark.parametrize("T", [1, 2])
def test_a_nan_among_logits_of_minus_infinity(T):
    x, w, y, _ = inputs(T, 64, 300, "bf16", ignored=0.0)
    x = x.abs() + 0.25
    masked = torch.full((300, 64), -math.inf, device="cuda", dtype=torch.bfloat16)
    masked[177] = math.nan
    _, lse = run_forward(x, masked.t(), y)
    assert bool(lse.isnan().all())
