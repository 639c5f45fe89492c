"""dg_linear_ce and dg_linear_ce_grad with one and two rows against a [V x D] weight (dot products on the CUDA
cores), for logits that are not finite, and in several pieces.  Tolerances are those of test_gpu_linear_ce."""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_linear_ce import IGNORE, check_forward, check_grads, inputs, run_both, run_forward

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


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("D,V", [(8, 1), (256, 100), (264, 4001), (1032, 9000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_alpha_ignored_rows_and_types(T, D, V, dtype):
    run_both(T, D, V, dtype, out="f32", alpha=0.5, ignored=0.6)
    run_both(T, D, V, dtype, out="f32", alpha=-1.75, ignored=0.0)


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("fraction", [0.0, 0.1, 0.3, 0.8])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_several_pieces(T, fraction, out):
    # the gradient walks the vocabulary in pieces, the target in any of them
    for seed_width in (64, 72, 136):
        run_both(T, seed_width, 5003, "bf16", out=out, fraction=fraction, ignored=0.0)
    run_both(T, 64, 5003, "f16", out=out, alpha=0.75, fraction=fraction, ignored=0.0)


@pytest.mark.parametrize("v", [0, 255, 256, 300, 4999])
def test_targets_in_every_piece(v):
    x, w, _, dl = inputs(1, 64, 5000, "bf16", ignored=0.0)
    y = torch.full((1,), v, device="cuda")
    loss, lse = run_forward(x, w, y)
    check_forward(x, w, y, loss, lse)
    dx, dw = torch.empty(1, 64, device="cuda"), torch.empty(5000, 64, device="cuda").t()
    least, _ = dg.dg_linear_ce_grad_workspace(dg.view(x), dg.view(w), dg.view(dx), dg.view(dw))
    ws = torch.empty(least, dtype=torch.uint8, device="cuda")
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE, workspace=ws)
    check_grads(x, w, y, dl, dx, dw)
