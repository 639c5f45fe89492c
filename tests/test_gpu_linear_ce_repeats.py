"""Runs of dg_linear_ce_grad are bit-identical whatever the workspace: dX summed over several pieces of the
vocabulary, by products whose k is split.  Tolerances are those of test_gpu_linear_ce."""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_linear_ce import DT, IGNORE, check_grads, inputs, run_forward

pytestmark = pytest.mark.gpu


def space(x, w, dx, dw, fraction):
    least, best = dg.dg_linear_ce_grad_workspace(dg.view(x), dg.view(w), dg.view(dx),
                                                 None if dw is None else dg.view(dw))
    return torch.empty(max(least, int(least + fraction * (best - least))), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("T,D,V,fractions", [
    (96, 128, 3000, (0.0, 0.3, 0.6, 0.9)),    # pieces below the best workspace
    (8192, 16, 50000, (1.0,)),                # two pieces at the best one
    (40, 24, 9000, (0.1, 0.5)),
    (300, 256, 8000, (0.2, 0.7)),
])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_several_pieces(T, D, V, fractions, out):
    x, w, y, dl = inputs(T, D, V, "bf16")
    _, lse = run_forward(x, w, y)
    dx = torch.empty(T, D, device="cuda", dtype=DT[out])
    dw = torch.empty(V, D, device="cuda", dtype=DT[out]).t()
    for fraction in fractions:
        ws = space(x, w, dx, dw, fraction)
        first = None
        for _ in range(8):
            dx.fill_(math.nan)
            dw.fill_(math.nan)
            dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE, workspace=ws)
            if first is None:
                first = dx.clone(), dw.clone()
                check_grads(x, w, y, dl, dx, dw)
            assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
