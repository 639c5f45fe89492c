"""linear_ce and linear_ce_grad of activations whose features are several dims (x_row_dims)."""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg


@pytest.mark.parametrize("shape,rd,rows", [((2, 3, 4, 8), 2, 6), ((2, 3, 32), 2, 6), ((5, 4, 8), 1, 5), ((4, 8), 0, 1)])
def test_one_target_per_row(shape, rd, rows):
    """The binding counts the rows by x_row_dims: as many targets pass it (and are refused by the library, for not
    being device memory), others do not."""
    x, w = torch.zeros(shape).bfloat16(), torch.zeros(32, 10).bfloat16()
    space = torch.zeros(1 << 16, dtype=torch.uint8)
    for n in (rows, rows + 1):
        y, f = torch.zeros(n, dtype=torch.int64), torch.zeros(n)
        with pytest.raises(dg.DgError if n == rows else ValueError):
            dg.linear_ce(x, w, y, f, f, stream=0, workspace=space, x_row_dims=rd)
        with pytest.raises(dg.DgError if n == rows else ValueError):
            dg.linear_ce_grad(x, w, y, f, f, x, w, stream=0, workspace=space, x_row_dims=rd)


@pytest.mark.gpu
def test_features_of_two_dims():
    # heads side by side, and heads apart in memory; tolerances are those of test_gpu_linear_ce
    from test_gpu_linear_ce import check_forward, check_grads

    B, T, H, E, V = 2, 7, 4, 16, 300
    g = torch.Generator().manual_seed(3)
    packed = torch.randn(B, T, H, E, generator=g).bfloat16().cuda()
    apart = packed.transpose(1, 2).contiguous().transpose(1, 2)
    w = (torch.randn(V, H * E, generator=g) / 8).bfloat16().cuda().t()
    y = torch.randint(0, V, (B * T,), generator=g).cuda()
    flat = packed.view(B * T, H * E)

    def both(x, rd):
        loss, lse = torch.empty(B * T, device="cuda"), torch.empty(B * T, device="cuda")
        dg.linear_ce(x, w, y, loss, lse, x_row_dims=rd)
        dx, dw = torch.full_like(x, math.nan), torch.empty(V, H * E, device="cuda").t()
        dg.linear_ce_grad(x, w, y, lse, torch.ones(1, device="cuda"), dx, dw, x_row_dims=rd)
        return loss, lse, dx.reshape(B * T, H * E), dw

    for x, rd in ((flat, 1), (packed, 2), (apart, 2)):
        loss, lse, dx, dw = both(x, rd)
        check_forward(flat, w, y, loss, lse)
        check_grads(flat, w, y, torch.ones(B * T, device="cuda"), dx, dw)
