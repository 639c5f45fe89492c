"""G of confident rows: dg_linear_ce_grad with the lse that dg_linear_ce wrote, at a long k.

Every row has a feature of its own that W does not use, so that dW holds G itself (in FP32: one term per sum, its
value G rounded to X's type), and one feature that is 0 in X and 1 in W, so that dX holds the rows' sums of G.

Tolerance.  With z' = z + d the logits that the device makes of a long sum (|d| <= dz), p' = exp(z' - lse') and
lse' their own lse, 1 - p' at a confident target is off by (1 - p) (exp(2 dz) - 1) only, however large dz |z| is:
the errors of the target's logit and of lse are the same one.  What comes on top does not depend on k: lse is held in
FP32 (2^-24 |lse|), the difference z' - lse' is rounded (2^-24 |z|), alpha z' too (2^-24 |z|), twice (both passes);
the sum of exponentials is off by at most (512 + V / 1024) 2^-24, exponentials by 2^-20; together
  e = 2^-22 (|z| + |lse|) + (512 + V / 1024) 2^-24 + 2^-19,
and a row's sum of G adds u sum |G| (u = eps / 2 for the rounding of each entry) and, F16, half a subnormal a column.
Other entries are off by p (e + exp(2 dz) - 1).
"""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_linear_ce import DT, IGNORE, run_forward

pytestmark = pytest.mark.gpu


def problem(T, D, V, dtype, top, order):
    """x [T x (D + T + 1)] and w whose target logits are about `top`, all of their products positive."""
    g = torch.Generator().manual_seed(T + D + V)
    pad = -(D + T + 1) % 8
    x = torch.zeros(T, D + T + 1 + pad)
    x[:, :D] = torch.randn(T, D, generator=g)
    x[:, D:D + T] = torch.eye(T)
    w = torch.zeros(V, D + T + 1 + pad)
    w[:, :D] = torch.randn(V, D, generator=g) / math.sqrt(D)
    y = torch.randperm(V, generator=g)[torch.arange(T) % V]
    for t in range(T):
        w[y[t], :D] = x[t, :D] * (top / D)
    w[:, D + T] = 1
    x, w = x.to(DT[dtype]).cuda(), w.to(DT[dtype]).cuda()
    return x, (w.t() if order == "vd" else w.t().contiguous()), y.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("order", ["vd", "dv"])
@pytest.mark.parametrize("T,D,V", [
    (2, 4000, 500),       # dot products ("vd")
    (40, 4000, 500),      # few rows and columns: logits of FP32 in pieces
    (70, 4000, 500), (300, 2000, 700), (200, 8000, 19000), (70, 900, 300),  # paired tiles
    (100, 4000, 40),      # fewer columns than the tensor stores take
])
def test_confident_rows_of_a_long_k(T, D, V, order, dtype):
    x, w, y = problem(min(T, V), D, V, dtype, 30.0, order)
    T = x.shape[0]
    z = x.double() @ w.double()
    S = x.double().abs() @ w.double().abs()
    lse64 = torch.logsumexp(z, 1, keepdim=True)
    loss, lse = run_forward(x, w, y)
    dl = torch.ones(1, device="cuda")
    dx, dw = torch.empty(x.shape, device="cuda"), torch.empty(w.shape, device="cuda")
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    assert dg.dg_sync_status() == dg.DG_OK
    G = dw[D:D + T].double()
    u = torch.finfo(x.dtype).eps / 2
    dz = (32 + x.shape[1] / 16) * 2.0 ** -23 * S
    e = 2.0 ** -22 * (z.abs() + lse64.abs()) + (512 + V / 1024) * 2.0 ** -24 + 2.0 ** -19
    grow = torch.exp(2 * dz.amax(1, keepdim=True)) - 1
    p = torch.exp(z - lse64)
    hit = torch.zeros_like(p, dtype=torch.bool).scatter_(1, y[:, None], True)
    rest = torch.where(hit, 0.0, p).sum(1, keepdim=True)      # 1 - p at the target, without cancellation
    want = torch.where(hit, -rest, p)
    tol = torch.where(hit, rest * grow + e, p * (e + grow))
    tol = tol + u * (want.abs() + tol) + 2.0 ** -33            # (F16 pieces: half a subnormal over the scale)
    err = (G - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), float(err[hit].max()))
    sums = dx[:, D + T].double()
    tol = e.gather(1, y[:, None])[:, 0] + u * 2 * rest[:, 0] * (1 + grow[:, 0]) + u * e.amax(1) + V * 2.0 ** -33 + \
        (64 + V / 16) * 2.0 ** -23 * 2 * (rest[:, 0] * (1 + grow[:, 0]) + e.amax(1))
    assert bool((sums.abs() <= tol).all()), (float((sums.abs() / tol).max()), float(sums.abs().max()))


@pytest.mark.parametrize("T,V", [(1, 500), (2, 500), (2, 9000)])
@pytest.mark.parametrize("share", [0.0, 0.3])
def test_few_rows_in_a_small_workspace(T, V, share):
    # lse made with the least workspace, the gradient with the best: the same dot products
    D = 4000
    x, w, y = problem(T, D, V, "bf16", 30.0, "vd")
    least, best = dg.dg_linear_ce_workspace(dg.view(x), dg.view(w))
    loss, lse = run_forward(x, w, y, workspace=torch.empty(least + int(share * (best - least)), dtype=torch.uint8,
                                                           device="cuda"))
    z = x.double() @ w.double()
    lse64 = torch.logsumexp(z, 1)
    # FP32 dot products: D / 256 terms a lane and five steps over the warp, 2^-24 each
    S = x.double().abs() @ w.double().abs()
    dz = (D / 256 * 8 + 5) * 2.0 ** -24 * S.amax(1)
    assert bool(((lse.double() - lse64).abs() <= dz + 2.0 ** -19 + (512 + V / 8) * 2.0 ** -24 + 2.0 ** -23 * lse64).all())
    dw = torch.empty(w.shape, device="cuda")
    dg.linear_ce_grad(x, w, y, lse, torch.ones(1, device="cuda"), None, dw, ignore_index=IGNORE)
    G = dw[D:D + T].double()
    hit = G.gather(1, y[:, None])[:, 0]
    # 1 - p is below 1e-8, and so are all terms but one of the sum of exponentials, which is 1: what is left is the
    # rounding of lse and of z - lse, and the exponential's of a number next to 0
    e = 2.0 ** -23 * (z.amax(1) + lse64) + 2.0 ** -21
    assert bool((hit.abs() <= e + 1e-8).all()), float(hit.abs().max())
