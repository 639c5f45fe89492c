"""dg_linear_ce_grad with F16 operands and a dloss that differs from row to row by many orders of magnitude.

Tolerance, element by element.  Row t's |dloss| is r times the largest, b; e is the exponent of r (r 2^-e in
[1/2, 1)), k that of the largest |x| of the row, and h = max(min(0, e + 10), min(0, -9 - k)) the power of two that dW's
copy of the row takes (h = e without dW).  An entry of G is rounded to F16 at the scale 2^14 r 2^-h / |dloss|: by u = 2^-11 of
itself or half a subnormal, 2^-25 of b 2^h 2^-14.  An element of the copy moves by half a subnormal, 2^-25, over 2^h,
or not at all.  The rest is as in test_gpu_linear_ce: logits, exponentials, FP32 sums, the output's rounding.
"""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_linear_ce import DT, IGNORE, logits, run_forward

pytestmark = pytest.mark.gpu


def check(x, w, y, dl, dx, dw):
    """dx [T x D] and dw [D x V] (either None) against the formula, in FP64."""
    z, dz = logits(x, w, 1.0)
    T, V = z.shape
    lse = torch.logsumexp(z, 1, keepdim=True)
    kept = y != IGNORE
    g = torch.where(kept, dl.double(), 0.0)[:, None]
    p = torch.exp(z - lse)
    one = torch.zeros_like(p).scatter_(1, torch.where(kept, y, 0)[:, None], 1.0)
    G = g * (p - one)
    b = g.abs().max()
    e = torch.frexp(g.abs() / b).exponent.clamp(max=0).double()
    xk = torch.where(kept[:, None], x.double(), 0.0)
    h = e
    if dw is not None:
        k = torch.frexp(xk.abs().amax(1, keepdim=True)).exponent.double()
        h = torch.maximum((e + 10).clamp(max=0), (-9 - k).clamp(max=0))
    u = 2.0 ** -11
    dG = (u + 2.0 ** -22) * G.abs() + g.abs() * p * (dz + lse.abs() * 2.0 ** -22 + 2.0 ** -20)
    dG = dG + torch.where(kept[:, None], b * 2.0 ** (h - 39.0), 0.0)

    def one_grad(got, a, bb, da, db, n):
        want, s = a @ bb, a.abs() @ bb.abs()
        tol = da @ bb.abs() + (0 if db is None else a.abs() @ db) + (64 + n / 16) * 2.0 ** -23 * s
        tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol) + \
            (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126)
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), (float((err / tol).max()), float(err.max()))

    if dx is not None:
        one_grad(dx, G, w.double().t(), dG, None, V)
        assert bool((dx[~kept] == 0).all())
    if dw is not None:
        dxk = torch.where((xk.abs() * 2.0 ** h < 2.0 ** -14) & (h < 0), 2.0 ** (-25.0 - h), 0.0)
        one_grad(dw.t(), G.t(), xk, dG.t(), dxk, T)


def problem(T, D, V, std, aligned, scale=1.0, seed=0):
    """Feature 0 is 0 in x and 1 in w: dX holds the rows' sums of G there."""
    g = torch.Generator().manual_seed(seed + T + D + V)
    x = torch.randn(T, D, generator=g) * scale
    x[:, 0] = 0
    w = torch.randn(V, D, generator=g) * (std / math.sqrt(D))
    w[:, 0] = 1
    x, w = x.half().cuda(), w.half().cuda()
    if not aligned:
        off = torch.zeros(T, D + 1, device="cuda").half()[:, 1:]
        off.copy_(x)
        x = off
    y = torch.randint(0, V, (T,), generator=g)
    y[T // 2] = IGNORE if T > 2 else y[T // 2]
    dl = 10.0 ** -(8.0 * torch.rand(T, generator=g)) * torch.where(torch.rand(T, generator=g) < 0.5, -1.0, 1.0)
    dl[0] = 0.75
    return x, w.t(), y.cuda(), dl.cuda()


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("outputs", ["both", "dx", "dw"])
@pytest.mark.parametrize("T,D,V", [(2, 64, 20000), (9, 64, 20000), (40, 1400, 900), (70, 136, 20000), (400, 264, 5000),
                                   (2100, 40, 700)])
def test_rows_of_every_magnitude(T, D, V, outputs, aligned):
    # logits close to one another: p near 1 / V in every column
    x, w, y, dl = problem(T, D, V, 0.05, aligned)
    _, lse = run_forward(x, w, y)
    for out in ("f32", "f16"):
        dx = torch.full((T, D), math.nan, device="cuda", dtype=DT[out]) if outputs != "dw" else None
        dw = torch.full((V, D), math.nan, device="cuda", dtype=DT[out]).t() if outputs != "dx" else None
        dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
        check(x, w, y, dl, dx, dw)


@pytest.mark.parametrize("scale", [2.0 ** -12, 1.0, 2.0 ** 10])
@pytest.mark.parametrize("fraction", [0.0, 0.4])
def test_sizes_of_x_and_several_pieces(scale, fraction):
    x, w, y, dl = problem(90, 128, 4000, 1.0 / max(scale, 1.0), True, scale)
    _, lse = run_forward(x, w, y)
    dx, dw = torch.empty(90, 128, device="cuda"), torch.empty(4000, 128, device="cuda").t()
    least, best = dg.dg_linear_ce_grad_workspace(dg.view(x), dg.view(w), dg.view(dx), dg.view(dw))
    ws = torch.empty(least + int(fraction * (best - least)), dtype=torch.uint8, device="cuda")
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE, workspace=ws)
    check(x, w, y, dl, dx, dw)


def test_rows_of_zero_nan_and_infinite_dloss():
    x, w, y, dl = problem(12, 64, 300, 1.0, True)
    _, lse = run_forward(x, w, y)
    dl[3], dl[7] = 0.0, 1e-40
    dx = torch.empty(12, 64, device="cuda")
    dw = torch.empty(300, 64, device="cuda").t()
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    check(x, w, y, torch.where(dl.abs() < 1e-38, 0.0, dl), torch.where(dl[:, None].abs() < 1e-38, 0.0, dx), dw)
    assert bool((dx[3] == 0).all()) and bool((dx[7].abs() < 1e-38).all())
    dl[5], dl[9] = math.nan, math.inf
    dg.linear_ce_grad(x, w, y, lse, dl, dx, None, ignore_index=IGNORE)
    rest = torch.ones(12, dtype=torch.bool, device="cuda")
    rest[[5, 9]] = False
    assert not bool(dx[5].isfinite().any()) and not bool(dx[9].isfinite().any())
    dl = torch.where(dl.abs() < 1e-38, 0.0, dl)
    check(x[rest], w, y[rest], dl[rest], torch.where(dl[rest][:, None] == 0, 0.0, dx[rest]), None)
