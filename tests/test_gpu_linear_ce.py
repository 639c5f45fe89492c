"""dg_linear_ce and dg_linear_ce_grad against their definitions in FP64.

Tolerances, with S[t][v] = |alpha| sum_d |x| |w| and g the upstream gradient:
  a logit's FP32 sum passes each product through at most 32 + D / 16 roundings
    (a tensor-core step sums 16; 2^-23 each, since it may truncate), or D + 1
    of 2^-24 on the CUDA cores: dz = (32 + D / 16) 2^-23 S, D 2^-24 S there;
  lse moves by at most max_v dz, the sum of exponentials by at most
    (512 + V / 1024) 2^-24 of itself (256 logits a thread, then pairs) and 2^-20
    for the exponentials and the logarithm, the result by 2^-23 (|lse| + |z|);
  G is off by u |G| (its rounding to X's type, u = eps / 2, 0 for F32; the
    division by the largest dloss and back adds 2^-22 |G|) plus
    |g| p (dz + |lse| 2^-22 + 2^-20) + (|g| + 1) 2^-126 (the hardware's power of
    two gives 0 for a result below 2^-126, so p is off by up to 2^-126 there,
    and G may be flushed below 2^-126 itself), and F16 pieces by half a
    subnormal, 2^-25 of 2^9 times smaller than the largest |g|;
  dX and dW pass that on through |W| and |X|, add (64 + n / 16) 2^-23 of
    sum |G| |W| (n terms: V or T; n 2^-24 on the CUDA cores), and round once.
"""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100


@pytest.fixture(autouse=True)
def _reset_options():
    yield
    dg.dg_set_option(dg.DG_OPT_FORCE_KIND, 0)
    dg.dg_set_option(dg.DG_OPT_CTA_PAIR, 1)


def inputs(T, D, V, dtype, ignored=0.2, seed=0, order="vd", std=2.0):
    g = torch.Generator().manual_seed(seed + T * 7 + D * 3 + V)
    x = torch.randn(T, D, generator=g).to(DT[dtype]).cuda()
    w = (torch.randn(V, D, generator=g) * (std / math.sqrt(max(D, 1)))).to(DT[dtype]).cuda()
    w = w.t() if order == "vd" else w.t().contiguous()
    y = torch.randint(0, V, (T,), generator=g)
    y = torch.where(torch.rand(T, generator=g) < ignored, torch.full_like(y, IGNORE), y).cuda()
    dl = torch.randn(T, generator=g).cuda()
    return x, w, y, dl


def logits(x, w, alpha):
    """(z, dz) in FP64."""
    D = x.shape[1]
    xd, wd = x.double(), w.double()
    S = abs(alpha) * (xd.abs() @ wd.abs())
    u = (D + 1) * 2.0 ** -24 if x.dtype == torch.float32 else (32 + D / 16) * 2.0 ** -23
    return alpha * (xd @ wd), u * S


def run_forward(x, w, y, alpha=1.0, **kw):
    rows = y.numel()
    loss = torch.full((rows,), math.nan, device="cuda")
    lse = torch.full((rows,), math.nan, device="cuda")
    dg.linear_ce(x, w, y, loss, lse, alpha=alpha, ignore_index=IGNORE, **kw)
    return loss, lse


def check_forward(x2, w, y, loss, lse, alpha=1.0):
    z, dz = logits(x2, w, alpha)
    V = w.shape[1]
    want = torch.logsumexp(z, 1)
    tol = dz.amax(1) + (512 + V / 1024) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -23 * want.abs()
    assert bool(((lse.double() - want).abs() <= tol).all()), float(((lse.double() - want).abs() - tol).max())
    kept = y != IGNORE
    hit = z.gather(1, torch.where(kept, y, 0)[:, None])[:, 0]
    tol = tol + dz.amax(1) + 2.0 ** -23 * hit.abs()
    err = (loss.double() - (want - hit)).abs()
    assert bool((err[kept] <= tol[kept]).all()), float((err - tol)[kept].max())
    assert bool((loss[~kept] == 0).all())
    return z, dz


def check_grads(x2, w, y, dl, dx, dw, alpha=1.0):
    """dx [T x D] and dw [D x V] (either None) against the formula."""
    z, dz = logits(x2, w, alpha)
    T, V = z.shape
    lse = torch.logsumexp(z, 1, keepdim=True)
    kept = (y != IGNORE) & (y >= 0) & (y < V)
    g = torch.where(kept, dl.double(), 0.0)[:, None]
    p = torch.exp(z - lse)
    one = torch.zeros_like(p).scatter_(1, torch.where(kept, y, 0)[:, None], 1.0)
    G = g * (p - one)
    u = 0.0 if x2.dtype == torch.float32 else torch.finfo(x2.dtype).eps / 2
    dG = (u + 2.0 ** -22) * G.abs() + g.abs() * p * (dz + lse.abs() * 2.0 ** -22 + 2.0 ** -20) + \
        (g.abs() + 1) * 2.0 ** -126
    if x2.dtype == torch.float16:
        dG = dG + torch.where(kept, 1.0, 0.0)[:, None].double() * g.abs().max() * 2.0 ** -34
    G0 = torch.where(kept[:, None], G, 0.0)
    xk = torch.where(kept[:, None], x2.double(), 0.0)

    def one_grad(got, a, b, da, n):
        want = alpha * (a @ b)
        s = abs(alpha) * (a.abs() @ b.abs())
        acc = n * 2.0 ** -24 + 2.0 ** -22 if x2.dtype == torch.float32 else (64 + n / 16) * 2.0 ** -23
        tol = abs(alpha) * (da.abs() @ b.abs()) + acc * s
        tol = tol + torch.finfo(got.dtype).eps / 2 * (want.abs() + tol) + \
            (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126)
        err = (got.double() - want).abs()
        assert bool((err <= tol).all()), (float((err - tol).max()), float(err.max()))

    if dx is not None:
        one_grad(dx, G0, w.double().t(), dG, V)
        assert bool((dx[~kept] == 0).all())
    if dw is not None:
        one_grad(dw.t(), G0.t(), xk, dG.t(), T)


def run_both(T, D, V, dtype, alpha=1.0, order="vd", out=None, fraction=None, ignored=0.2, std=2.0):
    """Forward and gradient of one problem, both checked; `fraction` of the best workspace for each."""
    x, w, y, dl = inputs(T, D, V, dtype, ignored, order=order, std=std)
    xv, wv = dg.view(x), dg.view(w)
    out = DT[out or dtype]
    dx = torch.full((T, D), math.nan, dtype=out, device="cuda")
    dw = torch.full((V, D), math.nan, dtype=out, device="cuda").t() if order == "vd" else \
        torch.full((D, V), math.nan, dtype=out, device="cuda")

    def space(sizes):
        if fraction is None:
            return None
        least, best = sizes
        return torch.empty(max(least, int(least + fraction * (best - least))), dtype=torch.uint8, device="cuda")

    loss, lse = run_forward(x, w, y, alpha, workspace=space(dg.dg_linear_ce_workspace(xv, wv)))
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, alpha=alpha, ignore_index=IGNORE,
                      workspace=space(dg.dg_linear_ce_grad_workspace(xv, wv, dg.view(dx), dg.view(dw))))
    assert dg.dg_sync_status() == dg.DG_OK
    check_forward(x, w, y, loss, lse, alpha)
    check_grads(x, w, y, dl, dx, dw, alpha)
    return loss, lse, dx, dw


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 33, 64, 65, 127, 129, 200, 257])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_numbers_of_rows(T, dtype):
    run_both(T, 128, 1000, dtype)


@pytest.mark.parametrize("V", [1, 2, 7, 8, 31, 255, 256, 257, 2047, 2049, 5003])
@pytest.mark.parametrize("order", ["vd", "dv"])
def test_sizes_of_the_vocabulary(V, order):
    run_both(19, 72, V, "bf16", order=order)


@pytest.mark.parametrize("D", [1, 3, 8, 17, 100, 1000, 2050])
@pytest.mark.parametrize("T", [3, 70, 300])
def test_widths(D, T):
    run_both(T, D, 520, "bf16")


@pytest.mark.parametrize("order", ["vd", "dv"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_paired_tiles(dtype, order):
    # enough rows and columns for the paired tensor-core tiles, with both edges inside a tile
    run_both(513, 320, 19300, dtype, alpha=0.75, order=order)


@pytest.mark.parametrize("T", [1, 4, 5, 31, 32, 100])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_paired_tiles_with_few_rows(T, out):
    run_both(T, 192, 19000, "bf16", out=out)


def test_very_wide_rows():
    run_both(3, 20000, 70, "bf16")
    run_both(130, 16392, 300, "f16", order="dv")


@pytest.mark.parametrize("T", [1, 2])
@pytest.mark.parametrize("D,V", [(8, 1), (8, 9), (256, 100), (264, 4001), (4096, 3000), (7680, 50), (9000, 70)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_and_two_rows(T, D, V, dtype):
    # dot products against a [V x D] weight, and what they leave to the tiles (wide rows)
    run_both(T, D, V, dtype, ignored=0.0)
    run_both(T, D, V, dtype, out="f32", alpha=0.5, ignored=0.6, order="dv")


@pytest.mark.parametrize("T,D,V", [(3000, 64, 300), (2500, 100, 65), (2049, 520, 1000), (5000, 32, 64), (700, 2048, 64)])
@pytest.mark.parametrize("order", ["vd", "dv"])
def test_small_layers_with_many_rows(T, D, V, order):
    # few tiles: k of dX and of dW split into planes of partial sums
    run_both(T, D, V, "f16", order=order)
    run_both(T, D, V, "bf16", order=order, out="f32", alpha=-0.25)


@pytest.mark.parametrize("V", [19000, 19201, 25600 + 40])
def test_pieces_that_end_in_few_columns(V):
    for fraction in (0.15, 0.5, 0.9):
        run_both(290, 64, V, "bf16", fraction=fraction)


def test_paired_and_plain_tiles_agree():
    x, w, y, dl = inputs(640, 256, 16640, "bf16")
    a = run_forward(x, w, y)
    dg.dg_set_option(dg.DG_OPT_CTA_PAIR, 0)
    b = run_forward(x, w, y)
    check_forward(x, w, y, *a)
    check_forward(x, w, y, *b)


def test_float32():
    run_both(37, 65, 300, "f32")
    run_both(5, 64, 129, "f32", alpha=-0.5, order="dv")


@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fraction", [0.0, 0.3])
def test_several_pieces_and_output_types(out, fraction):
    run_both(96, 128, 3000, "bf16", out=out, fraction=fraction)
    run_both(300, 128, 19000, "f16", out=out, fraction=fraction)


def test_every_row_ignored_and_no_rows():
    x, w, y, dl = inputs(12, 64, 100, "bf16")
    y.fill_(IGNORE)
    loss, lse = run_forward(x, w, y)
    dx, dw = torch.full_like(x, math.nan), torch.full_like(w, math.nan)
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    assert bool((loss == 0).all() and (dx == 0).all() and (dw == 0).all())
    empty = torch.empty(0, device="cuda")
    dg.linear_ce(x[:0], w, y[:0], empty, empty)
    dw.fill_(math.nan)
    dg.linear_ce_grad(x[:0], w, y[:0], empty, empty, x[:0].clone(), dw)
    assert bool((dw == 0).all())


def test_no_features():
    # D = 0: every logit is 0
    x, w = torch.empty(5, 0, device="cuda").bfloat16(), torch.empty(0, 40, device="cuda").bfloat16()
    y = torch.arange(5, device="cuda")
    loss, lse = run_forward(x, w, y)
    assert bool(((lse - math.log(40)).abs() < 1e-6).all() and torch.equal(loss, lse))


@pytest.mark.parametrize("T,V", [(2, 300), (40, 1200), (400, 19000)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_ignored_rows_may_hold_anything(T, V, bad):
    x, w, y, dl = inputs(T, 96, V, "bf16")
    y[::3] = IGNORE
    clean = x.clone()
    x[::3] = bad
    dl[::3] = math.nan
    loss, lse = run_forward(x, w, y)
    lse[::3] = math.nan
    dx, dw = torch.full_like(x, math.nan), torch.full_like(w, math.nan)
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    keep = y != IGNORE
    check_forward(clean[keep], w, y[keep], loss[keep], lse[keep])
    assert bool((loss[~keep] == 0).all())
    check_grads(clean, w, y, torch.where(keep, dl, 0.0), dx, dw)


@pytest.mark.parametrize("T,V", [(40, 1200), (400, 19000)])
def test_targets_out_of_range_are_reported(T, V):
    x, w, y, dl = inputs(T, 96, V, "bf16")
    y[3], y[5] = V, -7
    loss, lse = run_forward(x, w, y)
    assert dg.dg_sync_status() == dg.DG_ERR_VALUE
    assert dg.dg_sync_status() == dg.DG_OK
    assert bool(loss[[3, 5]].isnan().all())
    good = (y >= 0) & (y < V) | (y == IGNORE)
    check_forward(x[good], w, y[good], loss[good], lse[good])
    dx, dw = torch.full_like(x, math.nan), torch.full_like(w, math.nan)
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    assert dg.dg_sync_status() == dg.DG_ERR_VALUE
    check_grads(x, w, y, dl, dx, dw)


@pytest.mark.parametrize("T,V", [(24, 700), (512, 19000)])
def test_nan_and_infinite_rows_stay_alone(T, V):
    x, w, y, dl = inputs(T, 64, V, "bf16", ignored=0.0)
    x[4, 9] = math.nan
    x[6, 9] = math.inf
    loss, lse = run_forward(x, w, y)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[[4, 6]] = False
    assert bool(loss[[4, 6]].isnan().all())
    check_forward(x[rest], w, y[rest], loss[rest], lse[rest])


def test_columns_at_the_lowest_value():
    # a vocabulary padded with weights that push its logits to the type's lowest values
    T, D, V = 300, 64, 19000
    x, w, y, dl = inputs(T, D, V, "bf16")
    x = x.abs() + 0.25
    w = w.clone()
    w[:, 18000:] = torch.finfo(torch.bfloat16).min / 2 ** 12
    y = torch.where(y == IGNORE, y, y % 18000)
    loss, lse = run_forward(x, w, y)
    check_forward(x, w[:, :18000], y, loss, lse)
    w[:, 18000:] = -math.inf                      # logits of -infinity
    loss2, lse2 = run_forward(x, w, y)
    check_forward(x, w[:, :18000], y, loss2, lse2)


def test_confident_rows():
    # logits of +-60: probabilities of 1 and of 1e-50
    run_both(64, 64, 700, "bf16", std=60.0)
    run_both(300, 64, 19000, "f16", std=60.0)


@pytest.mark.parametrize("scale", [1e-7, 1.0, 3e4])
def test_float16_loss_scales(scale):
    x, w, y, dl = inputs(60, 128, 4000, "f16")
    dl = dl * scale
    _, lse = run_forward(x, w, y)
    dx, dw = torch.empty_like(x, dtype=torch.float32), torch.empty_like(w, dtype=torch.float32)
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    check_grads(x, w, y, dl, dx, dw)


def test_one_gradient_for_all_rows_and_one_output_only():
    x, w, y, _ = inputs(50, 128, 900, "bf16")
    _, lse = run_forward(x, w, y)
    n = int((y != IGNORE).sum())
    dl = torch.full((1,), 1.0 / n, device="cuda")
    dx, dw = torch.full_like(x, math.nan), torch.full_like(w, math.nan)
    dg.linear_ce_grad(x, w, y, lse, dl.expand(50), dx=dx, ignore_index=IGNORE)
    dg.linear_ce_grad(x, w, y, lse, dl, dw=dw, ignore_index=IGNORE)
    check_grads(x, w, y, dl.expand(50), dx, dw)


@pytest.mark.parametrize("T,V", [(5, 300), (70, 19000)])
def test_shifted_tokens_and_strided_outputs(T, V):
    # all tokens but each sequence's last one: the rows are two dims that do not merge
    B, D = 4, 128
    x, w, y, dl = inputs(B * T, D, V, "bf16")
    x3 = x.view(B, T, D)[:, :-1]
    rows = B * (T - 1)
    y, dl = y[:rows].contiguous(), dl[:rows].contiguous()
    loss, lse = run_forward(x3, w, y)
    flat = x3.reshape(rows, D)
    check_forward(flat, w, y, loss, lse)
    full = torch.full((B, T, D), -3.0, device="cuda").bfloat16()
    wide = torch.full((V, D + 8), -3.0, device="cuda").bfloat16()
    dg.linear_ce_grad(x3, w, y, lse, dl, full[:, :-1], wide[:, :D].t(), ignore_index=IGNORE)
    check_grads(flat, w, y, dl, full[:, :-1].reshape(rows, D), wide[:, :D].t())
    assert bool((full[:, -1] == -3).all() and (wide[:, D:] == -3).all())


@pytest.mark.parametrize("T,V", [(6, 300), (300, 19000)])
def test_one_row_for_all(T, V):
    # X expanded from one row, targets differ
    x, w, y, dl = inputs(T, 128, V, "bf16")
    xe = x[:1].expand(T, 128)
    loss, lse = run_forward(xe, w, y)
    check_forward(xe.contiguous(), w, y, loss, lse)
    dx, dw = torch.full_like(x, math.nan), torch.full_like(w, math.nan)
    dg.linear_ce_grad(xe, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    check_grads(xe.contiguous(), w, y, dl, dx, dw)


@pytest.mark.parametrize("T,V", [(33, 500), (400, 19000)])
def test_unaligned_operands(T, V):
    # rows that start at odd multiples of two bytes, in X, W and the gradients
    D = 101
    x, w, y, dl = inputs(T, D, V, "bf16")
    xo = torch.zeros(T, D + 2, device="cuda").bfloat16()[:, 1:D + 1]
    wo = torch.zeros(V, D + 2, device="cuda").bfloat16()[:, 1:D + 1]
    xo.copy_(x)
    wo.copy_(w.t())
    loss, lse = run_forward(xo, wo.t(), y)
    check_forward(x, w, y, loss, lse)
    dxo, dwo = torch.zeros_like(xo), torch.zeros_like(wo)
    dg.linear_ce_grad(xo, wo.t(), y, lse, dl, dxo, dwo.t(), ignore_index=IGNORE)
    check_grads(x, w, y, dl, dxo, dwo.t())


# W and dW whose rows do not start at multiples of 16 bytes: the products read and make copies of them.
def off_rows(kind, D, V, dtype):
    """An empty D x V matrix of the kind on the device, and its storage."""
    if kind == "steps":  # neither dimension contiguous
        store = torch.full((V, 2 * D + 3), 7.0, device="cuda", dtype=dtype)
        return store[:, 1:2 * D + 1:2].t(), store
    first, second = (V, D) if kind[:2] == "vd" else (D, V)
    pad = (kind[2:] == " even") * 2 + (kind[2:] == " odd") * 3
    store = torch.full((first, second + pad), 7.0, device="cuda", dtype=dtype)
    m = store[:, pad // 2:pad // 2 + second]
    return (m.t() if first == V else m), store


@pytest.mark.parametrize("T,D,V", [(1, 333, 70), (2, 1031, 900), (8, 100, 257), (70, 513, 1025), (300, 2, 3001),
                                   (300, 2050, 3001), (64, 4099, 501)])
@pytest.mark.parametrize("kind", ["vd", "vd even", "vd odd", "dv", "dv even", "dv odd", "steps"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows_off_sixteen_bytes(T, D, V, kind, out):
    x, w0, y, dl = inputs(T, D, V, "bf16")
    w, _ = off_rows(kind, D, V, torch.bfloat16)
    w.copy_(w0)
    dx = torch.empty(T, D, device="cuda", dtype=DT[out])
    dw, store = off_rows(kind, D, V, DT[out])
    written = torch.zeros_like(store, dtype=torch.bool)
    written.as_strided(dw.shape, dw.stride(), dw.storage_offset()).fill_(True)
    least, best = dg.dg_linear_ce_workspace(dg.view(x), dg.view(w))
    gleast, gbest = dg.dg_linear_ce_grad_workspace(dg.view(x), dg.view(w), dg.view(dx), dg.view(dw))
    for size, gsize in ((best, gbest), (least, gleast), ((least + best) // 2, (gleast + gbest) // 2)):
        loss, lse = run_forward(x, w, y, workspace=torch.empty(size, dtype=torch.uint8, device="cuda"))
        check_forward(x, w0, y, loss, lse)
        dx.fill_(math.nan)
        dw.fill_(math.nan)
        dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE,
                          workspace=torch.empty(gsize, dtype=torch.uint8, device="cuda"))
        check_grads(x, w0, y, dl, dx, dw)
        assert bool((store[~written] == 7).all())


@pytest.mark.parametrize("V", [513, 769, 65537, 66049, 98305, 99073, 131073])
@pytest.mark.parametrize("share", [0.0, 0.1, 0.4])
def test_last_piece_of_one_column(V, share):
    # W's columns contiguous and its rows aligned, so that no piece is copied
    T, D = 40, 16
    x, w0, y, dl = inputs(T, D, V, "bf16")
    w = torch.zeros(D, V + 7, device="cuda").bfloat16()[:, :V]
    w.copy_(w0)
    dx, dw = torch.empty_like(x), torch.empty(D, V + 7, device="cuda")[:, :V]
    least, best = dg.dg_linear_ce_workspace(dg.view(x), dg.view(w))
    space = torch.empty(least + int(share * (best - least)), dtype=torch.uint8, device="cuda")
    loss, lse = run_forward(x, w, y, workspace=space)
    check_forward(x, w0, y, loss, lse)
    least, best = dg.dg_linear_ce_grad_workspace(dg.view(x), dg.view(w), dg.view(dx), dg.view(dw))
    space = torch.empty(least + int(share * (best - least)), dtype=torch.uint8, device="cuda")
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE, workspace=space)
    check_grads(x, w0, y, dl, dx, dw)


def test_gradient_against_differences():
    # central differences of the library's own loss along random directions: with the direction scaled
    # so that no logit moves by more than 1 per unit, the third derivative of a row's loss is at most
    # 2 max|move - mean|^3 <= 16, the truncation h^2 / 6 * 16 a row; the losses' own error is below
    # 2^-18 a row, 2^-18 / h
    T, D, V, h = 6, 48, 200, 1.0 / 32
    x, w, y, dl = inputs(T, D, V, "f32")
    dl = dl.abs() + 0.5
    _, lse = run_forward(x, w, y)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    tol = float(dl.sum()) * (16 * h * h / 6 + 2.0 ** -18 / h)
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        u = torch.randn(T, D, generator=g).cuda()
        u /= (u @ w).abs().max()
        lo, hi = run_forward(x - h * u, w, y)[0], run_forward(x + h * u, w, y)[0]
        assert abs(float((dl * (hi - lo)).sum()) / (2 * h) - float((dx * u).sum())) <= tol
        u = torch.randn(V, D, generator=g).cuda().t()
        u = u / (x @ u).abs().max()
        lo, hi = run_forward(x, w - h * u, y)[0], run_forward(x, w + h * u, y)[0]
        assert abs(float((dl * (hi - lo)).sum()) / (2 * h) - float((dw * u).sum())) <= tol


@pytest.mark.parametrize("T,V", [(16, 900), (512, 19000)])
def test_streams_graphs_and_repeats(T, V):
    x, w, y, dl = inputs(T, 128, V, "f16")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    loss, lse = run_forward(x, w, y)
    dg.linear_ce_grad(x, w, y, lse, dl, dx, dw, ignore_index=IGNORE)
    torch.cuda.synchronize()
    # two streams, each with its own results and workspace
    outs = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        o = [torch.empty_like(loss), torch.empty_like(lse), torch.empty_like(dx), torch.empty_like(dw)]
        torch.cuda.synchronize()
        outs.append(o)
    for _ in range(3):
        for s, o in zip(streams, outs):
            dg.linear_ce(x, w, y, o[0], o[1], ignore_index=IGNORE, stream=s)
            dg.linear_ce_grad(x, w, y, o[1], dl, o[2], o[3], ignore_index=IGNORE, stream=s)
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, (loss, lse, dx, dw)):
            assert torch.equal(a, b)
    # captured once, replayed on new values
    o = outs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dg.linear_ce(x, w, y, o[0], o[1], ignore_index=IGNORE)
        dg.linear_ce_grad(x, w, y, o[1], dl, o[2], o[3], ignore_index=IGNORE)
    x2, _, y2, dl2 = inputs(T, 128, V, "f16", seed=9)
    x.copy_(x2), y.copy_(y2), dl.copy_(dl2)
    for a in o:
        a.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(x, w, y, o[0], o[1])
    check_grads(x, w, y, dl, o[2], o[3])


def test_trained_then_served_in_four_bits():
    """The operators together: an output layer trained with linear_ce and its gradient, its weight put into
    4 bits, and a token's logits from gemv_w4 against the loss of the same 4-bit weight."""
    T, D, V, group = 64, 256, 1000, 32
    x, w, y, _ = inputs(T, D, V, "bf16", ignored=0.1)
    weight = w.t().contiguous()
    dl = torch.full((1,), 1.0 / T, device="cuda")
    dweight = torch.empty(V, D, device="cuda")
    for _ in range(3):
        loss, lse = run_forward(x, weight.t(), y)
        dg.linear_ce_grad(x, weight.t(), y, lse, dl, dw=dweight.t(), ignore_index=IGNORE)
        check_grads(x, weight.t(), y, dl.expand(T), None, dweight.t())
        weight = (weight.float() - 2.0 * dweight).bfloat16()
    wg = weight.float().view(V, D // group, group)
    scales = (wg.abs().amax(2) / 7).bfloat16()
    q = (torch.round(wg / scales.float()[:, :, None]) + 8).clamp(0, 15).to(torch.uint8).view(V, D)
    codes = q[:, 0::2] | (q[:, 1::2] << 4)
    z = torch.empty(8, V, device="cuda")
    dg.gemv_w4(x[:8], codes, scales, z, group=group)
    w4 = (scales.float()[:, :, None] * (q.view(V, -1, group).float() - 8)).view(V, D)
    z64 = x[:8].double() @ w4.double().t()
    S = x[:8].double().abs() @ w4.double().abs().t()
    assert bool(((z.double() - z64).abs() <= (32 + D / 32) * 2.0 ** -23 * S + 2.0 ** -22 * z64.abs()).all())
    # the loss of the 4-bit weight (exact in FP32) through the FP32 path
    loss4, lse4 = run_forward(x[:8].float(), w4.t(), y[:8].contiguous())
    check_forward(x[:8].float(), w4.t(), y[:8], loss4, lse4)
    assert bool(((torch.logsumexp(z.double(), 1) - lse4.double()).abs() <= 1e-4).all())
