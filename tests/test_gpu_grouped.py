"""dg_gemm_grouped and dg_gemm_grouped_dw against their definitions in FP64.

Tolerance.  With S = |alpha| sum |a| |b| (scales included), a 16- or 8-bit
product is exact in FP32 and the tensor core adds 16 of them (32 of E4M3) per
step to the running sum; each step truncates, so it loses at most 2^-23 of the
running magnitude, and the 16 or 32 terms of a step no more than 32 times that
in all their alignments together over the whole sum's first step:
(32 + k / 16) 2^-23 S for a sum of k products.  F32 operands are summed by k
fused multiply-adds of 2^-24: less than (32 + k / 2) 2^-23 S.  The scales, beta
and the bias round five more times, at most 2^-22 (|z| + |beta c| + |bias|).
GeLU's slope is below 1.13 and its own error is 2^-20 |z| (FP32 outputs) or
2^-11 |z| (16-bit outputs, the hardware's tanh).  The store rounds by half a
step, eps / 2 of the value (F16: or half of its smallest subnormal, 2^-25).
"""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
ACT = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0),
       "gelu_tanh": lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))}
SIZES = {
    "one": [1],
    "few": [0, 1, 0, 7, 33, 0],
    "even": [16] * 8,
    "odd": [257, 0, 255, 300, 31, 2],
    "tall": [520, 1030],
    "none": [0, 0, 0],
    "many": [(7 * i) % 41 for i in range(70)],
}


def values(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(DT[dtype])


def padded(t, pad, offset=0):
    """The same values with `pad` elements of NaN behind each row, `offset` elements past an aligned address."""
    rows, cols = t.shape[:-1].numel(), t.shape[-1]
    nan = torch.full((offset + rows * (cols + pad) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    flat = nan.repeat_interleave(t.element_size()).view(t.dtype)
    strides, step = [1], cols + pad
    for s in reversed(t.shape[:-1]):
        strides.insert(0, step)
        step *= s
    v = torch.as_strided(flat, t.shape, strides, offset)
    v.copy_(t)
    return v


def offsets_of(sizes, front=0):
    return torch.tensor([front] + list(sizes), device="cuda").cumsum(0)


def check(got, want, tol, dtype):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    ok &= ~inf
    tol = tol + torch.finfo(dtype).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)
    err = (got - want).abs()
    assert bool((err[ok] <= tol[ok]).all()), float((err[ok] - tol[ok]).max())


def steps(k, dtype):
    return (32 + k / (2 if dtype == torch.float32 else 16)) * 2.0 ** -23


def rows_case(sizes, K, N, dtype="bf16", out="bf16", weight="nk", alpha=1.0, beta=0.0, scales=False, bias=False,
              act="none", front=0, behind=0, a=None, b=None, c=None, pad=0, off=0, stream=None):
    G, R = len(sizes), front + sum(sizes) + behind
    seed = R * 31 + K * 7 + N
    a = values((R, K), dtype, seed) if a is None else a
    if b is None:
        b = values((G, N, K) if weight == "nk" else (G, K, N), dtype, seed + 1, max(K, 1) ** -0.5 if dtype != "e4m3" else 1.0)
        b = padded(b, pad, off) if pad or off else b
        b = b.transpose(1, 2) if weight == "nk" else b
    if pad or off:
        a = padded(a, pad, off)
    c = values((R, N), out, seed + 2) if c is None else c
    c0 = c.clone()
    offsets = offsets_of(sizes, front)
    sa = torch.rand(R, device="cuda") + 0.5 if scales else None
    sb = torch.rand(G, N, device="cuda") - 0.5 if scales else None
    bs = torch.randn(G, N, device="cuda") if bias else None
    before = dg.dg_launch_count()
    dg.gemm_grouped(a, b, c, offsets, scale_a=sa, scale_b=sb, alpha=alpha, beta=beta, bias=bs, act=act, stream=stream)
    assert dg.dg_launch_count() == before + (R > 0)  # without rows there is nothing to do
    assert dg.dg_sync_status(stream) == dg.DG_OK
    ends = offsets.tolist()
    assert torch.equal(c[:ends[0]], c0[:ends[0]]) and torch.equal(c[ends[-1]:], c0[ends[-1]:])
    for g in range(G):
        r = slice(ends[g], ends[g + 1])
        x, w = a[r].double(), b[g].double()
        s = alpha * (1 if sa is None else sa[r, None].double()) * (1 if sb is None else sb[g].double())
        z = (x @ w) * s if alpha else torch.zeros_like(c0[r], dtype=torch.float64)
        S = (x.abs() @ w.abs()) * (abs(s) if isinstance(s, float) else s.abs()) if alpha else torch.zeros_like(z)
        bc = beta * c0[r].double() if beta else torch.zeros_like(z)
        bb = torch.zeros_like(z) if bs is None else bs[g].double().expand_as(z)
        z = z + bc + bb
        tol = steps(K, a.dtype) * S + 2.0 ** -22 * (z.abs() + bc.abs() + bb.abs())
        if act == "gelu_tanh":
            tol = 1.13 * tol + (2.0 ** -20 if out == "f32" else 2.0 ** -11) * z.abs()
        check(c[r], ACT[act](z), tol, c.dtype)
    return c


def dw_case(sizes, K, N, dtype="bf16", out="f32", weight="kn", alpha=1.0, beta=0.0, front=0, behind=0, x=None, dy=None,
            dw=None, pad=0):
    G, R = len(sizes), front + sum(sizes) + behind
    seed = R * 37 + K * 5 + N
    x = values((R, K), dtype, seed) if x is None else x
    dy = values((R, N), dtype, seed + 1) if dy is None else dy
    if pad:
        x, dy = padded(x, pad), padded(dy, pad)
    if dw is None:
        dw = values((G, N, K) if weight == "nk" else (G, K, N), out, seed + 2)
        dw = dw.transpose(1, 2) if weight == "nk" else dw
    if not beta:
        dw.fill_(math.nan)
    old = dw.clone()
    offsets = offsets_of(sizes, front)
    before = dg.dg_launch_count()
    dg.gemm_grouped_dw(x, dy, dw, offsets, alpha=alpha, beta=beta)
    assert dg.dg_launch_count() == before + 1
    assert dg.dg_sync_status() == dg.DG_OK
    ends = offsets.tolist()
    for g in range(G):
        r = slice(ends[g], ends[g + 1])
        a, b = x[r].double(), dy[r].double()
        z, S = alpha * (a.t() @ b), abs(alpha) * (a.abs().t() @ b.abs())
        bc = beta * old[g].double() if beta else torch.zeros_like(z)
        tol = steps(ends[g + 1] - ends[g], x.dtype) * S + 2.0 ** -22 * ((z + bc).abs() + bc.abs())
        check(dw[g], z + bc, tol, dw.dtype)
    return dw


# ------------------------------------------------------------------- by rows

@pytest.mark.parametrize("weight", ["nk", "kn"])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_rows_sizes(sizes, dtype, weight):
    rows_case(SIZES[sizes], 272, 304, dtype, "f32", weight)


@pytest.mark.parametrize("K", [1, 8, 16, 63, 64, 65, 127, 128, 129, 1001])
@pytest.mark.parametrize("weight", ["nk", "kn"])
def test_rows_k(K, weight):
    # rows padded to multiples of 16 bytes: K itself is any
    rows_case([3, 0, 70], K, 128, "f16", "f32", weight, pad=-K % 8 if weight == "nk" else 0,
              a=None if weight == "nk" else padded(values((73, K), "f16", 5), -K % 8))


@pytest.mark.parametrize("N", [1, 2, 31, 32, 33, 100, 255, 256, 257, 1000])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_rows_n(N, out):
    rows_case([5, 40, 0, 1], 128, N, "bf16", out)


@pytest.mark.parametrize("weight", ["nk", "kn"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_rows_types(dtype, out, weight):
    rows_case([40, 0, 3, 300], 144, 160, dtype, out, weight, scales=dtype == "e4m3")


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("beta", [0.0, -0.5])
@pytest.mark.parametrize("N", [192, 77])
def test_rows_epilogue(act, out, beta, N):
    rows_case([40, 0, 3, 65], 96, N, "bf16", out, alpha=1.5, beta=beta, scales=True, bias=True, act=act, front=2,
              behind=3)


@pytest.mark.parametrize("weight", ["nk", "kn"])
def test_rows_of_no_group_stay(weight):
    rows_case([10, 0, 90], 64, 200, front=7, behind=33, weight=weight)


@pytest.mark.parametrize("weight", ["nk", "kn"])
def test_rows_nothing_multiplied(weight):
    a = torch.full((50, 64), math.nan, device="cuda").bfloat16()
    b = torch.full((3, 64, 80), math.nan, device="cuda").bfloat16()
    rows_case([20, 0, 30], 64, 80, a=a, b=b, alpha=0.0, beta=0.5, bias=True)
    rows_case([20, 0, 30], 64, 80, a=a, b=b, alpha=0.0, beta=0.0)
    rows_case([20, 0, 30], 0, 80, beta=2.0, bias=True, act="relu", weight=weight)


def test_rows_keep_to_their_group():
    # NaN and infinities stay in their rows, columns and groups
    a = values((120, 128), "bf16", 1)
    b = values((4, 96, 128), "bf16", 2)
    a[17, 5], a[60, 9], a[110] = math.nan, math.inf, math.nan
    b[1] = math.nan  # a group without rows
    b[2, 50, 3] = -math.inf
    c = rows_case([40, 0, 60], 128, 96, a=a, b=b[:3].transpose(1, 2), behind=20)
    assert c[17].isnan().all() and not c[16].isnan().any()


def test_rows_strides():
    wide = values((90, 400), "bf16", 3)
    rows_case([50, 40], 200, 120, a=wide[:, 8:208])
    rows_case([25, 20], 200, 120, a=wide[::2, 8:208])
    # A whose columns are not contiguous, C with any strides, and rows at odd addresses: the CUDA cores
    rows_case([25, 20], 200, 120, a=values((200, 45), "bf16", 4).t())
    rows_case([25, 20], 77, 50)
    rows_case([25, 20], 80, 50, pad=1)
    rows_case([25, 20], 80, 50, off=3)
    c = values((45, 120, 2), "bf16", 5)
    other = c[:, :, 1].clone()
    rows_case([25, 20], 200, 120, c=c[:, :, 0])
    assert torch.equal(c[:, :, 1], other)
    c = values((120, 45), "f32", 6).t()
    rows_case([25, 20], 200, 120, c=c, out="f32")
    c = values((45, 131), "bf16", 7)[:, 3:123]
    rows_case([25, 20], 200, 120, c=c, beta=1.0)


def test_rows_weight_layouts():
    w = values((96, 3, 128), "bf16", 8)
    rows_case([10, 20, 30], 128, 96, b=w.permute(1, 2, 0))            # [N, groups, K]
    rows_case([10, 20, 30], 96, 128, b=w.permute(1, 0, 2))            # [K, groups, N]
    rows_case([10, 20, 30], 128, 96, b=w[:, 0].t().expand(3, 128, 96))  # one weight for all
    rows_case([10, 20], 128, 96, b=w[:, ::2].permute(1, 2, 0))
    big = values((5, 100, 136), "bf16", 9)
    rows_case([10, 20], 128, 96, b=big[1:4:2, 2:98, 8:].transpose(1, 2))  # slices of a larger stack


def test_rows_of_several_dims():
    # [batch, positions] of tokens, one of them sliced away; the CUDA cores on demand
    x = values((4, 9, 128), "bf16", 1)
    w, offsets = values((3, 96, 128), "bf16", 2), offsets_of([10, 0, 22])
    want = torch.empty(32, 96, device="cuda")
    dg.gemm_grouped(x[:, 1:].reshape(32, 128), w.transpose(1, 2), want, offsets)
    c = torch.empty(4, 8, 96, device="cuda")
    dg.gemm_grouped(x[:, 1:], w.transpose(1, 2), c, offsets)
    z = steps(128, torch.bfloat16) * 2 * (x[:, 1:].double().abs().sum(2).max() * w.double().abs().max())
    assert bool(((c.view(32, 96) - want).abs() <= z).all())
    dg.dg_set_option(dg.DG_OPT_FORCE_KIND, dg.DG_KIND_SIMT)
    try:
        rows_case([10, 0, 22], 128, 96, out="f32")
        dw_case([10, 0, 22], 128, 96)
    finally:
        dg.dg_set_option(dg.DG_OPT_FORCE_KIND, 0)
    assert dg.dg_sync_status() == dg.DG_OK


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [[2], [1, 1], [3, 0, 2, 1, 0, 0, 1, 1]])
def test_rows_single_tokens(rows, dtype):
    rows_case(rows, 1024, 2048, dtype)


def test_rows_deep():
    rows_case([300, 20], 8192, 256, out="f32")
    rows_case([5], 16384, 128, out="f32", weight="kn")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_sums_keep_their_precision(dtype):
    """F32 sums of many products.  A step of 16 truncates to 2^-23, 2^-24 of the sum on average, always towards zero:
    128 steps of an accumulator lose 128 * 2^-24 = 7.6e-6 of it at most, in the norm over many sums; 14336 products in
    one accumulator would lose seven times that."""
    x, w = values((200, 14336), dtype, 1), values((1, 300, 14336), dtype, 2, 2.0 ** -6)
    c = torch.empty(200, 300, device="cuda")
    dg.gemm_grouped(x, w.transpose(1, 2), c, offsets_of([200]))
    want = x.double() @ w[0].double().t()
    assert float((c.double() - want).norm() / want.norm()) <= 7.6e-6
    x, dy = values((16000, 300), dtype, 3), values((16000, 260), dtype, 4)
    x, dy = padded(x, 4), padded(dy, 4)
    dw = torch.empty(3, 300, 260, device="cuda")
    sizes = [12000, 100, 3900]
    dg.gemm_grouped_dw(x, dy, dw, offsets_of(sizes))
    assert dg.dg_sync_status() == dg.DG_OK
    for g, (a, b) in enumerate([(0, 12000), (12000, 12100), (12100, 16000)]):
        want = x[a:b].double().t() @ dy[a:b].double()
        assert float((dw[g].double() - want).norm() / want.norm()) <= 7.6e-6


def test_rows_most_groups():
    sizes = [(i * 7919) % 5 for i in range(1024)]
    rows_case(sizes, 64, 64)
    with pytest.raises(dg.DgError):
        rows_case([1] * 1025, 64, 64)


def test_rows_far_offsets():
    # C and A past 2^31 and 2^32 bytes
    R, K, N = 70000, 64, 16400
    c = torch.empty(R, N, device="cuda")
    sizes = [1, 34999, 0, 35000]
    a, b = values((R, K), "bf16", 1), values((4, N, K), "bf16", 2, 0.1)
    c.fill_(math.nan)
    dg.gemm_grouped(a, b.transpose(1, 2), c, offsets_of(sizes))
    assert dg.dg_sync_status() == dg.DG_OK
    for g, rows in ((0, [0]), (1, [1, 34999]), (3, [35000, 35017, 69999])):
        x, w = a[rows].double(), b[g].double()
        check(c[rows], x @ w.t(), steps(K, a.dtype) * (x.abs() @ w.abs().t()), c.dtype)
    assert not c.isnan().any()


# ---------------------------------------------------------------------- by k

@pytest.mark.parametrize("weight", ["nk", "kn"])
@pytest.mark.parametrize("sizes", SIZES)
def test_dw_sizes(sizes, weight):
    dw_case(SIZES[sizes], 264, 152, weight=weight)


@pytest.mark.parametrize("weight", ["nk", "kn"])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "e4m3", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_dw_types(dtype, out, weight):
    dw_case([40, 0, 3, 300], 144, 160, dtype, out, weight, alpha=0.5, beta=-2.0)


@pytest.mark.parametrize("size", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257])
def test_dw_ragged_sums(size):
    # what follows the group's last row is NaN
    x, dy = values((size + 200, 128), "bf16", 1), values((size + 200, 136), "bf16", 2)
    x[size:size + 100], dy[size:size + 100] = math.nan, math.inf
    dw_case([size], 128, 136, x=x, dy=dy, behind=200)


@pytest.mark.parametrize("K,N", [(1, 1), (8, 8), (7, 9), (128, 1), (100, 72), (129, 257), (1000, 64), (64, 1000)])
def test_dw_shapes(K, N):
    dw_case([30, 0, 100], K, N)
    dw_case([30, 0, 100], K, N, weight="nk", out="bf16")


def test_dw_strides():
    x, dy = values((100, 300), "bf16", 1), values((100, 400), "bf16", 2)
    dw_case([50, 50], 200, 120, x=x[:, 8:208], dy=dy[:, 16:136])
    dw_case([25, 25], 200, 120, x=x[::2, 8:208], dy=dy[1::2, 16:136])
    dw_case([50, 50], 200, 120, x=x[:, 3:203], dy=dy[:, 16:136])  # odd addresses: the CUDA cores
    dw_case([50, 50], 200, 120, x=values((200, 100), "bf16", 3).t(), dy=dy[:, :120])
    d = values((2, 210, 130), "f32", 4)
    keep = d.clone()
    dw_case([50, 50], 200, 120, x=x[:, 8:208], dy=dy[:, 16:136], dw=d[:, 3:203, 5:125], beta=1.0)
    assert torch.equal(d[:, :3], keep[:, :3]) and torch.equal(d[:, :, 125:], keep[:, :, 125:])
    d = values((200, 2, 120), "bf16", 5)
    dw_case([50, 50], 200, 120, x=x[:, 8:208], dy=dy[:, 16:136], dw=d.transpose(0, 1), out="bf16")


def test_dw_empty():
    dw_case([0, 0], 128, 64)
    dw_case([0, 0], 128, 64, beta=0.5)
    nan = torch.full((10, 128), math.nan, device="cuda").bfloat16()
    dw_case([0, 0], 128, 128, x=nan, dy=nan, behind=10)
    x = torch.empty(0, 128, device="cuda").bfloat16()
    dw_case([0, 0], 128, 128, x=x, dy=x, beta=3.0)
    # alpha 0 reads neither operand
    d = values((2, 128, 128), "f32", 1)
    old = d.clone()
    dg.gemm_grouped_dw(nan, nan, d, offsets_of([4, 6]), alpha=0.0, beta=2.0)
    assert dg.dg_sync_status() == dg.DG_OK and torch.equal(d, 2 * old)


def test_dw_deep():
    dw_case([9000, 100, 3000], 64, 64)


# ------------------------------------------------------------ used as they are

def test_gradients_against_differences():
    """dX and dW of sum(Y * D) for Y = grouped X W, against the change of that sum."""
    sizes, K, N = [40, 0, 25], 64, 48
    x, w = values((65, K), "f32", 1), values((3, K, N), "f32", 2)
    d = values((65, N), "f32", 3)
    offsets = offsets_of(sizes)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dg.gemm_grouped(d, w.transpose(1, 2), dx, offsets)
    dg.gemm_grouped_dw(x, d, dw, offsets)

    def total(x, w):
        return sum(float(((x[a:b] @ w[g]) * d[a:b].double()).sum()) for g, (a, b) in enumerate([(0, 40), (40, 40), (40, 65)]))

    dirx, dirw = values((65, K), "f32", 4).double(), values((3, K, N), "f32", 5).double()
    h = 2.0 ** -10  # the sum is bilinear: differences along one operand are exact but for FP64's rounding
    fx = (total(x.double() + h * dirx, w.double()) - total(x.double() - h * dirx, w.double())) / (2 * h)
    fw = (total(x.double(), w.double() + h * dirw) - total(x.double(), w.double() - h * dirw)) / (2 * h)
    # each FP32 gradient is off by (32 + k / 2) 2^-23 of its sum of magnitudes, k <= 64
    Sx = sum(float(((d[a:b].double().abs() @ w[g].double().abs().t()) * dirx[a:b].abs()).sum()) for g, (a, b) in enumerate([(0, 40), (40, 40), (40, 65)]))
    Sw = sum(float(((x[a:b].double().abs().t() @ d[a:b].double().abs()) * dirw[g].abs()).sum()) for g, (a, b) in enumerate([(0, 40), (40, 40), (40, 65)]))
    assert abs(float((dx.double() * dirx).sum()) - fx) <= 64 * 2.0 ** -23 * Sx
    assert abs(float((dw.double() * dirw).sum()) - fw) <= 64 * 2.0 ** -23 * Sw


@pytest.mark.parametrize("bad", [[0, 40, 30, 60], [0, 20, 70, 60], [-5, 10, 30, 60], [0, 10, 1 << 40, 60], [0, -1, 30, 60]])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_offsets_are_reported(bad, dtype):
    a, w = values((60, 64), dtype, 1), values((3, 64, 64), dtype, 2)
    offsets = torch.tensor(bad, device="cuda")
    c = torch.zeros(60, 64, device="cuda")
    dg.gemm_grouped(a, w, c, offsets)
    assert dg.dg_sync_status() == dg.DG_ERR_VALUE
    assert dg.dg_sync_status() == dg.DG_OK
    dw = torch.zeros(3, 64, 64, device="cuda")
    dg.gemm_grouped_dw(a, a, dw, offsets)
    assert dg.dg_sync_status() == dg.DG_ERR_VALUE
    # the groups whose own rows are right are computed all the same
    for g in range(3):
        if 0 <= bad[g] <= bad[g + 1] <= 60:
            x = a[bad[g]:bad[g + 1]].double()
            check(dw[g], x.t() @ x, steps(60, a.dtype) * (x.abs().t() @ x.abs()), dw.dtype)


def test_streams_and_graphs():
    sizes, K, N = [100, 0, 300, 57], 256, 384
    a, w, d = values((457, K), "bf16", 1), values((4, N, K), "bf16", 2), values((457, N), "bf16", 3)
    offsets = offsets_of(sizes)

    def layer(out, dx, dw, stream=None):
        dg.gemm_grouped(a, w.transpose(1, 2), out, offsets, stream=stream)
        dg.gemm_grouped(d, w, dx, offsets, stream=stream)
        dg.gemm_grouped_dw(a, d, dw.transpose(1, 2), offsets, stream=stream)

    def outputs():
        return (torch.full((457, N), math.nan, device="cuda").bfloat16(), torch.full((457, K), math.nan, device="cuda").bfloat16(),
                torch.full((4, N, K), math.nan, device="cuda").bfloat16())

    want = outputs()
    layer(*want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [outputs() for _ in range(4)]
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        layer(*o, stream=streams[i % 2])
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(x, y) for x, y in zip(o, want))
    # captured, then replayed on other offsets: the sizes are read when the graph runs
    graphs = []
    for o in got[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            layer(*o)
        graphs.append(graph)
    offsets.copy_(offsets_of([57, 300, 100, 0]))
    layer(*want)
    torch.cuda.synchronize()
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for o in got[:2]:
        assert all(torch.equal(x, y) for x, y in zip(o, want))
    assert dg.dg_sync_status() == dg.DG_OK


def test_bounded_waits():
    a, w = values((60, 256), "bf16", 1), values((2, 256, 256), "bf16", 2)
    offsets, c = offsets_of([30, 30]), torch.empty(60, 256, device="cuda")
    dg.gemm_grouped(a, w, c, offsets)
    assert dg.dg_sync_status() == dg.DG_OK
    want = c.clone()
    dg.dg_set_option(dg.DG_OPT_WAIT_TIMEOUT_MS, 20)
    dg.dg_set_option(dg.DG_OPT_TEST_STALL, 1)
    try:
        dg.gemm_grouped(a, w, c, offsets)
        assert dg.dg_sync_status() == dg.DG_ERR_TIMEOUT
        dw = torch.empty(2, 256, 256, device="cuda")
        dg.gemm_grouped_dw(a, a, dw, offsets)
        assert dg.dg_sync_status() == dg.DG_ERR_TIMEOUT
    finally:
        dg.dg_set_option(dg.DG_OPT_TEST_STALL, 0)
        dg.dg_set_option(dg.DG_OPT_WAIT_TIMEOUT_MS, 2000)
    dg.gemm_grouped(a, w, c, offsets)
    assert dg.dg_sync_status() == dg.DG_OK and torch.equal(c, want)


def test_layers_of_a_block():
    """The experts of a block and a linear cross entropy behind them, forward and backward."""
    T, D, H, V, sizes = 300, 128, 256, 1000, [50, 0, 130, 120]
    x, up, down = values((T, D), "bf16", 1), values((4, H, D), "bf16", 2, D ** -0.5), values((4, D, H), "bf16", 3, H ** -0.5)
    head, target = values((V, D), "bf16", 4, D ** -0.5), torch.arange(T, device="cuda") % V
    offsets = offsets_of(sizes)
    h, y = torch.empty(T, H, device="cuda").bfloat16(), torch.empty(T, D, device="cuda").bfloat16()
    dg.gemm_grouped(x, up.transpose(1, 2), h, offsets, act="relu")
    dg.gemm_grouped(h, down.transpose(1, 2), y, offsets)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dg.linear_ce(y, head.t(), target, loss, lse)
    dy, dhead = torch.empty_like(y), torch.empty_like(head)
    dg.linear_ce_grad(y, head.t(), target, lse, torch.full((1,), 1 / T, device="cuda"), dy, dhead.t())
    dh, ddown = torch.empty_like(h), torch.empty_like(down)
    dg.gemm_grouped(dy, down, dh, offsets)
    dg.gemm_grouped_dw(h, dy, ddown.transpose(1, 2), offsets)
    dh.mul_(h > 0)
    dup = torch.empty_like(up)
    dg.gemm_grouped_dw(x, dh, dup.transpose(1, 2), offsets)
    assert dg.dg_sync_status() == dg.DG_OK
    leaves = [t.double().requires_grad_() for t in (up, down, head)]
    ends = offsets.tolist()
    out = torch.cat([torch.relu(x[a:b].double() @ leaves[0][g].t()) @ leaves[1][g].t() for g, (a, b) in enumerate(zip(ends, ends[1:]))])
    want = torch.nn.functional.cross_entropy(out @ leaves[2].t(), target)
    want.backward()
    # each of the five roundings to BF16 on the way is 2^-9 of its value; ten of them, in the norm
    assert abs(float(loss.mean()) - want.item()) <= 10 * 2.0 ** -9 * want.item()
    for got, leaf in zip((dup, ddown, dhead), leaves):
        assert float((got.double() - leaf.grad).norm()) <= 10 * 2.0 ** -9 * float(leaf.grad.norm())
