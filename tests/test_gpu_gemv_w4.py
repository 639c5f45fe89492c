"""dg_gemv_w4 against its definition in FP64.

y = act(alpha * x W + beta * y + bias), W[k][n] = scale[n][k / group] *
(code[n][k] - zero[n][k / group]), at the sizes, layouts and values where a
kernel can go wrong: one k and one column, groups and rows that end inside a
tile, codes at any byte, strides of x and y, NaN and infinity.

Tolerance.  With S = |alpha| sum_k |x| |w|, the FP32 sum of one output passes a
product through at most 32 + K / 32 roundings (16 products per tensor-core
step, the steps of a warp's share of k, the groups' sums, the warps and the
cluster), each at most 2^-23 of the running magnitude (a tensor core may
truncate): (32 + K / 32) 2^-23 S.  Adding beta * y and the bias rounds three
more times, at most 2^-22 (|z| + |beta y| + |bias|).  GeLU's slope is below 1.13
and its own error is 2^-20 |z| (FP32 outputs) or 2^-11 |z| (16-bit outputs, the
hardware's tanh).  The store rounds by half a step, eps / 2 of the value
(F16: or half of its smallest subnormal, 2^-25).
"""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def weights(K, N, group, scale="bf16", zeros=False, seed=0, pad=(0, 0, 0), offset=0):
    """Random codes, scales and zeros on the GPU, with `pad` bytes/elements behind each row and the codes
    `offset` bytes past an aligned address.  Bytes of the padding, and an odd K's last high nibble, are 0xFF."""
    g = torch.Generator().manual_seed(seed + 7919 * K + N)
    nb, groups = (K + 1) // 2, -(-K // group)
    codes = torch.randint(0, 256, (N, nb), generator=g, dtype=torch.uint8)
    if K % 2:
        codes[:, -1] |= 0xF0
    flat = torch.full((offset + N * (nb + pad[0]) + 16,), 0xFF, dtype=torch.uint8, device="cuda")
    c = torch.as_strided(flat, (N, nb), (nb + pad[0], 1), offset)
    c.copy_(codes)
    s = torch.as_strided(torch.full((N * (groups + pad[1]) + 1,), math.nan, dtype=DT[scale], device="cuda"),
                         (N, groups), (groups + pad[1], 1))
    s.copy_((torch.rand(N, groups, generator=g) + 0.25) * torch.where(torch.rand(N, groups, generator=g) < 0.3, -1, 1))
    z = None
    if zeros:
        z = torch.as_strided(torch.full((N * (groups + pad[2]) + 1,), 0xFF, dtype=torch.uint8, device="cuda"),
                             (N, groups), (groups + pad[2], 1))
        z.copy_(torch.randint(0, 16, (N, groups), generator=g, dtype=torch.uint8))
    return c, s, z


def dense(codes, scales, zeros, group, K):
    """W [K x N] in FP64."""
    k = torch.arange(K, device="cuda")
    q = (codes[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
    z = 8 if zeros is None else (zeros[:, k // group].int() & 15)
    return ((q - z).double() * scales[:, k // group].double()).t()


ACT = {"none": lambda z: z, "relu": lambda z: z.clamp(min=0),
       "gelu_tanh": lambda z: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))}


def expected(x, W, y0, alpha, beta, bias, act):
    """(value, tolerance before the store)."""
    xd = x.double().reshape(-1, x.shape[-1])
    K = W.shape[0]
    S = abs(alpha) * (xd.abs() @ W.abs())
    by = beta * y0.double().reshape(xd.shape[0], -1) if beta else torch.zeros_like(S)
    b = torch.zeros_like(S) if bias is None else bias.double().expand_as(S)
    z = alpha * (xd @ W) + by + b
    tol = (32 + K / 32) * 2.0 ** -23 * S + 2.0 ** -22 * (z.abs() + by.abs() + b.abs())
    if act == "gelu_tanh":
        tol = 1.13 * tol + (2.0 ** -20 if y0.dtype == torch.float32 else 2.0 ** -11) * z.abs()
    return ACT[act](z), tol


def check(y, want, tol):
    got = y.double().reshape(want.shape)
    assert torch.equal(got.isnan(), want.isnan())
    ok = ~want.isnan()
    inf = want.isinf()
    assert torch.equal(got[inf & ok], want[inf & ok])
    ok &= ~inf
    tol = tol + torch.finfo(y.dtype).eps / 2 * (want.abs() + tol) + (2.0 ** -25 if y.dtype == torch.float16 else 0)
    err = (got - want).abs()
    assert bool((err[ok] <= tol[ok]).all()), float((err[ok] - tol[ok]).max())


def run_case(R, K, N, group, dtype="bf16", scale="bf16", zeros=False, out="bf16", alpha=1.0, beta=0.0, act="none",
             bias=False, pad=(0, 0, 0), offset=0, x=None, y=None):
    g = torch.Generator().manual_seed(R * 1000003 + K * 31 + N)
    codes, scales, zs = weights(K, N, group, scale, zeros, pad=pad, offset=offset)
    if x is None:
        x = torch.randn(R, K, generator=g).to(DT[dtype]).cuda()
    if y is None:
        y = torch.randn(R, N, generator=g).to(DT[out]).cuda() if beta else torch.full((R, N), math.nan, dtype=DT[out],
                                                                                      device="cuda")
    b = torch.randn(N, generator=g).cuda() if bias else None
    want, tol = expected(x, dense(codes, scales, zs, group, K), y.clone(), alpha, beta, b, act)
    before = dg.dg_launch_count()
    dg.gemv_w4(x, codes, scales, y, zeros=zs, group=group, alpha=alpha, beta=beta, bias=b, act=act)
    assert dg.dg_launch_count() > before
    assert dg.dg_sync_status() == dg.DG_OK
    check(y, want, tol)
    return y


@pytest.mark.parametrize("R", range(1, 9))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_row_count(R, dtype):
    run_case(R, 640, 200, 128, dtype, zeros=True, out=dtype)


@pytest.mark.parametrize("K", [1, 2, 31, 32, 33, 63, 65, 100, 127, 128, 129, 255, 1000, 1024, 4097, 5000])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 384])
def test_sizes_of_k_and_group(K, group):
    run_case(3, K, 37, group, "f16", "f32", zeros=group % 64 == 0, out="f32")


@pytest.mark.parametrize("N", [1, 2, 7, 8, 15, 16, 17, 31, 33, 127, 1001])
@pytest.mark.parametrize("R", [1, 8])
def test_sizes_of_n(N, R):
    run_case(R, 288, N, 32, "bf16", "f16", zeros=True, out="f32")


@pytest.mark.parametrize("pad,offset", [((0, 0, 0), 1), ((3, 1, 2), 0), ((16, 5, 7), 4), ((12, 0, 1), 8),
                                        ((5, 2, 0), 3), ((0, 0, 0), 16)])
@pytest.mark.parametrize("K,group", [(256, 128), (1000, 64), (77, 32)])
def test_strides_and_alignment_of_the_weights(pad, offset, K, group):
    for R in (1, 5):
        run_case(R, K, 50, group, "bf16", "bf16", zeros=True, out="f32", pad=pad, offset=offset)


@pytest.mark.parametrize("K,N,R", [(4096, 1024, 1), (14336, 256, 8), (16384, 64, 2), (20000, 48, 4), (512, 4096, 1),
                                   (70000, 16, 8)])
@pytest.mark.parametrize("group", [32, 128, 1 << 20])
def test_long_k_and_wide_n(K, N, R, group):
    run_case(R, K, N, group, "bf16", "f32", zeros=True, out="f32")


@pytest.mark.parametrize("act", ["none", "relu", "gelu_tanh"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_epilogue(act, out):
    run_case(4, 512, 300, 64, "f16", "f16", out=out, alpha=0.125, beta=-0.5, act=act, bias=True)
    run_case(4, 512, 300, 128, "f16", "f16", zeros=True, out=out, alpha=-1.5, act=act, bias=True)


def test_alpha_zero_and_empty():
    y = torch.full((2, 5), 3.0, device="cuda")
    codes, scales, _ = weights(64, 5, 32)
    x = torch.full((2, 64), math.nan, device="cuda", dtype=torch.bfloat16)
    dg.gemv_w4(x, codes, scales, y, group=32, alpha=0.0, beta=2.0)
    assert torch.equal(y, torch.full_like(y, 6.0))
    dg.gemv_w4(x[:, :0], codes[:, :0], scales[:, :0], y, group=32, beta=0.0)  # K = 0
    assert torch.equal(y, torch.zeros_like(y))
    dg.gemv_w4(x[:0], codes, scales, y[:0], group=32)                         # no rows
    dg.gemv_w4(x, codes[:0], scales[:0], y[:, :0], group=32)                  # no columns


@pytest.mark.parametrize("group", [32, 128])
def test_views_of_x_and_y(group):
    K, N = 512, 96
    g = torch.Generator().manual_seed(5)
    base = torch.randn(K, 4, generator=g).bfloat16().cuda()
    run_case(4, K, N, group, x=base.t(), out="f32")                            # k strided
    wide = torch.randn(4, 3 * K, generator=g).bfloat16().cuda()
    run_case(4, K, N, group, x=wide[:, 1:K + 1], out="f32")                    # odd start
    run_case(4, K, N, group, x=wide[:, ::3][:, :K], out="f32")                 # every third element
    run_case(3, K, N, group, x=wide[:1, :K].expand(3, K), out="f32")           # one row for all
    yt = torch.full((N, 4), math.nan, device="cuda")
    run_case(4, K, N, group, x=base.t(), y=yt.t())                             # transposed output
    behind = torch.full((6, N + 3), -7.0, device="cuda")
    run_case(4, K, N, group, x=base.t(), y=behind[:4, 2:N + 2])
    assert bool((behind[4:] == -7).all() and (behind[:, :2] == -7).all() and (behind[:, N + 2:] == -7).all())


def test_one_dimensional_x_and_y():
    x = torch.randn(256, device="cuda").half()
    codes, scales, _ = weights(256, 40, 128)
    y = torch.empty(40, device="cuda")
    dg.gemv_w4(x, codes, scales, y)
    want, tol = expected(x, dense(codes, scales, None, 128, 256), y, 1.0, 0.0, None, "none")
    check(y, want, tol)


def test_shared_column():
    # a code stride of 0: every column reads the same codes, under its own scale
    K, N = 384, 64
    codes, scales, _ = weights(K, N, 128)
    one = codes[:1].expand(N, K // 2)
    x = torch.randn(2, K, device="cuda").bfloat16()
    y = torch.empty(2, N, device="cuda")
    dg.gemv_w4(x, one, scales, y)
    want, tol = expected(x, dense(one, scales, None, 128, K), y, 1.0, 0.0, None, "none")
    check(y, want, tol)


@pytest.mark.parametrize("group", [32, 128])
def test_nan_and_infinity_stay_where_they_belong(group):
    K, N, R = 1024, 80, 8
    codes, scales, zeros = weights(K, N, group, "f32", True)
    x = torch.randn(R, K, device="cuda").bfloat16()
    x[2, 77] = math.inf
    x[5, 1023] = math.nan
    scales[11, 0] = math.nan
    scales[12, -1] = math.inf
    y = torch.empty(R, N, device="cuda")
    dg.gemv_w4(x, codes, scales, y, zeros=zeros, group=group)
    k = torch.arange(K, device="cuda")
    q = ((codes[:, k // 2].int() >> (4 * (k % 2)).int()) & 15) - zeros[:, k // group].int()
    # the definition: group sums of x (code - zero), times the scale
    groups = -(-K // group)
    part = (x.double()[:, None, :] * q.double()[None]).view(R, N, groups, group).sum(3)
    want = (part * scales.double()[None]).sum(2)
    finite = want.isfinite()
    got = y.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got[want.isinf()], want[want.isinf()])
    assert bool(((got - want).abs()[finite] <= 1e-3).all())
    assert bool(finite[[0, 1, 3, 4, 6, 7]][:, :11].all()) and not bool(finite[2].any()) and not bool(finite[5].any())


def test_runs_are_bit_identical():
    args = (2, 8192, 512, 128)
    a = run_case(*args, zeros=True, out="f32")
    for _ in range(3):
        assert torch.equal(a, run_case(*args, zeros=True, out="f32"))


def test_streams_and_graph():
    K, N = 2048, 768
    codes, scales, zeros = weights(K, N, 64, "f32", True)
    W = dense(codes, scales, zeros, 64, K)
    xs = [torch.randn(r, K, device="cuda").half() for r in (1, 8)]
    ys = [torch.empty(r, N, device="cuda") for r in (1, 8)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for x, y, s in zip(xs, ys, streams):
            dg.gemv_w4(x, codes, scales, y, zeros=zeros, group=64, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        check(y, *expected(x, W, y, 1.0, 0.0, None, "none"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for x, y in zip(xs, ys):
            dg.gemv_w4(x, codes, scales, y, zeros=zeros, group=64)
    for x, y in zip(xs, ys):
        x.copy_(torch.randn_like(x))
        y.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(xs, ys):
        check(y, *expected(x, W, y, 1.0, 0.0, None, "none"))


def test_codes_past_four_gigabytes():
    # rows of codes 2^26 bytes apart: the last one starts past byte offset 2^32
    K, N = 4096, 70
    flat = torch.empty((N << 26), dtype=torch.uint8, device="cuda")
    codes = torch.as_strided(flat, (N, K // 2), (1 << 26, 1))
    small, scales, _ = weights(K, N, 128, "f32")
    codes.copy_(small)
    x = torch.randn(1, K, device="cuda").bfloat16()
    y = torch.empty(1, N, device="cuda")
    dg.gemv_w4(x, codes, scales, y)
    check(y, *expected(x, dense(small, scales, None, 128, K), y, 1.0, 0.0, None, "none"))
