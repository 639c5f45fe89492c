"""Long sums of dg_gemm_grouped and dg_gemm_grouped_dw, whatever the type of their outputs.

The tensor core truncates when it adds to an accumulator.  A step of 16 products loses at most 2^-23 of the running sum,
and its products' alignments no more than 32 times that over the whole sum (the bound of test_gpu_grouped.py), so an
accumulator of 2048 products is at most (32 + 128) 2^-23 low.  Sums of positive products show it: every step errs to the
same side, and one accumulator of 65536 would lose 32 times as much.  The rounding to 16 bits is to nearest: over n values
spread through a binade its mean is 0, with a deviation of eps / 2 / sqrt(3 n), of which six are allowed.
"""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PART = (32 + 128) * 2.0 ** -23


def positive(shape, dtype, seed, spread=None):
    """Magnitudes of normal values; rows, or columns (spread = 0, 1), times factors in [1, 2)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda").abs()
    if spread is not None:
        x = x * (1 + torch.rand([n if d == spread else 1 for d, n in enumerate(shape)], generator=g, device="cuda"))
    return x.to(dtype)


def check_mean(got, want):
    err = float(((got.double() - want) / want).mean())
    rounding = 0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2 / (3 * got.numel()) ** 0.5
    assert abs(err) <= PART + 2.0 ** -23 + 6 * rounding, err


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("weight", ["nk", "kn"])
def test_rows_long_sums(dtype, out, weight):
    K, sizes = 65536, [200, 0, 57]
    x = positive((257, K), DT[dtype], 1, 0)
    w = positive((3, 300, K) if weight == "nk" else (3, K, 304), DT[dtype], 2)
    w = w.transpose(1, 2) if weight == "nk" else w
    c = torch.empty(257, w.shape[2], device="cuda", dtype=DT[out])
    dg.gemm_grouped(x, w, c, torch.tensor([0] + sizes, device="cuda").cumsum(0), alpha=2.0 ** -8)
    assert dg.dg_sync_status() == dg.DG_OK
    for r, g in ((slice(0, 200), 0), (slice(200, 257), 2)):
        check_mean(c[r], 2.0 ** -8 * (x[r].double() @ w[g].double()))


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dw_long_sums(dtype, out):
    sizes = [65536, 100]
    x, dy = positive((65636, 200), DT[dtype], 3, 1), positive((65636, 256), DT[dtype], 4)
    dw = torch.empty(2, 200, 256, device="cuda", dtype=DT[out])
    dg.gemm_grouped_dw(x, dy, dw, torch.tensor([0] + sizes, device="cuda").cumsum(0), alpha=2.0 ** -8)
    assert dg.dg_sync_status() == dg.DG_OK
    for r, g in ((slice(0, 65536), 0), (slice(65536, 65636), 1)):
        check_mean(dw[g], 2.0 ** -8 * (x[r].double().t() @ dy[r].double()))


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_sums_of_one_part_and_of_several_in_turn(out):
    """Each pair of CTAs takes several tiles, of sums of every number of parts."""
    sizes = [100, 5000, 0, 2048, 2049, 9000, 3, 4096, 1, 6145]
    R, K, N = sum(sizes), 512, 2048
    x, dy = torch.randn(R, K, device="cuda").bfloat16(), torch.randn(R, N, device="cuda").bfloat16()
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0)
    dw = torch.full((len(sizes), K, N), torch.nan, device="cuda", dtype=DT[out])
    dg.gemm_grouped_dw(x, dy, dw, offsets)
    again = torch.full_like(dw, torch.nan)
    dg.gemm_grouped_dw(x, dy, again, offsets)
    assert dg.dg_sync_status() == dg.DG_OK and torch.equal(dw, again)
    ends = offsets.tolist()
    for g in range(len(sizes)):
        a, b = x[ends[g]:ends[g + 1]].double(), dy[ends[g]:ends[g + 1]].double()
        want, S = a.t() @ b, a.abs().t() @ b.abs()
        tol = PART * S + 2.0 ** -22 * want.abs()
        tol = tol + torch.finfo(dw.dtype).eps / 2 * (want.abs() + tol)
        assert bool(((dw[g].double() - want).abs() <= tol).all()), g


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weight", ["nk", "kn"])
def test_rows_long_sums_of_e4m3(out, weight):
    """Parts of 4096: as many steps, of 32 products each."""
    K, sizes = 65536, [200, 0, 57]
    x = positive((257, K), torch.float8_e4m3fn, 1, 0)
    w = positive((3, 300, K) if weight == "nk" else (3, K, 304), torch.float8_e4m3fn, 2)
    w = w.transpose(1, 2) if weight == "nk" else w
    c = torch.empty(257, w.shape[2], device="cuda", dtype=DT[out])
    dg.gemm_grouped(x, w, c, torch.tensor([0] + sizes, device="cuda").cumsum(0), alpha=2.0 ** -8)
    assert dg.dg_sync_status() == dg.DG_OK
    for r, g in ((slice(0, 200), 0), (slice(200, 257), 2)):
        check_mean(c[r], 2.0 ** -8 * (x[r].double() @ w[g].double()))
