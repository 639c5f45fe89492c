"""Long sums of dg_gemm_mx4 in each of its forms (CTAs, pairs of them, clusters that share k).

The tensor core truncates as it adds, at most 2^-23 of the running sum in each step of 64 k, and the alignment of the
products to the sum costs no more than 32 times that over a whole accumulator: an accumulator of 16384 is at most
(32 + 256) 2^-23 low, and adding the pieces up rounds to nearest.
"""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

pytestmark = pytest.mark.gpu

# M, N: pairs, CTAs, clusters
FORMS = {"pairs": (512, 2048), "ctas": (100, 9000), "clusters": (8, 256)}


def operand(R, K, block, seed, mask, scales):
    """Random codes under `mask`, random scales out of `scales`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes, _ = dg.empty_mx4(R, K, block)
    codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8) & mask)
    if K % 2:
        codes[:, -1] &= 15
    at = torch.randint(0, len(scales), (dg.dg_mx4_scale_bytes(R, K, block),), generator=g, device="cuda", dtype=torch.uint8)
    return codes, torch.tensor(scales, device="cuda", dtype=torch.uint8)[at.long()]


def first_rows(q, rows, K, block):
    """The values of the first rows (128 at most), in FP64: a code under its scale is exact in FP32."""
    y = torch.empty(min(rows, q[0].shape[0]), K, device="cuda")
    n = dg.dg_mx4_scale_bytes(len(y), K, block)
    return dg.dequantize_mx4(q[0][:len(y)], q[1][:n], y, block=block).double()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("form", FORMS)
def test_long_sums(form, block):
    (M, N), K = FORMS[form], 262144
    scales = list(range(40, 73)) if block == 16 else list(range(123, 131))
    a, b = operand(M, K, block, 1, 0x77, scales), operand(N, K, block, 2, 0x77, scales)
    c = torch.empty(M, N, device="cuda")
    dg.gemm_mx4(dg.mx4(*a, K=K, block=block), dg.mx4(*b, K=K, block=block), c)
    assert dg.dg_sync_status() == dg.DG_OK
    want = first_rows(a, 64, K, block) @ first_rows(b, 128, K, block).t()
    got = c[:64, :128].double()
    err = (got - want) / want
    assert float(err.abs().max()) <= (32 + 256) * 2.0 ** -23 + 16 * 2.0 ** -24, float(err.mean())


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("K", [16384 + 2, 3 * 16384 - 31, 8 * 16384 + 33, 9 * 16384])
@pytest.mark.parametrize("form", FORMS)
def test_pieces_and_their_epilogue(form, K, block):
    """Sums that are exact in FP32 (multiples of 1 / 16 below 2^19): pieces of every length, beta, bias and activation once."""
    M, N = FORMS[form]
    scales = [0x30, 0x38, 0x40] if block == 16 else [126, 127, 128]  # 1/2, 1, 2
    a, b = operand(M, K, block, 3, 0xFF, scales), operand(N, K, block, 4, 0xFF, scales)
    c = torch.randint(-50, 51, (M, N), device="cuda").float()
    bias = torch.randint(-50, 51, (N,), device="cuda").float()
    want = 0.5 * (first_rows(a, 64, K, block) @ first_rows(b, 128, K, block).t())
    m, n = want.shape
    want = (want - 2 * c[:m, :n].double() + bias[:n].double()).clamp(min=0)
    dg.gemm_mx4(dg.mx4(*a, K=K, block=block), dg.mx4(*b, K=K, block=block), c, alpha=0.5, beta=-2.0, bias=bias, act="relu")
    assert dg.dg_sync_status() == dg.DG_OK
    assert torch.equal(c[:m, :n].double(), want)
