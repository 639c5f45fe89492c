"""Quantising and reading back more rows, or more k, than one grid has: second turns of the kernels' outer loops.

The row kernels take 65532 quarters of 32 rows, 2097024 rows; the kernels for any view 65535 times 32 k.
"""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_mx4 import quantised, read_codes, tile_index, values_of

pytestmark = pytest.mark.gpu


def values(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("odd", [False, True])
def test_rows(odd, block):
    border, K = 2097024, 40
    R = border + 333
    # odd: rows at every second multiple of 2 bytes, which go through shared memory
    x = values((R, K + 1), 1)[:, 1:] if odd else values((R, K), 1)
    codes, scales = dg.empty_mx4(R, K, block)
    codes.fill_(0xEE)
    scales.fill_(0xEE)
    dg.quantize_mx4(x, codes, scales, block=block)
    y = torch.full((R, K + 1), torch.nan, device="cuda").bfloat16()[:, 1:] if odd else torch.empty_like(x)
    dg.dequantize_mx4(codes, scales, y, block=block)
    assert dg.dg_sync_status() == dg.DG_OK
    n = -(-K // block)
    for r0, r1 in ((0, 200), (border - 128, border + 128), (R - 150, R)):
        want, s = quantised(x[r0:r1], block)
        assert torch.equal(read_codes(codes[r0:r1], K), want)
        at = tile_index(R, n)[r0:r1]
        assert torch.equal(scales.cpu()[at], s)
        first = r0 // 128  # whole tiles of scales from that of the first row on
        back = values_of(codes[first * 128:r1], scales[first * ((n + 3) // 4) * 512:], K, block)
        assert torch.equal(y[r0:r1], back[r0 - first * 128:].bfloat16())


@pytest.mark.parametrize("block", [16, 32])
def test_turned_k(block):
    border, R = 65535 * 32, 3
    K = border + 1000
    x = values((K, R), 2).t()
    codes, scales = dg.empty_mx4(R, K, block)
    dg.quantize_mx4(x, codes, scales, block=block)
    y = torch.full((K, R), torch.nan, device="cuda").bfloat16().t()
    dg.dequantize_mx4(codes, scales, y, block=block)
    assert dg.dg_sync_status() == dg.DG_OK
    at = tile_index(R, -(-K // block))
    for k0, k1 in ((0, 640), (border - 640, border + 640), (border + 640, K)):
        want, s = quantised(x[:, k0:k1], block)
        assert torch.equal(read_codes(codes, K)[:, k0:k1], want)
        s_at = at[:, k0 // block:-(-k1 // block)]
        assert torch.equal(scales.cpu()[s_at], s)
    assert torch.equal(y, values_of(codes, scales, K, block).bfloat16())
