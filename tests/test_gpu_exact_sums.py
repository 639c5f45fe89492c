"""Products whose sums are exact in FP32, compared for equality: a block of k that is lost or counted twice, a scale of the
wrong block or a sum of fewer bits cannot hide in a tolerance.

4-bit: codes under scales of 1/2, 1 and 2 are multiples of 1/4, their products multiples of 1/16; a sum of k random ones
stays far below 2^20 at the k used here.  E4M3 and BF16: integers up to 8 and 15, sums below 2^24.
"""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_mx4_sums import operand

pytestmark = pytest.mark.gpu

# M, N by the form that a long k takes: pairs of CTAs, single CTAs, clusters that share k; whole and partial tiles
FORMS = {"pairs": (512, 2048), "pairs-odd": (777, 2100), "ctas": (100, 9000), "clusters": (8, 256), "clusters-odd": (33, 300),
         "one": (1, 4096)}


def values(q, K, block):
    y = torch.empty(q[0].shape[0], K, device="cuda")
    return dg.dequantize_mx4(*q, y, block=block).double()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("K", [1, 64, 100, 255, 1000, 2049, 4096, 14336, 16384])
@pytest.mark.parametrize("form", FORMS)
def test_mx4(form, K, block):
    M, N = FORMS[form]
    scales = [0x30, 0x38, 0x40] if block == 16 else [126, 127, 128]
    a, b = operand(M, K, block, K, 0xFF, scales), operand(N, K, block, K + 1, 0xFF, scales)
    c = torch.full((M, N), torch.nan, device="cuda")
    dg.gemm_mx4(dg.mx4(*a, K=K, block=block), dg.mx4(*b, K=K, block=block), c)
    assert dg.dg_sync_status() == dg.DG_OK
    assert torch.equal(c.double(), values(a, K, block) @ values(b, K, block).t())


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.bfloat16])
@pytest.mark.parametrize("weight", ["nk", "kn"])
@pytest.mark.parametrize("K", [16, 272, 4096, 4112, 14336])
def test_grouped(K, weight, dtype):
    g = torch.Generator(device="cuda").manual_seed(K)
    most, sizes, N = 8 if dtype == torch.float8_e4m3fn else 15, [300, 0, 33, 1, 90], 400
    x = torch.randint(-most, most + 1, (sum(sizes), K), generator=g, device="cuda").to(dtype)
    w = torch.randint(-most, most + 1, (5, N, K) if weight == "nk" else (5, K, N), generator=g, device="cuda").to(dtype)
    w = w.transpose(1, 2) if weight == "nk" else w
    c = torch.full((sum(sizes), N), torch.nan, device="cuda")
    ends = torch.tensor([0] + sizes).cumsum(0)
    dg.gemm_grouped(x, w, c, ends.cuda())
    assert dg.dg_sync_status() == dg.DG_OK
    for i, (r0, r1) in enumerate(zip(ends.tolist(), ends.tolist()[1:])):
        assert torch.equal(c[r0:r1].double(), x[r0:r1].double() @ w[i].double()), i


def test_grouped_dw():
    g = torch.Generator(device="cuda").manual_seed(1)
    sizes, K, N = [5000, 0, 33, 1, 2048, 2100], 264, 400
    x = torch.randint(-15, 16, (sum(sizes), K), generator=g, device="cuda").bfloat16()
    dy = torch.randint(-15, 16, (sum(sizes), N), generator=g, device="cuda").bfloat16()
    dw = torch.full((len(sizes), K, N), torch.nan, device="cuda")
    ends = torch.tensor([0] + sizes).cumsum(0)
    dg.gemm_grouped_dw(x, dy, dw, ends.cuda())
    assert dg.dg_sync_status() == dg.DG_OK
    for i, (r0, r1) in enumerate(zip(ends.tolist(), ends.tolist()[1:])):
        assert torch.equal(dw[i].double(), x[r0:r1].double().t() @ dy[r0:r1].double()), i


@pytest.mark.parametrize("weight", ["nk", "kn"])
def test_long_e4m3_sums_keep_their_precision(weight):
    """Normal values: 128 steps of an accumulator cut at most 2^-24 of the sum each, in the norm over many sums."""
    K = 14336
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(200, K, generator=g, device="cuda").to(torch.float8_e4m3fn)
    w = torch.randn((1, 304, K) if weight == "nk" else (1, K, 304), generator=g, device="cuda").to(torch.float8_e4m3fn)
    w = w.transpose(1, 2) if weight == "nk" else w
    c = torch.empty(200, 304, device="cuda")
    dg.gemm_grouped(x, w, c, torch.tensor([0, 200], device="cuda"))
    want = x.double() @ w[0].double()
    assert float((c.double() - want).norm() / want.norm()) <= 128 * 2.0 ** -24


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("form", FORMS)
def test_long_mx4_sums_keep_their_precision(form, block):
    """Scales spread over some binades: 256 steps of an accumulator of 16384, as above."""
    (M, N), K = FORMS[form], 14336
    scales = list(range(40, 73)) if block == 16 else list(range(123, 131))
    a, b = operand(M, K, block, 1, 0xFF, scales), operand(N, K, block, 2, 0xFF, scales)
    c = torch.empty(M, N, device="cuda")
    dg.gemm_mx4(dg.mx4(*a, K=K, block=block), dg.mx4(*b, K=K, block=block), c)
    want = values(a, K, block) @ values(b, K, block).t()
    assert float((c.double() - want).norm() / want.norm()) <= 256 * 2.0 ** -24
