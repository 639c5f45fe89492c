"""Host-only checks of the grouped products and the 4-bit floats: exports, refusals, sizes.  Pointers are plain
aligned integers; every call here returns before it would touch a device."""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

FAKE = 1 << 40


def mat(rows, cols, dtype="bf16", base=FAKE, es=2, rs=None, cs=None):
    return dg.make_view(base, (rows, cols), (cols * es if rs is None else rs, es if cs is None else cs), 1, dtype)


def stack(G, K, N, dtype="bf16", base=FAKE, es=2, strides=None, row_dims=2):
    return dg.make_view(base, (G, K, N), strides or (K * N * es, N * es, es), row_dims, dtype)


def rows(A=None, B=None, C=None, offsets=FAKE, groups=3, alpha=1.0, beta=0.0, sa=None, sb=None, epi=None):
    return dg.dg_gemm_grouped(A or mat(10, 64), B or stack(3, 64, 32), C or mat(10, 32), offsets, groups, alpha, beta, sa,
                              sb, epi, 0)


def by_k(X=None, dY=None, dW=None, offsets=FAKE, groups=3, alpha=1.0, beta=0.0):
    return dg.dg_gemm_grouped_dw(X or mat(10, 64), dY or mat(10, 32), dW or stack(3, 64, 32, "f32", es=4), offsets, groups,
                                 alpha, beta, 0)


def mx4(rows=16, K=64, block=32, codes=FAKE, scales=FAKE, stride=None, scale=None, reserved=0):
    q = dg.dg_mx4()
    q.codes, q.scales, q.scale, q.rows, q.K, q.block, q.reserved = codes, scales, scale, rows, K, block, reserved
    q.code_stride = max(16, (K + 31) // 32 * 16) if stride is None else stride
    return q


def gemm(A=None, B=None, C=None, alpha=1.0, beta=0.0, epi=None):
    return dg.dg_gemm_mx4(A or mx4(), B or mx4(8), C or mat(16, 8), alpha, beta, epi, 0)


def test_exports():
    for n in ("dg_gemm_grouped", "dg_gemm_grouped_dw", "dg_quantize_mx4", "dg_dequantize_mx4", "dg_gemm_mx4",
              "dg_mx4_scale_bytes"):
        assert hasattr(dg.lib, n)


@pytest.mark.parametrize("call", [rows, by_k])
def test_grouped_refusals(call):
    assert call(offsets=None) == dg.DG_ERR_NULL
    assert call(offsets=FAKE + 4) == dg.DG_ERR_ALIGN
    assert call(groups=-1) == dg.DG_ERR_SHAPE
    assert call(groups=2) == dg.DG_ERR_SHAPE
    assert call(alpha=math.nan) == dg.DG_ERR_VALUE
    assert call(beta=-math.inf) == dg.DG_ERR_VALUE


def test_rows_refusals():
    assert rows(A=mat(10, 63)) == dg.DG_ERR_SHAPE
    assert rows(C=mat(9, 32)) == dg.DG_ERR_SHAPE
    assert rows(C=mat(10, 31)) == dg.DG_ERR_SHAPE
    assert rows(B=stack(3, 64, 32, row_dims=1)) == dg.DG_ERR_NDIM
    assert rows(B=mat(3, 64 * 32)) == dg.DG_ERR_NDIM
    assert rows(B=stack(3, 64, 32, "f16")) == dg.DG_ERR_DTYPE
    assert rows(C=mat(10, 32, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert rows(C=mat(10, 32, rs=0)) == dg.DG_ERR_STRIDE
    assert rows(A=mat(10, 64, base=FAKE + 1)) == dg.DG_ERR_ALIGN
    assert rows(A=mat(10, 64, rs=-128)) == dg.DG_ERR_STRIDE
    assert rows(sa=FAKE + 2) == dg.DG_ERR_ALIGN
    assert rows(sb=FAKE + 1) == dg.DG_ERR_ALIGN
    assert rows(epi=dg.epilogue(FAKE + 3)) == dg.DG_ERR_ALIGN
    assert rows(epi=dg.epilogue(None, 9)) == dg.DG_ERR_VALUE
    assert rows(B=stack(1025, 64, 32), groups=1025) == dg.DG_ERR_UNSUPPORTED
    big = (1 << 31) - (1 << 13) + 1
    assert rows(A=mat(big, 64), C=mat(big, 32)) == dg.DG_ERR_UNSUPPORTED
    # nothing to do
    assert rows(A=mat(0, 64), C=mat(0, 32)) == dg.DG_OK
    assert rows(B=stack(3, 64, 0), C=mat(10, 0)) == dg.DG_OK
    assert rows(B=stack(0, 64, 32), groups=0, offsets=None) == dg.DG_OK


def test_dw_refusals():
    assert by_k(dY=mat(9, 32)) == dg.DG_ERR_SHAPE
    assert by_k(X=mat(10, 63)) == dg.DG_ERR_SHAPE
    assert by_k(dY=mat(10, 31)) == dg.DG_ERR_SHAPE
    assert by_k(dY=mat(10, 32, "f16")) == dg.DG_ERR_DTYPE
    assert by_k(dW=stack(3, 64, 32, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert by_k(dW=stack(3, 64, 32, "f32", es=4, strides=(0, 128, 4))) == dg.DG_ERR_STRIDE
    assert by_k(dW=stack(3, 64, 32, "f32", es=4, row_dims=1)) == dg.DG_ERR_NDIM
    assert by_k(dW=mat(192, 32, "f32", es=4)) == dg.DG_ERR_NDIM
    assert by_k(dW=stack(0, 64, 32, "f32", es=4), groups=0, offsets=None) == dg.DG_OK
    assert by_k(X=mat(10, 0), dW=stack(3, 0, 32, "f32", es=4)) == dg.DG_OK


def test_scale_bytes():
    assert dg.dg_mx4_scale_bytes(1, 1, 32) == 512
    assert dg.dg_mx4_scale_bytes(128, 128, 32) == 512
    assert dg.dg_mx4_scale_bytes(129, 128, 32) == 1024
    assert dg.dg_mx4_scale_bytes(128, 129, 32) == 1024
    assert dg.dg_mx4_scale_bytes(128, 129, 16) == 1536
    assert dg.dg_mx4_scale_bytes(0, 64, 16) == dg.dg_mx4_scale_bytes(64, 0, 16) == 0
    for bad in ((-1, 64, 32), (64, -1, 32), (64, 64, 8), (64, 64, 0), (1 << 31, 64, 32)):
        assert dg.dg_mx4_scale_bytes(*bad) == -1


@pytest.mark.parametrize("call", [lambda x, q: dg.dg_quantize_mx4(x, q, 0), lambda x, q: dg.dg_dequantize_mx4(q, x, 0)])
def test_quantise_refusals(call):
    x = mat(16, 64)
    for block in (0, 8, 31, 64, -32):
        assert call(x, mx4(block=block)) == dg.DG_ERR_VALUE
    assert call(x, mx4(reserved=1)) == dg.DG_ERR_VALUE
    assert call(x, mx4(K=63)) == dg.DG_ERR_SHAPE
    assert call(x, mx4(15)) == dg.DG_ERR_SHAPE
    assert call(x, mx4(-1)) == dg.DG_ERR_SHAPE
    assert call(x, mx4(codes=None)) == dg.DG_ERR_NULL
    assert call(x, mx4(scales=None)) == dg.DG_ERR_NULL
    assert call(x, mx4(scales=FAKE + 8)) == dg.DG_ERR_ALIGN
    assert call(x, mx4(scale=FAKE + 2)) == dg.DG_ERR_ALIGN
    assert call(x, mx4(stride=-16)) == dg.DG_ERR_STRIDE
    assert call(x, mx4(stride=1 << 62)) == dg.DG_ERR_STRIDE
    assert call(mat(16, 64, "e4m3", es=1), mx4()) == dg.DG_ERR_DTYPE
    assert call(mat(16, 64, base=FAKE + 1), mx4()) == dg.DG_ERR_ALIGN
    assert call(mat(0, 64), mx4(0)) == dg.DG_OK
    assert call(mat(16, 0), mx4(K=0)) == dg.DG_OK


def test_codes_that_overlap():
    assert dg.dg_quantize_mx4(mat(16, 64), mx4(stride=31), 0) == dg.DG_ERR_STRIDE
    assert dg.dg_dequantize_mx4(mx4(), mat(16, 64, rs=0), 0) == dg.DG_ERR_STRIDE


def test_product_refusals():
    assert gemm(A=mx4(block=16)) == dg.DG_ERR_VALUE
    assert gemm(A=mx4(K=128)) == dg.DG_ERR_SHAPE
    assert gemm(C=mat(15, 8)) == dg.DG_ERR_SHAPE
    assert gemm(C=mat(16, 9)) == dg.DG_ERR_SHAPE
    assert gemm(C=mat(16, 8, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert gemm(C=mat(16, 8, rs=0)) == dg.DG_ERR_STRIDE
    assert gemm(alpha=math.inf) == dg.DG_ERR_VALUE
    assert gemm(epi=dg.epilogue(None, -1)) == dg.DG_ERR_VALUE
    assert gemm(A=mx4(codes=FAKE + 8)) == dg.DG_ERR_ALIGN
    assert gemm(B=mx4(8, stride=40)) == dg.DG_ERR_ALIGN
    assert gemm(B=mx4(8, stride=0)) == dg.DG_ERR_UNSUPPORTED
    assert gemm(C=dg.make_view(FAKE, (4, 4, 8), (200, 48, 2), 2, "bf16")) == dg.DG_ERR_UNSUPPORTED
    assert gemm(A=mx4(0), C=mat(0, 8)) == dg.DG_OK
    assert gemm(B=mx4(0), C=mat(16, 0)) == dg.DG_OK


def test_binding_refusals():
    x, w, c = torch.zeros(4, 8).bfloat16(), torch.zeros(2, 8, 6).bfloat16(), torch.zeros(4, 6)
    offsets = torch.tensor([0, 1, 4])
    with pytest.raises(ValueError):
        dg.gemm_grouped(x, w, c, offsets.int())
    with pytest.raises(ValueError):
        dg.gemm_grouped(x, w, c, offsets[:2])
    with pytest.raises(ValueError):
        dg.gemm_grouped(x, w, c, torch.tensor([0, 0, 1, 1, 4, 4])[::2])
    with pytest.raises(ValueError):
        dg.gemm_grouped(x, w, c, offsets, scale_a=torch.zeros(3))
    with pytest.raises(ValueError):
        dg.gemm_grouped(x, w, c, offsets, scale_b=torch.zeros(6))
    with pytest.raises(ValueError):
        dg.gemm_grouped(x, w, c, offsets, bias=torch.zeros(2, 6).double())
    with pytest.raises(ValueError):
        dg.gemm_grouped_dw(x, c.bfloat16(), w[0], offsets)
    codes, scales = torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    assert dg.mx4(codes, scales).K == 32 and dg.mx4(codes, scales, K=31).K == 31
    with pytest.raises(TypeError):
        dg.mx4(codes.int(), scales)
    with pytest.raises(ValueError):
        dg.mx4(codes, scales, K=29)
    with pytest.raises(ValueError):
        dg.mx4(codes, scales[:256])
    with pytest.raises(ValueError):
        dg.mx4(codes, scales, block=8)
    with pytest.raises(ValueError):
        dg.mx4(codes.t(), scales)
    with pytest.raises(ValueError):
        dg.mx4(codes, scales, scale=torch.zeros(2))
    c, s = dg.empty_mx4(5, 100, 16, device="cpu")
    assert c.shape == (5, 50) and c.stride(0) % 16 == 0 and s.numel() == dg.dg_mx4_scale_bytes(5, 100, 16)
