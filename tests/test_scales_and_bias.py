"""Host-only: scales and biases that a kernel would read past their end, or off their alignment, are refused by every
entry point that takes them.  Pointers are plain integers; each call returns before it would touch a device."""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

FAKE = 1 << 40


def mat(rows, cols, dtype="bf16", es=2):
    return dg.make_view(FAKE, (rows, cols), (cols * es, es), 1, dtype)


def call(name, scale_a=None, scale_b=None, bias=None):
    A, B, C = mat(16, 64), mat(64, 8), mat(16, 8)
    if name == "gemm":
        return dg.dg_gemm(A, B, C, 1.0, 0.0, scale_a, scale_b, 0)
    if name == "static":
        import ctypes

        return dg.lib.dg_gemm_static(ctypes.byref(A), ctypes.byref(B), ctypes.byref(C), 1.0, 0.0, scale_a, scale_b, None)
    if name == "autotune":
        return dg.dg_autotune(A, B, C, 1.0, 0.0, scale_a, scale_b, dg.epilogue(bias), 0)[0]
    return dg.dg_gemm_ex(A, B, C, 1.0, 0.0, scale_a, scale_b, dg.epilogue(bias), 0)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_alignment(off):
    for name in ("gemm", "static", "autotune", "gemm_ex"):
        assert call(name, scale_a=FAKE + off) == dg.DG_ERR_ALIGN
        assert call(name, scale_b=FAKE + off) == dg.DG_ERR_ALIGN
    for name in ("autotune", "gemm_ex"):
        assert call(name, bias=FAKE + off) == dg.DG_ERR_ALIGN
    W = dg.dg_w4()
    W.codes, W.scales, W.K, W.N, W.code_stride, W.scale_stride, W.group, W.scale_dtype = FAKE, FAKE, 64, 8, 32, 4, 32, dg.DG_BF16
    assert dg.dg_gemv_w4(mat(1, 64), W, mat(1, 8), 1.0, 0.0, dg.epilogue(FAKE + off), 0) == dg.DG_ERR_ALIGN


def bad(n):
    return [torch.zeros(n).bfloat16(), torch.zeros(n).double(), torch.zeros(n - 1), torch.zeros(2 * n)[::2], torch.zeros(1).expand(n)]


def test_binding():
    a, b = torch.zeros(16, 64).bfloat16(), torch.zeros(64, 8).bfloat16()
    for c in (torch.zeros(16, 8), mat(16, 8)):
        for t in bad(8):
            with pytest.raises(ValueError):
                dg.gemm(a, b, c, bias=t)
            with pytest.raises(ValueError):
                dg.gemm(a, b, c, scale_b=t)
        for t in bad(16):
            with pytest.raises(ValueError):
                dg.gemm(a, b, c, scale_a=t)
    # columns of several dims
    for t in bad(8):
        with pytest.raises(ValueError):
            dg.gemm(a, b, torch.zeros(16, 2, 4), bias=t)
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.ones(8, 2)
    for t in bad(8):
        with pytest.raises(ValueError):
            dg.gemv_w4(a[:1], codes, scales, torch.zeros(1, 8), group=32, bias=t)
