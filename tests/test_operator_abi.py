"""Host-only checks of dg_gemv_w4, dg_linear_ce and dg_linear_ce_grad: exports,
refusals in the order the header gives, workspace sizes.  Pointers are plain
aligned integers; every call here returns before it would touch a device."""
import ctypes
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

FAKE = 1 << 40


def mat(rows, cols, dtype="bf16", base=FAKE, es=2, rs=None, cs=None):
    return dg.make_view(base, (rows, cols), (cols * es if rs is None else rs, es if cs is None else cs), 1, dtype)


def w4(K=256, N=64, group=128, scale_dtype=dg.DG_BF16, zeros=None, **kw):
    w = dg.dg_w4()
    w.codes, w.scales, w.zeros = FAKE, FAKE, zeros
    w.K, w.N, w.group, w.scale_dtype = K, N, group, scale_dtype
    w.code_stride, w.scale_stride, w.zero_stride = (K + 1) // 2, 2 * (-(-K // group) if group > 0 else 1), 4
    for k, v in kw.items():
        if k == "reserved":
            w.reserved[1] = v
        else:
            setattr(w, k, v)
    return w


def gemv(x=None, W=None, y=None, alpha=1.0, beta=0.0, epi=None):
    x = mat(2, 256) if x is None else x
    y = mat(2, 64, "f32", es=4) if y is None else y
    return dg.dg_gemv_w4(x, w4() if W is None else W, y, alpha, beta, epi, 0)


def test_exports():
    for n in ("dg_gemv_w4", "dg_linear_ce", "dg_linear_ce_grad", "dg_linear_ce_workspace",
              "dg_linear_ce_grad_workspace"):
        assert hasattr(dg.lib, n)


def test_gemv_w4_refusals():
    L = dg.lib
    x, W, y = mat(2, 256), w4(), mat(2, 64, "f32", es=4)
    b = ctypes.byref
    assert L.dg_gemv_w4(None, b(W), b(y), 1.0, 0.0, None, None) == dg.DG_ERR_NULL
    assert L.dg_gemv_w4(b(x), None, b(y), 1.0, 0.0, None, None) == dg.DG_ERR_NULL
    assert L.dg_gemv_w4(b(x), b(W), None, 1.0, 0.0, None, None) == dg.DG_ERR_NULL
    assert gemv(W=w4(codes=None)) == dg.DG_ERR_NULL
    assert gemv(W=w4(scales=None)) == dg.DG_ERR_NULL
    assert gemv(x=mat(9, 256), y=mat(9, 64, "f32", es=4)) == dg.DG_ERR_UNSUPPORTED
    assert gemv(x=mat(2, 255)) == dg.DG_ERR_SHAPE
    assert gemv(y=mat(2, 63, "f32", es=4)) == dg.DG_ERR_SHAPE
    assert gemv(y=mat(3, 64, "f32", es=4)) == dg.DG_ERR_SHAPE
    assert gemv(W=w4(N=-1)) == dg.DG_ERR_SHAPE
    assert gemv(x=mat(2, 256, "f32", es=4)) == dg.DG_ERR_DTYPE
    assert gemv(x=mat(2, 256, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert gemv(y=mat(2, 64, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert gemv(W=w4(scale_dtype=dg.DG_E4M3)) == dg.DG_ERR_DTYPE
    for group in (0, -32, 1, 16, 33, 48):
        assert gemv(W=w4(group=group)) == dg.DG_ERR_VALUE
    assert gemv(W=w4(reserved=1)) == dg.DG_ERR_VALUE
    assert gemv(alpha=math.nan) == dg.DG_ERR_VALUE
    assert gemv(beta=math.inf) == dg.DG_ERR_VALUE
    assert gemv(epi=dg.epilogue(None, 7)) == dg.DG_ERR_VALUE
    assert gemv(W=w4(code_stride=-1)) == dg.DG_ERR_STRIDE
    assert gemv(W=w4(scale_stride=-2)) == dg.DG_ERR_STRIDE
    assert gemv(W=w4(zeros=FAKE, zero_stride=-1)) == dg.DG_ERR_STRIDE
    assert gemv(W=w4(code_stride=1 << 60)) == dg.DG_ERR_STRIDE
    assert gemv(y=mat(2, 64, "f32", es=4, rs=0)) == dg.DG_ERR_STRIDE
    assert gemv(W=w4(scales=FAKE + 1)) == dg.DG_ERR_ALIGN
    assert gemv(W=w4(scale_stride=5)) == dg.DG_ERR_ALIGN
    # nothing to do
    assert gemv(x=mat(0, 256), y=mat(0, 64, "f32", es=4)) == dg.DG_OK
    assert gemv(W=w4(N=0), y=mat(2, 0, "f32", es=4)) == dg.DG_OK


def test_gemv_w4_binding_refusals():
    codes, scales = torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1)
    with pytest.raises(TypeError):
        dg.w4(codes.int(), scales)
    with pytest.raises(ValueError):
        dg.w4(codes, scales, K=130)
    with pytest.raises(ValueError):
        dg.w4(codes, scales, group=64)
    with pytest.raises(ValueError):
        dg.w4(codes, scales, zeros=torch.zeros(8, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        dg.w4(torch.zeros(64, 8, dtype=torch.uint8).t(), scales)
    assert dg.w4(codes, scales).K == 128 and dg.w4(codes, scales, K=127).K == 127


def ce(X=None, W=None, target=FAKE, alpha=1.0, loss=FAKE, lse=FAKE, ws=FAKE, size=1 << 40):
    X = mat(4, 64) if X is None else X
    W = mat(64, 100) if W is None else W
    return dg.dg_linear_ce(X, W, target, -100, alpha, loss, lse, ws, size, 0)


def grad(X=None, W=None, target=FAKE, alpha=1.0, lse=FAKE, dl=FAKE, stride=4, dX=True, dW=True, ws=FAKE,
         size=1 << 40):
    X = mat(4, 64) if X is None else X
    W = mat(64, 100) if W is None else W
    dX = mat(4, 64) if dX is True else dX
    dW = mat(64, 100) if dW is True else dW
    return dg.dg_linear_ce_grad(X, W, target, -100, alpha, lse, dl, stride, dX, dW, ws, size, 0)


@pytest.mark.parametrize("call", [ce, grad])
def test_linear_ce_refusals(call):
    assert call(W=mat(63, 100)) == dg.DG_ERR_SHAPE
    assert call(W=mat(64, 0), **({"dW": None} if call is grad else {})) == dg.DG_ERR_SHAPE
    assert call(W=mat(64, 100, "f16")) == dg.DG_ERR_DTYPE
    assert call(X=mat(4, 64, "e4m3", es=1), W=mat(64, 100, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert call(alpha=math.inf) == dg.DG_ERR_VALUE
    assert call(target=None) == dg.DG_ERR_NULL
    assert call(lse=None) == dg.DG_ERR_NULL
    assert call(ws=None) == dg.DG_ERR_NULL
    assert call(target=FAKE + 4) == dg.DG_ERR_ALIGN
    assert call(lse=FAKE + 2) == dg.DG_ERR_ALIGN
    assert call(ws=FAKE + 128) == dg.DG_ERR_ALIGN
    assert call(size=0) == dg.DG_ERR_SHAPE
    assert call(X=mat(4, 64, base=FAKE + 1)) == dg.DG_ERR_ALIGN
    # W's columns as two dims that do not merge
    W3 = dg.make_view(FAKE, (64, 5, 20), (400, 50, 2), 1, "bf16")
    assert call(W=W3) == dg.DG_ERR_UNSUPPORTED


def test_linear_ce_refusals_of_its_own():
    assert ce(loss=None) == dg.DG_ERR_NULL
    assert ce(loss=FAKE + 1) == dg.DG_ERR_ALIGN
    assert ce(X=mat(0, 64)) == dg.DG_OK
    assert grad(dl=None) == dg.DG_ERR_NULL
    assert grad(dX=None, dW=None) == dg.DG_ERR_NULL
    assert grad(stride=8) == dg.DG_ERR_STRIDE
    assert grad(dX=mat(4, 63)) == dg.DG_ERR_SHAPE
    assert grad(dW=mat(100, 64)) == dg.DG_ERR_SHAPE
    assert grad(dX=mat(4, 64, "e4m3", es=1)) == dg.DG_ERR_DTYPE
    assert grad(dW=mat(64, 100, "f32", es=4, rs=0)) == dg.DG_ERR_STRIDE


def test_workspace_sizes():
    X, W = mat(4096, 1024), mat(1024, 32000)
    least, best = dg.dg_linear_ce_workspace(X, W)
    assert 0 < least <= best < 1 << 30
    gl, gb = dg.dg_linear_ce_grad_workspace(X, W, mat(4096, 1024), mat(1024, 32000))
    assert 0 < gl <= gb < 1 << 31
    assert ce(X=X, W=W, size=least - 1) == dg.DG_ERR_SHAPE
    # far below the logits themselves
    assert least < 4096 * 32000 * 2 // 8
    with pytest.raises(dg.DgError):
        dg.dg_linear_ce_workspace(X, mat(1000, 32000))


def test_linear_ce_binding_refusals():
    x, w = torch.zeros(4, 8).bfloat16(), torch.zeros(8, 10).bfloat16()
    y, f = torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError):
        dg.linear_ce(x, w, y.int(), f, f)
    with pytest.raises(ValueError):
        dg.linear_ce(x, w, y[:3], f, f)
    with pytest.raises(ValueError):
        dg.linear_ce(x, w, torch.zeros(8, dtype=torch.int64)[::2], f, f)
    with pytest.raises(ValueError):
        dg.linear_ce(x, w, y, f.double(), f)
    with pytest.raises(ValueError):
        dg.linear_ce_grad(x, w, y, f, torch.zeros(3), x, w)
    with pytest.raises(ValueError):
        dg.linear_ce_grad(x, w, y, f, f.double(), x, w)
