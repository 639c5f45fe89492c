"""Host-only: a bias of dg_gemm_mx4 that a kernel would read past its end, or off its alignment, is refused."""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

FAKE = 1 << 40


def operand(rows):
    q = dg.dg_mx4()
    q.codes, q.scales, q.rows, q.K, q.code_stride, q.block = FAKE, FAKE, rows, 64, 32, 32
    return q


@pytest.mark.parametrize("off", [1, 2, 3])
def test_alignment(off):
    c = dg.make_view(FAKE, (16, 8), (32, 4), 1, "f32")
    assert dg.dg_gemm_mx4(operand(16), operand(8), c, 1.0, 0.0, dg.epilogue(FAKE + off), 0) == dg.DG_ERR_ALIGN


@pytest.mark.parametrize("bias", [torch.zeros(8).bfloat16(), torch.zeros(8).half(), torch.zeros(8).double(), torch.zeros(7),
                                  torch.zeros(9), torch.zeros(16)[::2], torch.zeros(8, dtype=torch.int32)])
def test_binding(bias):
    with pytest.raises(ValueError):
        dg.gemm_mx4(operand(16), operand(8), dg.make_view(FAKE, (16, 8), (32, 4), 1, "f32"), bias=bias)
