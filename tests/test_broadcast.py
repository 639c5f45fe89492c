"""Operands with a broadcast (zero-stride) dim, which a tensor map cannot
describe: read through the thread loads, they give the same product as their
contiguous copies."""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

FAKE = 1 << 40


def test_a_broadcast_dim_is_not_a_tensor_map():
    for shape, stride in (((300, 64), (0, 2)), ((64, 300), (2, 0))):
        assert dg.dg_analyse_view(dg.make_view(FAKE, shape, stride, 1, "bf16")).tma_ok == 0
    # a zero stride on a dim of one element says nothing
    assert dg.dg_analyse_view(dg.make_view(FAKE, (1, 64), (0, 2), 1, "bf16")).tma_ok == 1


def test_a_weight_of_one_row_does_not_stream_through_a_map():
    x = dg.make_view(FAKE, (1, 512), (1024, 2), 1, "bf16")
    y = dg.make_view(FAKE, (1, 1024), (2048, 2), 1, "bf16")
    W = dg.make_view(FAKE, (512, 1024), (0, 2), 1, "bf16")
    assert dg.dg_plan(x, W, y, num_sms=148).as_dict()["kind_name"] != "gemv_n"


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 5, 64, 300])
@pytest.mark.parametrize("which", ["a_rows", "b_rows", "b_cols"])
def test_broadcast_operands(M, which):
    K, N = 256, 1024
    g = torch.Generator().manual_seed(M)
    a = torch.randn(M, K, generator=g).bfloat16().cuda()
    b = torch.randn(K, N, generator=g).bfloat16().cuda()
    if which == "a_rows":
        a = a[:1].expand(M, K)
    elif which == "b_rows":
        b = b[:1].expand(K, N)
    else:
        b = b[:, :1].expand(K, N)
    c = torch.empty(M, N, device="cuda")
    dg.gemm(a, b, c)
    assert dg.dg_sync_status() == dg.DG_OK
    ref = a.double() @ b.double()
    S = a.double().abs() @ b.double().abs()
    # the parity tests' bound for FP32 outputs
    assert bool(((c.double() - ref).abs() <= 5e-4 * S + 2.0 ** -22 * ref.abs()).all())
