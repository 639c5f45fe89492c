"""Offsets that decrease and then overlap: no row of C is computed twice, whatever they say, and every group of
dg_gemm_grouped_dw has the rows that its own offsets name.

Inputs are small integers and powers of two, so that all sums are exact and compared for equality.
"""
import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rows_of(offsets, R):
    """The rows of each group of dg_gemm_grouped."""
    out, end = [], 0
    for a, b in zip(offsets, offsets[1:]):
        if not 0 <= a <= b <= R or a == b:
            out.append((0, 0))
            continue
        out.append((a, b) if a >= end else (0, 0))
        end = max(end, b)
    return out


@pytest.mark.parametrize("offsets", [
    [0, 60, 0, 60, 0, 60],
    [10, 50, 20, 60, 55, 60],                       # an overlap with the end of an earlier group
    [30, 60, 0, 30, 60],                            # behind it, an earlier part of the rows
    [0, 60] * 512 + [0],                            # many more rows than there are, over all of the groups
    [50, 50, 10, 60],                               # an empty group is in front of nothing
    [0, 10, -1, 10, 40, 1 << 40, 40, 60],
    [0, 70, 0, 20, 10, 60],                         # what leaves the rows is in front of nothing either
    [0] * 40 + [30, 20, 40] + [40] * 40 + [60, 50, 60],
])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_overlapping_groups(offsets, dtype):
    R, K, N, G = 60, 64, 40, len(offsets) - 1
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randint(-3, 4, (R, K), generator=g, device="cuda").to(DT[dtype])
    w = torch.randint(-3, 4, (G, K, N), generator=g, device="cuda").to(DT[dtype])
    c = torch.randint(-9, 10, (R, N), generator=g, device="cuda").float()
    want = c.double()
    for i, (a, b) in enumerate(rows_of(offsets, R)):
        want[a:b] = 2 * want[a:b] + x[a:b].double() @ w[i].double()
    at = torch.tensor(offsets, device="cuda")
    dg.gemm_grouped(x, w, c, at, beta=2.0)
    assert dg.dg_sync_status() == dg.DG_ERR_VALUE and dg.dg_sync_status() == dg.DG_OK
    assert torch.equal(c.double(), want)
    dy = torch.randint(-3, 4, (R, N), generator=g, device="cuda").to(DT[dtype])
    dw = torch.ones(G, K, N, device="cuda")
    dg.gemm_grouped_dw(x, dy, dw, at, beta=2.0)
    assert dg.dg_sync_status() == dg.DG_ERR_VALUE and dg.dg_sync_status() == dg.DG_OK
    for i, (a, b) in enumerate(zip(offsets, offsets[1:])):
        a, b = (a, b) if 0 <= a <= b <= R else (0, 0)
        assert torch.equal(dw[i].double(), 2 + x[a:b].double().t() @ dy[a:b].double()), i


def test_rows_in_order_are_not_reported():
    at = torch.tensor([5, 5, 20, 20, 60], device="cuda")
    x, w, c = torch.ones(60, 64, device="cuda").bfloat16(), torch.ones(4, 64, 40, device="cuda").bfloat16(), torch.zeros(60, 40, device="cuda")
    dg.gemm_grouped(x, w, c, at)
    assert dg.dg_sync_status() == dg.DG_OK
    assert (c[:5] == 0).all() and (c[5:] == 64).all()
