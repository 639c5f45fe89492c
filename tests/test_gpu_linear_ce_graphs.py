"""Captured gradients keep to their own workspaces: two graphs captured on one stream, replayed on two at once."""
import math

import pytest
import torch

import tcgen05_tmem_gemm_b200 as dg
from test_gpu_linear_ce import IGNORE, inputs, run_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _reset_options():
    yield
    dg.dg_set_option(dg.DG_OPT_STREAM_K, 0)


@pytest.mark.parametrize("stream_k", [0, 1])
def test_two_graphs_of_one_stream_at_once(stream_k):
    # products of more tiles than pairs of SMs, with a partial last wave
    T, D, V = 4096, 4096, 2000
    dg.dg_set_option(dg.DG_OPT_STREAM_K, stream_k)
    stream = torch.cuda.Stream()
    # a product of the caller's own, which with Stream-K leaves the stream a workspace
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    c = torch.empty(4096, 4096, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()
    dg.gemm(a, a, c, stream=stream)
    torch.cuda.synchronize()
    problems, graphs, wanted = [], [], []
    for seed in (1, 2):
        x, w, y, dl = inputs(T, D, V, "bf16", seed=seed)
        _, lse = run_forward(x, w, y)
        dx, dw = torch.empty_like(x), torch.empty(V, D, device="cuda").bfloat16()
        dg.linear_ce_grad(x, w, y, lse, dl, dx, dw.t(), ignore_index=IGNORE)
        wanted.append((dx.clone(), dw.clone()))
        best = dg.dg_linear_ce_grad_workspace(dg.view(x), dg.view(w), dg.view(dx), dg.view(dw.t()))[1]
        ws = torch.empty(best, dtype=torch.uint8, device="cuda")
        problems.append((x, w, y, lse, dl, dx, dw, ws))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            dg.linear_ce_grad(x, w, y, lse, dl, dx, dw.t(), ignore_index=IGNORE, workspace=ws)
        graphs.append(graph)
    sides = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for p in problems:
            p[5].fill_(math.nan)
            p[6].fill_(math.nan)
        torch.cuda.synchronize()
        for side, graph in zip(sides, graphs):
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for p, (dx, dw) in zip(problems, wanted):
            assert torch.equal(p[5], dx) and torch.equal(p[6], dw)
    assert dg.dg_sync_status() == dg.DG_OK
