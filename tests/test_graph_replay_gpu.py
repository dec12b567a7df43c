"""One captured call of a layer, replayed on other values of the same buffers: each replay's output is
that of a call made for it, whatever an earlier replay left in the workspace."""
from __future__ import annotations

import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L

pytestmark = pytest.mark.gpu


def values(M, K, i):
    """Other outlier columns, another count of them and another size each time."""
    g = torch.Generator(device="cuda").manual_seed(100 * i + M)
    x = (torch.randn((M, K), generator=g, device="cuda") * (0.2 + 0.2 * i)).clamp(-5, 5)
    x[:, torch.arange(i + 1, device="cuda") * 31 + 7 * i] = 10.0 + i
    return x.half()


def weights(N, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    return L.llmint8_quantize_weight_colwise((torch.randn((N, K), generator=g, device="cuda") * 0.02).half())


def replays(X, call, out, want):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for i in range(6):
        new = values(*X.shape, i)
        X.copy_(new)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want(new)), i


@pytest.mark.parametrize("M,N,K", [(1, 1024, 1024), (1, 4096, 4096), (8, 528, 4112), (16, 4096, 4096),
                                   (16, 16384, 16384), (8, 49152, 12288), (100, 1024, 4096), (300, 1024, 4096)])
def test_int8_layer(M, N, K):
    CB, SCB = weights(N, K)
    X = values(M, K, 9)
    ws = torch.empty(L.llmint8_linear_workspace_size(M, N, K, 64), dtype=torch.uint8, device="cuda")
    Y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    replays(X, lambda: L.llmint8_linear(X, CB, SCB, max_outliers=64, Y=Y, workspace=ws), Y,
            lambda x: L.llmint8_linear(x, CB, SCB, max_outliers=64))
    assert L.llmint8_device_status(ws) == L.OK


def test_int8_layer_without_a_workspace():
    CB, SCB = weights(2048, 4096)
    X, Y = values(4, 4096, 9), torch.empty((4, 2048), dtype=torch.float16, device="cuda")
    replays(X, lambda: L.llmint8_linear_noalloc(X, CB, SCB, max_outliers=64, Y=Y), Y,
            lambda x: L.llmint8_linear(x, CB, SCB, max_outliers=64))


def test_two_graphs_of_one_workspace_in_turn():
    M, N, K = 8, 2048, 4096
    CB, SCB = weights(N, K)
    ws = torch.empty(L.llmint8_linear_workspace_size(M, N, K, 64), dtype=torch.uint8, device="cuda")
    X = [values(M, K, i) for i in (1, 2)]
    Y = [torch.empty((M, N), dtype=torch.float16, device="cuda") for _ in X]
    want = [L.llmint8_linear(x, CB, SCB, max_outliers=64) for x in X]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in X]
    for g, x, y in zip(graphs, X, Y):
        with torch.cuda.graph(g):
            L.llmint8_linear(x, CB, SCB, max_outliers=64, Y=y, workspace=ws)
    for turn in (0, 0, 1, 1, 0, 1):
        Y[turn].fill_(float("nan"))
        graphs[turn].replay()
        torch.cuda.synchronize()
        assert torch.equal(Y[turn], want[turn])


@pytest.mark.parametrize("M", [1, 8, 16, 300])
def test_mxfp4_layer(M):
    N, K = 2048, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    W = L.llmint8_mxfp4_quantize((torch.randn((N, K), generator=g, device="cuda") * 0.02).half())
    X, Y = values(M, K, 9), torch.empty((M, N), dtype=torch.float16, device="cuda")
    ws = torch.empty(L.llmint8_mxfp4_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    replays(X, lambda: L.llmint8_mxfp4_linear(X, *W, Y=Y, workspace=ws), Y, lambda x: L.llmint8_mxfp4_linear(x, *W))
