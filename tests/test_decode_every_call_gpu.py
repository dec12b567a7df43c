"""Every one of many decode calls, back to back, gives the first one's output: a weight stage read before its
copy has landed shows once in a thousand calls or so, and not always as a call that times out."""
from __future__ import annotations

import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L

pytestmark = pytest.mark.gpu


# as many stages as fit would be odd; an odd number of stages a tile over several tiles; both with 16 rows
@pytest.mark.parametrize("M,N,K", [(1, 49152, 12288), (1, 40000, 8448), (16, 40000, 8448)])
def test_every_call(M, N, K):
    cap, batch = 64, 50
    g = torch.Generator(device="cuda").manual_seed(N + M)
    W = (torch.randn((N, K), device="cuda", generator=g) * 0.01).half()
    CB, SCB = L.llmint8_quantize_weight_colwise(W)
    del W
    X = torch.randn((M, K), device="cuda", generator=g).half()
    X[:, [5, 700, 5000]] = 10
    ws = torch.empty(L.llmint8_linear_workspace_size(M, N, K, cap), dtype=torch.uint8, device="cuda")
    want = L.llmint8_linear(X, CB, SCB, max_outliers=cap, workspace=ws).clone()
    assert L.llmint8_device_status(ws) == L.OK
    Y = torch.empty((batch, M, N), dtype=torch.float16, device="cuda")
    wrong = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(6000 // batch):
        Y.fill_(float("nan"))
        for i in range(batch):
            L.llmint8_linear(X, CB, SCB, max_outliers=cap, Y=Y[i], workspace=ws)
        wrong += (Y != want).flatten(1).any(1).sum()
    assert int(wrong) == 0 and L.llmint8_device_status(ws) == L.OK
