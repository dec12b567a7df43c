"""The residual norm between int8 layers: what it hands to the int8 layer, held to the oracle."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L
from int8_quantized_02_b200 import synth
from oracle import oracle

from .gpu_util import assert_y_close, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K,N", [(1, 512, 256), (20, 512, 256), (130, 1056, 512), (300, 4096, 1024)])
@pytest.mark.parametrize("norm", ["rms", "layer"])
def test_norm_then_int8_layer(M, K, N, norm):
    g = torch.Generator().manual_seed(M)
    X = synth.activations(M, K, 4, 6.0, 20.0, 0.75, M)[0]
    res = dev(X)
    w = (1 + 0.2 * torch.randn(K, generator=g)).half().cuda()
    W = synth.weight(N, K, 0.02, seed=N)
    CB, SCB = L.llmint8_quantize_weight_colwise(dev(W))
    H, Y = L.llmint8_residual_norm(dev(X), residual=res, norm=norm, weight=w, scale=0.5)
    y = L.llmint8_linear(Y, CB, SCB, threshold=6.0, max_outliers=K)
    CB_o, SCB_o = oracle.quantize_weight_colwise(W)
    assert np.array_equal(host(CB), CB_o)
    assert_y_close(host(y), oracle.linear(host(Y), CB_o, SCB_o, threshold=6.0))
