"""A wait limit of 1 ns: every way out of the products' pipelines is taken, each call ends and says
so, nothing but its output is touched, and the next call is right."""
from __future__ import annotations

import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L

pytestmark = pytest.mark.gpu


@pytest.fixture
def tiny_limit():
    L.llmint8_set_wait_timeout_ns(0)
    yield lambda: L.llmint8_set_wait_timeout_ns(1)
    L.llmint8_set_wait_timeout_ns(0)


def run_out(limit, call, ws, out):
    """The statuses of three calls under the limit; `out` is Y with a row on either side of it."""
    want = call().clone()
    assert L.llmint8_device_status(ws) == L.OK
    limit()
    seen = []
    for _ in range(3):
        call()
        seen.append(L.llmint8_device_status(ws))
    L.llmint8_set_wait_timeout_ns(0)
    assert (out[0] == 7).all() and (out[-1] == 7).all()
    assert torch.equal(call(), want) and L.llmint8_device_status(ws) == L.OK
    return seen


# one CTA to a band; clusters of 4 and of 8; three CTAs to an SM; tiles of 16, 32 and 64 rows; X quantised
# in the product (up to 8 rows) and before it; CTA pairs
@pytest.mark.parametrize("M,N,K", [(8, 16384, 4096), (1, 4096, 4096), (8, 512, 16384), (8, 49152, 12288),
                                   (16, 4096, 8192), (32, 1024, 16384), (64, 16384, 4096), (200, 512, 16384),
                                   (1500, 1024, 16384), (3000, 4096, 4096)])
def test_mxfp4(M, N, K, tiny_limit):
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn((M, K), generator=g, device="cuda").half()
    WC = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    WS = torch.full(L.mxfp4_scales_shape(N, K), 120, dtype=torch.uint8, device="cuda")
    ws = torch.empty(L.llmint8_mxfp4_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.full((M + 2, N), 7.0, dtype=torch.float16, device="cuda")
    seen = run_out(tiny_limit, lambda: L.llmint8_mxfp4_linear(X, WC, WS, Y=out[1:M + 1], workspace=ws), ws, out)
    assert set(seen) <= {L.OK, L.ERR_TIMEOUT} and L.ERR_TIMEOUT in seen


# single CTAs, CTA pairs (outlier columns in the epilogue, and on the tensor cores), the decode kernel
@pytest.mark.parametrize("M,N,K,outliers", [(100, 512, 16384, 3), (200, 512, 16384, 3), (1500, 1024, 16384, 0),
                                            (3000, 4096, 4096, 3), (3000, 4096, 4096, 40), (16, 4096, 4096, 3)])
def test_int8(M, N, K, outliers, tiny_limit):
    g = torch.Generator(device="cuda").manual_seed(M)
    X = torch.randn((M, K), generator=g, device="cuda").half().clamp(-5, 5)
    X[:, 7:7 + 5 * outliers:5] = 10
    CB = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8, device="cuda")
    SCB = torch.rand(N, generator=g, device="cuda") * 0.1
    ws = torch.empty(L.llmint8_linear_workspace_size(M, N, K, 64), dtype=torch.uint8, device="cuda")
    out = torch.full((M + 2, N), 7.0, dtype=torch.float16, device="cuda")
    seen = run_out(tiny_limit, lambda: L.llmint8_linear(X, CB, SCB, max_outliers=64, Y=out[1:M + 1], workspace=ws),
                   ws, out)
    assert set(seen) <= {L.OK, L.ERR_TIMEOUT} and L.ERR_TIMEOUT in seen
