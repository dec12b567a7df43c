"""Products whose one launch takes more than a second, at the largest K: what limits the kernels' waits
must not be counted over the whole launch.  Operands of few values, so that every output is known
exactly."""
from __future__ import annotations

import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L

pytestmark = pytest.mark.gpu

K = 131072


@pytest.fixture
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 115e9:
        pytest.skip("needs 115 GB")
    yield
    torch.cuda.empty_cache()


def rows_equal(Y, row):
    return all(bool((Y[i:i + 4096] == row).all()) for i in range(0, Y.shape[0], 4096))


def test_mxfp4(room):
    M = N = 188000                  # 9.3e15 operations, over a second at the tensor cores' full rate
    # X is 1, W's row n one value of the format times 2^-7: sums of multiples of 2^-8 up to 6144, exact
    XC = torch.full((M, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    XS = torch.full(L.mxfp4_scales_shape(M, K), 127, dtype=torch.uint8, device="cuda")
    code = torch.arange(N, device="cuda") % 15
    WC = (code * 17).to(torch.uint8)[:, None].expand(N, K // 2).contiguous()
    WS = torch.full(L.mxfp4_scales_shape(N, K), 120, dtype=torch.uint8, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    Y = L.llmint8_mxfp4_linear_quantized(XC, XS, WC, WS, workspace=ws)
    assert L.llmint8_device_status(ws) == L.OK
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    value = torch.cat((grid, -grid))[code]
    assert rows_equal(Y, (value * (K / 128)).half())


def test_int8(room):
    M = N = 134000                  # 4.7e15 operations
    X = torch.ones((M, K), dtype=torch.float16, device="cuda")
    CB = ((torch.arange(N, device="cuda") % 255) - 127).to(torch.int8)[:, None].expand(N, K).contiguous()
    SCB = torch.full((N,), 2.0 ** -6, device="cuda")
    ws = torch.empty(L.llmint8_linear_workspace_size(M, N, K, 64), dtype=torch.uint8, device="cuda")
    Y = L.llmint8_linear(X, CB, SCB, max_outliers=64, workspace=ws)
    assert L.llmint8_device_status(ws) == L.OK
    # C = 127 K cb, below 2^31: Y = K cb / 127 * 2^-6, with fp32's roundings before fp16's
    want = K / 64 * CB[:, 0].double() / 127
    assert ((Y[0].double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -21) + 2.0 ** -25).all()
    assert rows_equal(Y, Y[0])
