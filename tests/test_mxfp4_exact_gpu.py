"""MXFP4 products whose every sum fits fp32 and the output type, compared bit for bit: at the largest K a
bound on fp32's roundings is wider than what a block, or a whole k-tile, adds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L
from tests import mx_util as mx

pytestmark = pytest.mark.gpu

GRID = np.concatenate([mx.GRID, -mx.GRID])


def mxfp4(codes, scales):
    """Plain codes [R, K] and scale bytes [R, K/32] on the device."""
    return torch.from_numpy(mx.pack(codes)).cuda(), torch.from_numpy(mx.tile(scales)).cuda()


# the band kernel with tiles of 16, 32 and 64 rows, k split over 1 to 8 CTAs; CTA pairs
SHAPES = [(1, 130, 131072), (8, 40, 131072), (16, 300, 131072), (20, 130, 131040), (64, 130, 131072),
          (9, 20000, 4128), (1300, 1003, 131072), (900, 1500, 8224)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_every_block_counts(M, N, K, dtype):
    """Each row of X has one code in each of 32 blocks and zeros elsewhere; over the rows, and calls
    where they are few, every block of K has its turn.  The weight is everywhere, each of its blocks with
    a power of two of its own that X's block undoes.  So a sum has 32 products, multiples of 1/4 up to 36:
    exact in fp32 whatever the order, and rounded once for Y."""
    rng = np.random.default_rng(M + N)
    blocks = K // 32
    W = rng.integers(0, 16, (N, K), dtype=np.uint8)
    e = rng.integers(-20, 21, blocks)
    WC, WS = mxfp4(W, np.broadcast_to(127 + e, (N, blocks)).astype(np.uint8))
    xs = np.broadcast_to(127 - e, (M, blocks)).astype(np.uint8)
    order = rng.permutation(blocks)
    calls = -(-blocks // (32 * M))
    for call in range(calls):
        X = np.zeros((M, K), np.uint8)
        want = np.zeros((M, N))
        for m in range(M):
            at = np.sort(np.take(order, np.arange(32) + 32 * (call * M + m), mode="wrap")) * 32 + \
                rng.integers(0, 32, 32)
            X[m, at] = rng.integers(1, 8, 32) + 8 * rng.integers(0, 2, 32)
            want[m] = GRID[W[:, at]] @ GRID[X[m, at]]
        Y = L.llmint8_mxfp4_linear_quantized(*mxfp4(X, xs), WC, WS, dtype=dtype)
        assert torch.equal(Y, torch.from_numpy(want).to(dtype).cuda()), call
