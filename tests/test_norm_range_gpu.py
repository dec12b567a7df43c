"""The residual norm over bf16's whole range: rows whose squares leave fp32's, at both ends, and what
stands beside them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L
from tests import mx_util as mx

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
# exponents of rows: bf16's subnormals, squares that vanish, ordinary ones, squares that overflow, and
# rows whose very sum does
POWERS = [-131, -126, -100, -75, -64, -50, -10, 0, 20, 63, 64, 65, 100, 120, 125]


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(M, K, seed, powers=POWERS):
    """Row m of size 2^powers[m], and of a mean of that size too."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn((M, K), generator=g).clamp(-3.5, 3.5).double() + 1
    p = torch.tensor([powers[m % len(powers)] for m in range(M)], dtype=torch.float64)
    return (v * torch.exp2(p)[:, None]).bfloat16().cuda()


def check(x, a, H, Y, scale=1.0):
    d = lambda k: None if a.get(k) is None else f64(a[k])  # noqa: E731
    h, ht, y, yt = mx.residual_norm(f64(x), d("residual"), a.get("post_norm"), d("post_weight"), None,
                                    None, scale, a["norm"], d("weight"), None, a["eps"],
                                    "bfloat16" if x.dtype == BF16 else "float16")
    assert np.isfinite(y).all()
    if H is not None:
        assert (np.abs(f64(H) - h) <= ht).all()
    off = np.abs(f64(Y) - y)
    assert (off <= yt).all(), (np.nonzero((off > yt).any(1))[0], (off / yt).max())


# every number of threads to a row, rows that fill their threads' chunks and rows that do not
SHAPES = [(15, 32), (15, 1056), (15, 4096), (15, 12288), (15, 32768), (200, 256), (200, 288), (200, 1024),
          (200, 1568), (160, 4096), (160, 12288), (160, 16384), (160, 17408)]


@pytest.mark.parametrize("norm,post", [("rms", None), ("layer", None), ("rms", "rms"), ("layer", "layer")])
@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("eps", [0.0, 1e-31, 1e-5])
def test_rows_of_any_size(M, K, norm, post, eps):
    x = rows(M, K, seed=M + K)
    g = torch.Generator().manual_seed(K)
    w = (1 + 0.2 * torch.randn(K, generator=g)).bfloat16().cuda()
    a = {"norm": norm, "post_norm": post, "eps": eps, "weight": w, "post_weight": w if post else None}
    H, Y = L.llmint8_residual_norm(x, **a)
    check(x, a, H, Y)
    _, codes, scales = L.llmint8_residual_norm_mxfp4(x, **a)
    want = L.llmint8_mxfp4_quantize(Y)
    assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


@pytest.mark.parametrize("M,K", [(15, 4096), (200, 256), (200, 1024), (160, 12288)])
def test_ordinary_rows_beside_them_do_not_change(M, K):
    x = rows(M, K, seed=1, powers=[0, 100, 0, -100])
    plain = rows(M, K, seed=1, powers=[0])
    for norm in ("rms", "layer"):
        Y = L.llmint8_residual_norm(x, norm=norm, eps=1e-5)[1]
        assert torch.equal(Y[::2], L.llmint8_residual_norm(plain, norm=norm, eps=1e-5)[1][::2])


def test_a_scale_that_leaves_fp16():
    """h beyond the 16-bit type is an infinity in H; its norm is that of the unrounded h."""
    x = torch.randn((20, 1024), generator=torch.Generator().manual_seed(2)).half().cuda()
    a = {"norm": "rms", "eps": 1e-6}
    H, Y = L.llmint8_residual_norm(x, scale=2.0 ** 90, **a)
    check(x, a, None, Y, scale=2.0 ** 90)
    assert torch.isinf(H[x.abs() > 1e-3]).all()


def test_infinities_and_nan_stay_what_they_were():
    x = rows(6, 512, seed=3, powers=[0])
    x[1, 5], x[2, 6], x[3, 7] = float("inf"), -float("inf"), float("nan")
    Y = L.llmint8_residual_norm(x, norm="rms", eps=1e-5)[1]
    fine = L.llmint8_residual_norm(x[4:], norm="rms", eps=1e-5)[1]
    assert torch.equal(Y[4:], fine) and torch.isfinite(Y[0]).all() and torch.isnan(Y[3]).all()
    for m, k in ((1, 5), (2, 6)):                    # v / inf: 0, and nothing for the infinity itself
        assert torch.isnan(Y[m, k]) and (Y[m, :k] == 0).all() and (Y[m, k + 1:] == 0).all()
    Y = L.llmint8_residual_norm(x, norm="layer", eps=1e-5)[1]
    assert torch.isnan(Y[1:4]).all() and torch.isfinite(Y[[0, 4, 5]]).all()
    zero = torch.zeros((3, 512), dtype=BF16, device="cuda")
    assert (L.llmint8_residual_norm(zero, norm="rms", eps=1e-31)[1] == 0).all()


@pytest.mark.parametrize("norm,post", [("rms", None), ("layer", "rms"), (None, "layer"), ("layer", None)])
@pytest.mark.parametrize("M,K", [(15, 4096), (200, 288), (200, 1024), (160, 12288), (160, 17408)])
def test_in_place(M, K, norm, post):
    """H over the residual and Y over X, and the other way round, whichever norm a row is scaled for."""
    x = rows(M, K, seed=4)
    res = rows(M, K, seed=5, powers=POWERS[::-1][1:] + [0])
    a = {"norm": norm, "post_norm": post, "eps": 0.0, "scale": 0.75}
    H, Y = L.llmint8_residual_norm(x, residual=res, **a)
    for swap in (False, True):
        xx, rr = x.clone(), res.clone()
        h, y = (xx, rr) if swap else (rr, xx)
        got = L.llmint8_residual_norm(xx, residual=rr, H=h, Y=y if norm else None, **a)
        assert torch.equal(H, got[0]) and (norm is None or torch.equal(Y, got[1]))


@pytest.mark.parametrize("M,K", [(15, 4096), (200, 288), (200, 1024), (160, 12288)])
@pytest.mark.parametrize("post", ["rms", "layer"])
def test_all_that_follows_a_scaled_post_norm(M, K, post):
    """Gate, scale, residual and both norms' vectors behind a PostNorm of rows of any size."""
    g = torch.Generator().manual_seed(7)
    put = lambda t: t.bfloat16().cuda()  # noqa: E731
    x = rows(M, K, seed=6)
    a = {"norm": "rms", "post_norm": post, "eps": 0.0, "scale": 0.75, "residual": put(torch.randn((M, K), generator=g)),
         "weight": put(1 + 0.2 * torch.randn(K, generator=g)), "bias": put(0.3 * torch.randn(K, generator=g)),
         "post_weight": put(1 + 0.2 * torch.randn(K, generator=g)),
         "post_bias": put(0.3 * torch.randn(K, generator=g)), "gate": put(torch.randn((M // 5, K), generator=g))}
    H, Y = L.llmint8_residual_norm(x, **a)
    d = {k: f64(v) for k, v in a.items() if isinstance(v, torch.Tensor)}
    h, ht, y, yt = mx.residual_norm(f64(x), d["residual"], post, d["post_weight"], d["post_bias"], d["gate"],
                                    0.75, "rms", d["weight"], d["bias"], 0.0, "bfloat16")
    assert (np.abs(f64(H) - h) <= ht).all() and (np.abs(f64(Y) - y) <= yt).all()
