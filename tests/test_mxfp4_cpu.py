"""The MXFP4 calls and the residual norm without a GPU: the format's oracle pinned by hand, the
layout helpers, and every refusal that comes before a launch."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

from int8_quantized_02_b200 import build as build_mod
from int8_quantized_02_b200 import llmint8 as L
from tests import mx_util as mx

FAKE = ctypes.c_void_p(1 << 20)      # aligned, never dereferenced: the checks come first
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return L.load()


def test_oracle_by_hand():
    x = np.zeros((1, 64))
    # max 6 = 1.5 * 4: scale 2^(2 - 2) = 1
    x[0, :12] = [6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -5, -.25, .26, 7.9 / 2]
    codes, s = mx.quantize(x)
    assert s.tolist() == [[127, 0]]
    assert mx.values(codes, s)[0, :12].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -4, 0, .5, 4]
    x[0, 0] = 7.9                       # beyond 6: the largest code
    assert mx.round_trip(x)[0, 0] == 6
    x[0, 0] = 8                         # the next power of two: scale 2
    codes, s = mx.quantize(x)
    assert s[0, 0] == 128 and mx.values(codes, s)[0, 0] == 8
    x[0, 40] = np.inf
    assert np.isnan(mx.round_trip(x)[0, 32:]).all() and np.isfinite(mx.round_trip(x)[0, :32]).all()


@pytest.mark.parametrize("R,K", [(1, 32), (130, 288), (256, 512), (300, 96)])
def test_scale_tiles(R, K):
    s = np.random.default_rng(R).integers(0, 255, (R, K // 32), dtype=np.uint8)
    t = L.mxfp4_tile_scales(torch.from_numpy(s))
    assert tuple(t.shape) == L.mxfp4_scales_shape(R, K)
    assert np.array_equal(t.numpy(), mx.tile(s))
    assert np.array_equal(L.mxfp4_untile_scales(t, R, K).numpy(), s)
    assert L.llmint8_mxfp4_scales_size(R, K) == t.numel()


def test_sizes(lib):
    assert L.llmint8_mxfp4_scales_size(0, 64) == 0
    for bad in (0, 16, 48, 131072 + 32):
        assert L.llmint8_mxfp4_scales_size(128, bad) == 0
        assert L.llmint8_mxfp4_linear_workspace_size(16, 128, bad) == 0
    assert L.llmint8_mxfp4_linear_workspace_size(-1, 128, 64) == 0
    assert L.llmint8_mxfp4_linear_workspace_size(16, 0, 64) == 0
    assert L.llmint8_mxfp4_linear_workspace_size(16, 1, 64) >= 256 + 16 * 32 + 1024


def test_quantize_refusals(lib):
    f = lib.llmint8_mxfp4_quantize
    call = lambda x=FAKE, dt=0, R=4, K=64, ld=64, c=FAKE, s=FAKE: f(x, dt, R, K, ld, c, s, None)  # noqa: E731
    for dt in (-1, 3):
        assert call(dt=dt) == L.ERR_INVALID_ARG
    for K in (0, -32, 16, 48, 131072 + 32):
        assert call(K=K, ld=1 << 20) == L.ERR_UNSUPPORTED_SHAPE
    for R in (-1, 1 << 31):
        assert call(R=R) == L.ERR_UNSUPPORTED_SHAPE
    assert call(x=None) == call(c=None) == call(s=None) == L.ERR_INVALID_ARG
    assert call(x=ODD) == call(c=ODD) == call(s=ODD) == L.ERR_INVALID_ARG
    assert call(ld=32) == call(ld=68) == L.ERR_INVALID_ARG     # too short, off 16 bytes
    assert call(ld=(1 << 63) - 8) == call(ld=1 << 30) == L.ERR_INVALID_ARG
    assert f(None, 0, 0, 64, 64, None, None, None) == L.OK     # no rows: nothing to do


def test_dequant_refusals(lib):
    f = lib.llmint8_mxfp4_dequant
    assert f(FAKE, FAKE, 4, 64, FAKE, 3, None) == L.ERR_INVALID_ARG
    assert f(FAKE, FAKE, 4, 48, FAKE, 0, None) == L.ERR_UNSUPPORTED_SHAPE
    assert f(FAKE, FAKE, -4, 64, FAKE, 0, None) == L.ERR_UNSUPPORTED_SHAPE
    for bad in (None, ODD):
        assert f(bad, FAKE, 4, 64, FAKE, 0, None) == L.ERR_INVALID_ARG
        assert f(FAKE, bad, 4, 64, FAKE, 0, None) == L.ERR_INVALID_ARG
        assert f(FAKE, FAKE, 4, 64, bad, 0, None) == L.ERR_INVALID_ARG
    assert f(None, None, 0, 64, None, 0, None) == L.OK


def test_linear_refusals(lib):
    def call(x=FAKE, dt=0, M=4, K=64, ld=64, wc=FAKE, ws=FAKE, N=8, b=None, y=FAKE, w=FAKE,
             n=1 << 30):
        return lib.llmint8_mxfp4_linear(x, dt, M, K, ld, wc, ws, N, b, y, w, n, None)

    def quantized(xc=FAKE, xs=FAKE, M=4, K=64, wc=FAKE, ws=FAKE, N=8, b=None, y=FAKE, dt=0, w=FAKE,
                  n=256):
        return lib.llmint8_mxfp4_linear_quantized(xc, xs, M, K, wc, ws, N, b, y, dt, w, n, None)

    for f in (call, quantized):
        for dt in (-1, 2, 3):                      # no fp32 layer
            assert f(dt=dt) == L.ERR_INVALID_ARG
        assert f(K=48) == f(K=0) == f(K=131072 + 32) == L.ERR_UNSUPPORTED_SHAPE
        assert f(M=-1) == f(N=0) == f(N=-5) == f(M=1 << 31) == f(N=1 << 31) == \
            L.ERR_UNSUPPORTED_SHAPE
        for bad in (None, ODD):
            assert f(wc=bad) == f(ws=bad) == f(y=bad) == f(w=bad) == L.ERR_INVALID_ARG
        assert f(b=ODD) == L.ERR_INVALID_ARG
        assert f(n=255) == L.ERR_WORKSPACE_TOO_SMALL
        assert f(M=0) == L.OK
    assert call(n=L.llmint8_mxfp4_linear_workspace_size(4, 8, 64) - 1) == \
        L.ERR_WORKSPACE_TOO_SMALL
    assert call(x=None) == call(x=ODD) == call(ld=56) == call(ld=68) == L.ERR_INVALID_ARG
    assert quantized(xc=None) == quantized(xs=ODD) == L.ERR_INVALID_ARG


def test_outputs_that_overlap_are_refused(lib):
    at = lambda off: ctypes.c_void_p((1 << 20) + off)  # noqa: E731
    far = ctypes.c_void_p(1 << 30)
    bad = L.ERR_INVALID_ARG
    q = lib.llmint8_mxfp4_quantize
    assert q(at(0), 0, 4, 64, 64, at(496), far, None) == bad       # codes in X's last row
    assert q(at(0), 0, 4, 64, 64, far, at(0), None) == bad
    assert q(at(0), 0, 4, 64, 64, far, far, None) == bad
    d = lib.llmint8_mxfp4_dequant
    assert d(at(0), far, 4, 64, at(112), 0, None) == bad
    assert d(far, at(0), 4, 64, at(1008), 0, None) == bad

    def linear(x=at(0), wc=at(1 << 16), ws=at(2 << 16), y=at(3 << 16), b=None, w=at(4 << 16)):
        return lib.llmint8_mxfp4_linear(x, 0, 4, 64, 64, wc, ws, 8, b, y, w, 4096, None)
    assert linear(y=at(496)) == linear(y=at((1 << 16) + 240)) == linear(y=at((2 << 16) + 1008)) == bad
    assert linear(b=at((3 << 16) + 48)) == linear(w=at((3 << 16) + 48)) == linear(w=at(0)) == bad
    f = lib.llmint8_mxfp4_linear_quantized
    assert f(at(0), far, 4, 64, at(1 << 16), at(2 << 16), 8, None, at(112), 0, at(4 << 16), 256,
             None) == bad

    def norm(H=at(1 << 16), Y=at(2 << 16), c=None, s=None, ldx=64, w=None):
        return lib.llmint8_residual_norm(at(0), 0, 4, 64, ldx, at(3 << 16), 64, 0, None, None, None,
                                         1, ctypes.c_float(1), 1, w, None, ctypes.c_float(0), H, Y,
                                         c, s, None)
    assert norm(H=at(16)) == norm(Y=at((3 << 16) + 16)) == bad     # shifted against X, the residual
    assert norm(H=at(0), ldx=72) == bad                            # X's buffer, but not X's rows
    assert norm(H=at(1 << 16), Y=at(1 << 16)) == norm(H=at(0), Y=at(0)) == bad
    assert norm(c=at(0), s=far) == norm(c=far, s=at((3 << 16) + 496)) == bad
    assert norm(w=at((2 << 16) + 496)) == bad


def test_residual_norm_refusals(lib):
    nan, inf = float("nan"), float("inf")

    def call(x=FAKE, dt=0, M=4, K=64, ld=64, r=FAKE, ldr=64, post=0, pw=None, pb=None, g=None, G=1,
             scale=1.0, norm=1, w=None, b=None, eps=1e-6, H=FAKE, Y=FAKE, c=None, s=None):
        return lib.llmint8_residual_norm(x, dt, M, K, ld, r, ldr, post, pw, pb, g, G,
                                         ctypes.c_float(scale), norm, w, b, ctypes.c_float(eps),
                                         H, Y, c, s, None)

    bad = L.ERR_INVALID_ARG
    assert call(dt=2) == call(norm=3) == call(norm=-1) == call(post=3) == bad
    assert call(eps=-1.0) == call(eps=nan) == call(eps=inf) == bad
    assert call(K=48) == call(K=32768 + 32, ld=1 << 20, ldr=1 << 20) == call(M=-1) == \
        L.ERR_UNSUPPORTED_SHAPE
    assert call(x=None) == call(x=ODD) == call(r=ODD) == call(H=ODD) == call(Y=ODD) == bad
    assert call(ld=32) == call(ldr=32) == call(ld=68) == call(ldr=68) == bad
    assert call(post=1, pw=ODD) == call(post=1, pb=ODD) == call(w=ODD) == call(b=ODD) == bad
    assert call(pw=FAKE) == call(pb=FAKE) == bad            # a post norm's, without one
    assert call(g=ODD) == call(g=FAKE, G=3) == call(g=FAKE, G=0) == bad
    assert call(c=FAKE) == call(s=FAKE) == call(c=ODD, s=FAKE) == bad
    assert call(norm=0) == call(norm=0, Y=None, w=FAKE) == bad      # no norm, yet a Y, a weight
    assert call(Y=None) == call(norm=0, H=None, Y=None) == bad      # nothing to write
    assert call(M=0) == L.OK


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.float16)
    with pytest.raises(ValueError, match="CUDA"):
        L.llmint8_mxfp4_quantize(x)
    with pytest.raises(TypeError):
        L.llmint8_mxfp4_quantize(x.double())
    with pytest.raises(TypeError):
        L.llmint8_mxfp4_linear(x.float(), None, None)
    with pytest.raises(ValueError, match="two dimensions"):
        L.llmint8_residual_norm(x[0])
    with pytest.raises(ValueError):
        L.mxfp4_tile_scales(x)
    with pytest.raises(ValueError):
        L.mxfp4_untile_scales(torch.zeros((1, 1, 512), dtype=torch.uint8), 4, 64)
