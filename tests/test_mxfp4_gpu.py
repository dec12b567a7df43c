"""MXFP4 quantisation, product and the residual norm on the GPU against their 64-bit statements
(mx_util): codes and scales bit for bit, products and norms within derived bounds."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from int8_quantized_02_b200 import llmint8 as L
from tests import mx_util as mx

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
NAME = {F16: "float16", BF16: "bfloat16", F32: "float32"}


def f64(t):
    return t.detach().double().cpu().numpy()


def matrix(M, K, dtype, seed=0, spread=3.0):
    """N(0, 1) rows of sizes spread over powers of two, with a few large columns."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=g) * torch.exp2(spread * torch.randn((M, 1), generator=g))
    x[:, torch.randint(0, K, (3,), generator=g)] *= 12
    return x.to(dtype).cuda()


def assert_mx(codes, scales, x):
    """codes, scales (device) are exactly x's, NaN blocks' codes apart; padding is 0."""
    want, s = mx.quantize(f64(x))
    assert np.array_equal(scales.cpu().numpy(), mx.tile(s))
    got = mx.unpack(codes.cpu().numpy())
    fine = np.repeat(s != 255, 32, 1)
    # a negative value that rounds to zero keeps its sign in the code
    assert np.array_equal(got[fine], want[fine])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 4096), (3, 96), (127, 256), (129, 288), (300, 2080),
                                 (1000, 1024), (5000, 8192)])
def test_quantize(R, K, dtype):
    x = matrix(R, K, dtype, seed=R + K)
    codes, scales = L.llmint8_mxfp4_quantize(x)
    assert_mx(codes, scales, x)
    again = L.llmint8_mxfp4_quantize(x)
    assert torch.equal(codes, again[0]) and torch.equal(scales, again[1])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_edges(dtype):
    """Ties, the format's ends, zeros of both signs, subnormals, infinities and NaN."""
    x = torch.zeros((8, 128), dtype=torch.float64)
    x[0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -6, -.25, -.75, -1.25, -1.75,
                              -2.5, -3.5, -5])
    x[1, :4] = torch.tensor([7.99, -7.99, 1e-7, -0.0])
    fi = torch.finfo(dtype)
    x[2, :3] = torch.tensor([fi.max, -fi.max, fi.tiny])
    x[3, :3] = torch.tensor([fi.smallest_normal, fi.smallest_normal / 2, -fi.smallest_normal / 4])
    x[4, 5], x[4, 40], x[4, 70] = float("inf"), float("nan"), -float("inf")
    x[5] = -0.0
    x[6, 32:64] = torch.exp2(torch.arange(32.0, dtype=torch.float64) - 20)
    x = x.to(dtype).cuda()
    codes, scales = L.llmint8_mxfp4_quantize(x)
    assert_mx(codes, scales, x)
    v = L.llmint8_mxfp4_dequant(codes, scales, dtype=F32)
    assert torch.isnan(v[4, :96]).all() and (v[4, 96:] == 0).all()


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("R,K", [(1, 32), (130, 288), (2000, 2080)])
def test_dequant(R, K, dtype):
    rng = np.random.default_rng(R)
    codes = rng.integers(0, 16, (R, K), dtype=np.uint8)
    s = rng.integers(0, 256, (R, K // 32), dtype=np.uint8)        # every scale, NaN included
    v = L.llmint8_mxfp4_dequant(torch.from_numpy(mx.pack(codes)).cuda(),
                                torch.from_numpy(mx.tile(s)).cuda(), dtype=dtype)
    want = torch.from_numpy(mx.values(codes, s)).float()          # 3 bits: exact, or infinite
    want = want.to(dtype)
    got = v.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(1.0, 2.0, -2.0), want.nan_to_num(1.0, 2.0, -2.0))


def test_quantize_takes_row_pitches_and_leaves_the_rest():
    big = matrix(50, 512, F16)
    x = big[:, 64:64 + 288]
    for rows in (x, x[::2], x[7:8]):
        codes, scales = L.llmint8_mxfp4_quantize(rows)
        assert_mx(codes, scales, rows)
    guard = torch.full((60, 144), 77, dtype=torch.uint8, device="cuda")
    L.llmint8_mxfp4_quantize(x, codes=guard[5:55])
    assert (guard[:5] == 77).all() and (guard[55:] == 77).all()
    with pytest.raises(ValueError):
        L.llmint8_mxfp4_quantize(big[:, 4:4 + 288])                # rows off 16 bytes
    with pytest.raises(ValueError):
        L.llmint8_mxfp4_quantize(big.t())
    with pytest.raises(ValueError):
        L.llmint8_mxfp4_quantize(big[:1].expand(4, 512))
    assert L.llmint8_mxfp4_quantize(big[:0])[0].shape == (0, 256)


# ------------------------------------------------------------------------------ product ------

def layer(M, N, K, dtype, bias=True, seed=0):
    x = matrix(M, K, dtype, seed, spread=1.0)
    w = matrix(N, K, dtype, seed + 1, spread=1.0)
    b = torch.randn(N, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda() if bias \
        else None
    return x, w, b, L.llmint8_mxfp4_quantize(w)


def assert_product(y, x, w, b, dtype):
    want, tol = mx.product(mx.round_trip(f64(x)), mx.round_trip(f64(w)),
                           None if b is None else f64(b), NAME[dtype])
    off = np.abs(f64(y) - want)
    assert y.shape == want.shape and np.isfinite(off).all()
    assert (off <= tol).all(), (off / tol).max()


SHAPES = [(1, 1, 32), (1, 130, 131072), (3, 200, 8224), (7, 96, 2080), (8, 130, 4096), (8, 257, 16416), (9, 300, 4128), (15, 1000, 2080), (16, 77, 16416), (11, 4096, 8192), (1, 1024, 1024), (2, 130, 64), (5, 129, 96), (16, 512, 4096), (17, 300, 288),
          (33, 128, 544), (64, 257, 1056), (65, 96, 2080), (128, 640, 512), (129, 1000, 320),
          (255, 77, 800), (256, 256, 256), (257, 256, 32), (300, 1003, 2080), (513, 520, 96),
          (700, 31, 1312), (1000, 2050, 512), (100, 16000, 96), (1200, 1003, 288),
          (1300, 2500, 1056),
          # enough bands for three CTAs to an SM, and more k-tiles than their stages
          (2, 38100, 1568), (12, 38100, 1056), (16, 38100, 1568), (20, 38100, 1056), (50, 38100, 1056)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K, dtype):
    x, w, b, (wc, ws) = layer(M, N, K, dtype, bias=(M + N) % 2 == 0, seed=M)
    need = L.llmint8_mxfp4_linear_workspace_size(M, N, K)
    # scales of X that no row has are whatever the workspace held: the NaN scale here
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    y = L.llmint8_mxfp4_linear(x, wc, ws, bias=b, workspace=work)
    assert_product(y, x, w, b, dtype)
    assert L.llmint8_device_status(work) == L.OK
    again = L.llmint8_mxfp4_linear(x, wc, ws, bias=b)
    assert torch.equal(y, again)
    xc, xs = L.llmint8_mxfp4_quantize(x)
    assert torch.equal(y, L.llmint8_mxfp4_linear_quantized(xc, xs, wc, ws, bias=b, dtype=dtype))


@pytest.mark.parametrize("M", [9, 100, 4000])
def test_linear_takes_row_pitches_and_leaves_the_rest(M):
    N, K = 333, 288
    big = matrix(M, K + 64, BF16)
    x, w = big[:, 32:32 + K], matrix(N, K, BF16, seed=5, spread=1.0)
    wc, ws = L.llmint8_mxfp4_quantize(w)
    out = torch.full((M + 2, N), 7.0, dtype=BF16, device="cuda").view(-1)
    at = (N + 7) // 8 * 8                       # outputs start on 16 bytes
    y = out[at:at + M * N].view(M, N)
    L.llmint8_mxfp4_linear(x, wc, ws, Y=y)
    assert_product(y, x, w, None, BF16)
    assert (out[:at] == 7).all() and (out[at + M * N:] == 7).all()
    assert L.llmint8_mxfp4_linear(x[:0], wc, ws).shape == (0, N)


@pytest.mark.parametrize("M", [4, 300, 5000])
def test_a_row_or_channel_of_nan_stays_alone(M):
    N, K = 200, 320
    x, w, b, _ = layer(M, N, K, F16)
    x[1, 7] = float("inf")                      # one block of row 1
    w[3, 40] = float("nan")                     # one block of channel 3
    wc, ws = L.llmint8_mxfp4_quantize(w)
    y = L.llmint8_mxfp4_linear(x, wc, ws, bias=b)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[1] = True
    bad[:, 3] = True
    assert torch.equal(torch.isnan(y), bad)
    x[1, 7] = 0
    w[3, 40] = 0
    x[1, :32], w[3, 32:64] = 0, 0
    want, tol = mx.product(mx.round_trip(f64(x)), mx.round_trip(f64(w)), f64(b), "float16")
    fine = ~bad.cpu().numpy()
    assert (np.abs(f64(y) - want) <= tol)[fine].all()


def test_linear_past_two_to_the_31_outputs():
    M, N, K = 70000, 31000, 32                  # 2.17e9 outputs
    x, w = matrix(M, K, F16, spread=1.0), matrix(N, K, F16, seed=3, spread=1.0)
    y = L.llmint8_mxfp4_linear(x, *L.llmint8_mxfp4_quantize(w))
    for rows in (slice(0, 3), slice(35000, 35003), slice(M - 3, M)):
        assert_product(y[rows], x[rows], w, None, F16)


# --------------------------------------------------------------------------------- norm ------

def norm_inputs(M, K, dtype, norm, post, gate, residual, affine, seed=0):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    put = lambda t: t.to(dtype).cuda()  # noqa: E731
    a = {"norm": norm, "post_norm": post, "scale": 0.7, "eps": 1e-5}
    x = put(rand(M, K) * torch.exp2(2 * rand(M, 1)) + rand(M, 1))
    if residual:
        a["residual"] = put(3 * rand(M, K) + 1)
    if affine:
        if norm:
            a["weight"] = put(1 + 0.2 * rand(K))
            a["bias"] = put(0.3 * rand(K))
        if post:
            a["post_weight"] = put(1 + 0.2 * rand(K))
            a["post_bias"] = put(0.3 * rand(K))
    if gate:
        a["gate"] = put(rand(gate, K))
    return x, a


def assert_norm(H, Y, x, a, dtype):
    d = lambda k: None if a.get(k) is None else f64(a[k])  # noqa: E731
    gate = d("gate")
    if gate is not None and gate.ndim == 1:
        gate = gate[None]
    h, ht, y, yt = mx.residual_norm(f64(x), d("residual"), a["post_norm"], d("post_weight"),
                                    d("post_bias"), gate, a["scale"], a["norm"], d("weight"),
                                    d("bias"), a["eps"], NAME[dtype])
    assert (np.abs(f64(H) - h) <= ht).all(), (np.abs(f64(H) - h) / ht).max()
    if a["norm"]:
        assert (np.abs(f64(Y) - y) <= yt).all(), (np.abs(f64(Y) - y) / yt).max()
    else:
        assert Y is None


NORMS = [("rms", None, 0, True, True), ("layer", None, 0, True, True), ("rms", "rms", 1, True, True),
         ("layer", "layer", 1, True, True), ("rms", "layer", "M", True, False),
         (None, "rms", 1, True, True), ("layer", None, 0, False, False), ("rms", None, 2, True, True)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("norm,post,gate,residual,affine", NORMS)
@pytest.mark.parametrize("M,K", [(1, 32), (2, 4096), (6, 288), (130, 2080), (300, 1056),
                                 (200, 12288), (2, 32768), (160, 17408), (150, 16384),
                                 (151, 14368), (149, 768)])
def test_residual_norm(M, K, norm, post, gate, residual, affine, dtype):
    gate = M if gate == "M" or (gate and M % gate) else gate
    x, a = norm_inputs(M, K, dtype, norm, post, gate, residual, affine, seed=M + K)
    H, Y = L.llmint8_residual_norm(x, **a)
    assert_norm(H, Y, x, a, dtype)
    if norm:
        H2, codes, scales = L.llmint8_residual_norm_mxfp4(x, **a)
        want = L.llmint8_mxfp4_quantize(Y)
        assert torch.equal(H, H2)
        assert torch.equal(codes, want[0]) and torch.equal(scales, want[1])


def test_residual_norm_in_place_and_with_pitches():
    M, K = 70, 1056
    x, a = norm_inputs(M, K, BF16, "rms", "rms", 1, True, True)
    H, Y = L.llmint8_residual_norm(x, **a)
    wide = torch.zeros((M, K + 32), dtype=BF16, device="cuda")
    wide[:, 16:16 + K] = x
    wider = torch.zeros((2 * M, K), dtype=BF16, device="cuda")
    wider[::2] = a["residual"]
    H2, Y2 = L.llmint8_residual_norm(wide[:, 16:16 + K], **{**a, "residual": wider[::2]})
    assert torch.equal(H, H2) and torch.equal(Y, Y2)
    res, xx = a["residual"].clone(), x.clone()
    L.llmint8_residual_norm(xx, **{**a, "residual": res}, H=res, Y=xx)
    assert torch.equal(H, res) and torch.equal(Y, xx)


def test_residual_norm_extremes():
    """Rows of zeros, of one value, and with a NaN or an infinity, which stay alone."""
    x = torch.randn((6, 512), device="cuda").half()
    x[0] = 0
    x[1] = 3
    x[2, 5] = float("nan")
    x[3, 6] = float("inf")
    clean = L.llmint8_residual_norm(x[4:], norm="layer", eps=1e-5)[1]
    H, Y = L.llmint8_residual_norm(x, norm="layer", eps=1e-5)
    assert (Y[0] == 0).all() and (Y[1] == 0).all()
    assert torch.isnan(Y[2]).all() and torch.isnan(Y[3]).all()
    assert torch.equal(Y[4:], clean)
    H, codes, scales = L.llmint8_residual_norm_mxfp4(x, norm="layer", eps=1e-5)
    assert (L.mxfp4_untile_scales(scales, 6, 512)[2:4] == 255).all()


# ------------------------------------------------------------------- as they would be used ----

def block(x, res, w1, w2, a):
    """Two blocks' worth: norm -> product -> norm with the residual -> product."""
    h, c, s = L.llmint8_residual_norm_mxfp4(x, residual=res, **a)
    y = L.llmint8_mxfp4_linear_quantized(c, s, *w1, dtype=x.dtype)
    h, c, s = L.llmint8_residual_norm_mxfp4(y, residual=h, post_norm="rms", **a)
    return h, L.llmint8_mxfp4_linear_quantized(c, s, *w2, dtype=x.dtype)


@pytest.mark.parametrize("M", [1, 40, 300, 1400])
def test_a_run_of_them_together(M):
    K, N = 512, 1003
    g = torch.Generator().manual_seed(M)
    x = torch.randn((M, K), generator=g).half().cuda()
    res = torch.randn((M, K), generator=g).half().cuda()
    W1 = (0.05 * torch.randn((K, K), generator=g)).half().cuda()
    W2 = (0.05 * torch.randn((N, K), generator=g)).half().cuda()
    a = {"norm": "rms", "eps": 1e-5, "weight": (1 + 0.1 * torch.randn(K, generator=g)).half().cuda()}
    w1, w2 = L.llmint8_mxfp4_quantize(W1), L.llmint8_mxfp4_quantize(W2)
    h, y = block(x, res, w1, w2, a)
    # step by step, each step from the values that the step before it stored
    H1, Y1 = L.llmint8_residual_norm(x, residual=res, **a)
    assert_norm(H1, Y1, x, {**a, "residual": res, "post_norm": None, "scale": 1.0}, F16)
    Z1 = L.llmint8_mxfp4_linear(Y1, *w1)
    assert_product(Z1, Y1, W1, None, F16)
    H2, Y2 = L.llmint8_residual_norm(Z1, residual=H1, post_norm="rms", **a)
    assert_norm(H2, Y2, Z1, {**a, "residual": H1, "post_norm": "rms", "scale": 1.0}, F16)
    Z2 = L.llmint8_mxfp4_linear(Y2, *w2)
    assert_product(Z2, Y2, W2, None, F16)
    assert torch.equal(h, H2) and torch.equal(y, Z2)


def test_the_layer_between_int8_layers():
    """The norm's 16-bit output feeds the int8 layer as any fp16 matrix does."""
    M, K, N = 20, 512, 256
    x, a = norm_inputs(M, K, F16, "rms", None, 0, True, True)
    CB, SCB = L.llmint8_quantize_weight_colwise(matrix(N, K, F16, seed=2, spread=0.1) * 0.02)
    H, Y = L.llmint8_residual_norm(x, **a)
    y = L.llmint8_linear(Y, CB, SCB)
    assert torch.equal(y, L.llmint8_linear(Y.clone(), CB, SCB)) and torch.isfinite(y).all()


def test_streams_graphs_and_plans():
    M, K, N = 24, 1024, 520
    x, w, b, (wc, ws) = layer(M, N, K, F16)
    a = {"norm": "rms", "residual": x.clone()}
    want = L.llmint8_mxfp4_linear(x, wc, ws, bias=b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = L.llmint8_mxfp4_linear(x, wc, ws, bias=b, stream=side)
    hs = L.llmint8_residual_norm(x, **a, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    assert all(torch.equal(p, q) for p, q in zip(hs, L.llmint8_residual_norm(x, **a)))
    plan = L.Mxfp4LinearPlan(x, wc, ws, bias=b)
    assert torch.equal(plan(), want)

    # captured: two products and a norm; replayed on other values of the same buffers
    big = matrix(2000, K, F16, seed=9, spread=1.0)
    static, static_big = x.clone(), big.clone()
    graph = torch.cuda.CUDAGraph()
    for _ in range(2):
        L.llmint8_mxfp4_linear(static, wc, ws, bias=b)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = L.llmint8_mxfp4_linear(static, wc, ws, bias=b)
        out_big = L.llmint8_mxfp4_linear(static_big, wc, ws)
        H, c, s = L.llmint8_residual_norm_mxfp4(static, norm="layer")
        out_norm = L.llmint8_mxfp4_linear_quantized(c, s, wc, ws)
    for seed in (1, 2):
        new = matrix(M, K, F16, seed=seed)
        static.copy_(new)
        static_big.copy_(matrix(2000, K, F16, seed=seed + 20, spread=1.0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, L.llmint8_mxfp4_linear(new, wc, ws, bias=b))
        assert torch.equal(out_big, L.llmint8_mxfp4_linear(static_big, wc, ws))
        Y = L.llmint8_residual_norm(new, norm="layer")[1]
        assert torch.equal(out_norm, L.llmint8_mxfp4_linear(Y, wc, ws))


def test_a_stream_argument_inside_a_capture():
    x, w, b, (wc, ws) = layer(20, 520, 512, F16)
    want = L.llmint8_mxfp4_linear(x, wc, ws, bias=b)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        y = L.llmint8_mxfp4_linear(x, wc, ws, bias=b, stream=side)
        q = L.llmint8_mxfp4_quantize(x, stream=side)
        v = L.llmint8_mxfp4_dequant(*q, stream=side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    assert torch.equal(v, L.llmint8_mxfp4_dequant(*L.llmint8_mxfp4_quantize(x)))


def test_inputs_dropped_while_another_stream_works():
    """Temporaries handed to a call on another stream keep their memory until that stream is done."""
    x, w, b, (wc, ws) = layer(2000, 2048, 2048, F16, seed=3)
    want = L.llmint8_mxfp4_linear(x, wc, ws)
    side = torch.cuda.Stream()
    got = []
    for _ in range(10):
        temp = x.clone()
        side.wait_stream(torch.cuda.current_stream())
        got.append(L.llmint8_mxfp4_linear(temp, wc, ws, stream=side))
        del temp
        torch.full_like(x, 7.0)                 # would take the memory of the one dropped
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


def test_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    layers = [layer(m, 2048, 2048, F16, seed=m) for m in (8, 200, 1500)]
    want = [L.llmint8_mxfp4_linear(x, *q, bias=b) for x, w, b, q in layers]
    streams = [torch.cuda.Stream() for _ in layers]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(20):
        got.append([L.llmint8_mxfp4_linear(x, *q, bias=b, stream=s)
                    for s, (x, w, b, q) in zip(streams, layers)])
    torch.cuda.synchronize()
    for ys in got:
        assert all(torch.equal(y, v) for y, v in zip(ys, want))


def test_binding_checks_shapes_and_types():
    x, w, b, (wc, ws) = layer(4, 64, 256, F16)
    with pytest.raises(ValueError):
        L.llmint8_mxfp4_linear(x[:, :128], wc, ws)
    with pytest.raises(ValueError):
        L.llmint8_mxfp4_linear(x, wc, ws[:, :, :512])
    with pytest.raises(TypeError):
        L.llmint8_mxfp4_linear(x, wc, ws, bias=b.float())
    with pytest.raises(TypeError):
        L.llmint8_mxfp4_linear(x.bfloat16(), wc, ws, bias=b)
    with pytest.raises(L.LLMInt8Error):
        L.llmint8_mxfp4_linear(x, wc, ws, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(L.LLMInt8Error):
        L.llmint8_mxfp4_quantize(x[:, :48].contiguous())
    with pytest.raises(ValueError):
        L.llmint8_residual_norm(x, gate=torch.zeros((3, 256), dtype=F16, device="cuda"))
    with pytest.raises(TypeError):
        L.llmint8_residual_norm(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        L.llmint8_residual_norm(x, norm="batch")


@pytest.mark.parametrize("M", [8, 1500])
def test_a_wait_that_runs_out_is_reported(M):
    """A bound of 1 ns makes waits give up: the call ends, says so, and the next one is right.  (The
    few microseconds that a band's waits last may pass before the clock is first read; the
    accumulator of a pair takes tens of them with K = 16384.)"""
    N, K = (4096, 4096) if M == 8 else (1024, 16384)
    x, w, b, (wc, ws) = layer(M, N, K, F16)
    work = torch.empty(L.llmint8_mxfp4_linear_workspace_size(M, N, K), dtype=torch.uint8,
                       device="cuda")
    seen = set()
    L.llmint8_set_wait_timeout_ns(1)
    try:
        for _ in range(3):
            L.llmint8_mxfp4_linear(x, wc, ws, workspace=work)
            seen.add(L.llmint8_device_status(work))
    finally:
        L.llmint8_set_wait_timeout_ns(0)
    assert seen <= {L.OK, L.ERR_TIMEOUT} and (M == 8 or L.ERR_TIMEOUT in seen)
    y = L.llmint8_mxfp4_linear(x, wc, ws, workspace=work)
    assert L.llmint8_device_status(work) == L.OK
    assert_product(y[:4], x[:4], w, None, F16)
