"""64-bit statements of MXFP4, its product and the residual norm, for the tests: plain numpy, from
the definitions in include/llmint8.h."""
from __future__ import annotations

import numpy as np

GRID = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float64)
VALUES = np.concatenate([GRID, -GRID])


def quantize(x: np.ndarray):
    """x [R, K] -> (codes uint8 [R, K], scale bytes uint8 [R, K/32]), both in plain order; codes of
    NaN blocks are unspecified (0 here)."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    v = x.reshape(R, K // 32, 32)
    top = np.abs(v).max(-1)
    bad = ~np.isfinite(top)
    e = np.frexp(np.where(bad | (top == 0), 1.0, top))[1] - 1      # floor(log2 top)
    e = np.where(top == 0, -127, np.maximum(e - 2, -127))
    with np.errstate(invalid="ignore"):
        a = np.ldexp(v, -e[..., None])
    m = np.where(np.isfinite(a), np.abs(a), 0.0)
    # index of the nearest grid value; a tie goes to the even index
    mid = (GRID[:-1] + GRID[1:]) / 2
    i = (m[..., None] > mid).sum(-1)
    for k in range(1, 7, 2):                # between an odd k and k + 1, a tie goes up
        i = np.where(m == mid[k], k + 1, i)
    codes = (i + 8 * np.signbit(a)).astype(np.uint8)
    codes[bad] = 0
    return codes.reshape(R, K), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Plain codes [R, K] and scale bytes [R, K/32] -> fp64 [R, K]."""
    R, K = codes.shape
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (VALUES[codes].reshape(R, K // 32, 32) * s[..., None]).reshape(R, K)


def round_trip(x: np.ndarray) -> np.ndarray:
    return values(*quantize(x))


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    R, half = packed.shape
    out = np.empty((R, 2 * half), np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def tile(scales: np.ndarray) -> np.ndarray:
    """Scale bytes [R, K/32] in tiles, byte by byte as the header states; padding 0."""
    R, B = scales.shape
    out = np.zeros((-(-R // 128), -(-B // 8), 1024), np.uint8)
    r, b = np.meshgrid(np.arange(R), np.arange(B), indexing="ij")
    out[r // 128, b // 8, 512 * (b % 8 // 4) + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4] = scales
    return out


# Half a step of rounding to the type, relative to the value, and half its smallest step.
HALF_EPS = {"float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}


def product(xq: np.ndarray, wq: np.ndarray, bias, dtype: str):
    """(Y, tolerance) of xq . wq^T + bias for fp64 values of MXFP4 matrices.

    The 32 products of a block are multiples of 1/4 up to 36 times one power of two, so their sum
    is exact in fp32; each of the K / 32 such sums is then added to an accumulator whose size
    never passes sum |x w|, with at most one step (2^-23, truncation allowed) lost each time;
    adding the parts of up to 8 CTAs, and the bias, is 9 additions more; the output is rounded once."""
    y = xq @ wq.T
    size = np.abs(xq) @ np.abs(wq).T
    if bias is not None:
        y = y + bias
        size = size + np.abs(bias)
    rel, least = HALF_EPS[dtype]
    steps = xq.shape[1] // 32 + 9
    return y, np.abs(y) * rel + least + size * steps * 2.0 ** -23 * (1 + rel)


U = 2.0 ** -24        # half a step of fp32


def norm(v, kind, w, b, eps, err):
    """(norm of the rows of v, bound of the fp32 evaluation's error), given the error bound `err`
    of v itself.  A row's sum is taken in at most 32 + 10 additions one after another, each of at
    most U of the sum of magnitudes; 64 U covers them and the few operations of each element."""
    if kind is None:
        return v, err
    c = 64 * U
    mean = v.mean(1, keepdims=True) if kind == "layer" else 0.0
    mean_err = (c * np.abs(v).mean(1, keepdims=True) + err.mean(1, keepdims=True)) \
        if kind == "layer" else 0.0
    d = v - mean
    d_err = err + mean_err + U * np.abs(d)
    r = 1 / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    # d(1/r^2) = 2 mean(d d_err): relative error of r
    r_rel = c + r * r * (np.abs(d) * d_err).mean(1, keepdims=True) + \
        r * r * (d_err * d_err).mean(1, keepdims=True)
    w = np.ones(v.shape[1]) if w is None else w
    b = np.zeros(v.shape[1]) if b is None else b
    y = d * r * w
    out_err = (d_err * r * np.abs(w)) * (1 + r_rel) + np.abs(y) * (r_rel + 4 * U)
    return y + b, out_err + U * np.abs(y + b)


def residual_norm(x, residual, post, post_w, post_b, gate, scale, kind, w, b, eps, dtype):
    """(H, its tolerance, Y, its tolerance), fp64."""
    t, err = norm(x, post, post_w, post_b, eps, np.zeros_like(x))
    scale = float(np.float32(scale))
    if gate is not None:
        g = np.repeat(gate, x.shape[0] // gate.shape[0], 0)
        t, err = t * g, err * np.abs(g) + U * np.abs(t * g)
    h = t * scale + (0 if residual is None else residual)
    err = err * abs(scale) + U * np.abs(h)
    rel, least = HALF_EPS[dtype]
    y, y_err = norm(h, kind, w, b, eps, err)
    return (h, np.abs(h) * rel + least + err * (1 + rel),
            y, np.abs(y) * rel + least + y_err * (1 + rel))
