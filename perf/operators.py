"""The 4-bit microscaled (MXFP4) operators and the residual norm that feeds them: cases, plain
forms, the library's calls and a 64-bit statement of each definition.

Formats.  An MXFP4 matrix of R rows and K columns (K a multiple of 32) is
  codes  uint8 [R, K/2]: element k of a row in the low (k even) or high (k odd) half of byte k/2,
         an e2m1 code (sign, 2 exponent bits, 1 mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6);
  scales uint8 [ceil(R/128), ceil(K/256), 1024]: one e8m0 scale 2^(s - 127) (255 = NaN) for each 32
         consecutive elements of a row, in tiles of 128 rows x 256 columns; inside a tile, block b
         (of 8) of row r lies at byte 512 (b / 4) + 16 (r % 32) + 4 (r / 32) + b % 4.
Quantisation takes 2^(floor(log2 max|x|) - 2) as a block's scale, rounds x / scale to the nearest
e2m1 value (ties to the even code, beyond 6 to 6), and gives a block with a NaN or an infinity the
NaN scale.

Kinds of case:
  quantize  values -> codes and scales -> values again (both operators of the format)
  linear    Y = q(X) . W^T + bias, W held as MXFP4, X quantised in the call
  norm      H = residual + scale * gate * PostNorm(X);  Y = Norm(H)
  block     norm, its Y left as MXFP4 only, and the product that takes it: H and the product
"""
import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's activations, the smallest call
        dict(name="quantize_1x1024_f16", kind="quantize", R=1, K=1024, dtype="f16"),
        # the weight of the 6.7B-class FFN, quantised when a model is loaded
        dict(name="quantize_16384x4096_f16", kind="quantize", R=16384, K=4096, dtype="f16"),
        # a ragged batch of bf16 activations
        dict(name="quantize_1237x2848_bf16", kind="quantize", R=1237, K=2848, dtype="bf16"),
        # the tiny workload's layer for one token: latency alone
        dict(name="linear_1x1024x1024_f16", kind="linear", M=1, N=1024, K=1024, dtype="f16", bias=True),
        # decode step of the 6.7B-class FFN, 16 sequences
        dict(name="linear_16x16384x4096_f16", kind="linear", M=16, N=16384, K=4096, dtype="f16", bias=False),
        # decode step of the 175B-class projection
        dict(name="linear_8x49152x12288_bf16", kind="linear", M=8, N=49152, K=12288, dtype="bf16", bias=False),
        # a short prompt into an odd vocabulary-like width, with a bias
        dict(name="linear_333x5003x2080_bf16", kind="linear", M=333, N=5003, K=2080, dtype="bf16", bias=True),
        # prefill of the 175B-class projection, the largest
        dict(name="linear_4096x49152x12288_f16", kind="linear", M=4096, N=49152, K=12288, dtype="f16", bias=False),
        # between two blocks, one token of each of 4 sequences: RMS norms on both sides, a gate
        dict(name="norm_4x4096_bf16", kind="norm", M=4, K=4096, dtype="bf16", norm="rms", post="rms", gate=1),
        # ... the prefill of 4096 tokens at the 175B class's width, layer norm before the block only
        dict(name="norm_4096x12288_f16", kind="norm", M=4096, K=12288, dtype="f16", norm="layer", post="none", gate=0),
        # the step from one block into the next one's first product, a decode batch
        dict(name="block_8x16384x4096_f16", kind="block", M=8, N=16384, K=4096, dtype="f16", norm="rms", post="rms", gate=1),
        # ... and the 6.7B-class prefill, a gate for each of 4 sequences
        dict(name="block_2048x16384x4096_bf16", kind="block", M=2048, N=16384, K=4096, dtype="bf16", norm="rms", post="rms", gate=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quantize", "linear", "linear", "norm", "block"])
    dtype = rng.choice(["f16", "bf16"])
    if kind == "quantize":
        K = 32 * _log(rng, 1, 512)
        return dict(kind=kind, R=_log(rng, 1, min(65536, 200_000_000 // K)), K=K, dtype=rng.choice(["f16", "bf16", "f32"]))
    if kind == "linear":
        return dict(kind=kind, M=_log(rng, 1, 4096), N=_log(rng, 1, 49152), K=32 * _log(rng, 1, 384), dtype=dtype,
                    bias=rng.random() < 0.5)
    M, gate = _log(rng, 1, 4096), rng.choice([0, 1, 2])
    M += M % 2 if gate == 2 else 0
    case = dict(kind=kind, M=M, K=32 * _log(rng, 1, 512), dtype=dtype, norm=rng.choice(["rms", "layer"]),
                post=rng.choice(["none", "rms", "layer"]), gate=gate)
    if kind == "block":
        case["N"] = _log(rng, 1, 16384)
    return case


# ------------------------------------------------------------------------------ inputs -------

def _activations(g, M, K, dtype):
    """N(0, 1) with a few large feature columns on three quarters of the rows."""
    x = torch.randn((M, K), generator=g, device="cuda")
    cols = torch.randint(0, K, (6,), generator=g, device="cuda")
    big = 6 + 14 * torch.rand((M, 6), generator=g, device="cuda")
    big = torch.where(torch.rand((M, 6), generator=g, device="cuda") < 0.5, -big, big)
    x[:, cols] = torch.where(torch.rand((M, 6), generator=g, device="cuda") < 0.75, big, x[:, cols])
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, K = _DT[case["dtype"]], case["K"]
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["kind"] == "quantize":
        s["X"] = _activations(g, case["R"], K, dt)
        return s
    s["X"] = _activations(g, case["M"], K, dt)
    if "N" in case:
        # a layer's weight as a loaded model holds it: quantised already
        s["WC"], s["WS"] = _quantize(torch.randn((case["N"], K), generator=g, device="cuda").mul_(0.02).to(dt))
    if case["kind"] == "linear":
        s["bias"] = rand(case["N"]).mul_(0.1).to(dt) if case["bias"] else None
        return s
    layer = case["norm"] == "layer"
    s["residual"] = rand(case["M"], K).mul_(2).to(dt)
    s["weight"] = (1 + 0.1 * rand(K)).to(dt)
    s["nbias"] = (0.1 * rand(K)).to(dt) if layer else None
    s["post_weight"] = (1 + 0.1 * rand(K)).to(dt) if case["post"] != "none" else None
    s["post_bias"] = (0.1 * rand(K)).to(dt) if case["post"] == "layer" else None
    s["gate"] = torch.sigmoid(rand(case["gate"], K)).to(dt) if case["gate"] else None
    s["scale"] = 0.75
    s["eps"] = 1e-5
    return s


# ------------------------------------------------------------- the plain forms (32 bits) ------

def _blocks(x):
    """x [R, K] -> (codes as integers 0..15 [R, K/32, 32], scale bytes [R, K/32])."""
    v = x.float().reshape(x.shape[0], -1, 32)
    amax = v.abs().amax(-1)
    bad = ~torch.isfinite(amax)
    s = torch.clamp(torch.frexp(torch.where(bad, 1.0, amax))[1] - 3, min=-127)
    s = torch.where(amax == 0, -127, s)
    a = v * (127 - s << 23).view(torch.float32)[..., None]          # v / 2^s
    m = a.abs()
    # twice the magnitude on the grid 0 1 2 3 4 | 6 8 | 12, ties to the even code
    step = torch.where(m < 2, 1.0, torch.where(m < 4, 2.0, 4.0))
    q = torch.clamp(torch.round(2 * m / step) * step, max=12.0)
    code = torch.where(q <= 4, q, torch.where(q <= 8, q / 2 + 2, 7.0)).to(torch.uint8)
    code = torch.where(torch.isnan(m), 0, code) + 8 * torch.signbit(a).to(torch.uint8)
    return code, torch.where(bad, 255, s + 127).to(torch.uint8)


def _tiled(s):
    """Scale bytes [R, K/32] -> the tiled layout; what pads them is 0."""
    R, B = s.shape
    rt, kt = -(-R // 128), -(-B // 8)
    p = torch.zeros((rt * 128, kt * 8), dtype=torch.uint8, device=s.device)
    p[:R, :B] = s
    return p.view(rt, 4, 32, kt, 2, 4).permute(0, 3, 4, 2, 1, 5).reshape(rt, kt, 1024).contiguous()


def _untiled(t, R, B):
    rt, kt = t.shape[:2]
    return t.view(rt, kt, 2, 32, 4, 4).permute(0, 4, 3, 1, 2, 5).reshape(rt * 128, kt * 8)[:R, :B]


def _quantize(x):
    code, s = _blocks(x)
    code = code.reshape(x.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), _tiled(s)


def _values(code, s):
    """Codes [R, K/32, 32] and scale bytes [R, K/32] -> fp32 [R, K]."""
    e, m = (code >> 1 & 3).float(), (code & 1).float()
    mag = torch.where(e == 0, m / 2, torch.exp2(e - 1) * (1 + m / 2))
    v = torch.where(code >= 8, -mag, mag)
    bits = torch.where(s == 0, 1 << 22, s.to(torch.int32) << 23)     # 2^(s - 127), 2^-127 a subnormal
    scale = torch.where(s == 255, math.nan, bits.view(torch.float32))
    return (v * scale[..., None]).reshape(code.shape[0], -1)


def _dequantize(codes, scales):
    R, half = codes.shape
    code = torch.stack((codes & 15, codes >> 4), -1).reshape(R, -1, 32)
    return _values(code, _untiled(scales, R, half // 16))


def _round_trip(x):
    return _values(*_blocks(x))


def _norm(x, kind, w, b, eps):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    if w is not None:
        y = y * w.float()
    return y if b is None else y + b.float()


def _residual_norm(s):
    c, t = s["case"], s["X"].float()
    if c["post"] != "none":
        t = _norm(t, c["post"], s["post_weight"], s["post_bias"], s["eps"])
    if s["gate"] is not None:
        t = t * s["gate"].float().repeat_interleave(c["M"] // c["gate"], 0)
    h = s["residual"].float() + s["scale"] * t
    return h, _norm(h, c["norm"], s["weight"], s["nbias"], s["eps"])


def run(state):
    c, X = state["case"], state["X"]
    if own:
        return _run_own(state)
    if c["kind"] == "quantize":
        return _dequantize(*_quantize(X)).to(X.dtype)
    if c["kind"] == "linear":
        y = _round_trip(X) @ _dequantize(state["WC"], state["WS"]).T
        return (y if state["bias"] is None else y + state["bias"].float()).to(X.dtype)
    h, y = _residual_norm(state)
    if c["kind"] == "norm":
        return {"H": h.to(X.dtype), "Y": y.to(X.dtype)}
    y = _round_trip(y.to(X.dtype)) @ _dequantize(state["WC"], state["WS"]).T
    return {"H": h.to(X.dtype), "Y": y.to(X.dtype)}


# ----------------------------------------------------------------------- the library's calls ---

def _run_own(s):
    from int8_quantized_02_b200 import llmint8 as L
    c, X = s["case"], s["X"]
    if c["kind"] == "quantize":
        codes, scales = L.llmint8_mxfp4_quantize(X)
        return L.llmint8_mxfp4_dequant(codes, scales, dtype=X.dtype)
    if c["kind"] == "linear":
        return L.llmint8_mxfp4_linear(X, s["WC"], s["WS"], bias=s["bias"])
    args = dict(residual=s["residual"], weight=s["weight"], bias=s["nbias"], norm=c["norm"],
                post_norm=None if c["post"] == "none" else c["post"], post_weight=s["post_weight"],
                post_bias=s["post_bias"], gate=s["gate"], scale=s["scale"], eps=s["eps"])
    if c["kind"] == "norm":
        H, Y = L.llmint8_residual_norm(X, **args)
        return {"H": H, "Y": Y}
    H, codes, scales = L.llmint8_residual_norm_mxfp4(X, **args)
    return {"H": H, "Y": L.llmint8_mxfp4_linear_quantized(codes, scales, s["WC"], s["WS"], dtype=X.dtype)}


# ------------------------------------------------------------------------- floors and truth ----

def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    K, half = case["K"], 17 * case["K"] // 32          # codes and scales of a row
    if case["kind"] == "quantize":
        # there and back: values read, codes written, codes read, values written
        return {"bytes": case["R"] * (2 * size * K + 2 * half), "flops": 4 * case["R"] * K}
    M, N = case["M"], case.get("N", 0)
    product = {"bytes": N * half + size * M * N, "flops": 2 * M * N * K}
    if case["kind"] == "linear":
        return {"bytes": size * M * K + product["bytes"] + (size * N if case["bias"] else 0), "flops": product["flops"]}
    rows = 3 if case["kind"] == "block" else 4         # X, residual, H (and Y)
    vectors = 1 + (case["norm"] == "layer") + (case["post"] != "none") + (case["post"] == "layer") + case["gate"]
    return {"bytes": size * K * (rows * M + vectors) + product["bytes"], "flops": 12 * M * K + product["flops"]}


_GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_quantized(x):
    """x fp64 [R, K] -> the fp64 values that its MXFP4 form stands for: each element to the nearest
    of the format's values, a tie to the one with the even code."""
    v = x.reshape(x.shape[0], -1, 32)
    top = v.abs().max(-1, keepdim=True).values
    fine = torch.isfinite(top)
    power = torch.clamp((torch.where(fine & (top > 0), top, 1.0).view(torch.int64) >> 52) - 1023 - 2, min=-127)
    unit = (power + 1023 << 52).view(torch.float64)
    m = (v / unit).abs()
    got = torch.zeros_like(m)
    for i in range(7):
        middle = (_GRID[i] + _GRID[i + 1]) / 2
        got = torch.where((m >= middle) if i % 2 else (m > middle), _GRID[i + 1], got)
    return torch.where(fine, torch.sign(v) * got * unit, math.nan).reshape(x.shape)


def _exact_weight(codes, scales):
    """fp64 [N, K] from the codes and the tiled scales, by index."""
    N, half = codes.shape
    dev = codes.device
    table = torch.tensor(_GRID + [-v for v in _GRID], dtype=torch.float64, device=dev)
    powers = (torch.arange(256, device=dev) - 127 + 1023 << 52).view(torch.float64)
    powers[255] = math.nan
    r, b = torch.arange(N, device=dev)[:, None], torch.arange(half // 16, device=dev)[None, :]
    flat = (r // 128 * scales.shape[1] + b // 8) * 1024 + b % 8 // 4 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    unit = powers[scales.reshape(-1)[flat].to(torch.int32)]
    out = torch.empty((N, half // 16, 16, 2), dtype=torch.float64, device=dev)
    c = codes.to(torch.int32).reshape(N, half // 16, 16)
    out[..., 0] = table[c % 16]
    out[..., 1] = table[c // 16]
    return out.mul_(unit[..., None, None]).reshape(N, half * 2)


def _exact_norm(x, kind, w, b, eps):
    if kind == "none":
        return x
    if kind == "layer":
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        y = (x - mean) / torch.sqrt(var + eps)
    else:
        y = x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + eps)
    y = y * w.double()
    return y if b is None else y + b.double()


def exact(case, seed):
    s = prepare(case, seed)
    x = s["X"].double()
    if case["kind"] == "quantize":
        return _exact_quantized(x)
    if case["kind"] == "linear":
        y = _exact_quantized(x) @ _exact_weight(s["WC"], s["WS"]).T
        return y if s["bias"] is None else y + s["bias"].double()
    t = _exact_norm(x, case["post"], s["post_weight"], s["post_bias"], s["eps"])
    if case["gate"]:
        rows = torch.arange(case["M"], device=x.device) // (case["M"] // case["gate"])
        t = t * s["gate"].double()[rows]
    h = s["residual"].double() + s["scale"] * t
    y = _exact_norm(h, case["norm"], s["weight"], s["nbias"], s["eps"])
    if case["kind"] == "norm":
        return {"H": h, "Y": y}
    # what enters the product is quantised from the 16-bit values
    y = _exact_quantized(y.to(_DT[case["dtype"]]).double())
    return {"H": h, "Y": y @ _exact_weight(s["WC"], s["WS"]).T}
