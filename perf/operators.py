"""The 8-bit serving operators of the encoder tower, as cases to time and to compare.

linear    matrix product of e4m3 operands with a power-of-two scale for each block of
          128 elements along K:  out = act(A W^T + bias), stored as bf16, as fp32, or
          again as e4m3 with scales
norm      RMS norm or LayerNorm of a residual stream, with the addition of the last
          sub-layer's output, to e4m3 with scales
quantize  rows of bf16 or fp32 values to e4m3 with scales

The 8-bit format: row r of a [rows, cols] matrix is cut into blocks of 128 columns
(the last one may be shorter). A block has the scale 2^e, where e is the least whole
number with amax <= 448 * 2^e, and not below -126; amax is the largest finite magnitude
of the block. The block's elements are value / 2^e rounded to e4m3, ties to even; a NaN
or an infinity becomes e4m3's NaN. Scales are held as e8m0, in rows padded to a multiple
of four bytes.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one position through fc1 of the Whisper-large block: the smallest call, all latency
        {"name": "linear_token", "op": "linear", "m": 1, "n": 5120, "k": 1280, "out": "bf16", "gelu": True, "bias": True},
        # 1 s of audio (50 positions) through the medium tower's fused QKV projection
        {"name": "linear_chunk", "op": "linear", "m": 50, "n": 3840, "k": 1024, "out": "bf16", "gelu": False, "bias": True},
        # an odd number of packed positions and an odd projector: ragged in every size
        {"name": "linear_odd", "op": "linear", "m": 777, "n": 1360, "k": 1104, "out": "fp8", "gelu": True, "bias": True},
        # one 30 s clip through fc2, output kept in fp32
        {"name": "linear_clip_fp32", "op": "linear", "m": 1500, "n": 1280, "k": 5120, "out": "fp32", "gelu": False, "bias": True},
        # 16 clips of 30 s through fc1 with GELU, the output quantised for fc2: the largest
        {"name": "linear_fc1_fp8", "op": "linear", "m": 24000, "n": 5120, "k": 1280, "out": "fp8", "gelu": True, "bias": True},
        # a ragged batch through the QKV projection of the Whisper-large block
        {"name": "linear_qkv", "op": "linear", "m": 18737, "n": 3840, "k": 1280, "out": "bf16", "gelu": False, "bias": True},
        # one position of a bf16 stream, with the addition
        {"name": "norm_token", "op": "norm", "rows": 1, "d": 1280, "kind": "rms", "x": "bf16", "delta": "bf16"},
        # one clip through the medium tower's LayerNorm
        {"name": "norm_clip", "op": "norm", "rows": 1500, "d": 1024, "kind": "layer", "x": "fp32", "delta": "none"},
        # 16 clips, fp32 stream, the out-projection's bf16 output added
        {"name": "norm_batch", "op": "norm", "rows": 24000, "d": 1280, "kind": "rms", "x": "fp32", "delta": "bf16"},
        # a wide bf16 stream with a last block that is not full
        {"name": "norm_wide", "op": "norm", "rows": 8191, "d": 4016, "kind": "rms", "x": "bf16", "delta": "bf16"},
        # fc1's weight, laid out when a tower is made
        {"name": "quantize_weight", "op": "quantize", "rows": 5120, "cols": 1280, "x": "bf16"},
        # the attention output of 32 clips before the out-projection
        {"name": "quantize_batch", "op": "quantize", "rows": 48000, "cols": 1280, "x": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    """A multiple of `step` in lo .. hi, spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "quantize"])
    if op == "linear":
        n, k = _log_int(rng, 128, 5120, 16), _log_int(rng, 128, 5120, 16)
        most = min(24000, 24000 * 5120 * 1280 // (n * k))
        m = _log_int(rng, 1, most)
        return {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(["bf16", "fp32", "fp8"]),
                "gelu": rng.random() < 0.5, "bias": rng.random() < 0.8}
    width = _log_int(rng, 128, 4096, 16)
    rows = _log_int(rng, 1, min(48000, 24000 * 1280 // width))
    if op == "norm":
        return {"op": op, "rows": rows, "d": width, "kind": rng.choice(["rms", "layer"]),
                "x": rng.choice(["bf16", "fp32"]), "delta": rng.choice(["bf16", "fp32", "none"])}
    return {"op": op, "rows": rows, "cols": width, "x": rng.choice(["bf16", "fp32"])}


# ------------------------------------------------------------------------ inputs
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}


def _pitch(cols):
    return -(-(-(-cols // BLOCK)) // 4) * 4


def _activations(g, rows, cols):
    """Normal values under a spread of channel sizes, with a few channels far above the rest."""
    size = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    loud = torch.rand(cols, generator=g, device="cuda") < 0.01
    return torch.randn(rows, cols, generator=g, device="cuda") * torch.where(loud, 20 * size, size)


def _scale_rows(rows, cols, exponents=None):
    """Storage of a scale matrix, e8m0 in padded rows."""
    s = torch.full((rows, _pitch(cols)), 127, dtype=torch.uint8, device="cuda")
    if exponents is not None:
        s[:, :exponents.shape[1]] = exponents
    return s.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": case}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        for name, t in (("a", _activations(g, m, k)),
                        ("w", torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k))):
            q, e = _to_fp8(t)
            s[name], s[name + "_scales"] = q, _scale_rows(t.shape[0], k, e.view(torch.uint8))
        s["bias"] = 0.1 * torch.randn(n, generator=g, device="cuda") if case["bias"] else None
        s["out"] = torch.empty(m, n, dtype=_TYPES[case["out"]], device="cuda")
        s["out_scales"] = _scale_rows(m, n) if case["out"] == "fp8" else None
        return s
    rows, cols = case["rows"], case["d" if case["op"] == "norm" else "cols"]
    s["x"] = _activations(g, rows, cols).to(_TYPES[case["x"]])
    s["q"] = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
    s["scales"] = _scale_rows(rows, cols)
    if case["op"] == "norm":
        s["delta"] = None
        if case["delta"] != "none":
            s["delta"] = (0.3 * torch.randn(rows, cols, generator=g, device="cuda")).to(_TYPES[case["delta"]])
        s["x_out"] = torch.empty_like(s["x"]) if s["delta"] is not None else None
        s["gamma"] = 1 + 0.1 * torch.randn(cols, generator=g, device="cuda")
        s["beta"] = 0.1 * torch.randn(cols, generator=g, device="cuda") if case["kind"] == "layer" else None
    return s


# ------------------------------------------------------------------- plain forms
def _to_fp8(y):
    """(q e4m3, scales e8m0) of fp32 rows."""
    rows, cols = y.shape
    blocks = -(-cols // BLOCK)
    t = torch.nn.functional.pad(y, (0, blocks * BLOCK - cols)).view(rows, blocks, BLOCK)
    amax = torch.where(torch.isfinite(t), t.abs(), 0.0).amax(dim=2)
    m, e = torch.frexp(amax)                       # amax = m 2^e, 1/2 <= m < 1;  448 = 0.875 * 2^9
    e = torch.clamp(e - 9 + (m > 0.875), min=-126)
    e = torch.where(amax > 0, e, -126)
    q = torch.ldexp(t, -e[:, :, None])
    q = torch.where(torch.isfinite(q), q, float("nan")).to(torch.float8_e4m3fn)
    return q.view(rows, blocks * BLOCK)[:, :cols].contiguous(), (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _from_fp8(q, scales):
    """fp32 values of an e4m3 matrix with scales."""
    s = scales.float().repeat_interleave(BLOCK, dim=1)[:, :q.shape[1]]
    return q.float() * s


def _plain_linear(s):
    case = s["case"]
    y = _from_fp8(s["a"], s["a_scales"]) @ _from_fp8(s["w"], s["w_scales"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if case["gelu"]:
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    return _to_fp8(y) if case["out"] == "fp8" else y.to(_TYPES[case["out"]])


def _plain_norm(s):
    case, x = s["case"], s["x"]
    if s["delta"] is not None:
        x = (x.float() + s["delta"].float()).to(x.dtype)
    y = x.float()
    if case["kind"] == "layer":
        y = y - y.mean(dim=1, keepdim=True)
    y = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + 1e-5) * s["gamma"]
    if s["beta"] is not None:
        y = y + s["beta"]
    q, scales = _to_fp8(y)
    return (q, scales, x) if s["delta"] is not None else (q, scales)


def run(s):
    case = s["case"]
    if own:
        import audio_encoder_tower_b200 as E
        if case["op"] == "linear":
            r = E.linear_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], bias=s["bias"], gelu=case["gelu"],
                             out=s["out"], out_scales=s["out_scales"])
            return (r[0], r[1][:, :-(-case["n"] // BLOCK)]) if case["out"] == "fp8" else r
        if case["op"] == "norm":
            q, scales, x = E.norm_fp8(s["x"], s["gamma"], s["beta"], delta=s["delta"], kind=case["kind"], eps=1e-5,
                                      x_out=s["x_out"], q=s["q"], scales=s["scales"])
            scales = scales[:, :-(-case["d"] // BLOCK)]
            return (q, scales, x) if s["delta"] is not None else (q, scales)
        q, scales = E.quantize_fp8(s["x"], q=s["q"], scales=s["scales"])
        return q, scales[:, :-(-case["cols"] // BLOCK)]
    if case["op"] == "linear":
        return _plain_linear(s)
    if case["op"] == "norm":
        return _plain_norm(s)
    return _to_fp8(s["x"].float())


# -------------------------------------------------------------- work and 64 bits
def work(case):
    size = {"bf16": 2, "fp32": 4, "fp8": 1, "none": 0}
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        kb, nb = -(-k // BLOCK), -(-n // BLOCK)
        out = m * n * size[case["out"]] + (m * nb if case["out"] == "fp8" else 0)
        return {"bytes": (m + n) * (k + kb) + 4 * n * case["bias"] + out, "flops": 2 * m * n * k}
    if case["op"] == "norm":
        n, d = case["rows"] * case["d"], case["d"]
        moved = size[case["x"]] * (2 if case["delta"] != "none" else 1) + size[case["delta"]] + 1
        return {"bytes": n * moved + case["rows"] * -(-d // BLOCK) + 4 * d * (2 if case["kind"] == "layer" else 1),
                "flops": 8 * n}
    n = case["rows"] * case["cols"]
    return {"bytes": n * (size[case["x"]] + 1) + case["rows"] * -(-case["cols"] // BLOCK), "flops": 3 * n}


def _scaled64(y):
    """What each e4m3 element of float64 rows stands for before its rounding: value / 2^e,
    with the power of two found by counting up from the block's largest magnitude."""
    out = torch.empty_like(y)
    for c in range(0, y.shape[1], BLOCK):
        b = y[:, c:c + BLOCK]
        top = b.abs().amax(dim=1, keepdim=True).clamp(min=E4M3_MAX * 2.0 ** -126)
        e = torch.ceil(torch.log2(top / E4M3_MAX))
        e = torch.where(top > E4M3_MAX * torch.exp2(e), e + 1, e)
        e = torch.where(top <= E4M3_MAX * torch.exp2(e - 1), e - 1, e)
        out[:, c:c + BLOCK] = b * torch.exp2(-e)
    return out


def exact(case, seed):
    """In 64 bits; an e4m3 output as value / scale before its rounding. A scale is a rounding
    upwards to a power of two and has no value of its own."""
    s = prepare(case, seed)
    if case["op"] == "linear":
        wide = []
        for name in ("a", "w"):
            q = s[name].double()
            for b in range(-(-case["k"] // BLOCK)):
                q[:, b * BLOCK:(b + 1) * BLOCK] *= s[name + "_scales"][:, b:b + 1].double()
            wide.append(q)
        y = torch.einsum("mk,nk->mn", *wide)
        if s["bias"] is not None:
            y += s["bias"].double()
        if case["gelu"]:
            y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
        return (_scaled64(y), None) if case["out"] == "fp8" else y
    x = s["x"].double()
    if case["op"] == "quantize":
        return _scaled64(x), None
    if s["delta"] is not None:
        x = x + s["delta"].double()
    stored = x if s["delta"] is None else x.to(s["x"].dtype).double()   # the norm is that of the stored stream
    y = stored
    mean = y.mean(dim=1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(y[:, :1])
    var = ((y - mean) ** 2).sum(dim=1, keepdim=True) / case["d"]
    y = (y - mean) * torch.rsqrt(var + 1e-5) * s["gamma"].double()
    if s["beta"] is not None:
        y = y + s["beta"].double()
    return (_scaled64(y), None, x) if s["delta"] is not None else (_scaled64(y), None)
