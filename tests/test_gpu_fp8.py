"""The 8-bit operators on the GPU against the float64 oracle (oracle/fp8.py):
quantisation bit for bit, the norm and the matrix product within what their fp32
arithmetic and the final rounding can be off by."""
import math

import numpy as np
import pytest

import oracle.fp8 as F8

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24          # fp32: half a step, relative
HALF = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4, "fp32": 2.0 ** -24}


def _t(a, dtype=None):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).to(device="cuda", dtype=dtype or torch.float32)


def _deq(q, scales):
    """(float64 values, exponents) of a device matrix in the 8-bit format; checks the padding bytes."""
    import torch
    nb = -(-q.shape[1] // 128)
    by = scales.view(torch.uint8).cpu().numpy().astype(np.int64)
    assert np.all(by[:, nb:] == 127)
    e = by[:, :nb] - 127
    return q.cpu().to(torch.float64).numpy() * F8.spread(e, q.shape[1]), e


def _rows(rng, rows, cols):
    """Rows whose blocks differ in size by up to 2^60, with zero rows and zero blocks."""
    x = rng.standard_normal((rows, cols)) * F8.spread(rng.integers(-30, 31, (rows, -(-cols // 128))), cols)
    if rows > 2:
        x[1] = 0
        x[2, :min(cols, 128)] = 0
    return x.astype(np.float32)


# -------------------------------------------------------------------- quantise
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 128), (2, 144), (5, 512), (7, 1040), (33, 1280), (4, 1168),
                                       (2, 4096), (1, 65536)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize(rows, cols, dtype):
    import torch
    from audio_encoder_tower_b200 import quantize_fp8
    x = _t(_rows(np.random.default_rng(rows * cols), rows, cols), torch.bfloat16 if dtype == "bf16" else None)
    q, s = quantize_fp8(x)
    got, e = _deq(q, s)
    want, we = F8.quantize(x.double().cpu().numpy())
    assert np.array_equal(e, we)
    assert np.array_equal(got, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_special_values(dtype):
    """Borders of the scale, the largest and smallest magnitudes, NaN and infinities beside finite values."""
    import torch
    from audio_encoder_tower_b200 import quantize_fp8
    tiny = 2.0 ** -126
    rows = [[448.0], [450.0], [-1.75, 1.0, 0.01], [3.3e38, 1.0, 1e30], [tiny, -tiny / 2], [2.0 ** -133],
            [np.inf, 3.0, -1.0], [-np.inf, np.nan, 1e-3], [np.nan], [0.0, -0.0], [1e-30, -1e-36, 1e-38]]
    x = np.zeros((len(rows), 272))
    for i, r in enumerate(rows):
        x[i, 7:7 + len(r)] = r
        x[i, 200], x[i, 271] = 5.0, -448.0      # the other blocks are not affected
    x = _t(x.astype(np.float32), torch.bfloat16 if dtype == "bf16" else None)
    q, s = quantize_fp8(x)
    got, e = _deq(q, s)
    want, we = F8.quantize(x.double().cpu().numpy())
    assert np.array_equal(e, we)
    assert np.array_equal(got, want, equal_nan=True)


def test_quantize_strides_and_neighbours():
    """Rows inside a wider matrix; rows of the outputs past the last one stay as they were."""
    import torch
    from audio_encoder_tower_b200 import quantize_fp8
    x = _t(_rows(np.random.default_rng(3), 9, 2000), torch.bfloat16)
    part = x[:, 8:8 + 656]
    q = torch.full((12, 656), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((12, 8), 0x55, dtype=torch.uint8, device="cuda")
    quantize_fp8(part, q=q[:9].view(torch.float8_e4m3fn), scales=s[:9])
    got, e = _deq(q[:9].view(torch.float8_e4m3fn), s[:9])
    want, we = F8.quantize(part.double().cpu().numpy())
    assert np.array_equal(e, we) and np.array_equal(got, want)
    assert bool((q[9:] == 0x55).all()) and bool((s[9:] == 0x55).all())


def test_quantize_past_32_bits():
    """More elements than 2^31: the last rows are where their offsets say."""
    import torch
    from audio_encoder_tower_b200 import quantize_fp8
    rows, cols = 1_700_000, 1280
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-3:] = _t(_rows(np.random.default_rng(5), 3, cols), torch.bfloat16)
    q, s = quantize_fp8(x)
    got, e = _deq(q[-3:], s[-3:])
    want, we = F8.quantize(x[-3:].double().cpu().numpy())
    assert np.array_equal(e, we) and np.array_equal(got, want)
    assert int(q[:-3].view(torch.uint8).max()) == 0


# ------------------------------------------------------------------------ norm
def _check_norm(got, e, y, slack):
    """Each value is within half an e4m3 step of some value within `slack` of y, and each
    scale is the least for an amax within `slack` of y's."""
    lo, hi = np.abs(y) - slack, np.abs(y) + slack
    elo, ehi = F8.exponents(np.maximum(lo, 0)), F8.exponents(hi)
    assert np.all((e >= elo) & (e <= ehi))
    step = np.maximum(HALF["fp8"] * hi, 2.0 ** -10 * F8.spread(e, y.shape[1]))   # subnormal step 2^-9
    assert np.all(np.abs(got - y) <= step + slack)


@pytest.mark.parametrize("rows,d", [(1, 16), (1, 1280), (9, 128), (5, 144), (17, 384), (8, 656), (3, 1024), (33, 1280),
                                    (6, 1536), (2, 2048), (5, 2064), (3, 4016), (2, 4112), (2, 8192)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("x_type,delta_type", [("bf16", "bf16"), ("fp32", "bf16"), ("fp32", None), ("bf16", "fp32")])
def test_norm(rows, d, kind, x_type, delta_type):
    import torch
    from audio_encoder_tower_b200 import norm_fp8
    T = {"bf16": torch.bfloat16, "fp32": torch.float32}
    rng = np.random.default_rng(rows * 10000 + d)
    x = _t((rng.standard_normal((rows, d)) * 3 + 0.5).astype(np.float32), T[x_type])
    delta = None if delta_type is None else _t(rng.standard_normal((rows, d)).astype(np.float32), T[delta_type])
    gamma = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    beta = (0.1 * rng.standard_normal(d)).astype(np.float32) if kind == "layer" else None
    before = x.clone()
    q, s, xo = norm_fp8(x, _t(gamma), None if beta is None else _t(beta), delta=delta, kind=kind)
    assert torch.equal(x, before)
    want_x = x if delta is None else (x.float() + delta.float()).to(x.dtype)
    assert torch.equal(xo, want_x)                        # one fp32 addition and one rounding: exact
    st = want_x.double().cpu().numpy()
    y = F8.norm(st, gamma, beta, kind)
    got, e = _deq(q, s)
    # fp32: a sum of n terms in a tree of lanes and registers is off by at most (n / 32 / WPR + 7) * E32 <= 80 E32
    # of the sum of magnitudes; half of that reaches the root, all of the mean's reaches x - mean; a handful of
    # roundings per element on top
    sd = np.sqrt(((st - (st.mean(1, keepdims=True) if kind == "layer" else 0)) ** 2).mean(1, keepdims=True) + 1e-5)
    core = np.abs(st) / sd * np.abs(gamma)
    slack = 60 * E32 * (core + (0 if beta is None else np.abs(beta)))
    if kind == "layer":
        slack = slack + 80 * E32 * np.abs(st).mean(1, keepdims=True) / sd * np.abs(gamma)
    _check_norm(got, e, y, slack)


@pytest.mark.parametrize("d", [16, 384, 512, 656, 1024, 1280, 1424, 1648, 2048, 2208, 4016, 5120, 5648, 7168, 8192])
@pytest.mark.parametrize("x_type,delta_type", [("bf16", None), ("fp32", None), ("bf16", "bf16"), ("fp32", "fp32")])
def test_norm_many_rows(d, x_type, delta_type):
    """More rows than run at once take a kernel with other registers: the same bits, special rows among them,
    in place, and rows behind the last one stay."""
    import torch
    from audio_encoder_tower_b200 import norm_fp8
    rows = 14001 if d < 256 else 6001 if d <= 2048 else 1501
    T = {"bf16": torch.bfloat16, "fp32": torch.float32}
    g = torch.Generator("cuda").manual_seed(d)
    rand = lambda *s: torch.randn(*s, device="cuda", dtype=torch.float32, generator=g)
    x = rand(rows + 2, d).to(T[x_type])
    delta = None if delta_type is None else rand(rows + 2, d).to(T[delta_type])
    x[rows // 2], x[7, d - 1], x[rows - 1, 3] = 0, float("nan"), float("inf")
    gamma, beta = rand(d), rand(d)
    for kind in ("rms", "layer"):
        y = x.clone()
        q = torch.full((rows + 2, d), 0x55, dtype=torch.uint8, device="cuda")
        s = torch.full((rows + 2, -(-d // 512) * 4), 0x55, dtype=torch.uint8, device="cuda")
        norm_fp8(y[:rows], gamma, beta, delta=None if delta is None else delta[:rows], kind=kind, x_out=y[:rows],
                 q=q[:rows].view(torch.float8_e4m3fn), scales=s[:rows])
        assert bool((q[rows:] == 0x55).all()) and bool((s[rows:] == 0x55).all())
        assert torch.equal(y[rows:], x[rows:])
        for r in [*range(0, rows, 499)]:      # few enough to run at once
            e = min(r + 499, rows)
            a, b, o = norm_fp8(x[r:e], gamma, beta, delta=None if delta is None else delta[r:e], kind=kind)
            assert torch.equal(a.view(torch.uint8), q[r:e]) and torch.equal(b.view(torch.uint8), s[r:e])
            assert torch.equal(o.view(torch.uint8), y[r:e].view(torch.uint8))


def test_norm_in_place_strides_and_neighbours():
    import torch
    from audio_encoder_tower_b200 import norm_fp8
    rng = np.random.default_rng(12)
    wide = _t(rng.standard_normal((10, 1500)).astype(np.float32), torch.bfloat16)
    dwide = _t(rng.standard_normal((7, 720)).astype(np.float32), torch.bfloat16)
    x, delta = wide[:7, 16:16 + 704], dwide[:, 8:712]
    gamma = _t(np.ones(704, np.float32))
    want = wide.clone()
    want[:7, 16:720] = (x.float() + delta.float()).to(torch.bfloat16)
    q, s, xo = norm_fp8(x, gamma, delta=delta, x_out=x)
    assert torch.equal(wide, want) and xo.data_ptr() == x.data_ptr()
    y = F8.norm(x.double().cpu().numpy(), np.ones(704))
    got, e = _deq(q, s)
    _check_norm(got, e, y, 60 * E32 * np.abs(y))


def test_norm_special_rows():
    """A zero row stays zero; a NaN or an infinity makes its own row NaN and no other."""
    import torch
    from audio_encoder_tower_b200 import norm_fp8
    rng = np.random.default_rng(13)
    x = rng.standard_normal((6, 1280)).astype(np.float32)
    x[1], x[2, 5], x[4, 1279] = 0, np.nan, np.inf
    for kind in ("rms", "layer"):
        q, s, _ = norm_fp8(_t(x), _t(np.ones(1280, np.float32)), kind=kind)
        got, e = _deq(q, s)
        assert np.all(got[1] == 0) and np.all(np.isfinite(got[[0, 1, 3, 5]]))
        assert np.isnan(got[2]).all()
        assert np.isnan(got[4, 1279])
        y = F8.norm(x[[0, 3, 5]], np.ones(1280), None, kind)
        _check_norm(got[[0, 3, 5]], e[[0, 3, 5]], y, 150 * E32 * (np.abs(y) + 1))


# ---------------------------------------------------------------- matrix product
def _operand(rng, rows, cols, spread=2, scale=1.0):
    """A device matrix in the 8-bit format with exactly known values: (q, scales, float64 values)."""
    from audio_encoder_tower_b200 import quantize_fp8
    x = rng.standard_normal((rows, cols)) * scale
    x = x * F8.spread(rng.integers(-spread, spread + 1, (rows, -(-cols // 128))), cols)
    q, s = quantize_fp8(_t(x.astype(np.float32)))
    return q, s, _deq(q, s)[0]


def _acc_slack(a, w, K):
    """What fp32 accumulation may be off by: each MMA of 32 products adds to the running sum
    with an error of at most two steps (2^-22) of the magnitudes seen so far."""
    return (K / 32 + 4) * 2.0 ** -22 * (np.abs(a) @ np.abs(w).T)


SHAPES = [(1, 16, 16), (1, 128, 128), (1, 1280, 1280), (3, 272, 144), (16, 512, 1104), (50, 384, 1024), (64, 144, 640),
          (100, 1360, 512), (127, 256, 656), (128, 400, 128), (129, 128, 2064), (200, 1280, 1280), (257, 640, 1280),
          (300, 272, 1168), (513, 1296, 272), (1000, 512, 528), (4000, 3840, 1280),
          # few rows at a long depth; units of both widths in turn on one pair of SMs, several each
          (33, 144, 2304), (90, 272, 4112), (400, 1280, 5120), (12000, 1360, 272), (7000, 1424, 144),
          # every height of tile with every split of K, then the 256 x 256 kernel on less than a wave of tiles
          (628, 144, 144), (39, 176, 144), (82, 144, 480), (49, 144, 1296), (1373, 144, 176), (598, 144, 672),
          (312, 144, 800), (81, 272, 2608), (1186, 432, 144), (1219, 144, 1680), (609, 144, 1840), (184, 576, 5168),
          (1300, 1296, 2064), (2600, 400, 128), (1537, 1040, 4112), (257, 4240, 528), (2000, 4240, 16)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "fp32", "fp8", "resid"])
def test_linear(M, N, K, out):
    import torch
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, sa, av = _operand(rng, M, K)
    w, sw, wv = _operand(rng, N, K, scale=1 / math.sqrt(K))
    bias = rng.standard_normal(N).astype(np.float32) if N != 512 else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gelu = out != "resid" and N % 256 == 0
    slack = _acc_slack(av, wv, K)
    y = F8.linear(av, wv, bias)
    slack = slack + 2 * E32 * (np.abs(y) + np.abs(y - (0 if bias is None else bias)))
    # GELU's slope is at most 1.13. fp32: erff and its product are a few steps of fp32 off. bf16: the
    # epilogue's form is within 1.1e-5 of GELU (relative) or 4.1e-11 |x|. e4m3: within 2.5e-4 for
    # |x| <= 5.5; beyond, form and GELU are both within Phi(-5.5) |x| = 1.9e-8 |x| of max(x, 0)
    if gelu:
        rel, tail = {"fp32": (8 * E32, 8 * E32), "bf16": (1.3e-5, 5e-11), "fp8": (2.6e-4, 2e-8)}[out]
        act = F8.linear(av, wv, bias, True)
        slack = 1.13 * slack + rel * np.abs(act) + tail * np.abs(y)
        y = act
    b = None if bias is None else _t(bias)
    if out == "resid":
        base = rng.standard_normal((M + 3, N)).astype(np.float32)
        buf = _t(base)
        r = linear_fp8(a, sa, w, sw, bias=b, resid=buf[:M], status=status)
        assert r.data_ptr() == buf.data_ptr() and np.array_equal(buf[M:].cpu().numpy(), base[M:])
        got = buf[:M].double().cpu().numpy()
        y = y + base[:M]
        assert np.all(np.abs(got - y) <= slack + 2 * E32 * (np.abs(y) + np.abs(base[:M])))
    elif out == "fp8":
        o = torch.full((M + 3, N), 0x55, dtype=torch.uint8, device="cuda")
        s = torch.full((M + 3, sw.shape[1] if N == K else -(-N // 512) * 4), 0x55, dtype=torch.uint8, device="cuda")
        q, so = linear_fp8(a, sa, w, sw, bias=b, out=o[:M].view(torch.float8_e4m3fn), out_scales=s[:M], gelu=gelu,
                           status=status)
        assert bool((o[M:] == 0x55).all()) and bool((s[M:] == 0x55).all())
        got, e = _deq(q, so)
        _check_norm(got, e, y, slack)
    else:
        T = torch.bfloat16 if out == "bf16" else torch.float32
        o = torch.full((M + 3, N), 7.0, dtype=T, device="cuda")
        linear_fp8(a, sa, w, sw, bias=b, out=o[:M], gelu=gelu, status=status)
        assert bool((o[M:] == 7).all())
        got = o[:M].double().cpu().numpy()
        assert np.all(np.abs(got - y) <= slack + HALF[out] * (np.abs(y) + slack))
    assert int(status) == 0


@pytest.mark.parametrize("M,N,K", [(5, 144, 640), (96, 272, 1168), (300, 512, 1280), (700, 1280, 528), (2000, 1280, 528),
                                   (184, 576, 5168)])
def test_linear_exact(M, N, K):
    """Small whole numbers under powers of two that differ from block to block: every partial sum
    is a number of fp32, so the result is the exact one in any order."""
    from audio_encoder_tower_b200 import linear_fp8, quantize_fp8
    rng = np.random.default_rng(K)
    v = []
    for rows in (M, N):
        x = rng.integers(-4, 5, (rows, K)) * F8.spread(rng.integers(-2, 3, (rows, -(-K // 128))), K)
        q, s = quantize_fp8(_t(x.astype(np.float32)))
        assert np.array_equal(_deq(q, s)[0], x)
        v.append((q, s, x))
    (a, sa, av), (w, sw, wv) = v
    got = linear_fp8(a, sa, w, sw, out_dtype="fp32").double().cpu().numpy()
    assert np.array_equal(got, av @ wv.T)


def test_linear_scales_far_apart():
    """Block scales from 2^-60 to 2^60 on both sides, one block of each row far above the rest."""
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(21)
    for M, N, K in ((40, 256, 1280), (400, 256, 1280), (2500, 1280, 640)):
        a, sa, av = _operand(rng, M, K, spread=30)
        w, sw, wv = _operand(rng, N, K, spread=30)
        got = linear_fp8(a, sa, w, sw, out_dtype="fp32").double().cpu().numpy()
        assert np.all(np.abs(got - av @ wv.T) <= _acc_slack(av, wv, K))


def test_linear_nan_stays_in_its_row():
    """A NaN element, or a NaN scale (byte 255), makes its row of A and its row of W NaN and nothing else."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(22)
    for M in (20, 300, 20000):
        a, sa, av = _operand(rng, M, 656)
        w, sw, wv = _operand(rng, 272, 656)
        a.view(torch.uint8)[3, 100] = 0x7F
        sa.view(torch.uint8)[7, 5] = 255
        w.view(torch.uint8)[271, 655] = 0xFF
        got = linear_fp8(a, sa, w, sw, out_dtype="fp32").double().cpu().numpy()
        nan = np.zeros((M, 272), bool)
        nan[3], nan[7], nan[:, 271] = True, True, True
        assert np.array_equal(np.isnan(got), nan)
        ok = ~nan
        assert np.all(np.abs(got - av @ wv.T)[ok] <= _acc_slack(av, wv, 656)[ok])
        # the same blocks in e4m3: NaN elements, the rest of the block as without them
        q, s = linear_fp8(a, sa, w, sw, out_dtype="fp8")
        got8, _ = _deq(q, s)
        assert np.array_equal(np.isnan(got8), nan)


@pytest.mark.parametrize("M", [20, 300, 2500])
def test_linear_overflow(M):
    """Sums past fp32's range are not finite (an infinity, or NaN where products of both signs are past it:
    each is 2^160 times a number near one here), NaN in e4m3, where the rest of the block keeps the scale
    of its largest finite value. M takes the kernel for few rows, narrow units and full ones."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(24)
    N, K = (1280, 256) if M == 2500 else (272, 256)
    a, sa, av = _operand(rng, M, K, spread=0)
    w, sw, wv = _operand(rng, N, K, spread=0)
    rows, cols = [3, M - 1], [7, 100, 130, N - 1]
    for r in rows:      # 2^80 * 2^80 overflows; either alone does not
        sa.view(torch.uint8)[r, :2] += 80
        av[r] *= 2.0 ** 80
    for c in cols:
        sw.view(torch.uint8)[c, :2] += 80
        wv[c] *= 2.0 ** 80
    y = av @ wv.T
    big = np.abs(y) > 3.5e38
    assert big.sum() == len(rows) * len(cols)
    for gelu in (False, True):
        for out in ("fp32", "bf16"):
            got = linear_fp8(a, sa, w, sw, out_dtype=out, gelu=gelu).double().cpu().numpy()
            ok = ~big
            ref = F8.linear(av, wv, None, gelu)
            assert np.all(np.isfinite(got[ok]))
            if not gelu:   # GELU takes minus infinity to zero
                assert not np.any(np.isfinite(got[big]))
            slack = 1.13 * _acc_slack(av, wv, K) + 1e-4 * np.abs(ref) + 5e-11 * np.abs(y)
            assert np.all(np.abs(got - ref)[ok] <= (slack + HALF[out] * (np.abs(ref) + slack))[ok])
    q, s = linear_fp8(a, sa, w, sw, out_dtype="fp8")
    got, e = _deq(q, s)
    assert np.array_equal(np.isnan(got), big)
    _check_norm(np.where(big, 0, got), e, np.where(big, 0, y), np.where(big, 0, _acc_slack(av, wv, K)))


def test_linear_row_does_not_depend_on_its_neighbours():
    """The same row, alone and among others, within a tile and in another one, gives the same bits per kernel
    variant, and the same call twice gives the same bits."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(23)
    a, sa, _ = _operand(rng, 900, 1280)
    w, sw, _ = _operand(rng, 512, 1280)
    full = linear_fp8(a, sa, w, sw, out_dtype="fp32")
    assert torch.equal(full, linear_fp8(a, sa, w, sw, out_dtype="fp32"))
    perm = torch.randperm(900, device="cuda")
    part = linear_fp8(a.view(torch.uint8)[perm].view(a.dtype), sa.view(torch.uint8)[perm].view(sa.dtype), w, sw,
                      out_dtype="fp32")
    assert torch.equal(part, full[perm])


def test_both_ways_from_python():
    """The short way (contiguous tensors, outputs given, the current stream) and the general one (the stream named)
    make the same call, and a refusal is the same with outputs given."""
    import torch
    from audio_encoder_tower_b200 import EncError, binding, linear_fp8, norm_fp8, quantize_fp8
    assert binding.fp8_scale_pitch(640) == 8
    rng = np.random.default_rng(41)
    x = _t(rng.standard_normal((70, 640)).astype(np.float32), torch.bfloat16)
    g, b = _t(rng.standard_normal(640).astype(np.float32)), _t(rng.standard_normal(640).astype(np.float32))
    w, sw, _ = _operand(rng, 272, 640)
    bias = _t(rng.standard_normal(272).astype(np.float32))
    cur = torch.cuda.current_stream()

    def outs():
        return (torch.empty(70, 640, dtype=torch.float8_e4m3fn, device="cuda"),
                torch.empty(70, 8, dtype=torch.float8_e8m0fnu, device="cuda"))

    def same(p, q):
        assert all(torch.equal(a.view(torch.uint8), c.view(torch.uint8)) for a, c in zip(p, q))

    q, s = quantize_fp8(x, *outs())
    assert binding._fast_quantize(x, q, s) == 0
    same((q, s), quantize_fp8(x, *outs(), stream=cur))
    for kind, delta in (("rms", x), ("layer", x.float()), ("rms", None)):
        xo = [torch.empty_like(x) if delta is not None else None for _ in range(2)]
        q1, s1 = outs()
        assert binding._fast_norm(0 if kind == "rms" else 1, x, g, b, delta, 1e-5, xo[0], q1, s1) == 0
        first = norm_fp8(x, g, b, delta=delta, kind=kind, x_out=xo[0], q=q1, scales=s1)
        q2, s2 = outs()
        same(first, norm_fp8(x, g, b, delta=delta, kind=kind, x_out=xo[1], q=q2, scales=s2, stream=cur))
    for T in (torch.bfloat16, torch.float32, torch.float8_e4m3fn):
        o = [torch.empty(70, 272, dtype=T, device="cuda") for _ in range(2)]
        so = [torch.empty(70, 4, dtype=torch.float8_e8m0fnu, device="cuda") if T == torch.float8_e4m3fn else None
              for _ in range(2)]
        assert binding._fast_linear(q, s, w, sw, bias, o[0], so[0], True) == 0
        first = linear_fp8(q, s, w, sw, bias=bias, out=o[0], out_scales=so[0], gelu=True)
        second = linear_fp8(q, s, w, sw, bias=bias, out=o[1], out_scales=so[1], gelu=True, stream=cur)
        same(*((first, second) if isinstance(first, tuple) else ((first,), (second,))))
    strided = x[:, :320]
    q3, s3 = quantize_fp8(strided, q=torch.empty(70, 320, dtype=torch.float8_e4m3fn, device="cuda"),
                          scales=torch.empty(70, 4, dtype=torch.float8_e8m0fnu, device="cuda"))
    same((q3, s3), quantize_fp8(strided.contiguous()))
    with pytest.raises(ValueError):
        quantize_fp8(x, q=q[:69], scales=s)
    with pytest.raises(ValueError):
        linear_fp8(q, s, w, sw, out=torch.empty(70, 272, dtype=torch.float16, device="cuda"))
    odd = torch.zeros(4, 24, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(EncError):
        quantize_fp8(odd, q=torch.empty(4, 24, dtype=torch.float8_e4m3fn, device="cuda"),
                     scales=torch.empty(4, 4, dtype=torch.float8_e8m0fnu, device="cuda"))


def test_no_rows():
    import torch
    from audio_encoder_tower_b200 import linear_fp8, norm_fp8, quantize_fp8
    x = torch.zeros(0, 256, dtype=torch.bfloat16, device="cuda")
    q, s = quantize_fp8(x)
    q2, s2, xo = norm_fp8(x, torch.ones(256, dtype=torch.float32, device="cuda"), delta=x)
    w, sw, _ = _operand(np.random.default_rng(1), 32, 256)
    assert linear_fp8(q, s, w, sw).shape == (0, 32) and q2.shape == (0, 256) and xo.shape == (0, 256)


# ------------------------------------------------------- together, streams, graphs
def _ffn(x, gamma, beta, w1, w2, resid, stream=None):
    """LayerNorm -> fc1 + GELU (e4m3 out) -> fc2 added to the stream: a block's feed-forward half."""
    from audio_encoder_tower_b200 import linear_fp8, norm_fp8
    q, s, _ = norm_fp8(x, gamma, beta, kind="layer", stream=stream)
    h, hs = linear_fp8(q, s, w1[0], w1[1], bias=w1[2], out_dtype="fp8", gelu=True, stream=stream)
    return linear_fp8(h, hs, w2[0], w2[1], bias=w2[2], resid=resid, stream=stream)


def _ffn_case(seed, rows, d=640, f=1296):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, d)).astype(np.float32)
    g, b = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32), (0.1 * rng.standard_normal(d)).astype(np.float32)
    w1 = _operand(rng, f, d, scale=1 / math.sqrt(d), spread=0)
    w2 = _operand(rng, d, f, scale=1 / math.sqrt(f), spread=0)
    b1, b2 = (0.1 * rng.standard_normal(n).astype(np.float32) for n in (f, d))
    return x, g, b, w1, w2, b1, b2


@pytest.mark.parametrize("rows", [1, 50, 333])
def test_feed_forward_chain(rows):
    """norm -> product with GELU -> product onto the stream, against the float64 formulas with the
    8-bit roundings in the same places. A value near the middle between two e4m3 values may fall on
    either side, so the result may differ by a few of those steps: compared in norm with the error
    that the roundings themselves cause."""
    import torch
    x, g, b, w1, w2, b1, b2 = _ffn_case(31, rows)
    xt = _t(x)
    _ffn(xt, _t(g), _t(b), (*w1[:2], _t(b1)), (*w2[:2], _t(b2)), xt)
    torch.cuda.synchronize()
    got = xt.double().cpu().numpy()
    y = F8.norm(x, g, b, "layer")
    exact = x + F8.linear(F8.linear(y, w1[2], b1, True), w2[2], b2)
    h, _ = F8.quantize(F8.linear(F8.quantize(y)[0], w1[2], b1, True))
    model = x + F8.linear(h, w2[2], b2)
    noise = np.linalg.norm(model - exact)
    assert np.linalg.norm(got - model) <= 0.1 * noise, (np.linalg.norm(got - model), noise)


def test_captured_and_replayed():
    """The chain captured into a graph and replayed on new data gives the eager call's bits."""
    import torch
    x, g, b, w1, w2, b1, b2 = _ffn_case(32, 70)
    dev = [_t(v) for v in (g, b, b1, b2)]
    args = (dev[0], dev[1], (*w1[:2], dev[2]), (*w2[:2], dev[3]))
    want = []
    for k in (1, 2):
        r = _t(x * k)
        want.append(_ffn(r.clone(), *args, resid=r).clone())
    buf, res = _t(x), _t(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _ffn(buf, *args, resid=res)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _ffn(buf, *args, resid=res)
    for k in (1, 2):
        buf.copy_(_t(x * k))
        res.copy_(buf)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(res, want[k - 1])


def test_two_streams_at_once():
    """Independent chains on two streams, started together, give what each gives alone."""
    import torch
    cases = []
    for seed in (33, 34):
        x, g, b, w1, w2, b1, b2 = _ffn_case(seed, 600)
        cases.append((_t(x), _t(g), _t(b), (*w1[:2], _t(b1)), (*w2[:2], _t(b2))))
    alone = [_ffn(*c, resid=c[0].clone()).clone() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    out = [c[0].clone() for c in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                out[i].copy_(c[0])
            _ffn(*c, resid=out[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i], alone[i])


FIRST_CALL = """
import torch
from audio_encoder_tower_b200 import linear_fp8, norm_fp8, quantize_fp8
g = torch.Generator("cuda").manual_seed(35)
rand = lambda *s: torch.randn(*s, device="cuda", dtype=torch.float32, generator=g)
wide, few, w, gamma = rand(700, 640), rand(5, 640), rand(384, 640), rand(640)
def run():
    wq = quantize_fp8(w)
    return [t.view(torch.uint8) for x in (wide, few)
            for q, s, _ in [norm_fp8(x, gamma, delta=x)]
            for t in (q, s, linear_fp8(q, s, *wq, out_dtype="fp32"), *linear_fp8(q, s, *wq, out_dtype="fp8", gelu=True))]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = run()
graph.replay()
eager = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, eager, strict=True))
print("same")
"""


def test_first_call_of_a_process_is_captured():
    """The one-time set-up of each kernel happens inside a capture as well."""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


@pytest.mark.parametrize("M,N,K", [(1024, 1280, 5120), (300, 272, 4112), (257, 4240, 1936), (12000, 768, 1040)])
def test_linear_scales_reach_both_ctas(M, N, K):
    """Scales that differ from block to block and from call to call, in calls queued one after another on pairs of
    SMs: a group of scales that came late to the second SM of a pair would leave the one before in its place, off by
    powers of two. All sums are whole numbers of 2^-6 below 2^24 of them, so every result is exact."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8, quantize_fp8
    g = torch.Generator("cuda").manual_seed(M + N + K)
    blocks = -(-K // 128)

    def operand(rows):
        v = torch.randint(-2, 3, (rows, K), generator=g, device="cuda").float()
        e = torch.randint(-3, 4, (rows, blocks), generator=g, device="cuda").float()
        x = v * torch.exp2(e).repeat_interleave(128, dim=1)[:, :K]
        return (*quantize_fp8(x), x.double())

    sets = [(operand(M), operand(N)) for _ in range(3)]
    outs = [torch.empty(M, N, dtype=torch.float32, device="cuda") for _ in range(9)]
    for i, o in enumerate(outs):
        (a, sa, _), (w, sw, _) = sets[i % 3]
        linear_fp8(a, sa, w, sw, out=o)
    for i, o in enumerate(outs):
        av, wv = sets[i % 3][0][2], sets[i % 3][1][2]
        assert float((av.abs() @ wv.abs().t()).max()) * 64 < 2 ** 24
        assert torch.equal(o.double(), av @ wv.t())


def _queue_and_free(shape, dtype):
    """Work on the current stream that starts late and writes and reads a tensor of that size, which is freed here:
    the copy that was read."""
    import torch
    torch.cuda._sleep(20_000_000)      # 10 ms and more
    return torch.full(shape, 1, dtype=torch.uint8 if dtype.itemsize == 1 else dtype, device="cuda").clone()


@pytest.mark.parametrize("as_handle", [False, True])
def test_new_outputs_on_a_named_stream(as_handle):
    """Outputs that a call on a named stream allocates are not memory in which the current stream still has work
    queued: that work would overwrite them, or they its data."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8, norm_fp8, quantize_fp8
    rng = np.random.default_rng(51)
    M, K, N = 4096, 2048, 2560
    x = _t(rng.standard_normal((M, K)).astype(np.float32), torch.bfloat16)
    w, sw, _ = _operand(rng, N, K)
    gamma = _t(np.ones(K, np.float32))
    a, sa = quantize_fp8(x)
    side = torch.cuda.Stream()
    name = side.cuda_stream if as_handle else side
    calls = [((M, K), torch.float8_e4m3fn, lambda s: quantize_fp8(x, stream=s)),
             ((M, K), torch.bfloat16, lambda s: norm_fp8(x, gamma, delta=x, stream=s)),
             ((M, N), torch.bfloat16, lambda s: (linear_fp8(a, sa, w, sw, stream=s),)),
             ((M, N), torch.float32, lambda s: (linear_fp8(a, sa, w, sw, out_dtype="fp32", stream=s),)),
             ((M, N), torch.float8_e4m3fn, lambda s: linear_fp8(a, sa, w, sw, out_dtype="fp8", stream=s))]
    for shape, dtype, call in calls:
        want = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        kept = _queue_and_free(shape, dtype)
        got = call(name)
        torch.cuda.synchronize()
        assert bool((kept == 1).all())
        assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(got, want, strict=True))


@pytest.mark.parametrize("M", [1, 20, 300, 2500])
def test_linear_overflow_with_gelu_in_e4m3(M):
    """With GELU as without it, a sum past fp32's range is NaN in e4m3, whatever its sign and whichever kernel M
    takes (few rows, narrow units, full ones), and the rest of its block keeps the scale of its finite values."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(52)
    N, K = (1280, 256) if M == 2500 else (272, 256)
    a, sa, av = _operand(rng, M, K, spread=0)
    w, sw, wv = _operand(rng, N, K, spread=0)
    row, cols = M - 1, [3, 7, 100, 130, 131, 133, N - 1]
    sa.view(torch.uint8)[row, :2] += 80     # 2^80 * 2^80 overflows; either alone does not
    av[row] *= 2.0 ** 80
    for c in cols:
        sw.view(torch.uint8)[c, :2] += 80
        wv[c] *= 2.0 ** 80
    wv[cols[::2]] *= -1
    w.view(torch.uint8)[cols[::2]] ^= 0x80
    y = av @ wv.T
    big = np.abs(y) > 3.5e38
    assert big.sum() == len(cols) and (y[big] > 0).any() and (y[big] < 0).any()
    q, s = linear_fp8(a, sa, w, sw, out_dtype="fp8", gelu=True)
    got, e = _deq(q, s)
    assert np.array_equal(np.isnan(got), big)
    y = np.where(big, 0, y)
    ref = F8.gelu(y)
    slack = 1.13 * _acc_slack(av, wv, K) + 2.6e-4 * np.abs(ref) + 2e-8 * np.abs(y)      # as in test_linear
    _check_norm(np.where(big, 0, got), e, ref, np.where(big, 0, slack))


@pytest.mark.parametrize("M,N,K", [(1, 144, 128), (20, 272, 144), (64, 656, 512), (300, 272, 656), (1300, 400, 272),
                                   (777, 1360, 1104), (5000, 1296, 528)])
@pytest.mark.parametrize("out", ["bf16", "fp32", "fp8"])
def test_linear_gelu_in_ragged_blocks(M, N, K, out):
    """GELU where the last block of columns is not full, values far below zero among them, on both kernels."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8
    rng = np.random.default_rng(M + N + K)
    a, sa, av = _operand(rng, M, K, scale=2)
    w, sw, wv = _operand(rng, N, K, scale=1 / math.sqrt(K))
    bias = (3 * rng.standard_normal(N)).astype(np.float32)
    bias[-16:] = -40                                   # GELU is zero in fp32 here
    y = F8.linear(av, wv, bias)
    ref = F8.gelu(y)
    rel, tail = {"fp32": (8 * E32, 8 * E32), "bf16": (1.3e-5, 5e-11), "fp8": (2.6e-4, 2e-8)}[out]   # as in test_linear
    slack = 1.13 * (_acc_slack(av, wv, K) + 2 * E32 * (np.abs(y) + np.abs(bias))) + rel * np.abs(ref) + tail * np.abs(y)
    r = linear_fp8(a, sa, w, sw, bias=_t(bias), out_dtype=out, gelu=True)
    if out == "fp8":
        got, e = _deq(*r)
        _check_norm(got, e, ref, slack)
    else:
        got = r.double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= slack + HALF[out] * (np.abs(ref) + slack))


def test_other_threads_run_while_a_launch_waits():
    """With the device's queue full a call waits for it to drain; other Python threads go on meanwhile."""
    import threading
    import time
    import torch
    from audio_encoder_tower_b200 import binding, quantize_fp8
    x = _t(np.ones((64, 256), np.float32))
    q, s = quantize_fp8(x)
    assert binding._fast_quantize(x, q, s) == 0
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.001)

    thread = threading.Thread(target=tick)
    thread.start()
    torch.cuda._sleep(2_000_000_000)            # a second and more
    t0, longest = time.perf_counter(), 0.0
    for _ in range(6000):
        t = time.perf_counter()
        quantize_fp8(x, q, s)
        longest = max(longest, time.perf_counter() - t)
    t1 = time.perf_counter()
    stop.set()
    thread.join()
    torch.cuda.synchronize()
    assert longest > 0.3                        # a call did wait
    seen = [t0] + [t for t in ticks if t0 < t < t1] + [t1]
    assert max(b - a for a, b in zip(seen, seen[1:])) < longest / 2


@pytest.mark.parametrize("d", [2208, 4016, 5120, 5648, 7168, 8192])
@pytest.mark.parametrize("x_type,delta_type", [("bf16", None), ("fp32", None), ("bf16", "bf16"), ("fp32", "fp32")])
def test_norm_many_wide_rows(d, x_type, delta_type):
    """The kernel for many rows of more than 16 blocks against the one for rows that run at once (here 100 of them: a
    block of four warps each, and an SM holds two), and its last rows against float64."""
    import torch
    from audio_encoder_tower_b200 import norm_fp8
    rows = 1501
    T = {"bf16": torch.bfloat16, "fp32": torch.float32}
    g = torch.Generator("cuda").manual_seed(d)
    x = (3 * torch.randn(rows, d, device="cuda", dtype=torch.float32, generator=g) + 0.5).to(T[x_type])
    delta = None
    if delta_type is not None:
        delta = torch.randn(rows, d, device="cuda", dtype=torch.float32, generator=g).to(T[delta_type])
    gamma, beta = (torch.randn(d, device="cuda", dtype=torch.float32, generator=g) for _ in range(2))
    for kind in ("rms", "layer"):
        q, s, o = norm_fp8(x, gamma, beta, delta=delta, kind=kind)
        for r in range(0, rows, 100):
            e = min(r + 100, rows)
            few = norm_fp8(x[r:e], gamma, beta, delta=None if delta is None else delta[r:e], kind=kind)
            assert all(torch.equal(a.view(torch.uint8), b[r:e].view(torch.uint8)) for a, b in zip(few, (q, s, o), strict=True))
        st = o[-20:].double().cpu().numpy()
        gm, bt = gamma.double().cpu().numpy(), beta.double().cpu().numpy()
        got, e = _deq(q[-20:], s[-20:])
        mean = st.mean(1, keepdims=True) if kind == "layer" else 0
        sd = np.sqrt(((st - mean) ** 2).mean(1, keepdims=True) + 1e-5)
        slack = 60 * E32 * (np.abs(st) / sd * np.abs(gm) + np.abs(bt))       # as in test_norm
        if kind == "layer":
            slack = slack + 80 * E32 * np.abs(st).mean(1, keepdims=True) / sd * np.abs(gm)
        _check_norm(got, e, F8.norm(st, gm, bt, kind), slack)


def test_captured_with_branches():
    """A capture in which the calls follow a join of two streams, a memset and a copy, replayed on new data."""
    import torch
    from audio_encoder_tower_b200 import linear_fp8, norm_fp8, quantize_fp8
    rng = np.random.default_rng(53)
    x, y = (_t(rng.standard_normal((700, 640)).astype(np.float32)) for _ in range(2))
    gamma = _t((1 + 0.1 * rng.standard_normal(640)).astype(np.float32))
    w, sw, _ = _operand(rng, 640, 640, scale=1 / 25)
    side = torch.cuda.Stream()
    out, copy = torch.empty_like(x), torch.empty_like(x)

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        a, sa = quantize_fp8(x)
        with torch.cuda.stream(side):
            b, sb, _ = norm_fp8(y, gamma)
            h = linear_fp8(b, sb, w, sw, out_dtype="fp32")
        main.wait_stream(side)
        n, sn, _ = norm_fp8(h, gamma, delta=x)             # after a join
        out.zero_()
        linear_fp8(a, sa, w, sw, resid=out)                # after a memset
        copy.copy_(out)
        m, sm = quantize_fp8(copy)                         # after a copy
        linear_fp8(n, sn, w, sw, resid=out)
        linear_fp8(m[:20], sm[:20], w, sw, resid=out[:20])
        return (a, b, h, n, m)                             # kept until the graph has run

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for k in (1, 2, 3):
        x.copy_(_t(rng.standard_normal((700, 640)).astype(np.float32)))
        y.copy_(x * k)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        run()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    del kept


@pytest.mark.parametrize("M", [1, 40])
def test_linear_deepest(M):
    """K past 2^28: the rows of both operands lie further apart than 32 bits of bytes reach, and the sums are short."""
    import torch
    from audio_encoder_tower_b200 import binding, linear_fp8
    K, N = 2 ** 28 + 48, 16
    if torch.cuda.mem_get_info()[0] < 20 * 2 ** 30:
        pytest.skip("needs 20 GB")
    mats = []
    for rows in (M, N):
        q = torch.zeros(rows, K, dtype=torch.uint8, device="cuda")
        q[:, K - 48:] = 0x38                                          # 1.0: the last block, of 48 columns
        q[:, ::2 ** 26] = 0x40                                        # 2.0: in blocks of every CTA's share
        s = torch.full((rows, binding.fp8_scale_pitch(K)), 127, dtype=torch.uint8, device="cuda")
        s[:, -(-K // 128) - 1] = 127 + torch.arange(rows, device="cuda", dtype=torch.uint8) % 8
        mats += [q.view(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = linear_fp8(*mats, out_dtype="fp32", status=status).double().cpu().numpy()
    last = 2.0 ** (np.arange(M) % 8)[:, None] * 2.0 ** (np.arange(N) % 8)[None, :]
    # 2^28 is the fifth multiple of 2^26, the first column of the last block
    assert np.array_equal(got, 4 * 4.0 + last * (47 + 4)) and int(status) == 0


@pytest.mark.parametrize("rows", [1, 2, 5, 7, 6002])
def test_norm_in_place_with_warps_past_the_last_row(rows):
    """In place the stream is read once, by the warps that own its rows: those past the last row read none of it, and
    give the same bits as a call that writes the stream elsewhere."""
    import torch
    from audio_encoder_tower_b200 import norm_fp8
    rng = np.random.default_rng(rows)
    x = _t(rng.standard_normal((rows, 1280)).astype(np.float32))
    delta = _t(rng.standard_normal((rows, 1280)).astype(np.float32), torch.bfloat16)
    gamma = _t(rng.standard_normal(1280).astype(np.float32))
    apart = norm_fp8(x, gamma, delta=delta)
    for _ in range(3):
        y = x.clone()
        q, s, o = norm_fp8(y, gamma, delta=delta, x_out=y)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(apart, (q, s, o), strict=True))
