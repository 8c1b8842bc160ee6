"""The 8-bit format and its operators in float64: e4m3 values with a power-of-two
scale for each block of 128 columns. Test infrastructure, no method of the GPU
path: the e4m3 grid is spelled out, exponents are found by comparison, and sums
are float64."""
import numpy as np

from .encoder import gelu

BLOCK = 128


def e4m3_grid() -> np.ndarray:
    """The 127 values >= 0 of e4m3: exponent field 0 is m/8 * 2^-6, field f is
    (1 + m/8) * 2^(f-7); field 15 with m = 7 is NaN and left out."""
    sub = [m / 8 * 2.0 ** -6 for m in range(8)]
    normal = [(1 + m / 8) * 2.0 ** (f - 7) for f in range(1, 16) for m in range(8) if not (f == 15 and m == 7)]
    return np.array(sub + normal)


_GRID = e4m3_grid()


def round_e4m3(v):
    """Nearest e4m3 value of |v| <= 448, ties to the even code; NaN and infinities give NaN."""
    v = np.asarray(v, np.float64)
    a = np.where(np.isfinite(v), np.abs(v), 0.0)
    hi = np.clip(np.searchsorted(_GRID, a), 1, len(_GRID) - 1)
    lo = hi - 1
    up, down = _GRID[hi] - a, a - _GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.where(np.isfinite(v), np.copysign(_GRID[code], v), np.nan)


def exponents(x):
    """[rows, blocks] least e >= -126 with amax <= 448 * 2^e over the finite values of each block."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    a = np.zeros((rows, nb * BLOCK))
    a[:, :cols] = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = a.reshape(rows, nb, BLOCK).max(axis=2)
    ladder = 448.0 * 2.0 ** np.arange(-126, 128)            # exact in float64
    return np.searchsorted(ladder, amax) - 126


def spread(e, cols):
    """2^e of every element of a [rows, cols] matrix with block exponents e."""
    return np.repeat(2.0 ** e.astype(np.float64), BLOCK, axis=1)[:, :cols]


def quantize(x):
    """(values q * 2^e, exponents e) of x in the 8-bit format."""
    e = exponents(x)
    s = spread(e, x.shape[1])
    return round_e4m3(np.asarray(x, np.float64) / s) * s, e


def norm(x, gamma, beta=None, kind="rms", eps=1e-5):
    x = np.asarray(x, np.float64)
    if kind == "layer":
        x = x - x.mean(axis=1, keepdims=True)
    y = x / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    return y if beta is None else y + np.asarray(beta, np.float64)


def linear(a, w, bias=None, with_gelu=False):
    """act(a w^T + bias) of dequantised float64 operands."""
    y = np.asarray(a, np.float64) @ np.asarray(w, np.float64).T
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    return gelu(y) if with_gelu else y
