"""The 8-bit operators without a GPU: the oracle's format pinned to PyTorch's e4m3
casts and to closed forms, and every refusal of the C calls and of the Python
functions (they return before anything reaches a device)."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle.fp8 as F8
from audio_encoder_tower_b200 import binding as B
from audio_encoder_tower_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED = B.ENC_OK, B.ENC_ERR_INVALID_ARG, B.ENC_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.load_library()


# ------------------------------------------------------------------ the oracle
def test_grid_is_e4m3():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert np.array_equal(F8.e4m3_grid(), codes.double().numpy())


def test_rounding_is_torchs():
    grid = F8.e4m3_grid()
    mid = (grid[1:] + grid[:-1]) / 2
    rng = np.random.default_rng(0)
    v = np.concatenate([grid, mid, mid * (1 + 2 ** -20), mid * (1 - 2 ** -20), rng.uniform(-448, 448, 5000),
                        rng.standard_normal(5000) * 0.01]).astype(np.float32)
    v = np.concatenate([v, -v])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(F8.round_e4m3(v), want)
    assert np.isnan(F8.round_e4m3([np.nan, np.inf, -np.inf])).all()


@pytest.mark.parametrize("amax,e", [(448.0, 0), (448.0000001, 1), (1.75, -8), (1.7500001, -7), (1.0, -8), (0.0, -126),
                                    (2.0 ** -149, -126), (448 * 2.0 ** -126, -126), (449 * 2.0 ** -126, -125),
                                    (float(np.finfo(np.float32).max), 120)])
def test_exponent_is_the_least(amax, e):
    x = np.zeros((1, 16))
    x[0, 5] = -amax
    assert F8.exponents(x)[0, 0] == e


def test_quantize_keeps_blocks_apart():
    x = np.ones((2, 144))
    x[0, 3], x[0, 130], x[1, 140] = 1e6, np.inf, np.nan
    v, e = F8.quantize(x)
    assert e.tolist() == [[12, -8], [-8, -8]]
    assert np.isnan(v[0, 130]) and np.isnan(v[1, 140])
    assert np.all(v[0, 131:] == 1) and np.all(v[1, :140] == 1)


# ------------------------------------------------------------------- refusals
@pytest.mark.parametrize("cols,pitch", [(-5, 0), (0, 0), (1, 4), (128, 4), (512, 4), (513, 8), (1280, 12), (5120, 40)])
def test_scale_pitch(lib, cols, pitch):
    assert lib.enc_fp8_scale_pitch(cols) == pitch
    if cols > 0:
        assert B.fp8_scale_pitch(cols) == pitch


A = 1 << 20   # an aligned address that nothing reads: these calls return before a launch


@pytest.mark.parametrize("change,want", [
    (dict(rows=0), OK), (dict(rows=0, x=None, q=None), OK), (dict(rows=-1), INVALID), (dict(cols=0), INVALID),
    (dict(cols=24), UNSUPPORTED), (dict(cols=65552, ldx=65552), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(dtype=-1), INVALID), (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(scales=None), INVALID),
    (dict(x=A + 8), INVALID), (dict(q=A + 4), INVALID), (dict(scales=A + 2), INVALID), (dict(ldx=127), INVALID),
    (dict(ldx=130), INVALID), (dict(ldx=0), INVALID), (dict(ldx=-128), INVALID), (dict(dtype=1, ldx=130), INVALID)])
def test_quantize_refusals(lib, change, want):
    a = dict(x=A, dtype=0, ldx=128, rows=4, cols=128, q=A, scales=A) | change
    assert lib.enc_quantize_fp8(a["x"], a["dtype"], a["ldx"], a["rows"], a["cols"], a["q"], a["scales"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(rows=0), OK), (dict(rows=-1), INVALID), (dict(kind=2), INVALID), (dict(kind=-1), INVALID),
    (dict(d=0), INVALID), (dict(d=24), UNSUPPORTED), (dict(d=8208), UNSUPPORTED), (dict(eps=0.0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(dtype=2), INVALID), (dict(x=None), INVALID),
    (dict(gamma=None), INVALID), (dict(gamma=A + 4), INVALID), (dict(beta=A + 4), INVALID), (dict(q=None), INVALID),
    (dict(scales=None), INVALID), (dict(delta=3 * A, ddtype=2), INVALID), (dict(delta=3 * A, ldd=120), INVALID),
    (dict(delta=3 * A + 8), INVALID), (dict(xo=A, ldxo=256), INVALID), (dict(xo=5 * A, ldxo=100), INVALID),
    (dict(xo=5 * A + 2), INVALID), (dict(delta=3 * A, xo=3 * A), INVALID), (dict(ldx=64), INVALID)])
def test_norm_refusals(lib, change, want):
    a = dict(kind=0, x=A, dtype=0, ldx=128, delta=None, ddtype=0, ldd=128, gamma=A, beta=None, eps=1e-5, rows=4, d=128,
             xo=None, ldxo=128, q=A, scales=A) | change
    assert lib.enc_norm_fp8(a["kind"], a["x"], a["dtype"], a["ldx"], a["delta"], a["ddtype"], a["ldd"], a["gamma"],
                            a["beta"], a["eps"], a["rows"], a["d"], a["xo"], a["ldxo"], a["q"], a["scales"],
                            None) == want


@pytest.mark.parametrize("change,want", [
    (dict(M=0), OK), (dict(M=0, a=None, out=None), OK), (dict(M=-1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(K=24), UNSUPPORTED), (dict(N=40), UNSUPPORTED),
    (dict(M=2 ** 31 - 1), UNSUPPORTED), (dict(M=2 ** 30, N=2 ** 20), UNSUPPORTED),
    (dict(N=2 ** 31 - 16), UNSUPPORTED), (dict(kind=4), INVALID),
    (dict(kind=-1), INVALID), (dict(kind=3, gelu=1), INVALID), (dict(kind=2), INVALID), (dict(a=None), INVALID),
    (dict(sa=None), INVALID), (dict(w=None), INVALID), (dict(sw=None), INVALID), (dict(out=None), INVALID),
    (dict(a=A + 8), INVALID), (dict(w=A + 8), INVALID), (dict(out=A + 8), INVALID), (dict(bias=A + 8), INVALID),
    (dict(sa=A + 1), INVALID), (dict(sw=A + 2), INVALID)])
def test_linear_refusals(lib, change, want):
    a = dict(a=A, sa=A, w=A, sw=A, bias=None, out=A, so=None, kind=0, M=4, N=128, K=128, gelu=0) | change
    assert lib.enc_linear_fp8(a["a"], a["sa"], a["w"], a["sw"], a["bias"], a["out"], a["so"], a["kind"], a["M"],
                              a["N"], a["K"], a["gelu"], None, None) == want


def _mat(rows, cols):
    return (torch.zeros(rows, cols, dtype=torch.uint8).view(torch.float8_e4m3fn),
            torch.zeros(rows, B.fp8_scale_pitch(cols), dtype=torch.uint8).view(torch.float8_e8m0fnu))


def test_python_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    g = torch.ones(256, dtype=torch.float32)
    q, s = _mat(4, 256)
    w, sw = _mat(32, 256)
    bad = [
        lambda: B.quantize_fp8(x),                                         # not on a CUDA device
        lambda: B.quantize_fp8(x.half()),
        lambda: B.quantize_fp8(x[0]),
        lambda: B.quantize_fp8(x.t()),
        lambda: B.quantize_fp8(x, q=q[:3]),
        lambda: B.quantize_fp8(x, scales=s[:, :2]),
        lambda: B.quantize_fp8(x, scales=s.float()),
        lambda: B.norm_fp8(x, g, kind="batch"),
        lambda: B.norm_fp8(x, None),
        lambda: B.norm_fp8(x, g[:128]),
        lambda: B.norm_fp8(x, g.double()),
        lambda: B.norm_fp8(x, g, beta=g[None]),
        lambda: B.norm_fp8(x, g, delta=x[:2]),
        lambda: B.norm_fp8(x, g, delta=x.double()),
        lambda: B.norm_fp8(x, g, x_out=x.float()),
        lambda: B.linear_fp8(q, s, w, sw),
        lambda: B.linear_fp8(q.float(), s, w, sw),
        lambda: B.linear_fp8(q, s, w[:, :128], sw),
        lambda: B.linear_fp8(q, sw, w, sw),
        lambda: B.linear_fp8(q, s, w, sw, bias=g),
        lambda: B.linear_fp8(q, s, w, sw, out_dtype="fp16"),
        lambda: B.linear_fp8(q, s, w, sw, out=torch.zeros(4, 32, dtype=torch.half)),
        lambda: B.linear_fp8(q, s, w, sw, out=torch.zeros(4, 16, dtype=torch.float32)),
        lambda: B.linear_fp8(q, s, w, sw, out=torch.zeros(4, 32, dtype=torch.float32), out_dtype="bf16"),
        lambda: B.linear_fp8(q, s, w, sw, out=torch.zeros(4, 32, dtype=torch.float32), out_scales=s),
        lambda: B.linear_fp8(q, s, w, sw, resid=torch.zeros(4, 32, dtype=torch.float32), gelu=True),
        lambda: B.linear_fp8(q, s, w, sw, resid=torch.zeros(4, 32).bfloat16()),
        lambda: B.linear_fp8(q, s, w, sw, status=torch.zeros(1, dtype=torch.int64)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")


def test_fastcall_leaves_anything_unusual_to_the_general_path():
    """-1, without a call and without an exception, for wrong counts, types, devices and tensor subclasses."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    assert build.build_fastcall() is not None
    B._bind_torch()
    q, s = _mat(4, 256)
    x, g = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.float32)
    o = torch.zeros(4, 4, dtype=torch.bfloat16)
    with FakeTensorMode():
        fq = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda")
        fs = torch.empty(4, 4, dtype=torch.float8_e8m0fnu, device="cuda")
        fx, fo = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 4, device="cuda")
    calls = [(B._fast_quantize, a) for a in [(), (x,), (x, q, s), (None, q, s), (x, None, None), (1, 2, 3), (fx, fq, fs)]]
    calls += [(B._fast_norm, a) for a in [(), (0, x, g, None, None, 1e-5, None, q, s), ("rms",) + (None,) * 8,
                                          (0, fx, fx, None, None, 1e-5, None, fq, fs), (0,) * 9]]
    calls += [(B._fast_linear, a) for a in [(), (q, s, q, s, None, o, None, False), (q, s, q, s, None, o, None, 1),
                                            (fq, fs, fq, fs, None, fo, None, False), (None,) * 8]]
    for f, a in calls:
        assert f(*a) == -1


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs gcc")
def test_header_is_c99(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "enc_fp8.h"\nint main(void) { return enc_fp8_scale_pitch(1280) == 12 ? 0 : 1; }\n')
    lib = build.build()
    exe = str(tmp_path / "t")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", exe, "-L", os.path.dirname(lib), "-lenc_b200",
                        "-Wl,-rpath," + os.path.dirname(lib)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert subprocess.run([exe], timeout=60).returncode == 0


def test_enum_values_match_the_header():
    src = open(os.path.join(ROOT, "include", "enc_fp8.h")).read()
    for name, value in (("ENC_NORM_RMS", B.ENC_NORM_RMS), ("ENC_NORM_LAYER", B.ENC_NORM_LAYER),
                        ("ENC_FP8_OUT_BF16", B.ENC_FP8_OUT_BF16), ("ENC_FP8_OUT_FP32", B.ENC_FP8_OUT_FP32),
                        ("ENC_FP8_OUT_FP8", B.ENC_FP8_OUT_FP8), ("ENC_FP8_OUT_RESID", B.ENC_FP8_OUT_RESID)):
        assert f"{name} = {value}" in src
    assert ctypes.sizeof(ctypes.c_int64) == 8


# ------------------------------------------------------- the short call's module
@pytest.mark.parametrize("compiler", ["fails", "missing"])
def test_library_builds_where_the_short_call_does_not(lib, tmp_path, monkeypatch, compiler):
    """build() warns and takes an old module away; the library is there and the calls go through ctypes."""
    bin_dir = tmp_path / "bin"
    bin_dir.mkdir()
    if compiler == "fails":
        (bin_dir / "g++").write_text("#!/bin/sh\necho no c10_cuda >&2\nexit 1\n")
        (bin_dir / "g++").chmod(0o755)
    module = tmp_path / "_fastcall.so"
    module.write_bytes(b"of another build")
    monkeypatch.setattr(build, "FASTCALL", str(module))
    monkeypatch.setattr(build, "FASTCALL_STAMP", str(tmp_path / "stamp"))
    monkeypatch.setenv("PATH", str(bin_dir))
    with pytest.warns(UserWarning, match="ctypes"):
        assert build.build() == build.LIB
    assert not module.exists()
    with pytest.raises((OSError, RuntimeError)):
        build.build_fastcall()


def test_short_call_is_rebuilt_for_another_pytorch(lib, tmp_path, monkeypatch):
    calls = []

    def compiled(cmd, **_):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "wb").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", compiled)
    monkeypatch.setattr(build, "FASTCALL", str(tmp_path / "_fastcall.so"))
    monkeypatch.setattr(build, "FASTCALL_STAMP", str(tmp_path / "stamp"))
    assert build.build_fastcall() and build.build_fastcall() and len(calls) == 1
    assert any(torch.__version__ in arg for arg in calls[0])
    (tmp_path / "stamp").write_text("0.0.1")
    assert build.build_fastcall() and len(calls) == 2


def test_short_call_of_another_pytorch_is_not_used(lib, monkeypatch):
    import types
    import audio_encoder_tower_b200 as package
    B._bind_torch()
    assert B._fast_quantize.__name__ == "quantize"
    other = types.SimpleNamespace(torch_version="0.0.1", quantize=None, norm=None, linear=None)
    with monkeypatch.context() as m:
        m.setattr(package, "_fastcall", other)
        B._bind_torch()
        assert B._fast_quantize(1, 2, 3) == -1 and B._fast_norm() == -1 and B._fast_linear() == -1
    B._bind_torch()
    assert B._fast_quantize.__name__ == "quantize"


@pytest.mark.parametrize("K", [2 ** 31 - 512, 2 ** 31 - 128, 2 ** 31 - 112, 2 ** 31 - 16])
def test_linear_refuses_a_depth_past_its_range(lib, K):
    """Past 2^31 - 128 the number of blocks overflowed to a negative one, and nothing was summed."""
    assert lib.enc_linear_fp8(A, A, A, A, None, A, None, 0, 4, 128, K, 0, None, None) == UNSUPPORTED
