"""ctypes binding of the encoder C ABI (include/enc.h).

Argument marshalling only: every step of the forward pass runs in the CUDA
kernels of libenc_b200.so. PyTorch provides device memory and streams.
The library must be built (python -m audio_encoder_tower_b200.build); there is
no fallback of any kind when it is missing.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libenc_b200.so")

ENC_OK, ENC_ERR_INVALID_ARG, ENC_ERR_UNSUPPORTED, ENC_ERR_OOM, ENC_ERR_CUDA, ENC_ERR_TIMEOUT, \
    ENC_ERR_DEVICE_CHECK = range(7)
ENC_DTYPE_BF16, ENC_DTYPE_FP32 = 0, 1

EXPORTED = ["enc_create", "enc_forward", "enc_output_positions", "enc_get_status", "enc_destroy",
            "enc_status_string", "enc_device_bytes", "enc_linear_bf16", "enc_attention_bf16",
            "enc_profile_enable", "enc_profile_collect", "enc_launch_count", "enc_forward_static_scratch",
            "enc_frontend_create", "enc_frontend_log_mel", "enc_frontend_destroy",
            "enc_cache_create", "enc_forward_cached", "enc_cache_size", "enc_cache_destroy", "enc_cache_content_keys",
            "enc_clip_flops", "enc_shard_plan", "enc_selftest_timeout", "enc_check_guards",
            "enc_guard_selftest", "enc_fp8_scale_pitch", "enc_quantize_fp8", "enc_norm_fp8", "enc_linear_fp8"]
ENC_FLAG_GUARD, ENC_FLAG_FP8 = 1, 2
ENC_NORM_RMS, ENC_NORM_LAYER = 0, 1
ENC_FP8_OUT_BF16, ENC_FP8_OUT_FP32, ENC_FP8_OUT_FP8, ENC_FP8_OUT_RESID = range(4)

KERNEL_CLASSES = ["mel", "conv1", "conv2", "ln", "qkv", "attn", "out", "fc1", "fc2", "final", "proj1", "proj2",
                  "zero"]


class EncError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


class EncConfig(ctypes.Structure):
    _fields_ = [("n_mels", ctypes.c_int32), ("d_model", ctypes.c_int32), ("n_layers", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("ffn_dim", ctypes.c_int32),
                ("max_frames", ctypes.c_int32), ("max_batch", ctypes.c_int32), ("pool_step", ctypes.c_int32),
                ("proj_hidden", ctypes.c_int32), ("proj_out", ctypes.c_int32), ("ln_eps", ctypes.c_float),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32), ("attn_chunk", ctypes.c_int32)]


_VP = ctypes.c_void_p
_VPP = ctypes.POINTER(ctypes.c_void_p)
LAYER_FIELDS = ["ln1_g", "ln1_b", "q_w", "q_b", "k_w", "k_b", "v_w", "v_b", "o_w", "o_b", "ln2_g", "ln2_b",
                "fc1_w", "fc1_b", "fc2_w", "fc2_b"]


class EncKernelTimes(ctypes.Structure):
    _fields_ = [("ms", ctypes.c_double * 13), ("flops", ctypes.c_double * 13), ("launches", ctypes.c_int64 * 13)]


class EncWeights(ctypes.Structure):
    _fields_ = ([("conv1_w", _VP), ("conv1_b", _VP), ("conv2_w", _VP), ("conv2_b", _VP)] +
                [(f, _VPP) for f in LAYER_FIELDS] +
                [("lnpost_g", _VP), ("lnpost_b", _VP), ("proj1_w", _VP), ("proj1_b", _VP),
                 ("proj2_w", _VP), ("proj2_b", _VP)])


_LIB = None


def load_library(path: str = LIB_PATH):
    """Load libenc_b200.so and declare the signatures of every exported call."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m audio_encoder_tower_b200.build`")
    lib = ctypes.CDLL(path)
    i32p = ctypes.POINTER(ctypes.c_int32)
    lib.enc_create.argtypes = [ctypes.POINTER(EncConfig), ctypes.POINTER(EncWeights), ctypes.POINTER(ctypes.c_void_p)]
    lib.enc_create.restype = ctypes.c_int
    lib.enc_forward.argtypes = [_VP, _VP, i32p, ctypes.c_int32, _VP, _VP]
    lib.enc_forward.restype = ctypes.c_int
    lib.enc_output_positions.argtypes = [_VP, ctypes.c_int32, i32p, i32p, i32p, i32p]
    lib.enc_output_positions.restype = ctypes.c_int
    lib.enc_get_status.argtypes = [_VP, _VP]
    lib.enc_get_status.restype = ctypes.c_int
    lib.enc_destroy.argtypes = [_VP]
    lib.enc_destroy.restype = None
    lib.enc_status_string.argtypes = [ctypes.c_int]
    lib.enc_status_string.restype = ctypes.c_char_p
    lib.enc_device_bytes.argtypes = [_VP]
    lib.enc_device_bytes.restype = ctypes.c_size_t
    lib.enc_linear_bf16.argtypes = [_VP, _VP, _VP, _VP, _VP, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.c_int32, _VP, _VP]
    lib.enc_linear_bf16.restype = ctypes.c_int
    lib.enc_attention_bf16.argtypes = [_VP, _VP, _VP, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                       ctypes.c_int32, _VP, _VP]
    lib.enc_attention_bf16.restype = ctypes.c_int
    lib.enc_profile_enable.argtypes = [_VP, ctypes.c_int32]
    lib.enc_profile_enable.restype = ctypes.c_int
    lib.enc_profile_collect.argtypes = [_VP, ctypes.POINTER(EncKernelTimes)]
    lib.enc_profile_collect.restype = ctypes.c_int
    lib.enc_launch_count.argtypes = [_VP]
    lib.enc_launch_count.restype = ctypes.c_int64
    lib.enc_forward_static_scratch.argtypes = [_VP, _VP, i32p, ctypes.c_int32, _VP, _VP]
    lib.enc_forward_static_scratch.restype = ctypes.c_int
    lib.enc_frontend_create.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)]
    lib.enc_frontend_create.restype = ctypes.c_int
    lib.enc_frontend_log_mel.argtypes = [_VP, _VP, ctypes.c_int32, _VP, ctypes.c_int32, _VP]
    lib.enc_frontend_log_mel.restype = ctypes.c_int
    lib.enc_frontend_destroy.argtypes = [_VP]
    lib.enc_frontend_destroy.restype = None
    lib.enc_cache_create.argtypes = [_VP, ctypes.c_int32, ctypes.POINTER(ctypes.c_void_p)]
    lib.enc_cache_create.restype = ctypes.c_int
    lib.enc_forward_cached.argtypes = [_VP, _VP, i32p, ctypes.POINTER(ctypes.c_uint64), ctypes.c_int32, _VP, i32p,
                                       _VP]
    lib.enc_forward_cached.restype = ctypes.c_int
    lib.enc_cache_content_keys.argtypes = [_VP, _VP, i32p, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint64), _VP]
    lib.enc_cache_content_keys.restype = ctypes.c_int
    lib.enc_cache_size.argtypes = [_VP]
    lib.enc_cache_size.restype = ctypes.c_int32
    lib.enc_cache_destroy.argtypes = [_VP]
    lib.enc_cache_destroy.restype = None
    lib.enc_check_guards.argtypes = [_VP, ctypes.c_char_p, ctypes.c_size_t]
    lib.enc_check_guards.restype = ctypes.c_int
    lib.enc_guard_selftest.argtypes = [_VP, ctypes.c_int32, ctypes.c_int64]
    lib.enc_guard_selftest.restype = ctypes.c_int
    lib.enc_selftest_timeout.argtypes = [_VP, ctypes.c_int64, _VP]
    lib.enc_selftest_timeout.restype = ctypes.c_int
    lib.enc_clip_flops.argtypes = [ctypes.POINTER(EncConfig), ctypes.c_int32, ctypes.POINTER(ctypes.c_double)]
    lib.enc_clip_flops.restype = ctypes.c_int
    lib.enc_shard_plan.argtypes = [ctypes.POINTER(EncConfig), i32p, ctypes.c_int32, ctypes.c_int32, i32p, i32p, i32p,
                                   ctypes.POINTER(ctypes.c_double)]
    lib.enc_shard_plan.restype = ctypes.c_int
    lib.enc_fp8_scale_pitch.argtypes = [ctypes.c_int32]
    lib.enc_fp8_scale_pitch.restype = ctypes.c_int32
    lib.enc_quantize_fp8.argtypes = [_VP, ctypes.c_int32, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, _VP, _VP,
                                     _VP]
    lib.enc_quantize_fp8.restype = ctypes.c_int
    lib.enc_norm_fp8.argtypes = [ctypes.c_int32, _VP, ctypes.c_int32, ctypes.c_int64, _VP, ctypes.c_int32,
                                 ctypes.c_int64, _VP, _VP, ctypes.c_float, ctypes.c_int32, ctypes.c_int32, _VP,
                                 ctypes.c_int64, _VP, _VP, _VP]
    lib.enc_norm_fp8.restype = ctypes.c_int
    lib.enc_linear_fp8.argtypes = [_VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                   ctypes.c_int32, ctypes.c_int32, _VP, _VP]
    lib.enc_linear_fp8.restype = ctypes.c_int
    _LIB = lib
    return lib


def status_string(code: int) -> str:
    return load_library().enc_status_string(int(code)).decode()


def _check(code: int, what: str):
    if code != ENC_OK:
        raise EncError(code, what)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _stream_handle(stream) -> int | None:
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _new_output(shape, dtype, device, stream):
    """A tensor for a call on `stream` (None: the current one) to write. It comes from that
    stream's memory, for a block that the current stream has freed may still have work queued there;
    the current stream is recorded as a user, so that it may read the result until it is freed."""
    import torch
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_stream_handle(stream), device=device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=device)
    out.record_stream(torch.cuda.current_stream(device))
    return out


def encoder_config(*, n_mels, d_model, n_layers, n_heads, ffn_dim, max_frames, max_batch, dtype="bf16",
                   pool_step=1, proj_hidden=0, proj_out=0, ln_eps=1e-5, head_dim=64, attn_chunk=0,
                   guard=False, fp8=False) -> EncConfig:
    """The enc_config struct of a tower geometry (dtype "bf16" or "fp32"); guard sets
    ENC_FLAG_GUARD, fp8 sets ENC_FLAG_FP8 (the blocks' linear layers in e4m3; dtype "bf16")."""
    return EncConfig(n_mels, d_model, n_layers, n_heads, head_dim, ffn_dim, max_frames, max_batch, pool_step,
                     proj_hidden, proj_out, ln_eps, ENC_DTYPE_BF16 if dtype == "bf16" else ENC_DTYPE_FP32,
                     (ENC_FLAG_GUARD if guard else 0) | (ENC_FLAG_FP8 if fp8 else 0), attn_chunk)


def clip_flops(cfg: EncConfig, length: int) -> float:
    """Algorithmic FLOPs of one clip of `length` valid frames (enc_clip_flops)."""
    v = ctypes.c_double()
    _check(load_library().enc_clip_flops(ctypes.byref(cfg), int(length), ctypes.byref(v)), "enc_clip_flops")
    return float(v.value)


def shard_plan(cfg: EncConfig, lengths, world: int):
    """Split clips over `world` ranks of cfg.max_batch clips each (enc_shard_plan).

    lengths: [B] valid frames per clip, or an int B for B full-length clips.
    Returns (rank_of [B], index_of [B], rank_count [world], rank_flops [world]).
    """
    i32p = ctypes.POINTER(ctypes.c_int32)
    if isinstance(lengths, (int, np.integer)):
        B, ln = int(lengths), None
    else:
        ln = np.ascontiguousarray(np.asarray(lengths, dtype=np.int32))
        B = int(ln.shape[0])
    rank_of = np.zeros(B, np.int32)
    index_of = np.zeros(B, np.int32)
    count = np.zeros(max(int(world), 1), np.int32)
    flops = np.zeros(max(int(world), 1), np.float64)
    _check(load_library().enc_shard_plan(ctypes.byref(cfg), None if ln is None else ln.ctypes.data_as(i32p), B,
                                         int(world), rank_of.ctypes.data_as(i32p), index_of.ctypes.data_as(i32p),
                                         count.ctypes.data_as(i32p),
                                         flops.ctypes.data_as(ctypes.POINTER(ctypes.c_double))), "enc_shard_plan")
    return rank_of, index_of, count, flops


class Encoder:
    """One encoder handle (enc_create / enc_forward / enc_destroy).

    weights: dict of device tensors in PyTorch layouts named as in enc.h
    ("conv1_w", "layers.{l}.q_w", "lnpost_g", "proj1_w", ...), dtype matching
    `dtype` ("bf16" or "fp32"). They may be freed after construction.
    fp8=True runs the blocks' linear layers on e4m3 operands (ENC_FLAG_FP8).
    """

    def __init__(self, *, n_mels, d_model, n_layers, n_heads, ffn_dim, max_frames, max_batch, dtype="bf16",
                 pool_step=1, proj_hidden=0, proj_out=0, ln_eps=1e-5, head_dim=64, attn_chunk=0, guard=False,
                 fp8=False, weights: dict):
        self.lib = load_library()
        self.cfg = encoder_config(n_mels=n_mels, d_model=d_model, n_layers=n_layers, n_heads=n_heads,
                                  ffn_dim=ffn_dim, max_frames=max_frames, max_batch=max_batch, dtype=dtype,
                                  pool_step=pool_step, proj_hidden=proj_hidden, proj_out=proj_out, ln_eps=ln_eps,
                                  head_dim=head_dim, attn_chunk=attn_chunk, guard=guard, fp8=fp8)
        w = EncWeights()
        for f in ("conv1_w", "conv1_b", "conv2_w", "conv2_b", "lnpost_g", "lnpost_b",
                  "proj1_w", "proj1_b", "proj2_w", "proj2_b"):
            setattr(w, f, _ptr(weights.get(f)))
        keep = []
        for f in LAYER_FIELDS:
            arr = (ctypes.c_void_p * max(n_layers, 1))()
            for l in range(n_layers):
                arr[l] = _ptr(weights.get(f"layers.{l}.{f}"))
            keep.append(arr)
            setattr(w, f, ctypes.cast(arr, _VPP))
        h = ctypes.c_void_p()
        _check(self.lib.enc_create(ctypes.byref(self.cfg), ctypes.byref(w), ctypes.byref(h)), "enc_create")
        self.handle = h
        self.dtype = dtype

    # ----------------------------------------------------------- geometry
    def output_positions(self, B: int, lengths=None):
        """(n_out [B] int32, p_out, d_out) for a batch, from the library."""
        n_out = np.zeros(B, np.int32)
        p = ctypes.c_int32()
        dd = ctypes.c_int32()
        lp = None
        if lengths is not None:
            lengths = np.ascontiguousarray(lengths, dtype=np.int32)
            lp = lengths.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        _check(self.lib.enc_output_positions(self.handle, B, lp, n_out.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                                             ctypes.byref(p), ctypes.byref(dd)), "enc_output_positions")
        return n_out, p.value, dd.value

    # ------------------------------------------------------------ forward
    def forward(self, mel, lengths=None, out=None, stream=None):
        """Enqueue the forward pass of mel [B, n_mels, T] (device) on `stream`.

        Returns `out` [B, P_out, d_out] (allocated with torch when not given).
        """
        B = int(mel.shape[0])
        if out is None:
            _, p_out, d_out = self.output_positions(B, lengths)
            out = _new_output((B, p_out, d_out), mel.dtype, mel.device, stream)
        lp = None
        if lengths is not None:
            self._len = np.ascontiguousarray(lengths, dtype=np.int32)
            lp = self._len.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        _check(self.lib.enc_forward(self.handle, _ptr(mel), lp, B, _ptr(out), _stream_handle(stream)),
               "enc_forward")
        return out

    def forward_static_scratch(self, mel, lengths=None, out=None, stream=None):
        """enc_forward_static_scratch: the same forward with its workspace in the
        library's fixed 64 MiB static device array (no device allocation in the call).

        `out` must be given by callers that cannot allocate; when omitted it is
        allocated here with torch for convenience.
        """
        B = int(mel.shape[0])
        if out is None:
            _, p_out, d_out = self.output_positions(B, lengths)
            out = _new_output((B, p_out, d_out), mel.dtype, mel.device, stream)
        lp = None
        if lengths is not None:
            self._len = np.ascontiguousarray(lengths, dtype=np.int32)
            lp = self._len.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
        _check(self.lib.enc_forward_static_scratch(self.handle, _ptr(mel), lp, B, _ptr(out),
                                                   _stream_handle(stream)), "enc_forward_static_scratch")
        return out

    def status(self, stream=None):
        """Synchronise `stream` and raise if a device-side check or wait failed."""
        _check(self.lib.enc_get_status(self.handle, _stream_handle(stream)), "enc_get_status")

    def check_guards(self):
        """enc_check_guards (handles created with guard=True): raise EncError naming the
        buffer and offset if a kernel wrote into a guard region around a workspace buffer."""
        msg = ctypes.create_string_buffer(256)
        code = self.lib.enc_check_guards(self.handle, msg, 256)
        if code != ENC_OK:
            raise EncError(code, "enc_check_guards: " + msg.value.decode())

    def guard_selftest(self, buffer: int, offset: int):
        """enc_guard_selftest: one guard byte changed from the host is reported, then restored."""
        _check(self.lib.enc_guard_selftest(self.handle, int(buffer), int(offset)), "enc_guard_selftest")

    def selftest_timeout(self, limit_ns: int, stream=None):
        """Enqueue the failure-detection self-test (enc_selftest_timeout): a bounded
        wait that runs out after limit_ns; the next status() raises ENC_ERR_TIMEOUT."""
        _check(self.lib.enc_selftest_timeout(self.handle, int(limit_ns), _stream_handle(stream)),
               "enc_selftest_timeout")

    def profile(self, enable: bool):
        """Bracket every kernel of the following forwards with CUDA events."""
        _check(self.lib.enc_profile_enable(self.handle, 1 if enable else 0), "enc_profile_enable")

    def collect_profile(self) -> dict:
        """{class: (ms, flops, launches)} summed since the last collect (waits for the events)."""
        t = EncKernelTimes()
        _check(self.lib.enc_profile_collect(self.handle, ctypes.byref(t)), "enc_profile_collect")
        return {k: (t.ms[i], t.flops[i], int(t.launches[i])) for i, k in enumerate(KERNEL_CLASSES)
                if t.launches[i]}

    def launch_count(self) -> int:
        return int(self.lib.enc_launch_count(self.handle))

    def device_bytes(self) -> int:
        return int(self.lib.enc_device_bytes(self.handle))

    def close(self):
        if getattr(self, "handle", None):
            self.lib.enc_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------- single-kernel calls
def linear_bf16(A, W, bias=None, out=None, resid=None, gelu=False, status=None, stream=None):
    """out = act(A W^T + bias) on the tensor cores (bf16 in/out), or resid += A W^T + bias."""
    import torch
    M, K = A.shape
    N = W.shape[0]
    if out is None and resid is None:
        out = _new_output((M, N), torch.bfloat16, A.device, stream)
    _check(load_library().enc_linear_bf16(_ptr(A), _ptr(W), _ptr(bias), _ptr(out), _ptr(resid), M, N, K,
                                          1 if gelu else 0, _ptr(status), _stream_handle(stream)),
           "enc_linear_bf16")
    return out if resid is None else resid


def attention_bf16(qkv, cu, max_n, n_heads, out=None, status=None, stream=None):
    """Packed-clip bidirectional attention: qkv [R, 3d] bf16, cu device int32 [B+1]."""
    import torch
    R = qkv.shape[0]
    d = 64 * n_heads
    if out is None:
        out = _new_output((R, d), torch.bfloat16, qkv.device, stream)
    _check(load_library().enc_attention_bf16(_ptr(qkv), _ptr(out), _ptr(cu), int(R), int(cu.numel()) - 1,
                                             int(max_n), int(n_heads), _ptr(status), _stream_handle(stream)),
           "enc_attention_bf16")
    return out


# ------------------------------------------------------ 8-bit (e4m3) operators
def fp8_scale_pitch(cols: int) -> int:
    """Bytes of one row of a scale matrix: ceil(cols / 128) rounded up to a multiple of four."""
    return (int(cols) + 511) // 512 * 4


def _expect(ok, what: str):
    if not ok:
        raise ValueError(what)


# What the 8-bit functions use of torch, looked up once. A call through ctypes costs 8 to 12 us of
# host time, more than a small launch takes on the device, so their usual case (outputs given, the
# current stream, contiguous tensors) goes through the module _fastcall (csrc/fastcall.cpp) where
# that has been built: 0 from it means launched, anything else takes the way below it.
_torch = _BF16 = _FP32 = _E4M3 = _E8M0 = _U8 = _raw_stream = _cur_device = None
_fast_quantize = _fast_norm = _fast_linear = None


def _bind_torch():
    global _torch, _BF16, _FP32, _E4M3, _E8M0, _U8, _raw_stream, _cur_device
    global _fast_quantize, _fast_norm, _fast_linear
    import torch
    _BF16, _FP32, _U8 = torch.bfloat16, torch.float32, torch.uint8
    _E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    _raw_stream, _cur_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    load_library()
    try:
        from . import _fastcall
        if getattr(_fastcall, "torch_version", None) != torch.__version__:
            raise ImportError("built against another PyTorch")
        _fast_quantize, _fast_norm, _fast_linear = _fastcall.quantize, _fastcall.norm, _fastcall.linear
    except ImportError:
        _fast_quantize = _fast_norm = _fast_linear = lambda *args: -1
    _torch = torch


def _fp8_call(fn, what, device, stream, *args):
    """fn(*args, stream handle) on `device` (an ordinal, made current). stream=None is the
    device's current stream."""
    if device < 0:
        raise ValueError("the tensors must be on a CUDA device")
    if device != _cur_device():
        with _torch.cuda.device(device):
            return _fp8_call(fn, what, device, stream, *args)
    code = fn(*args, _raw_stream(device) if stream is None else _stream_handle(stream))
    if code != ENC_OK:
        raise EncError(code, what)


def _row_stride(t, shape, device, what: str):
    """(enc_dtype, row stride) of a bf16 or fp32 matrix of that shape whose rows are contiguous."""
    dt = t.dtype
    if (dt == _BF16 or dt == _FP32) and t.shape == shape and t.get_device() == device:
        code = ENC_DTYPE_BF16 if dt == _BF16 else ENC_DTYPE_FP32
        if t.is_contiguous():
            return code, shape[1]
        rs, cs = t.stride()
        if cs == 1 or shape[1] <= 1:
            return code, (rs if shape[0] > 1 else shape[1])
    raise ValueError(f"{what} must be a bf16 or fp32 {list(shape)} matrix with contiguous rows on device {device}")


def _matrix_shape(t, what: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what} must be a matrix")
    return shape


def _check_fp8(q, scales, rows, cols, device, what: str):
    """An e4m3 [rows, cols] matrix with its block scales, both contiguous and on `device`."""
    st = scales.dtype
    if q.dtype == _E4M3 and q.shape == (rows, cols) and q.get_device() == device and q.is_contiguous() and \
            (st == _E8M0 or st == _U8) and scales.shape == (rows, (cols + 511) // 512 * 4) and \
            scales.get_device() == device and scales.is_contiguous():
        return
    raise ValueError(f"{what} must be a contiguous float8_e4m3fn [{rows}, {cols}] tensor on device {device}, and its "
                     f"scales a contiguous float8_e8m0fnu [{rows}, {fp8_scale_pitch(cols)}] tensor there")


def _fp8_out(q, scales, rows, cols, like, stream, what: str):
    """(q, scales): the caller's output matrix, or a new one beside `like` for a call on `stream`."""
    if q is None:
        q = _new_output((rows, cols), _E4M3, like.device, stream)
    if scales is None:
        scales = _new_output((rows, fp8_scale_pitch(cols)), _E8M0, like.device, stream)
    _check_fp8(q, scales, rows, cols, like.get_device(), what)
    return q, scales


def _check_vector(v, n, device, what: str):
    """A contiguous fp32 [n] vector on `device`, or None."""
    if v is not None and (v.dtype != _FP32 or v.shape != (n,) or not v.is_contiguous()
                          or v.get_device() != device):
        raise ValueError(f"{what} must be a contiguous fp32 [{n}] tensor on device {device}")


def quantize_fp8(x, q=None, scales=None, stream=None):
    """Rows of x [rows, cols] (bf16 or fp32, cols a multiple of 16) as e4m3 with a power-of-two
    scale for each block of 128 columns (enc_quantize_fp8).

    Returns (q float8_e4m3fn [rows, cols], scales float8_e8m0fnu [rows, fp8_scale_pitch(cols)]):
    element (r, c) stands for q[r, c] * scales[r, c // 128].
    """
    if _torch is None:
        _bind_torch()
    if stream is None and q is not None and _fast_quantize(x, q, scales) == ENC_OK:
        return q, scales
    dev = x.get_device()
    rows, cols = shape = _matrix_shape(x, "x")
    dtype, ldx = _row_stride(x, shape, dev, "x")
    q, scales = _fp8_out(q, scales, rows, cols, x, stream, "q")
    _fp8_call(_LIB.enc_quantize_fp8, "enc_quantize_fp8", dev, stream, x.data_ptr(), dtype, ldx, rows,
              cols, q.data_ptr(), scales.data_ptr())
    return q, scales


def norm_fp8(x, gamma, beta=None, delta=None, kind="rms", eps=1e-5, x_out=None, q=None, scales=None, stream=None):
    """RMS norm (kind "rms") or LayerNorm ("layer") of the residual stream x [rows, d] (bf16 or
    fp32) after the addition of delta [rows, d] (bf16, fp32 or None), as e4m3 with block scales
    (enc_norm_fp8).

    Returns (q, scales, x_out): x_out is the stream after the addition, in x's type; without a
    delta it is x itself, and x_out=x updates the stream in place. gamma, beta: fp32 [d].
    """
    if _torch is None:
        _bind_torch()
    if gamma is None or (kind != "rms" and kind != "layer"):
        raise ValueError('gamma is required, and kind must be "rms" or "layer"')
    number = ENC_NORM_RMS if kind == "rms" else ENC_NORM_LAYER
    if stream is None and q is not None and (delta is None or x_out is not None) and \
            _fast_norm(number, x, gamma, beta, delta, eps, x_out, q, scales) == ENC_OK:
        return q, scales, x if x_out is None else x_out
    dev = x.get_device()
    rows, d = shape = _matrix_shape(x, "x")
    dtype, ldx = _row_stride(x, shape, dev, "x")
    _check_vector(gamma, d, dev, "gamma")
    _check_vector(beta, d, dev, "beta")
    q, scales = _fp8_out(q, scales, rows, d, x, stream, "q")
    ddtype, ldd, ldxo = ENC_DTYPE_BF16, d, d
    if delta is not None:
        ddtype, ldd = _row_stride(delta, shape, dev, "delta")
        if x_out is None:
            x_out = _new_output((rows, d), x.dtype, x.device, stream)
    if x_out is not None:
        odtype, ldxo = _row_stride(x_out, shape, dev, "x_out")
        if odtype != dtype:
            raise ValueError("x_out must have x's type")
    _fp8_call(_LIB.enc_norm_fp8, "enc_norm_fp8", dev, stream,
              number, x.data_ptr(), dtype, ldx,
              None if delta is None else delta.data_ptr(), ddtype, ldd, gamma.data_ptr(),
              None if beta is None else beta.data_ptr(), eps, rows, d, None if x_out is None else x_out.data_ptr(),
              ldxo, q.data_ptr(), scales.data_ptr())
    return q, scales, x if x_out is None else x_out


def linear_fp8(a, a_scales, w, w_scales, bias=None, out=None, out_dtype=None, out_scales=None, resid=None, gelu=False,
               status=None, stream=None):
    """act(A W^T + bias) of e4m3 matrices with block scales (as quantize_fp8 and norm_fp8 give
    them), a [M, K] and w [N, K], K and N multiples of 16 (enc_linear_fp8).

    The result's type is out's, or out_dtype ("bf16" when neither is given, "fp32" or "fp8"):
    returns out, or (out, out_scales) for e4m3. With resid (fp32 [M, N]) the product and the
    bias are added to it instead, and resid is returned. bias: fp32 [N].
    """
    if _torch is None:
        _bind_torch()
    if out is not None and stream is None and resid is None and out_dtype is None and status is None and \
            _fast_linear(a, a_scales, w, w_scales, bias, out, out_scales, gelu) == ENC_OK:
        return out if out_scales is None else (out, out_scales)
    dev = a.get_device()
    M, K = _matrix_shape(a, "a")
    N = _matrix_shape(w, "w")[0]
    _check_fp8(a, a_scales, M, K, dev, "a")
    _check_fp8(w, w_scales, N, K, dev, "w")
    _check_vector(bias, N, dev, "bias")
    if resid is not None:
        _expect(out is None and out_dtype is None and out_scales is None and not gelu,
                "resid takes no out, out_dtype, out_scales or gelu")
        kind, tdt, dst = ENC_FP8_OUT_RESID, _FP32, resid
    else:
        if out_dtype is None:
            tdt = _BF16 if out is None else out.dtype
        else:
            tdt = {"bf16": _BF16, "fp32": _FP32, "fp8": _E4M3}.get(out_dtype)
        if tdt == _E4M3:
            out, out_scales = _fp8_out(out, out_scales, M, N, a, stream, "out")
            kind = ENC_FP8_OUT_FP8
        else:
            kind = ENC_FP8_OUT_BF16 if tdt == _BF16 else ENC_FP8_OUT_FP32
            _expect(kind == ENC_FP8_OUT_BF16 or tdt == _FP32, 'the output type must be "bf16", "fp32" or "fp8"')
            _expect(out_scales is None, "out_scales belong to an e4m3 output")
            if out is None:
                out = _new_output((M, N), tdt, a.device, stream)
        dst = out
    if status is not None and (status.dtype != _torch.int32 or status.numel() < 1 or status.get_device() != dev):
        raise ValueError(f"status must be an int32 tensor on device {dev}")
    if dst.dtype != tdt or dst.shape != (M, N) or dst.get_device() != dev or not dst.is_contiguous():
        raise ValueError(f"the output must be a contiguous {tdt} [{M}, {N}] tensor on device {dev}")
    _fp8_call(_LIB.enc_linear_fp8, "enc_linear_fp8", dev, stream, a.data_ptr(), a_scales.data_ptr(),
              w.data_ptr(), w_scales.data_ptr(), None if bias is None else bias.data_ptr(), dst.data_ptr(),
              None if out_scales is None else out_scales.data_ptr(), kind, M, N, K, 1 if gelu else 0,
              None if status is None else status.data_ptr())
    return (out, out_scales) if kind == ENC_FP8_OUT_FP8 else dst


class Frontend:
    """Log-mel front end (enc_frontend_create / enc_frontend_log_mel / enc_frontend_destroy):
    30 s clips of 16 kHz audio, fp32 [B, 480000] on the device -> [B, n_mels, 3000]."""

    SAMPLES, FRAMES = 480000, 3000

    def __init__(self, n_mels: int = 128, max_batch: int = 16):
        self.lib = load_library()
        h = ctypes.c_void_p()
        _check(self.lib.enc_frontend_create(int(n_mels), int(max_batch), ctypes.byref(h)), "enc_frontend_create")
        self.h, self.n_mels, self.max_batch = h, int(n_mels), int(max_batch)

    def log_mel(self, audio, out=None, dtype="bf16", stream=None):
        import torch
        B = audio.shape[0]
        if audio.dtype != torch.float32 or tuple(audio.shape[1:]) != (self.SAMPLES,) or not audio.is_contiguous():
            raise ValueError("audio must be a contiguous fp32 [B, 480000] device tensor")
        tdt = torch.bfloat16 if dtype == "bf16" else torch.float32
        if out is None:
            out = _new_output((B, self.n_mels, self.FRAMES), tdt, audio.device, stream)
        _check(self.lib.enc_frontend_log_mel(self.h, _ptr(audio), int(B), _ptr(out), 0 if dtype == "bf16" else 1,
                                             _stream_handle(stream)), "enc_frontend_log_mel")
        return out

    def close(self):
        if self.h:
            self.lib.enc_frontend_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Cache:
    """Embeddings cache in front of an Encoder (enc_cache_create / enc_forward_cached):
    outputs looked up by a 64-bit key per clip that identifies its mel and length."""

    def __init__(self, encoder: "Encoder", capacity: int):
        self.lib = load_library()
        self.encoder = encoder
        h = ctypes.c_void_p()
        _check(self.lib.enc_cache_create(encoder.handle, int(capacity), ctypes.byref(h)), "enc_cache_create")
        self.h = h

    def content_keys(self, mel, lengths=None, stream=None) -> np.ndarray:
        """enc_cache_content_keys: [B] uint64 keys hashed from each clip's length and
        valid mel frames on the device (waits for `stream`)."""
        B = int(mel.shape[0])
        ln = None if lengths is None else np.ascontiguousarray(np.asarray(lengths, dtype=np.int32))
        keys = np.zeros(B, dtype=np.uint64)
        i32p = ctypes.POINTER(ctypes.c_int32)
        _check(self.lib.enc_cache_content_keys(self.h, _ptr(mel), None if ln is None else ln.ctypes.data_as(i32p),
                                               B, keys.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)),
                                               _stream_handle(stream)), "enc_cache_content_keys")
        return keys

    def forward(self, mel, keys=None, lengths=None, out=None, stream=None):
        """Returns (out, hits): hits[b] = 1 where clip b's output came from the cache.
        keys=None derives each clip's key from its content (content_keys)."""
        B = int(mel.shape[0])
        if keys is None:
            keys = self.content_keys(mel, lengths, stream)
        if out is None:
            _, p_out, d_out = self.encoder.output_positions(B, lengths)
            out = _new_output((B, p_out, d_out), mel.dtype, mel.device, stream)
        k = np.ascontiguousarray(np.asarray(keys, dtype=np.uint64))
        if k.shape != (B,):
            raise ValueError("one key per clip")
        ln = None if lengths is None else np.ascontiguousarray(np.asarray(lengths, dtype=np.int32))
        hits = np.zeros(B, dtype=np.int32)
        i32p = ctypes.POINTER(ctypes.c_int32)
        _check(self.lib.enc_forward_cached(self.h, _ptr(mel), None if ln is None else ln.ctypes.data_as(i32p),
                                           k.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), int(B), _ptr(out),
                                           hits.ctypes.data_as(i32p), _stream_handle(stream)), "enc_forward_cached")
        return out, hits

    def size(self) -> int:
        return int(self.lib.enc_cache_size(self.h))

    def close(self):
        if self.h:
            self.lib.enc_cache_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
