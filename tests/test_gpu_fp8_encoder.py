"""The encoder with its linear layers in e4m3 (ENC_FLAG_FP8) against the oracle.

The bound is the size of those roundings on the same clip, from the rounding-point
model (oracle/fp8_model.py): the library's values differ from the model's by fp32
and bf16 steps, so some e4m3 roundings fall the other way, but they are as many and
as large. As for the bf16 stress case: relative Frobenius error <= 1.4x the model's
+ 2e-3, max-abs <= 2x the model's."""
import numpy as np
import pytest

import oracle as O
import synthetic as S
from oracle.fp8_model import encode_clip_fp8
from tests.encoder_cases import compare, oracle_clip, run_gpu, to_device

pytestmark = pytest.mark.gpu


def _small(name, **kw):
    base = dict(name=name, n_mels=80, d_model=256, n_layers=2, n_heads=4, ffn_dim=512, frames=333, batch=3,
                dtype="bf16", seed=11)
    base.update(kw)
    return S.EncoderConfig(**base)


def _encoder(cfg, w, **kw):
    from audio_encoder_tower_b200 import Encoder
    args = dict(n_mels=cfg.n_mels, d_model=cfg.d_model, n_layers=cfg.n_layers, n_heads=cfg.n_heads,
                ffn_dim=cfg.ffn_dim, max_frames=cfg.frames, max_batch=cfg.batch, dtype=cfg.dtype,
                pool_step=cfg.pool_step, proj_hidden=cfg.proj_hidden, proj_out=cfg.proj_out, ln_eps=cfg.ln_eps,
                attn_chunk=cfg.attn_chunk, guard=True, fp8=True, weights=w)
    return Encoder(**(args | kw))


def _check(cfg, w, mel, got, length, n_out):
    ref = oracle_clip(cfg, w, mel, length)
    band = compare(cfg, encode_clip_fp8(cfg, w, mel, length), ref, n_out)
    m = compare(cfg, got, ref, n_out)
    assert m["rel_fro"] <= 1.4 * band["rel_fro"] + 2e-3 and m["max_abs"] <= 2.0 * band["max_abs"], (m, band)
    return m, band


CASES = [
    (_small("ragged"), [333, 200, 1]),
    (_small("even", frames=400, n_mels=128), [400, 399, 256]),
    (_small("narrow", d_model=128, n_heads=2, ffn_dim=384), [333, 129, 2]),
    (_small("pool_proj", pool_step=2, proj_hidden=256, proj_out=384, d_model=384, n_heads=6), [333, 50, 3]),
    (_small("pool4", pool_step=4), [333, 302, 9]),
    (_small("chunk", attn_chunk=50), [333, 201, 99]),
]


@pytest.mark.parametrize("cfg,lengths", CASES, ids=[c.name for c, _ in CASES])
def test_small_configs(cfg, lengths):
    w, mel = S.make_weights(cfg), S.make_mel(cfg)
    enc = _encoder(cfg, to_device(cfg, w))
    got = run_gpu(enc, cfg, mel, np.array(lengths, np.int32))
    n_out, _, _ = enc.output_positions(cfg.batch, np.array(lengths, np.int32))
    enc.close()
    for b, ln in enumerate(lengths):
        _check(cfg, w, mel[b], got[b], ln, int(n_out[b]))


def test_whisper_large_width_sampled():
    """Two blocks at Whisper-large width on one full 30 s clip of a batch of three: the shapes of the
    real products (1500 positions per clip, K of 1280 and 5120)."""
    cfg = S.CONFIGS["large_b16"].replace(n_layers=2, batch=3)
    w, mel = S.make_weights(cfg), S.make_mel(cfg)
    enc = _encoder(cfg, to_device(cfg, w))
    got = run_gpu(enc, cfg, mel, None)
    enc.close()
    _check(cfg, w, mel[1], got[1], cfg.frames, 1500)


def test_batch_and_frame_mask_invariance():
    """Clip b alone == clip b in a batch, frames past a clip's length change nothing, and a second
    forward gives the same (bit-exact)."""
    cfg = _small("inv", batch=4, frames=300)
    lengths = np.array([300, 150, 77, 299], np.int32)
    mel = S.make_mel(cfg)
    enc = _encoder(cfg, to_device(cfg, S.make_weights(cfg)))
    full = run_gpu(enc, cfg, mel, lengths)
    np.testing.assert_array_equal(run_gpu(enc, cfg, mel[2:3], lengths[2:3])[0], full[2])
    mel2 = mel.copy()
    for b, ln in enumerate(lengths):
        mel2[b, :, ln:] = S.round_bf16(np.full((cfg.n_mels, cfg.frames - ln), 7.0, np.float32))
    np.testing.assert_array_equal(run_gpu(enc, cfg, mel2, lengths), full)
    enc.close()


def test_static_scratch_and_cache():
    """The other ways into the forward: without allocation, and through the cache."""
    import torch
    from audio_encoder_tower_b200 import Cache
    cfg = _small("ways", batch=2, frames=301)
    lengths = np.array([301, 77], np.int32)
    enc = _encoder(cfg, to_device(cfg, S.make_weights(cfg)))
    mel = torch.from_numpy(S.make_mel(cfg)).to("cuda", torch.bfloat16)
    ref = enc.forward(mel, lengths).clone()
    enc.status()
    free0 = torch.cuda.mem_get_info()[0]
    out = torch.full_like(ref, float("nan"))
    enc.forward_static_scratch(mel, lengths, out)
    enc.status()
    assert torch.equal(out, ref) and torch.cuda.mem_get_info()[0] == free0
    assert torch.equal(enc.forward(mel, lengths), ref)
    cache = Cache(enc, 4)
    for want_hits in (0, 1):
        got, hits = cache.forward(mel, lengths=lengths)
        enc.status()
        assert list(hits) == [want_hits] * 2 and torch.equal(got, ref)
    cache.close()
    enc.check_guards()
    enc.close()


def test_weights_at_any_address():
    """Weights that are views at odd element offsets of one buffer give the same output."""
    import torch
    cfg = _small("views", n_layers=1, batch=1)
    w = to_device(cfg, S.make_weights(cfg))
    moved = {}
    for k, v in w.items():
        buf = torch.empty(v.numel() + 3, dtype=v.dtype, device="cuda")
        buf[3:] = v.reshape(-1)
        moved[k] = buf[3:].view(v.shape)
    mel = S.make_mel(cfg)
    outs = []
    for weights in (w, moved):
        enc = _encoder(cfg, weights)
        outs.append(run_gpu(enc, cfg, mel, None))
        enc.close()
    np.testing.assert_array_equal(outs[0], outs[1])


def test_allocation_failures_and_refusals(monkeypatch):
    """Every device allocation of an fp8 handle failing in turn leaves nothing behind; fp32 has no e4m3 layers."""
    import torch
    from audio_encoder_tower_b200 import EncError
    cfg = _small("alloc", n_layers=1, batch=1, frames=100)
    w = to_device(cfg, S.make_weights(cfg))
    _encoder(cfg, w).close()
    torch.cuda.synchronize()
    free0 = torch.cuda.mem_get_info()[0]
    failed = 0
    for n in range(1, 200):
        monkeypatch.setenv("ENC_FAIL_ALLOC", str(n))
        try:
            _encoder(cfg, w).close()
            break
        except EncError as e:
            assert e.code == 3
            failed += 1
    monkeypatch.delenv("ENC_FAIL_ALLOC")
    assert failed >= 30
    assert abs(torch.cuda.mem_get_info()[0] - free0) < (8 << 20)
    with pytest.raises(EncError) as ei:
        _encoder(cfg.replace(dtype="fp32"), {k: v.float() for k, v in w.items()})
    assert ei.value.code == 1


def test_smaller_than_bf16():
    """e4m3 weights and activations take less device memory than bf16 ones."""
    cfg = _small("size", d_model=512, n_heads=8, ffn_dim=2048)
    w = to_device(cfg, S.make_weights(cfg))
    sizes = []
    for fp8 in (False, True):
        enc = _encoder(cfg, w, fp8=fp8, guard=False)
        sizes.append(enc.device_bytes())
        enc.close()
    assert sizes[1] < sizes[0]
