"""Pins of the e4m3 rounding-point model (oracle/fp8_model.py), CPU only."""
import numpy as np
import pytest

import oracle as O
import synthetic as S
from oracle.bf16_model import encode_clip_bf16
from oracle.fp8_model import encode_clip_fp8


def _small(name, **kw):
    base = dict(name=name, n_mels=80, d_model=256, n_layers=2, n_heads=4, ffn_dim=512, frames=333, batch=3,
                dtype="bf16", seed=11)
    base.update(kw)
    return S.EncoderConfig(**base)


def _rel(cfg, lengths, model, **kw):
    w, mel = S.make_weights(cfg), S.make_mel(cfg)
    out = []
    for b, ln in enumerate(lengths):
        n = O.valid_output_rows(cfg, ln)
        ref = O.encode_clip(cfg, w, mel[b], ln)[:n]
        out.append(float(np.linalg.norm(model(cfg, w, mel[b], ln, **kw)[:n] - ref) / np.linalg.norm(ref)))
    return out


@pytest.mark.parametrize("cfg,lengths", [
    (_small("std"), [333, 200, 1]),
    (_small("pp", pool_step=2, proj_hidden=256, proj_out=128, frames=120), [120, 51, 4]),
    (_small("ck", attn_chunk=7, frames=90), [90, 33, 2])], ids=["std", "pool_proj", "chunk"])
def test_without_rounding_the_model_is_the_oracle(cfg, lengths):
    assert max(_rel(cfg, lengths, encode_clip_fp8, rounding=False)) < 1e-12


def test_band_at_the_workloads_scale():
    """N(0, 0.02) weights, two blocks: e4m3 has 4 significant bits against bf16's 8, and only the
    blocks round to it, so the error is 4 to 16 times bf16's, one or two per cent."""
    cfg, lengths = _small("std"), [333, 200, 1]
    for e8, e16 in zip(_rel(cfg, lengths, encode_clip_fp8), _rel(cfg, lengths, encode_clip_bf16)):
        assert 4 * e16 < e8 < 16 * e16 and 3e-3 < e8 < 3e-2, (e8, e16)
