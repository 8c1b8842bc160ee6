"""Rounding-point model of the encoder with its linear layers in e4m3 (TEST
INFRASTRUCTURE): oracle/bf16_model.py's steps with the roundings of ENC_FLAG_FP8.

In the encoder blocks the operands of the q/k/v, output, fc1 and fc2 products are
rounded to e4m3 with a power-of-two scale per block of 128 elements (oracle/fp8.py):
the weights once, the LayerNorm outputs and the GELU output from their unrounded
values, the attention output from its bf16 value. Everything else rounds to bf16 as
in the bf16 model (conv1 output, q / k / v, probabilities, attention output,
projector operands, final output); sums, statistics and the residual stream do not
round. With rounding=False the model is the oracle's computation.
"""
from __future__ import annotations

import numpy as np

from . import fp8 as F8
from .bf16_model import _attention, _chunked, _identity, round_bf16
from .encoder import (avg_pool, conv1d, encoder_positions, gelu, layer_norm, layer_weights, linear,
                      pooled_positions, sinusoids, valid_positions)


def encode_clip_fp8(cfg, w: dict, mel: np.ndarray, length: int, rounding: bool = True) -> np.ndarray:
    """oracle.encode_clip with ENC_FLAG_FP8's rounding points; rows past the valid count are 0."""
    rb = round_bf16 if rounding else _identity
    r8 = (lambda x: F8.quantize(x)[0]) if rounding else _identity
    chunk = getattr(cfg, "attn_chunk", 0)
    n = valid_positions(length)
    x = np.array(mel, dtype=np.float64)
    x[:, length:] = 0.0
    y1 = rb(gelu(conv1d(x, w["conv1_w"], w["conv1_b"], 1)))
    h = gelu(conv1d(y1, w["conv2_w"], w["conv2_b"], 2)).T
    x = (h + sinusoids(h.shape[0], h.shape[1]))[:n]
    for l in range(cfg.n_layers):
        lw = layer_weights(w, l)
        w8 = {k: r8(lw[k]) for k in ("q_w", "k_w", "v_w", "o_w", "fc1_w", "fc2_w")}
        a = r8(layer_norm(x, lw["ln1_g"], lw["ln1_b"], cfg.ln_eps))
        q = rb(linear(a, w8["q_w"], lw["q_b"]))
        k = rb(linear(a, w8["k_w"], None))
        v = rb(linear(a, w8["v_w"], lw["v_b"]))
        att = (_chunked(q, k, v, cfg.n_heads, cfg.head_dim, chunk, rb) if chunk > 0
               else _attention(q, k, v, cfg.n_heads, cfg.head_dim, rb))
        x = x + linear(r8(rb(att)), w8["o_w"], lw["o_b"])
        a = r8(layer_norm(x, lw["ln2_g"], lw["ln2_b"], cfg.ln_eps))
        f = r8(gelu(linear(a, w8["fc1_w"], lw["fc1_b"])))
        x = x + linear(f, w8["fc2_w"], lw["fc2_b"])
    y = layer_norm(x, w["lnpost_g"], w["lnpost_b"], cfg.ln_eps)
    if cfg.pool_step > 1:
        y = avg_pool(y, cfg.pool_step)
    if cfg.proj_hidden:
        e = rb(y)
        p1 = rb(gelu(linear(e, w["proj1_w"], w["proj1_b"])))
        y = linear(p1, w["proj2_w"], w["proj2_b"])
    p_out = pooled_positions(encoder_positions(mel.shape[1]), cfg.pool_step)
    out = np.zeros((p_out, y.shape[1]), np.float64)
    out[: y.shape[0]] = rb(y)
    return out
