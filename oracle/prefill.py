"""The operators around the decode, restated plainly in float64 (test
infrastructure): rotation of keys and queries, expansion of cached rows,
attention of packed prompts, value projection.

Rotation: fp32 steps as the library defines them, so its results are exact.
Everything else is computed in float64 and left unrounded, next to the
magnitude sums that bound a lower-precision sum's error.
"""
from __future__ import annotations

import numpy as np

from .kv_insert import bf16_bits_to_f64, f32, f64_to_bf16_bits

D_LATENT = 512
PAGE = 64


def angle_table(max_pos: int, base: float = 10000.0) -> np.ndarray:
    """fp32 [max_pos, 64]: 32 cosines and 32 sines of pos * base^(-i/32)."""
    a = np.arange(max_pos, dtype=np.float64)[:, None] * base ** (-np.arange(32, dtype=np.float64) / 32)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


def rotate(x_bits: np.ndarray, cos_sin: np.ndarray, interleaved: bool) -> np.ndarray:
    """bf16 bits [..., 64] rotated by cos_sin rows [..., 64] -> bf16 bits."""
    x = f32(bf16_bits_to_f64(x_bits))
    c, s = cos_sin[..., :32], cos_sin[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    ra = (a * c).astype(np.float32) - (b * s).astype(np.float32)
    rb = (a * s).astype(np.float32) + (b * c).astype(np.float32)
    y = np.empty(np.broadcast_shapes(x.shape, ra.shape[:-1] + (64,)), np.float32)
    if interleaved:
        y[..., 0::2], y[..., 1::2] = ra, rb
    else:
        y[..., :32], y[..., 32:] = ra, rb
    return f64_to_bf16_bits(y.astype(np.float64)).reshape(y.shape)


def expand(latent: np.ndarray, w_uk: np.ndarray, w_uv: np.ndarray):
    """Latent rows [n, 512] and weights [H, 128, 512] (float64) -> (kv
    [n, H, 256], sum of |products|)."""
    w = np.concatenate([w_uk, w_uv], 1)
    return np.einsum("nl,hpl->nhp", latent, w), np.einsum("nl,hpl->nhp", np.abs(latent), np.abs(w))


def attention(q, k_nope, k_pe, v, scale: float, causal: bool):
    """One sequence in float64: q [nq, H, 192], k_nope and v [nk, H, 128], k_pe
    [nk, 64] -> dict of out [nq, H, 128], lse [nq, H], spread (sum of weights
    times |v|), top (largest |score| of a row) and mag (largest scale * sum
    |q k| of a row).  Keys that a row does not see take no part in it, whatever
    they hold."""
    nq, H, _ = q.shape
    nk = v.shape[0]
    out, spread = np.zeros((nq, H, 128)), np.zeros((nq, H, 128))
    lse, top, mag = np.full((nq, H), -np.inf), np.zeros((nq, H)), np.zeros((nq, H))
    for i in range(nq):
        n = max(0, min(nk, nk - nq + i + 1)) if causal else nk
        if n == 0:
            continue
        for h in range(H):
            k = np.concatenate([k_nope[:n, h], k_pe[:n]], 1)
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (k @ q[i, h])
                m = s.max()
                w = np.exp(s - m)
                z = w.sum()
                lse[i, h] = m + np.log(z)
                w /= z
                out[i, h] = w @ v[:n, h]
                spread[i, h] = w @ np.abs(v[:n, h])
                top[i, h] = np.abs(s).max()
                mag[i, h] = scale * (np.abs(k) @ np.abs(q[i, h])).max()
    return dict(out=out, lse=lse, spread=spread, top=top, mag=mag)


def value_project(attn: np.ndarray, w_uv: np.ndarray):
    """attn [n, H, 512], w_uv [H, 128, 512] (float64) -> (out [n, H, 128], sum
    of |products|)."""
    return np.einsum("nhl,hvl->nhv", attn, w_uv), np.einsum("nhl,hvl->nhv", np.abs(attn), np.abs(w_uv))
