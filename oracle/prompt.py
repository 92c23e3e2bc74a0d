"""Oracle of the prompt-side calls: rotary positions, the cache append and dense
chunk attention, in float64.

Test infrastructure only.  The rotary layouts and context scalings are the
published ones (rotary embedding, position interpolation, YaRN's by-parts and
base rules); RMS norm y = x w / sqrt(mean(x^2) + eps) is rounded once to bf16;
the FP4 write is the codec oracle's; attention is a plain softmax over every
visible position of the dequantized cache.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import codec


def rope_frequencies(rot, theta, scaling="plain", factor=1.0, orig_ctx=0.0, turns_lo=1.0, turns_hi=32.0):
    """Angle per position of each of the rot / 2 pairs."""
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2)) if rot > 2 else theta
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        turns = orig_ctx * f / (2 * math.pi)
        k = np.clip((turns - turns_lo) / (turns_hi - turns_lo), 0.0, 1.0)
        f = f * k + f / factor * (1.0 - k)
    return f


def rope(x, pos, freqs, half, mscale=1.0, inverse=False):
    """x [tokens, heads, rot], pos [tokens]: every pair turned by pos * f."""
    x = np.asarray(x, np.float64)
    a = np.asarray(pos, np.float64)[:, None, None] * freqs
    c, s = np.cos(a) * mscale, np.sin(a) * mscale * (-1.0 if inverse else 1.0)
    n = len(freqs)
    y = np.empty_like(x)
    iu, iv = (np.arange(n), np.arange(n) + n) if half else (2 * np.arange(n), 2 * np.arange(n) + 1)
    u, v = x[..., iu], x[..., iv]
    y[..., iu] = u * c - v * s
    y[..., iv] = u * s + v * c
    return y


def to_bf16(v):
    """float64 rounded once to bf16 (nearest, ties to even), as float64; normal range."""
    m, e = np.frexp(np.asarray(v, np.float64))
    return np.ldexp(np.rint(m * 256.0), e - 8)


def rms_norm_bf16(x, w, eps):
    """x [n, d], w [d] (bf16 values) -> bf16 values."""
    x = np.asarray(x, np.float64)
    return to_bf16(x * np.asarray(w, np.float64) / np.sqrt(np.mean(x * x, axis=1, keepdims=True) + eps))


def append_row_values(x, w, eps):
    """(latent bf16 values, codes, scales) of projection rows x [n, 576]."""
    lat = np.asarray(x, np.float64)[:, :512]
    if w is not None:
        lat = rms_norm_bf16(lat, w, eps)
    codes, scales = codec.quantize_rows(lat)
    return lat, codes, scales


def dense_attention(q, latent, rope_k, positions, scale, window=0, causal=True):
    """One sequence.  q [n, H, 576], latent [N, 512], rope_k [N, 64], positions [n]
    (each token's own).  Returns out [n, H, 512], lse [n, H] and the two sums that
    bound a kernel's rounding: sum_t p_t |v_t| and max_t |scale| sum_i |q_i k_ti|."""
    key = np.concatenate([latent, rope_k], axis=1)
    N = key.shape[0]
    n, H, _ = q.shape
    out = np.zeros((n, H, 512))
    lse = np.full((n, H), -np.inf)
    spread = np.zeros((n, H, 512))
    mass = np.zeros((n, H))
    t = np.arange(N)
    for i in range(n):
        see = np.ones(N, bool)
        if causal:
            see = t <= positions[i]
            if window > 0:
                see &= t > positions[i] - window
        if not see.any():
            continue
        k, v = key[see], latent[see]
        s = scale * (q[i] @ k.T)
        m = s.max(axis=1, keepdims=True)
        p = np.exp(s - m)
        z = p.sum(axis=1, keepdims=True)
        p = p / z
        out[i] = p @ v
        lse[i] = (m + np.log(z))[:, 0]
        spread[i] = p @ np.abs(v)
        mass[i] = abs(scale) * (np.abs(q[i]) @ np.abs(k).T).max(axis=1)
    return out, lse, spread, mass
