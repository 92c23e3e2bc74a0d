"""Oracle of the window-side calls, in float64: attention over a sliding window of exact
rows with first positions that stay visible, its join with another attention, and the
indexer keys' append.

Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

from oracle import codec, prompt


def window_attention(q, kv, positions, scale, window, sinks=0):
    """One sequence.  q [n, H, 576], kv [N, 576] (row t: position t), positions [n].
    Returns out [n, H, 512], lse [n, H] and the two sums that bound a kernel's rounding:
    sum_t p_t |v_t| and max_t |scale| sum_i |q_i k_ti|."""
    n, H, _ = q.shape
    out = np.zeros((n, H, 512))
    lse = np.full((n, H), -np.inf)
    spread = np.zeros((n, H, 512))
    mass = np.zeros((n, H))
    t = np.arange(kv.shape[0])
    for i, p in enumerate(positions):
        see = (t <= p) & ((t > p - window) | (t < sinks))
        if not see.any():
            continue
        k = kv[see]
        s = scale * (q[i] @ k.T)
        m = s.max(axis=1, keepdims=True)
        e = np.exp(s - m)
        z = e.sum(axis=1, keepdims=True)
        w = e / z
        out[i] = w @ k[:, :512]
        lse[i] = (m + np.log(z))[:, 0]
        spread[i] = w @ np.abs(k[:, :512])
        mass[i] = abs(scale) * (np.abs(q[i]) @ np.abs(k).T).max(axis=1)
    return out, lse, spread, mass


def join(out_a, lse_a, out_b, lse_b):
    """Two softmaxes over different rows as one: (out, lse, weight of a, weight of b)."""
    lse = np.logaddexp(lse_a, lse_b)
    safe = np.where(np.isneginf(lse), 0.0, lse)
    wa, wb = np.exp(lse_a - safe), np.exp(lse_b - safe)
    return wa[..., None] * out_a + wb[..., None] * out_b, lse, wa, wb


def key_rows(x, norm, w=None, b=None, eps=1e-6, pos=None, freqs=None, half=False, mscale=1.0, offset=0):
    """Normed and rotated keys of x [n, d]; also a bound of their size per channel: what a rounding
    of 2^-24 at each step can be relative to."""
    x = np.asarray(x, np.float64)
    size, top = np.abs(x), np.abs(x).max(axis=1, keepdims=True)
    if norm == "layer":
        x = x - x.mean(axis=1, keepdims=True)
    if norm != "none":
        r = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + eps)
        if norm == "layer":                    # a rounding of the row's size in the mean, and so in the root
            size = top + np.abs(x) * (1 + top * r)
        x, size = x * r * w, size * r * np.abs(w)
    if b is not None:
        x, size = x + b, size + np.abs(b)
    if freqs is not None:
        k = 2 * len(freqs)
        x = x.copy()
        x[:, offset:offset + k] = prompt.rope(x[:, None, offset:offset + k], pos, freqs, half, mscale)[:, 0]
        part = size[:, offset:offset + k]
        n = len(freqs)
        pair = (part[:, :n] + part[:, n:]) if half else (part[:, 0::2] + part[:, 1::2])
        size[:, offset:offset + k] = mscale * (np.concatenate([pair, pair], 1) if half else np.repeat(pair, 2, 1))
    return x, size
