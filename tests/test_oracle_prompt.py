"""Pins of the prompt-side oracle (CPU): rotary positions, norm, dense attention;
positions and cache rows of a chunk."""
import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import prompt as op


def test_rotation_keeps_lengths_and_adds_angles():
    r = np.random.default_rng(0)
    f = op.rope_frequencies(64, 10000.0)
    x = r.standard_normal((5, 2, 64))
    for half in (False, True):
        a = op.rope(x, np.array([3, 9, 1000, 0, 7]), f, half)
        np.testing.assert_allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
        b = op.rope(op.rope(x, np.full(5, 11), f, half), np.full(5, 31), f, half)
        np.testing.assert_allclose(b, op.rope(x, np.full(5, 42), f, half), rtol=1e-11, atol=1e-12)
        back = op.rope(a, np.array([3, 9, 1000, 0, 7]), f, half, inverse=True)
        np.testing.assert_allclose(back, x, rtol=1e-12, atol=1e-13)


def test_scores_depend_on_the_distance_alone():
    r = np.random.default_rng(1)
    f = op.rope_frequencies(64, 10000.0, "parts", 16.0, 4096.0)
    q, k = r.standard_normal((2, 1, 1, 64))
    at = lambda p, s: (op.rope(q, [p], f, True) * op.rope(k, [p - s], f, True)).sum()
    assert abs(at(100, 37) - at(90000, 37)) < 1e-9


def test_scaled_frequencies():
    f = op.rope_frequencies(64, 10000.0)
    np.testing.assert_allclose(op.rope_frequencies(64, 10000.0, "linear", 8.0), f / 8)
    p = op.rope_frequencies(64, 10000.0, "parts", 16.0, 4096.0, 1.0, 32.0)
    turns = 4096.0 * f / (2 * np.pi)
    np.testing.assert_allclose(p[turns >= 32], f[turns >= 32])
    np.testing.assert_allclose(p[turns <= 1], f[turns <= 1] / 16)
    assert np.all((p <= f) & (p >= f / 16))
    b = op.rope_frequencies(64, 10000.0, "base", 4.0)
    assert b[0] == 1.0 and abs(b[-1] - f[-1] / 4) < 1e-15      # the slowest pair is stretched by the factor


def test_bf16_rounding_is_torchs():
    v = np.concatenate([np.random.default_rng(2).standard_normal(5000) * 10.0 ** np.arange(-10, 10).repeat(250), [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8]])
    v32 = v.astype(np.float32)
    np.testing.assert_array_equal(op.to_bf16(v32.astype(np.float64)), torch.from_numpy(v32).to(torch.bfloat16).double().numpy())


def test_dense_attention_is_the_sparse_one_with_every_position():
    r = np.random.default_rng(3)
    lat, rk = r.standard_normal((40, 512)), r.standard_normal((40, 64))
    q = r.standard_normal((1, 3, 576))
    o, l, _, _ = op.dense_attention(q, lat, rk, np.array([39]), 0.04)
    so, sl = oatt.sparse_attn_decode(q[0], lat, rk, np.arange(40), np.zeros((0, 576)), 0, 0.04)
    np.testing.assert_allclose(o[0], so, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(l[0], sl, rtol=1e-13)
    o, l, _, _ = op.dense_attention(q, lat, rk, np.array([-1]), 0.04)
    assert np.all(o == 0) and np.all(np.isneginf(l))
    o, l, _, _ = op.dense_attention(q, lat, rk, np.array([30]), 0.04, window=1)
    np.testing.assert_allclose(o[0], np.broadcast_to(lat[30], (3, 512)), rtol=1e-14)


def test_positions_and_rows_of_a_chunk():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300.prefill import cache_rows
    start = torch.tensor([0, 3, 3, 5], dtype=torch.int32)
    ctx = torch.tensor([70, 10, 1], dtype=torch.int32)
    table = torch.tensor([[4, 2], [0, 0], [7, 1]], dtype=torch.int32)
    pos, rows = cache_rows(ctx, start, table)
    assert pos.tolist() == [67, 68, 69, -1, 0]
    assert rows.tolist() == [2 * 64 + 3, 2 * 64 + 4, 2 * 64 + 5, -1, 7 * 64]
    pos, rows = cache_rows(ctx, start, max_ctx=100)
    assert rows.tolist() == [67, 68, 69, -1, 200]
