"""Pins of the window-side oracle (CPU)."""
import numpy as np

from oracle import prompt as op
from oracle import window as ow


def test_window_attention_is_the_dense_one_with_that_mask():
    r = np.random.default_rng(0)
    kv, q = r.standard_normal((90, 576)), r.standard_normal((4, 3, 576))
    pos = np.array([0, 5, 40, 89])
    for window in (1, 7, 200):
        o, l, s, m = ow.window_attention(q, kv, pos, 0.04, window)
        do, dl, ds, dm = op.dense_attention(q, kv[:, :512], kv[:, 512:], pos, 0.04, window)
        for a, b in ((o, do), (l, dl), (s, ds), (m, dm)):
            np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-14)


def test_sinks_stay_visible_and_are_seen_once():
    r = np.random.default_rng(1)
    kv, q = r.standard_normal((60, 576)), r.standard_normal((1, 2, 576))
    o, l, _, _ = ow.window_attention(q, kv, [50], 0.04, 5, sinks=3)
    see = [0, 1, 2, 46, 47, 48, 49, 50]
    so, sl, _, _ = ow.window_attention(q, kv[see], [7], 0.04, 100)
    np.testing.assert_allclose(o, so, rtol=1e-12)
    np.testing.assert_allclose(l, sl, rtol=1e-12)
    a = ow.window_attention(q, kv, [20], 0.04, 100, sinks=40)       # sinks behind the token are not seen
    b = ow.window_attention(q, kv, [20], 0.04, 100)
    np.testing.assert_array_equal(a[0], b[0])
    o, l, _, _ = ow.window_attention(q, kv, [-1], 0.04, 5, sinks=3)
    assert np.all(o == 0) and np.all(np.isneginf(l))


def test_joining_parts_is_one_softmax():
    r = np.random.default_rng(2)
    kv, q = r.standard_normal((80, 576)), r.standard_normal((1, 4, 576))
    whole = ow.window_attention(q, kv, [79], 0.04, 1000)
    a = ow.window_attention(q, kv[:50], [49], 0.04, 1000)
    b = ow.window_attention(q, kv[50:], [29], 0.04, 1000)
    o, l, wa, wb = ow.join(a[0], a[1], b[0], b[1])
    np.testing.assert_allclose(o, whole[0], rtol=1e-11, atol=1e-14)
    np.testing.assert_allclose(l, whole[1], rtol=1e-13)
    np.testing.assert_allclose(wa + wb, 1.0)
    none = np.full_like(a[1], -np.inf)
    o, l, _, _ = ow.join(0 * a[0], none, b[0], b[1])
    np.testing.assert_allclose(o, b[0])
    assert np.all(np.isneginf(ow.join(0 * a[0], none, 0 * b[0], none)[1]))


def test_key_norms():
    r = np.random.default_rng(3)
    x = 5 + r.standard_normal((6, 128))
    y, size = ow.key_rows(x, "layer", np.ones(128), np.zeros(128), 1e-12)
    np.testing.assert_allclose(y.mean(1), 0, atol=1e-12)
    np.testing.assert_allclose(y.std(1), 1, rtol=1e-9)
    y, _ = ow.key_rows(x, "rms", np.full(128, 2.0), eps=0.0)
    np.testing.assert_allclose(np.sqrt((y * y).mean(1)), 2.0)
    f = op.rope_frequencies(32, 10000.0)
    z, _ = ow.key_rows(x, "none", pos=np.arange(6), freqs=f, offset=8)
    np.testing.assert_array_equal(z[:, :8], x[:, :8])
    np.testing.assert_array_equal(z[:, 40:], x[:, 40:])
    np.testing.assert_array_equal(z[0], x[0])
    np.testing.assert_allclose(np.linalg.norm(z, axis=1), np.linalg.norm(x, axis=1))
