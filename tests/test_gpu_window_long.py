"""Window attention of many tokens over long windows (tiles of 256 rows on four SMs) against the float64 oracle:
the tolerances and problems of the window attention's tests, in the sizes that take this kernel."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from tests.test_gpu_window import SCALE, Problem

pytestmark = pytest.mark.gpu


def kernels(fn):
    csa2.profile_enable(True)
    try:
        fn()
        torch.cuda.synchronize()
        return set(csa2.profile_read())
    finally:
        csa2.profile_enable(False)


def test_this_kernel_runs():
    p = Problem([200], [700], window=300, seed=1)
    assert kernels(p.run) == {"window_attn_long"}
    p.check()


@pytest.mark.parametrize("heads,q_lens,ctx", [(64, [260], [1000]), (64, [200, 1, 0, 77], [200, 700, 64, 1500]),
                                              (7, [1500, 900], [1600, 900]), (40, [300, 5, 3], [300, 4, 900]),
                                              (16, [640, 63], [2000, 63]), (1, [10000], [12000])])
@pytest.mark.parametrize("window,sinks", [(200, 0), (640, 5), (1000, 130)])
def test_ragged_chunks(heads, q_lens, ctx, window, sinks):
    """Tiles that cross tokens, sequences without queries, one with more queries than context."""
    p = Problem(q_lens, ctx, heads=heads, window=window, sinks=sinks, seed=heads + window, gap=(2, 3), join=heads % 8 == 0)
    assert kernels(p.run) == {"window_attn_long"}
    p.check(some=12)


@pytest.mark.parametrize("window", [129, 191, 192, 193, 256, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 64, 300])
def test_window_and_sinks(window, sinks):
    Problem([170, 130], [900, 130], heads=64, window=window, sinks=sinks, seed=window + sinks).run().check(some=12)


@pytest.mark.parametrize("paged,ring", [(True, 0), (False, 0), (True, 9)])
@pytest.mark.parametrize("join", [True, False])
def test_caches(paged, ring, join):
    Problem([300, 100], [2000, 800], heads=64, window=200, paged=paged, ring=ring, seed=4, join=join).run().check()


@pytest.mark.parametrize("scale", [0.0, -SCALE, 1.0, 1e-6])
def test_scales(scale):
    Problem([160], [700], heads=64, window=250, seed=6).run(scale=scale).check(scale=scale)


def test_steep_rows():
    """Scores that pass the reference by much from block to block."""
    Problem([160], [900], heads=64, window=400, sinks=4, seed=7, q_size=30.0).run().check()


def test_many_tiles():
    p = Problem([900, 1400], [5000, 1400], heads=64, window=320, sinks=4, seed=8, join=True)
    p.run().check()
    first = (p.out.clone(), p.lse.clone())
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0], p.out) and torch.equal(first[1], p.lse)


def test_joined_in_place():
    a = Problem([200, 30], [900, 20], heads=64, window=300, sinks=3, seed=9, join=True)
    a.run()
    out, lse = a.prev.clone(), a.prev_lse.clone()
    csa2.csa2_window_attn_chunk(a.dims, a.B, a.q, a.d_start, a.kv, a.d_table, a.d_ctx, SCALE, a.W, out, lse, a.ws, sinks=a.S,
                                prev_out=out, prev_lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), a.out.view(torch.int16)) and torch.equal(lse, a.lse)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("channel", [3, 300, 511, 570])
def test_a_row_that_is_no_number(value, channel):
    """It reaches the tokens that see it, and no others."""
    p = Problem([170], [800], heads=64, window=250, sinks=2, seed=10)
    clean = Problem([170], [800], heads=64, window=250, sinks=2, seed=10).run()
    t = 700
    p.kv[int(p.row(0, np.array([t]))[0]), channel] = value
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0
    pos = np.arange(800 - 170, 800)
    sees = torch.from_numpy((t <= pos) & (t > pos - 250)).cuda()
    # Of a row with an infinity a score of -inf has weight 0: 0 * inf in the outputs is NaN where the infinity is
    # one of its values (channels below 512), and 0 where it is not: such rows may be numbers.
    got = torch.isnan(p.out[sees]).any(-1)
    if channel >= 512 and np.isinf(value):
        got |= p.q[sees][..., channel].float() * value * SCALE < 0
    assert bool(got.all())
    assert torch.equal(p.out[~sees], clean.out[~sees]) and torch.equal(p.lse[~sees], clean.lse[~sees])


def test_a_query_that_is_no_number():
    p = Problem([170], [800], heads=64, window=250, seed=11)
    clean = Problem([170], [800], heads=64, window=250, seed=11).run()
    p.q[50, 7, 100] = float("nan")
    p.run()
    torch.cuda.synchronize()
    bad = torch.zeros(170, 64, dtype=torch.bool, device="cuda")
    bad[50, 7] = True
    assert bool(torch.isnan(p.out[bad]).all()) and bool(torch.isnan(p.lse[bad]).all())
    assert torch.equal(p.out[~bad], clean.out[~bad]) and torch.equal(p.lse[~bad], clean.lse[~bad])


def test_bad_page_is_skipped_and_reported():
    p = Problem([170], [800], heads=64, window=250, seed=12)
    p.d_table[0, 9] = p.pages + 7
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0x02
    k, see = p.key[0], np.ones(800, bool)
    see[9 * 64:10 * 64] = False
    for i in (0, 60, 169):
        pos = 800 - 170 + i
        t = np.arange(800)
        s = see & (t <= pos) & (t > pos - 250)
        z = SCALE * (p.q64[i] @ k[s].T)
        w = np.exp(z - z.max(1, keepdims=True))
        o = (w / w.sum(1, keepdims=True)) @ k[s][:, :512]
        spread = (w / w.sum(1, keepdims=True)) @ np.abs(k[s][:, :512])
        mass = SCALE * (np.abs(p.q64[i]) @ np.abs(k[s]).T).max(1)
        wide = (2.0 ** -8 + 2 * 576 * 2.0 ** -22 * mass[:, None] + 25 * 2.0 ** -22) * spread
        assert np.all(np.abs(p.out[i].double().cpu().numpy() - o) <= 2.0 ** -8 * np.abs(o) + wide)


@pytest.mark.parametrize("starts", [[5, 3], [0, 171], [-1, 170]])
def test_starts_out_of_order_write_nothing(starts):
    p = Problem([170], [800], heads=64, window=250, seed=13)
    p.d_start.copy_(torch.tensor(starts, dtype=torch.int32))
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0x40
    assert bool((p.out == 9.0).all()) and bool((p.lse == 9.0).all())


def test_captured_with_other_lengths():
    """One graph, replayed with other starts in place; rows behind the last sequence stay as they were."""
    p = Problem([100, 100], [700, 600], heads=64, window=250, sinks=2, seed=14)
    p.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for lens in ([100, 100], [40, 60], [0, 100], [1, 1], [0, 0]):
        p.q_lens = lens
        p.starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
        p.d_start.copy_(torch.from_numpy(p.starts))
        p.out.fill_(9.0)
        p.lse.fill_(9.0)
        g.replay()
        p.check()


def test_two_streams():
    a, b = (Problem([170, 3], [900, 100], heads=64, window=300, seed=s, join=True) for s in (15, 16))
    torch.cuda.synchronize()
    for p in (a, b):
        p.run(stream=torch.cuda.Stream())
    a.check()
    b.check()
