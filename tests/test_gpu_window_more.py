"""Window attention where its forms meet: single positions, whole pages in one block, joins over many tiles,
blocks that are not full after calls that left something else in shared memory.  Problems and tolerances are those
of the window attention's tests."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from tests.test_gpu_window import SCALE, Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,n,window", [(64, 1, 128), (16, 7, 60), (64, 300, 128), (64, 300, 500), (7, 40, 200)])
def test_one_position_is_its_row(heads, n, window):
    """The first token of a prompt sees itself alone: its outputs are its row's values, bit for bit (its weight is 1
    to 2^-22 before it is rounded to bf16, and so is the sum), its lse the score."""
    p = Problem([n], [n], heads=heads, window=window, seed=n).run()
    torch.cuda.synchronize()
    row = p.kv[int(p.row(0, np.array([0]))[0]), :512]
    assert torch.equal(p.out[0], row.expand(heads, 512))
    score = SCALE * (p.q64[0] @ p.key[0][0])
    size = SCALE * (np.abs(p.q64[0]) @ np.abs(p.key[0][0]))
    assert np.all(np.abs(p.lse[0].double().cpu().numpy() - score) <= 576 * 2.0 ** -22 * size + 2.0 ** -20 * (1 + np.abs(score)))
    p.check()


@pytest.mark.parametrize("heads,lens,ctx", [(64, [1] * 9, [1, 2, 63, 64, 65, 66, 700, 129, 191]), (16, [4, 1, 70], [4, 300, 1000]),
                                            (64, [500, 220], [500, 900])])
@pytest.mark.parametrize("window", [1, 2, 33, 61, 62, 63, 64, 65, 66])
def test_windows_of_a_page(heads, lens, ctx, window):
    """At most a page and one position a tile: one block of whole pages, and just above it places of positions."""
    Problem(lens, ctx, heads=heads, window=window, seed=window, join=window % 2 == 0).run().check(some=12)


@pytest.mark.parametrize("heads,lens,ctx,window,sinks", [(64, [300, 1, 90], [300, 700, 2000], 128, 0), (16, [900, 700], [900, 4000], 113, 0),
                                                         (16, [900, 700], [900, 4000], 113, 9), (7, [2000], [2100], 64, 0),
                                                         (64, [200, 3], [900, 100], 150, 5), (40, [400], [1000], 127, 1)])
def test_joins_over_many_tiles(heads, lens, ctx, window, sinks):
    """In place and apart: the same bits."""
    p = Problem(lens, ctx, heads=heads, window=window, sinks=sinks, seed=heads, gap=(1, 2), join=True).run()
    p.check(some=16)
    out, lse = p.prev.clone(), p.prev_lse.clone()
    csa2.csa2_window_attn_chunk(p.dims, p.B, p.q, p.d_start, p.kv, p.d_table, p.d_ctx, SCALE, window, out, lse, p.ws, sinks=sinks,
                                prev_out=out, prev_lse=lse)
    torch.cuda.synchronize()
    inside = slice(int(p.starts[0]), int(p.starts[-1]))
    assert torch.equal(out[inside].view(torch.int16), p.out[inside].view(torch.int16)) and torch.equal(lse[inside], p.lse[inside])
    # rows before and behind the sequences as they were
    for t in (0, p.total - 2, p.total - 1):
        assert torch.equal(out[t], p.prev[t]) and torch.equal(lse[t], p.prev_lse[t])


@pytest.mark.parametrize("ctx,window,sinks", [([5, 1, 70], 128, 0), ([5, 1, 70], 60, 0), ([300, 400, 333], 150, 0), ([200, 130, 500], 100, 20)])
def test_after_rows_that_are_no_numbers(ctx, window, sinks):
    """Blocks with places that no row is copied to, after calls over rows of NaN on every SM: nothing of those stays."""
    bad = Problem([400], [900], heads=64, window=300, seed=1)
    bad.kv.fill_(float("nan"))
    p = Problem([1] * len(ctx), ctx, heads=64, window=window, sinks=sinks, seed=2)
    wide = Problem([800], [800], heads=64, window=128, seed=3)
    wide.kv.fill_(float("nan"))
    for _ in range(3):
        bad.run()
        wide.run()
        p.out.fill_(9.0)
        p.run().check()


def test_other_attention_of_rows_that_see_nothing():
    """Tokens without a position keep the other attention's results; those that neither has seen are 0 and -inf."""
    p = Problem([6, 200], [2, 200], heads=64, window=128, seed=5, join=True)
    p.prev_lse[1].fill_(-float("inf"))
    p.prev[1].fill_(float("nan"))
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.out[2:4], p.prev[2:4]) and torch.equal(p.lse[2:4], p.prev_lse[2:4])
    assert bool((p.out[1] == 0).all()) and bool(torch.isneginf(p.lse[1]).all())
