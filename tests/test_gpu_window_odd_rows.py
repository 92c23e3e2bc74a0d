"""Window attention over caches without pages whose sequences do not begin at a multiple of 64 rows (GPU): boxes of rows reach
into the next sequence and, at the last one, past the cache."""
import dataclasses

import numpy as np
import pytest
import torch

from tests.test_gpu_window import Problem

pytestmark = pytest.mark.gpu


def relaid(p, cap):
    """The same problem with `cap` rows a sequence, next to each other; rows that no token sees hold NaN."""
    kv = torch.full((p.B * cap, 576), float("nan"), dtype=torch.bfloat16, device="cuda")
    for b, c in enumerate(p.ctx):
        kv[b * cap:b * cap + c] = p.kv[b * p.cap:b * p.cap + c]
    p.kv, p.cap, p.dims = kv, cap, dataclasses.replace(p.dims, max_ctx=cap)
    return p


@pytest.mark.parametrize("q,ctx,cap", [([1], [1], 1), ([1, 1, 1], [37, 5, 36], 37), ([3, 0, 7], [100, 64, 99], 100), ([40, 60], [1000, 777], 1001)])
@pytest.mark.parametrize("heads,window,sinks", [(64, 128, 0), (16, 50, 3), (7, 300, 5), (16, 1000, 70)])
@pytest.mark.parametrize("join", [False, True])
def test_rows_side_by_side(q, ctx, cap, heads, window, sinks, join):
    relaid(Problem(q, ctx, heads=heads, window=window, sinks=sinks, paged=False, seed=cap + heads, join=join), cap).run().check()


@pytest.mark.parametrize("cap", [801, 830])
def test_many_rows(cap):
    relaid(Problem([170, 200], [800, 801], heads=64, window=250, sinks=70, paged=False, seed=cap, join=True), cap).run().check(some=12)
