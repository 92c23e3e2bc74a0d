"""Window attention with one position whose logit is far above or below the others (GPU), in every form of the call.

Below them it has no weight, above them all of it, whatever its size.  Tolerances as in the window attention's tests, with
the scores' error ds of the positions that can have weight only (logits within 40 of the largest: e^-40 of it is nothing
beside 2^-8).  Of a position with all the weight the output is its values to bf16, and its score off by less than
(576 + 4) 2^-22 of its terms' size, here next to |lse| itself: one term outweighs the others.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import prompt as op
from oracle import window as ow
from tests.test_gpu_window import SCALE, Problem

pytestmark = pytest.mark.gpu

# sequences' tokens and contexts, heads, window, sinks, joined
FORMS = {
    "one block": ([100], [400], 16, 50, 2, False),
    "one block, 64 heads": ([12], [300], 64, 100, 0, True),
    "one block, odd heads": ([90], [300], 7, 70, 3, False),
    "short context": ([3, 5], [40, 9], 24, 128, 0, True),
    "pages": ([70, 3], [900, 300], 16, 200, 5, False),
    "pages, joined": ([33], [500], 7, 300, 1, True),
    "split": ([3], [1500], 16, 1000, 5, False),
    "split, joined": ([2], [1500], 64, 1400, 0, True),
    "many rows": ([170], [800], 64, 250, 2, False),
    "many rows, joined": ([1500], [1600], 7, 400, 70, True),
}


def places(p):
    """Positions of the first sequence: its newest, where windows begin and end, at borders of pages, a sink."""
    n, c = p.q_lens[0], p.ctx[0]
    first = max(0, c - n - p.W + 1)
    t = [c - 1, c - n, c - 1 - n // 2, first, first + 7, (c - 1) // 64 * 64, (c - n // 2) // 64 * 64 - 1, c - p.W, c - p.W // 2] + [0] * (p.S > 0)
    return sorted({x for x in t if 0 <= x < c and p.seen[0][x]})


def check(p, tokens):
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0
    n, c = p.q_lens[0], p.ctx[0]
    t = np.arange(c)
    for i in tokens:
        at, pos = p.starts[0] + i, c - n + i
        see = (t <= pos) & ((t > pos - p.W) | (t < p.S))
        k = p.key[0][see]
        z = SCALE * (p.q64[at] @ k.T)
        ro, rl, spread, _ = (v[0] for v in ow.window_attention(p.q64[at:at + 1], p.key[0], [pos], SCALE, p.W, p.S))
        near = z > z.max(1, keepdims=True) - 40
        alone = near.sum(1) == 1
        mass = SCALE * np.where(near, np.abs(p.q64[at]) @ np.abs(k).T, 0).max(1)
        ds = 576 * 2.0 ** -22 * mass
        acc = (-(-min(c, p.W + p.S + 64) // 128) + 20) * 2.0 ** -22
        wide = (2.0 ** -8 + 2 * np.where(alone, 0, ds)[:, None] + acc) * spread
        tol_l = ds + acc + 2.0 ** -22 * (4 + np.abs(rl))
        if p.prev is not None:
            po, pl = p.prev64[at], p.prev_lse[at].double().cpu().numpy()
            jo, jl, wa, wb = ow.join(ro, rl, po, pl)
            # the weights' error, that of lse, is nothing where one of the two has none left beside the other
            off = (2 * np.where(np.abs(rl - pl) > 60 + 2 * tol_l, 0, tol_l) + 2.0 ** -20)[:, None] * (wa[:, None] * np.abs(ro) + wb[:, None] * np.abs(po))
            wide, ro, rl = wa[:, None] * wide + off, jo, jl
        err = np.abs(p.out[at].double().cpu().numpy() - ro)
        assert np.all(err <= 2.0 ** -8 * np.abs(ro) + wide), (i, float(np.nanmax(err)))
        assert np.all(np.abs(p.lse[at].double().cpu().numpy() - rl) <= tol_l), i


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("size", [3e3, 1e9, 1e13, 1e30])
def test_one_far_logit(form, size):
    q, c, heads, window, sinks, join = FORMS[form]
    p = Problem(q, c, heads=heads, window=window, sinks=sinks, seed=heads + window, join=join)
    n = q[0]
    for t in places(p):
        at = int(p.row(0, np.array([t]))[0])
        kept = p.kv[at, 570].clone(), p.key[0][t, 570]
        p.kv[at, 570] = size
        p.key[0][t, 570] = op.to_bf16(np.array([size]))[0]
        p.run()
        first = max(0, t - (c[0] - n))                       # its first token, those beside it, the last that sees it
        check(p, sorted({i for i in (first - 1, first, first + 1, first + window - 1, first + window, n // 2, n - 1) if 0 <= i < n}))
        p.kv[at, 570], p.key[0][t, 570] = kept
