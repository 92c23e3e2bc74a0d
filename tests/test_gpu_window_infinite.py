"""Infinities in the rows that tokens see, wherever the row lies in a tile and whichever form takes the call (GPU).

Among a row's rotary channels alone the formula says what they do: a logit of -inf is weight 0, as of a logit that is
finite and far below the others (the same bits); one of +inf leaves no number.  Among its values: no number in those
channels for any token that sees them.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from tests.test_gpu_window import SCALE, Problem

pytestmark = pytest.mark.gpu

# sequences' tokens and contexts, heads, window, sinks, joined: the forms of the call
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


def build(form):
    q, c, heads, window, sinks, join = FORMS[form]
    return Problem(q, c, heads=heads, window=window, sinks=sinks, seed=heads + window, join=join)


def result(p):
    p.out.fill_(9.0)
    p.lse.fill_(9.0)
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0
    return p.out.clone(), p.lse.clone()


def places(p):
    """Positions of the first sequence: its newest, where windows begin and end, at borders of pages, a sink."""
    n, c = p.q_lens[0], p.ctx[0]
    first = max(0, c - n - p.W + 1)
    t = [c - 1, c - n, c - 1 - n // 2, first, first + 7, (c - 1) // 64 * 64, (c - n // 2) // 64 * 64 - 1, c - p.W, c - p.W // 2] + [0] * (p.S > 0)
    return sorted({x for x in t if 0 <= x < c and p.seen[0][x]})


def sees(p, t):
    pos = np.arange(p.ctx[0] - p.q_lens[0], p.ctx[0])
    mask = torch.zeros(p.total, dtype=torch.bool)
    mask[int(p.starts[0]):int(p.starts[1])] = torch.from_numpy((t <= pos) & ((t > pos - p.W) | (t < p.S)))
    return mask.cuda()


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_rotary_channels(form, sign):
    p = build(form)
    clean = result(p)
    for t in places(p):
        at = int(p.row(0, np.array([t]))[0])
        kept = p.kv[at, 570].clone()
        p.kv[at, 570] = sign * 1e30
        low = result(p)
        p.kv[at, 570] = sign * float("inf")
        out, lse = result(p)
        p.kv[at, 570] = kept
        see = sees(p, t)
        logit = p.q[..., 570].float() * sign
        none, over = see[:, None] & (logit < 0), see[:, None] & (logit > 0)
        assert torch.equal(out[~see], clean[0][~see]) and torch.equal(lse[~see], clean[1][~see]), t
        assert torch.equal(out[none], low[0][none]) and torch.equal(lse[none], low[1][none]), t
        assert bool(torch.isnan(out[over]).all()) and not bool(torch.isfinite(lse[over]).any()), t


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_values_that_are_no_numbers(form, value):
    p = build(form)
    clean = result(p)
    for t in places(p):
        for channel in (17, 500):
            at = int(p.row(0, np.array([t]))[0])
            kept = p.kv[at, channel].clone()
            p.kv[at, channel] = value
            out, lse = result(p)
            p.kv[at, channel] = kept
            see = sees(p, t)
            assert torch.equal(out[~see], clean[0][~see]) and torch.equal(lse[~see], clean[1][~see]), (t, channel)
            assert bool(torch.isnan(out[see][..., channel]).all()), (t, channel)


def test_a_token_left_without_weight():
    """Only positions of weight 0: as a token that sees nothing."""
    p = Problem([1], [1], heads=16, seed=3)
    p.kv[int(p.row(0, np.array([0]))[0]), 570] = -float("inf")
    out, lse = result(p)
    none = p.q[0, :, 570].float() > 0
    assert bool((out[0][none] == 0).all()) and bool(torch.isneginf(lse[0][none]).all())
    assert bool(torch.isnan(out[0][~none]).all())
