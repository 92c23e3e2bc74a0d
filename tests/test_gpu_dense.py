"""GPU dense chunk attention over the FP4 cache against the float64 oracle.

Tolerances, per output element, derived from the kernel's roundings:
  scores: products of bf16 values, 576 terms summed in fp32 by the tensor core
    (taken as 2^-22 of the terms' size each, with truncation):  ds = 576 * 2^-22 M_r,
    M_r = max_t |scale| sum |q_i k_ti|;
  P: fp16, half a step 2^-11, and exp2 2^-22, with terms 2^-31 below the
    reference lost: at most N 2^-31 of the largest value;
  sum and accumulation in fp32: (blocks + 20) 2^-22;  output: bf16, 2^-8.
out: 2^-8 |o| + (2^-11 + 2 ds + (blocks + 20) 2^-22) sum_t p_t |v_t| + N 2^-31 max|v|
lse: ds + (blocks + 20) 2^-22 + 2^-22 |lse|
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import codec as ocodec
from oracle import prompt as op
from tests.helpers import bf16_f64

pytestmark = pytest.mark.gpu

SCALE = 1 / 24.0


class Problem:
    """A ragged batch over a paged or contiguous cache whose unused places hold NaN scales and rope keys."""

    def __init__(self, q_lens, ctx, heads=64, paged=True, seed=0, gap=(0, 0), q_size=1.0):
        r = np.random.default_rng(seed)
        self.q_lens, self.ctx, self.H = list(q_lens), list(ctx), heads
        B = len(ctx)
        cap = max(64, -(-max(ctx) // 64) * 64)
        if paged:
            need = [-(-c // 64) for c in ctx]
            pages = sum(need) + 5
            order = r.permutation(pages)
            self.table = np.full((B, max(1, max(need))), 0, np.int32)
            at = 0
            for b, k in enumerate(need):
                self.table[b, :k] = order[at:at + k]
                at += k
            rows = pages * 64
        else:
            self.table, pages, rows = None, 0, B * cap
        self.rows = rows
        self.row = [self._rows_of(b, c, cap) for b, c in enumerate(ctx)]
        lat = r.standard_normal((rows, 512)) * np.exp(0.5 * r.standard_normal(512))
        codes, scales = ocodec.quantize_rows(op.to_bf16(lat))
        self.latent = ocodec.dequantize_rows(codes, scales)
        self.rope = op.to_bf16(r.standard_normal((rows, 64)))
        used = np.zeros(rows, bool)
        for x in self.row:
            used[x] = True
        dc, ds, dr = codes.copy(), scales.copy(), self.rope.copy()
        dc[~used], ds[~used], dr[~used] = 0x77, 0x7F, np.nan
        self.codes = torch.from_numpy(dc).cuda()
        self.scales = torch.from_numpy(ds).cuda()
        self.kr = torch.from_numpy(dr).to(torch.bfloat16).cuda()
        self.starts = np.concatenate([[gap[0]], gap[0] + np.cumsum(q_lens)]).astype(np.int32)
        self.total = int(self.starts[-1]) + gap[1]
        self.q64 = op.to_bf16(r.standard_normal((self.total, heads, 576)) * q_size)
        self.q = torch.from_numpy(self.q64).to(torch.bfloat16).cuda()
        self.dims = csa2.Dims(heads=heads, max_ctx=cap, num_pages=pages if paged else 0,
                              max_pages=self.table.shape[1] if paged else 0)
        self.B = B
        self.out = torch.full((self.total, heads, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.total, heads), 9.0, dtype=torch.float32, device="cuda")
        self.ws = csa2.alloc_dense_attn_workspace(self.dims, B, self.total)
        self.d_table = torch.from_numpy(self.table).cuda() if paged else None
        self.d_ctx = torch.tensor(ctx, dtype=torch.int32).cuda()
        self.d_start = torch.from_numpy(self.starts).cuda()

    def _rows_of(self, b, c, cap):
        t = np.arange(c)
        return b * cap + t if self.table is None else self.table[b, t // 64].astype(np.int64) * 64 + t % 64

    def run(self, window=0, causal=True, scale=SCALE, stream=None):
        csa2.csa2_dense_attn_chunk(self.dims, self.B, self.q, self.d_start, self.codes, self.scales, self.kr, self.d_table,
                                   self.d_ctx, scale, self.out, self.lse, self.ws, window=window,
                                   flags=0 if causal else csa2.DENSE_ALL_POSITIONS, stream=stream)
        return self

    def check(self, window=0, causal=True, scale=SCALE, some=24):
        """`some` tokens of each sequence (first, last and spread ones) against the oracle."""
        torch.cuda.synchronize()
        assert csa2.get_device_status(self.ws) == 0
        o = self.out.double().cpu().numpy()
        l = self.lse.double().cpu().numpy()
        for b in range(self.B):
            n, N = self.q_lens[b], self.ctx[b]
            if n == 0:
                continue
            tok = np.unique(np.linspace(0, n - 1, min(n, some)).astype(int))
            at = self.starts[b] + tok
            lat, rk = self.latent[self.row[b]], self.rope[self.row[b]]
            ro, rl, spread, mass = op.dense_attention(self.q64[at], lat, rk, N - n + tok, scale, window, causal)
            ds = 576 * 2.0 ** -22 * mass
            acc = (-(-N // 64) + 20) * 2.0 ** -22
            big = np.abs(lat).max() if N else 0.0
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * ds[..., None] + acc) * spread + N * 2.0 ** -31 * big
            err = np.abs(o[at] - ro)
            assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-30)).max()))
            none = np.isneginf(rl)
            assert np.array_equal(np.isneginf(l[at]), none)
            e = np.abs(l[at][~none] - rl[~none])
            assert np.all(e <= ds[~none] + acc + 2.0 ** -22 * np.abs(rl[~none])), (b, float(e.max()))
        for t in list(range(0, self.starts[0])) + list(range(self.starts[-1], self.total)):
            assert np.all(o[t] == 9.0) and np.all(l[t] == 9.0)


@pytest.mark.parametrize("ctx", [1, 2, 63, 64, 65, 127, 128, 129, 200, 1000, 4097])
@pytest.mark.parametrize("heads", [1, 16, 64])
def test_one_token(ctx, heads):
    Problem([1], [ctx], heads=heads, seed=ctx).run().check()


@pytest.mark.parametrize("paged", [True, False])
def test_decode_batch(paged):
    c = [1, 300, 64, 2049, 777, 8000, 65, 128]
    Problem([1] * 8, c, paged=paged, seed=3).run().check()


@pytest.mark.parametrize("heads", [3, 7, 24, 40, 64])
def test_ragged_chunks(heads):
    """Tiles that cross tokens, sequences without queries, one with more queries than context."""
    Problem([5, 0, 130, 1, 33, 9], [700, 64, 130, 1, 1500, 4], heads=heads, seed=heads, gap=(2, 3)).run().check()


def test_whole_prompts():
    Problem([257, 64, 511], [257, 64, 511], seed=8).run().check()


@pytest.mark.parametrize("window", [1, 2, 64, 65, 200, 5000])
def test_window(window):
    Problem([70, 3, 1], [900, 130, 2500], heads=16, seed=window).run(window=window).check(window=window)


def test_all_positions():
    Problem([70, 200, 1], [900, 33, 2500], heads=16, seed=5).run(causal=False).check(causal=False)


@pytest.mark.parametrize("scale", [0.0, -SCALE, 1.0, 1e-6])
def test_scales(scale):
    Problem([9], [500], heads=16, seed=6).run(scale=scale).check(scale=scale)


def test_steep_rows():
    """Logits in the hundreds: the running reference rises often, most weights vanish."""
    Problem([40, 1], [3000, 9000], heads=64, seed=11, q_size=12.0).run().check()


def test_rising_logits_rescale_every_block():
    """Keys grow along the context, so every block passes the reference by more than the slack."""
    p = Problem([4], [64 * 12], heads=16, paged=False, seed=13)
    v = np.repeat(np.arange(12), 64)[:, None] * np.ones((1, 64))
    p.rope[:64 * 12] = op.to_bf16(v)
    p.kr[:64 * 12] = torch.from_numpy(p.rope[:64 * 12]).to(torch.bfloat16).cuda()
    p.q64[:, :, 512:] = 4.0
    p.q[:, :, 512:] = 4.0
    p.run().check()
    p.q64[:, :, 512:] = -4.0                               # falling: the first block holds everything
    p.q[:, :, 512:] = -4.0
    p.run().check()


def test_same_results_every_time_and_with_a_used_workspace():
    p = Problem([1, 20, 200], [9000, 3000, 400], seed=14)
    a = p.run().out.clone()
    la = p.lse.clone()
    small = Problem([3], [70], heads=16, seed=15)
    small.ws = p.ws                                       # another shape through the same workspace
    small.run().check()
    p.out.fill_(1)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.out, a) and torch.equal(p.lse, la)
    p.check()


def test_long_context_splits_over_every_pair():
    Problem([1, 2], [40000, 70000], heads=64, seed=16).run().check()


def test_graph_replay_with_new_lengths():
    """Lengths are read on the device: a captured call follows them."""
    p = Problem([1, 1, 1], [500, 64, 1000], heads=16, seed=17)
    full = p.row
    p.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p.run()
    for c in ([500, 64, 1000], [1, 64, 999], [450, 3, 64]):
        p.ctx = list(c)
        p.row = [r[:n] for r, n in zip(full, c)]
        p.d_ctx.copy_(torch.tensor(c, dtype=torch.int32))
        p.out.fill_(9)
        g.replay()
        p.check()


def test_two_calls_at_once():
    ps = [Problem([1, 5], [3000, 700], seed=s) for s in (18, 19)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(ps, streams):
            p.run(stream=s)
    for p in ps:
        p.check()


def test_bad_page_is_skipped_and_reported():
    p = Problem([2], [300], heads=16, seed=20)
    p.table[0, 1] = -5
    p.d_table[0, 1] = -5
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0x02
    keep = np.r_[0:64, 128:300]
    for i in range(2):
        see = keep[keep <= 298 + i]
        ro, rl, _, _ = op.dense_attention(p.q64[i:i + 1], p.latent[p.row[0][see]], p.rope[p.row[0][see]], np.array([10 ** 6]), SCALE)
        assert np.abs(p.out[i].double().cpu().numpy() - ro[0]).max() <= 2.0 ** -7 * np.abs(ro).max()
        assert np.abs(p.lse[i].double().cpu().numpy() - rl[0]).max() <= 1e-4
    csa2.clear_device_status(p.ws)


def test_bad_lengths_are_reported():
    p = Problem([2, 1], [300, 100], heads=16, seed=21)
    p.d_ctx[1] = p.dims.max_ctx + 1
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0x01
    assert torch.all(p.out[2] == 0) and torch.all(torch.isneginf(p.lse[2]))
    csa2.clear_device_status(p.ws)
    for bad in ([0, 3, 2], [-1, 2, 3], [0, 2, 90]):
        p = Problem([2, 1], [300, 100], heads=16, seed=21)
        p.d_start.copy_(torch.tensor(bad, dtype=torch.int32))
        p.run()
        torch.cuda.synchronize()
        assert csa2.get_device_status(p.ws) == 0x40, bad
        assert torch.isfinite(p.out.float()).all()


@pytest.mark.parametrize("q_lens,ctx,heads", [([6, 2], [200, 90], 64), ([1, 1], [200, 90], 16), ([40, 1], [130, 64], 16)])
def test_nan_reaches_only_the_tokens_that_see_it(q_lens, ctx, heads):
    p = Problem(q_lens, ctx, heads=heads, seed=30).run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    at = int(p.row[0][-1])                                 # seen by the last token of the first sequence only
    for scale_code, rope in ((0x7F, None), (0xFF, None), (None, float("nan"))):
        s, k = p.scales[at].clone(), p.kr[at].clone()
        if scale_code is not None:
            p.scales[at, 5] = scale_code
        if rope is not None:
            p.kr[at, 3] = rope
        p.run()
        torch.cuda.synchronize()
        t = q_lens[0] - 1
        assert torch.isnan(p.out[t].float()).all() and torch.isnan(p.lse[t]).all()
        others = [i for i in range(p.total) if i != t]
        assert torch.equal(p.out[others], clean[others]) and torch.equal(p.lse[others], clean_lse[others])
        p.scales[at], p.kr[at] = s, k
    assert torch.equal(p.run().out, clean)


@pytest.mark.parametrize("heads", [16, 64])
def test_nan_behind_the_window(heads):
    p = Problem([5, 1], [300, 200], heads=heads, seed=31).run(window=64)
    clean = p.out.clone()
    for b, n in ((0, 5), (1, 1)):
        gone = torch.from_numpy(p.row[b][:p.ctx[b] - n - 63]).cuda()         # the first token sees 64 from there on
        p.scales[gone] = 0x7F
        p.kr[gone] = float("nan")
    assert torch.equal(p.run(window=64).out, clean)
    p.check(window=64)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_query_rows_stay_alone(bad):
    p = Problem([3, 1], [200, 90], heads=16, seed=32).run()
    clean, clean_lse = p.out.clone(), p.lse.clone()
    p.q[1, 3, 17] = bad
    p.q[3, 15, 570] = bad
    p.run()
    torch.cuda.synchronize()
    rows = torch.ones(4, 16, dtype=torch.bool)
    rows[1, 3] = rows[3, 15] = False
    rows = rows.cuda()
    assert torch.equal(p.out[rows], clean[rows]) and torch.equal(p.lse[rows], clean_lse[rows])
    assert not torch.isfinite(p.out[~rows].float()).any()


def test_thousands_of_sequences():
    """More sequences and tiles than the plan's threads; empty queries and empty contexts among them."""
    r = np.random.default_rng(33)
    q = r.integers(0, 3, 1500)
    c = np.maximum(r.integers(0, 70, 1500), q - 1)
    Problem([int(x) for x in q], [int(x) for x in c], heads=3, seed=33, gap=(2, 1)).run().check()


def test_more_tiles_than_plan_threads():
    Problem([2800], [2900], heads=64, seed=34).run(window=70).check(window=70, some=6)
    Problem([60] * 600, [61] * 600, heads=5, seed=35).run().check(some=2)


def test_longest_window_and_more_queries_than_context():
    w = 2 ** 31 - 1
    p = Problem([70, 3, 5], [50, 2, 0], heads=16, seed=36).run(window=w)
    p.check(window=w)
    for bad in (2 ** 31, 2 ** 32 + 5, -1):
        with pytest.raises(csa2.Csa2Error):
            p.run(window=bad)


@pytest.mark.parametrize("heads,q_lens", [(16, [1, 1]), (64, [5, 100])])
def test_contiguous_cache_that_ends_inside_a_block(heads, q_lens):
    p = Problem(q_lens, [100, 100], heads=heads, paged=False, seed=37)
    short = lambda t: t.view(2, 128, -1)[:, :100].reshape(200, -1).contiguous()
    p.codes, p.scales, p.kr = short(p.codes), short(p.scales), short(p.kr)
    p.dims = csa2.Dims(heads=heads, max_ctx=100)
    p.run().check()


def test_other_stream_than_the_inputs():
    p = Problem([3], [400], heads=16, seed=38)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        p.run()
    p.check()
