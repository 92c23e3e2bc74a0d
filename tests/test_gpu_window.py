"""GPU window attention over exact rows against the float64 oracle.

Tolerances, per output element, derived from the kernel's roundings:
  scores: products of bf16 values, 576 terms summed in fp32 by the tensor core
    (taken as 2^-22 of the terms' size each, with truncation):  ds = 576 * 2^-22 M_r,
    M_r = max_t |scale| sum |q_i k_ti|;
  P: bf16, half a step 2^-8, and exp2 2^-22;
  sum and accumulation in fp32: (blocks + 20) 2^-22;  output: bf16, 2^-8.
out: 2^-8 |o| + (2^-8 + 2 ds + (blocks + 20) 2^-22) sum_t p_t |v_t|
lse: ds + (blocks + 20) 2^-22 + 2^-22 |lse|
Joined: the own part's bounds times its weight, the weights' error (that of lse, and 2^-20)
times both parts' sizes.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import prompt as op
from oracle import window as ow

pytestmark = pytest.mark.gpu

SCALE = 1 / 24.0


class Problem:
    """A ragged batch over a paged or contiguous cache; rows that no token sees hold NaN, pages that
    none sees have no id (or, with ring pages, come round)."""

    def __init__(self, q_lens, ctx, heads=64, window=128, sinks=0, paged=True, seed=0, gap=(0, 0), q_size=1.0, join=False,
                 ring=0):
        r = np.random.default_rng(seed)
        self.q_lens, self.ctx, self.H, self.W, self.S = list(q_lens), list(ctx), heads, window, sinks
        self.B = B = len(ctx)
        cap = max(64, -(-max(ctx) // 64) * 64)
        self.seen = []
        for n, c in zip(q_lens, ctx):
            s = np.zeros(c, bool)
            s[max(0, c - n - window + 1):] = True
            s[:sinks] = True
            self.seen.append(s)
        if ring:
            self.table = (np.arange(B)[:, None] * ring + np.arange(cap // 64) % ring).astype(np.int32)
            pages = B * ring
            rows = pages * 64
        elif paged:
            width = cap // 64
            self.table = np.full((B, width), -1, np.int32)
            need = [np.unique(np.nonzero(s)[0] // 64) for s in self.seen]
            pages = sum(len(x) for x in need) + 5
            order, at = r.permutation(pages), 0
            for b, x in enumerate(need):
                self.table[b, x] = order[at:at + len(x)]
                at += len(x)
            rows = pages * 64
        else:
            self.table, pages, rows = None, 0, B * cap
        self.cap, self.rows, self.pages = cap, rows, pages
        kv = np.full((rows, 576), np.nan)
        self.key = []                                       # per sequence, by position
        scale = np.exp(0.5 * r.standard_normal(576))
        for b, c in enumerate(ctx):
            k = op.to_bf16(r.standard_normal((c, 576)) * scale)
            at = np.nonzero(self.seen[b])[0]
            kv[self.row(b, at)] = k[at]
            self.key.append(k)
        self.kv64 = kv
        self.kv = torch.from_numpy(kv).to(torch.bfloat16).cuda()
        self.starts = np.concatenate([[gap[0]], gap[0] + np.cumsum(q_lens)]).astype(np.int32)
        self.total = int(self.starts[-1]) + gap[1]
        self.q64 = op.to_bf16(r.standard_normal((self.total, heads, 576)) * q_size)
        self.q = torch.from_numpy(self.q64).to(torch.bfloat16).cuda()
        self.dims = csa2.Dims(heads=heads, max_ctx=cap, num_pages=pages, max_pages=cap // 64 if pages else 0)
        self.prev = self.prev_lse = None
        if join:
            self.prev64 = op.to_bf16(0.3 * r.standard_normal((self.total, heads, 512)))
            self.prev = torch.from_numpy(self.prev64).to(torch.bfloat16).cuda()
            self.prev_lse = torch.from_numpy((4 + 3 * r.standard_normal((self.total, heads))).astype(np.float32)).cuda()
            self.prev_lse[0, 0] = -float("inf")
        self.out = torch.full((self.total, heads, 512), 9.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.total, heads), 9.0, dtype=torch.float32, device="cuda")
        self.ws = csa2.alloc_window_attn_workspace(self.dims, B, self.total)
        self.d_table = torch.from_numpy(self.table).cuda() if self.table is not None else None
        self.d_ctx = torch.tensor(ctx, dtype=torch.int32).cuda()
        self.d_start = torch.from_numpy(self.starts).cuda()

    def row(self, b, t):
        return b * self.cap + t if self.table is None else self.table[b, t // 64].astype(np.int64) * 64 + t % 64

    def run(self, scale=SCALE, stream=None):
        csa2.csa2_window_attn_chunk(self.dims, self.B, self.q, self.d_start, self.kv, self.d_table, self.d_ctx, scale, self.W,
                                    self.out, self.lse, self.ws, sinks=self.S, prev_out=self.prev, prev_lse=self.prev_lse,
                                    stream=stream)
        return self

    def check(self, scale=SCALE, some=24, status=0):
        """`some` tokens of each sequence (first, last and spread ones) against the oracle."""
        torch.cuda.synchronize()
        assert csa2.get_device_status(self.ws) == status
        o = self.out.double().cpu().numpy()
        l = self.lse.double().cpu().numpy()
        for b in range(self.B):
            n, N = self.q_lens[b], self.ctx[b]
            if n == 0:
                continue
            tok = np.unique(np.linspace(0, n - 1, min(n, some)).astype(int))
            at = self.starts[b] + tok
            ro, rl, spread, mass = ow.window_attention(self.q64[at], self.key[b], N - n + tok, scale, self.W, self.S)
            ds = 576 * 2.0 ** -22 * mass
            acc = (-(-min(N, self.W + self.S + 64) // 128) + 20) * 2.0 ** -22
            wide = (2.0 ** -8 + 2 * ds[..., None] + acc) * spread
            if self.prev is not None:
                po, pl = self.prev64[at], self.prev_lse.double().cpu().numpy()[at]
                jo, rl2, wa, wb = ow.join(ro, rl, po, pl)
                off = (2 * (ds + acc) + 2.0 ** -20)[..., None] * (wa[..., None] * np.abs(ro) + wb[..., None] * np.abs(po))
                wide, ro, rl = wa[..., None] * wide + off, jo, rl2
            err = np.abs(o[at] - ro)
            tol = 2.0 ** -8 * np.abs(ro) + wide
            assert np.all(err <= tol), (b, float((err / np.maximum(tol, 1e-30)).max()))
            none = np.isneginf(rl)
            assert np.array_equal(np.isneginf(l[at]), none)
            e = np.abs(l[at][~none] - rl[~none])
            assert np.all(e <= ds[~none] + acc + 2.0 ** -22 * (4 + np.abs(rl[~none]))), (b, float(e.max()))
        for t in list(range(0, self.starts[0])) + list(range(self.starts[-1], self.total)):
            assert np.all(o[t] == 9.0) and np.all(l[t] == 9.0)


@pytest.mark.parametrize("ctx", [1, 2, 63, 64, 65, 127, 128, 129, 130, 200, 1000])
@pytest.mark.parametrize("heads", [1, 7, 16, 64])
def test_one_token(ctx, heads):
    Problem([1], [ctx], heads=heads, seed=ctx).run().check()


@pytest.mark.parametrize("paged", [True, False])
@pytest.mark.parametrize("join", [True, False])
def test_decode_batch(paged, join):
    c = [1, 300, 64, 2049, 777, 8000, 65, 128]
    Problem([1] * 8, c, paged=paged, seed=3, join=join).run().check()


@pytest.mark.parametrize("heads", [3, 7, 24, 40, 64])
@pytest.mark.parametrize("join", [True, False])
def test_ragged_chunks(heads, join):
    """Tiles that cross tokens, sequences without queries, one with more queries than context."""
    Problem([5, 0, 130, 1, 33, 9], [700, 64, 130, 1, 1500, 4], heads=heads, seed=heads, gap=(2, 3), join=join).run().check()


def test_whole_prompts():
    Problem([257, 64, 511], [257, 64, 511], seed=8).run().check()


def test_more_tiles_than_sms():
    Problem([400, 7, 350], [400, 900, 390], heads=64, window=100, sinks=3, seed=9, join=True).run().check()


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 130, 200, 1000, 5000])
@pytest.mark.parametrize("sinks", [0, 1, 4, 64, 200])
def test_window_and_sinks(window, sinks):
    Problem([70, 3, 1], [900, 130, 2500], heads=16, window=window, sinks=sinks, seed=window + sinks).run().check(some=12)


@pytest.mark.parametrize("heads,lens,ctx", [(64, [1], [40000]), (16, [1, 2], [9000, 5000]), (64, [2, 1, 3], [6000, 100, 1]),
                                            (7, [1] * 70, [3000] * 70)])
@pytest.mark.parametrize("join", [True, False])
def test_long_windows_of_few_tokens_are_split(heads, lens, ctx, join):
    Problem(lens, ctx, heads=heads, window=5000, sinks=70, seed=len(lens), join=join).run().check()


@pytest.mark.parametrize("scale", [0.0, -SCALE, 1.0, 1e-6])
def test_scales(scale):
    Problem([9], [500], heads=16, seed=6).run(scale=scale).check(scale=scale)


def test_steep_rows():
    """Logits in the hundreds: most weights vanish, the reference rises."""
    Problem([40, 1], [3000, 2000], heads=64, window=1500, seed=11, q_size=12.0).run().check()


def test_rising_and_falling_logits():
    """Keys grow along the window, so every block passes the reference by more than the slack; then they fall."""
    p = Problem([4], [64 * 12], heads=16, window=64 * 12, paged=False, seed=13)
    v = op.to_bf16(np.repeat(np.arange(12), 64)[:, None] * np.ones((1, 64)))
    p.key[0][:, 512:] = v
    p.kv[:, 512:] = torch.from_numpy(v).to(torch.bfloat16).cuda()
    for s in (4.0, -4.0):
        p.q64[:, :, 512:] = s
        p.q[:, :, 512:] = s
        p.run().check()


@pytest.mark.parametrize("window,q", [(128, 1), (100, 20), (64, 40)])
def test_pages_that_come_round(window, q):
    """A ring of pages, the form in which a serving engine keeps a window."""
    p = Problem([q, q], [1000, 333], heads=16, window=window, ring=-(-(window + q + 62) // 64) + (window != 128), seed=window)
    for b in range(2):                                       # later positions have taken the places of earlier ones
        t = np.nonzero(p.seen[b])[0]
        assert len(np.unique(p.row(b, t))) == len(t)
    p.run().check()


def test_window_of_a_decode_step():
    """128 rows a sequence, position t in row t % 128: the sparse decode attention's window."""
    p = Problem([1, 1], [500, 90], heads=64, window=128, ring=2, seed=2)
    p.run().check()
    d = csa2.Dims(heads=64, topk=1, swa=128, max_ctx=64)
    none = torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    cache = [torch.zeros(128, w, dtype=torch.uint8, device="cuda") for w in (256, 32, 128)]
    out, lse = torch.zeros(2, 64, 512, device="cuda"), torch.zeros(2, 64, device="cuda")
    kv = torch.nan_to_num(p.kv).view(2, 128, 576)
    csa2.csa2_sparse_attn_decode(d, 2, csa2.MODE_FULL, p.q, cache[0], cache[1], cache[2].view(torch.bfloat16), None,
                                 torch.zeros(2, dtype=torch.int32, device="cuda"), none, kv,
                                 torch.tensor([128, 90], dtype=torch.int32, device="cuda"), SCALE, out, lse,
                                 csa2.alloc_workspace(d, 2))
    assert (out - p.out.float()).abs().max() <= 2.0 ** -6 * out.abs().max()
    assert (lse - p.lse).abs().max() <= 2e-5


def test_infinities_and_nan_stay_with_the_tokens_that_see_them():
    for bad in (float("nan"), float("inf"), -float("inf")):
        p = Problem([100], [400], heads=16, window=50, sinks=2, seed=21)
        clean = p.run().out.clone(), p.lse.clone()
        for t in (330, 370):
            p.kv[int(p.row(0, np.array([t]))[0]), 17] = bad
        p.q[40, 3, 5] = bad
        p.run()
        torch.cuda.synchronize()
        pos = torch.arange(300, 400)
        hit = torch.zeros(100, 16, dtype=torch.bool)
        for t in (330, 370):
            hit[(pos >= t) & (pos < t + 50)] = True
        rest = ~hit
        rest[40, 3] = False
        rest = rest.cuda()
        assert torch.equal(p.out[rest], clean[0][rest]) and torch.equal(p.lse[rest], clean[1][rest])
        assert torch.isnan(p.out[hit.cuda()][:, 17]).all()
        assert not torch.isfinite(p.out[40, 3]).any()


def test_rows_beside_a_batch_hold_anything():
    """Queries of padding tokens: NaN there reaches nothing."""
    p = Problem([3, 2], [70, 300], heads=16, seed=23, gap=(1, 2))
    p.q[0] = float("nan")
    p.q[-2:] = float("inf")
    p.run().check()


def test_same_results_every_time_and_with_a_used_workspace():
    p = Problem([1, 20, 200], [9000, 3000, 400], window=600, sinks=5, seed=14)
    a = p.run().out.clone()
    la = p.lse.clone()
    small = Problem([3], [4000], heads=16, window=3000, seed=15)
    small.ws = p.ws                                       # another shape through the same workspace
    small.run().check()
    p.out.fill_(9)
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(p.out, a) and torch.equal(p.lse, la)
    p.check()


def test_joined_in_place():
    for lens, ctx, W in (([5, 40], [100, 700], 128), ([1], [4000], 3000)):
        p = Problem(lens, ctx, heads=64, window=W, seed=16, join=True)
        p.run().check()
        out, lse = p.prev.clone(), p.prev_lse.clone()
        csa2.csa2_window_attn_chunk(p.dims, p.B, p.q, p.d_start, p.kv, p.d_table, p.d_ctx, SCALE, W, out, lse, p.ws,
                                    prev_out=out, prev_lse=lse)
        assert torch.equal(out, p.out) and torch.equal(lse, p.lse)


def test_a_joined_part_without_weight_may_be_anything():
    p = Problem([2, 3], [50, 2], heads=16, seed=17, join=True)
    p.prev_lse[:] = -float("inf")
    p.prev[:] = float("nan")
    p.run()
    q = Problem([2, 3], [50, 2], heads=16, seed=17)
    q.run().check()
    assert torch.equal(p.out, q.out) and torch.equal(p.lse, q.lse)


def test_graph_replay_with_new_lengths():
    """Lengths are read on the device: a captured call follows them."""
    for W in (128, 2000):
        p = Problem([1, 1, 1], [500, 64, 3000], heads=16, window=W, paged=False, seed=18)
        p.kv = torch.nan_to_num(p.kv)
        full = [k.copy() for k in p.key]
        for b in range(3):
            p.kv[b * p.cap:b * p.cap + p.ctx[b]] = torch.from_numpy(full[b]).to(torch.bfloat16).cuda()
        p.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run()
        for c in ([500, 64, 3000], [1, 64, 2999], [450, 3, 64]):
            p.ctx = list(c)
            p.key = [k[:n] for k, n in zip(full, c)]
            p.d_ctx.copy_(torch.tensor(c, dtype=torch.int32))
            p.out.fill_(9)
            g.replay()
            p.check()


def test_two_calls_at_once():
    ps = [Problem([1, 5], [3000, 700], window=700, seed=s) for s in (19, 20)]
    streams = [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for _ in range(3):
        for p, s in zip(ps, streams):
            p.run(stream=s)
    for p in ps:
        p.check()


def test_many_sequences():
    r = np.random.default_rng(5)
    lens = r.integers(0, 3, 2500).tolist()
    ctx = [int(n + r.integers(0, 90)) for n in lens]
    p = Problem(lens, [max(c, 1) for c in ctx], heads=5, window=40, sinks=2, seed=24)
    p.run().check()


def test_a_cache_past_2_31_bytes():
    p = Problem([2, 1], [200, 900], heads=16, window=300, seed=25)
    far = (1 << 31) // (64 * 1152) + 1000                  # pages before the ones in use
    kv = torch.empty((far + p.pages) * 64, 576, dtype=torch.bfloat16, device="cuda")
    kv[far * 64:] = p.kv
    p.kv = kv
    p.d_table = torch.where(p.d_table >= 0, p.d_table + far, p.d_table)
    p.dims.num_pages = far + p.pages
    p.run().check()


def test_bad_page_is_skipped_and_reported():
    p = Problem([2], [300], heads=16, window=290, seed=26)
    p.d_table[0, 1] = p.pages
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0x02
    t = np.arange(300)
    for i in range(2):
        see = (t <= 298 + i) & (t > 8 + i) & (t // 64 != 1)
        ro, rl, _, _ = ow.window_attention(p.q64[i:i + 1], p.key[0][see], [10 ** 6], SCALE, 1 << 30)
        assert np.abs(p.out[i].double().cpu().numpy() - ro[0]).max() <= 2.0 ** -6 * np.abs(ro).max()
        assert np.abs(p.lse[i].double().cpu().numpy() - rl[0]).max() <= 1e-4
    csa2.clear_device_status(p.ws)


def test_bad_lengths_and_starts_are_reported():
    p = Problem([2, 3], [100, 200], heads=16, seed=27)
    p.d_ctx[1] = p.cap + 1
    p.run()
    torch.cuda.synchronize()
    assert csa2.get_device_status(p.ws) == 0x01
    assert torch.all(p.out[2:] == 0) and torch.isneginf(p.lse[2:]).all()
    csa2.clear_device_status(p.ws)
    p.d_ctx[1] = 200
    for starts in ([0, 3, 2], [-1, 2, 5], [0, 2, 6], [0, 6, 5]):
        p.d_start.copy_(torch.tensor(starts, dtype=torch.int32))
        p.out.fill_(9)
        p.run()
        torch.cuda.synchronize()
        assert csa2.get_device_status(p.ws) == 0x40 and torch.all(p.out == 9)
        csa2.clear_device_status(p.ws)


def test_refusals():
    p = Problem([2], [100], heads=16, seed=28)

    def call(**kw):
        a = dict(q=p.q, start=p.d_start, kv=p.kv, table=p.d_table, ctx=p.d_ctx, window=128, out=p.out, lse=p.lse, ws=p.ws,
                 sinks=0, prev_out=None, prev_lse=None)
        a.update(kw)
        csa2.csa2_window_attn_chunk(p.dims, 1, a["q"], a["start"], a["kv"], a["table"], a["ctx"], SCALE, a["window"], a["out"],
                                    a["lse"], a["ws"], sinks=a["sinks"], prev_out=a["prev_out"], prev_lse=a["prev_lse"])
    call()
    for kw, code in ((dict(window=0), 1), (dict(sinks=-1), 1), (dict(window=1 << 21), 2), (dict(sinks=1 << 21), 2),
                     (dict(window=1 << 40), 1), (dict(q=p.q.float()), 1), (dict(kv=p.kv[:-1]), 1), (dict(kv=p.kv.cpu()), 1),
                     (dict(lse=p.lse.double()), 1), (dict(prev_out=p.out), 1), (dict(prev_lse=p.lse), 1),
                     (dict(ws=p.ws[:1024]), 3), (dict(start=p.d_start.long()), 1), (dict(out=p.q[..., :512]), 1)):
        with pytest.raises(csa2.Csa2Error) as e:
            call(**kw)
        assert e.value.code == code, kw
    # outputs over the other part's, by half
    both = torch.zeros(p.out.numel() + 512, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(csa2.Csa2Error):
        call(out=both[512:].view_as(p.out), prev_out=both[:-512].view_as(p.out), prev_lse=torch.zeros_like(p.lse))
