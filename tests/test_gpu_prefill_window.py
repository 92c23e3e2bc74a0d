"""A layer's new tokens through all that it has: FP4 rows, exact rows of a window and indexer keys written,
attention of the chunk over both kinds of rows in one softmax, and the decode step that follows.

The exact rows are compared bit for bit, the attention with the oracle on the rows as the kernels left
them.  Tolerance of the joined outputs: each part's own (the dense attention's and the window attention's
tests), times its weight, the weights' error (twice both log sums') times both parts' sizes, and the
last rounding.  The decode step: 2e-3 of a row's largest value, as in its own tests.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2, prefill, step
from oracle import attention as oat
from oracle import codec as ocodec
from oracle import indexer as oix
from oracle import prompt as op
from oracle import window as ow

pytestmark = pytest.mark.gpu

SCALE = 1 / 24.0
SWA = 128


def bf16(v):
    return torch.from_numpy(op.to_bf16(v)).to(torch.bfloat16)


class Layer:
    """Caches of one layer for sequences of the given final lengths; every token's projections and queries."""

    def __init__(self, lens, H, seed, window=128, sinks=0, ring=0):
        r = np.random.default_rng(seed)
        self.lens, self.H, self.window, self.sinks = lens, H, window, sinks
        B = len(lens)
        need = [-(-c // 64) for c in lens]
        self.table, self.win_table = np.zeros((B, max(need)), np.int32), np.zeros((B, max(need)), np.int32)
        pages = sum(need) + 2
        order, other, at = r.permutation(pages), r.permutation(pages), 0
        for b, k in enumerate(need):
            self.table[b, :k], self.win_table[b, :k] = order[at:at + k], other[at:at + k]
            at += k
        win_pages = pages
        if ring:                                             # pages of the window that come round
            self.win_table[:] = np.arange(B)[:, None] * ring + np.arange(max(need)) % ring
            win_pages = B * ring
        kw = dict(heads=H, max_ctx=max(need) * 64, max_pages=max(need))
        self.dims, self.win_dims = csa2.Dims(num_pages=pages, **kw), csa2.Dims(num_pages=win_pages, **kw)
        self.codes = torch.full((pages * 64, 256), 0x77, dtype=torch.uint8).cuda()
        self.scales = torch.full((pages * 64, 32), 0x7F, dtype=torch.uint8).cuda()
        self.kr = torch.full((pages * 64, 64), float("nan"), dtype=torch.bfloat16).cuda()
        self.kv = torch.full((win_pages * 64, 576), float("nan"), dtype=torch.bfloat16).cuda()
        self.swa = torch.full((B, SWA, 576), float("nan"), dtype=torch.bfloat16).cuda()
        self.idx = torch.full((pages * 64, 128), 0x7F, dtype=torch.uint8).cuda()
        self.d_table, self.d_win_table = torch.from_numpy(self.table).cuda(), torch.from_numpy(self.win_table).cuda()
        self.x = [bf16(r.standard_normal((n, 576))) for n in lens]
        self.q = [bf16(r.standard_normal((n, H, 576))) for n in lens]
        self.kx = [bf16(r.standard_normal((n, 128))) for n in lens]
        self.w = bf16(1 + 0.1 * r.standard_normal(512))
        self.kw, self.kb = bf16(1 + 0.1 * r.standard_normal(128)), bf16(0.1 * r.standard_normal(128))
        self.rope = csa2.Rope(layout=csa2.ROPE_HALF, scaling=csa2.ROPE_LINEAR, factor=4.0)
        self.done = [0] * B
        # every token's exact rows and rope part, by sequence, as they come out of the runs
        self.rows = [np.zeros((0, 576)) for _ in lens]

    def chunk(self, take):
        B, done = len(self.lens), self.done
        part = lambda xs: torch.cat([xs[b][done[b]:done[b] + take[b]] for b in range(B)]).cuda()
        start = torch.tensor(np.concatenate([[0], np.cumsum(take)]), dtype=torch.int32).cuda()
        ctx = torch.tensor([d + t for d, t in zip(done, take)], dtype=torch.int32).cuda()
        pos, rows = prefill.cache_rows(ctx, start, self.d_table)
        exact = prefill.ExactRows(self.kv, prefill.cache_rows(ctx, start, self.d_win_table)[1], self.window, self.sinks, self.win_dims,
                                  self.d_win_table, self.swa, prefill.window_rows(ctx, start, SWA))
        keys = prefill.IndexerKeys(part(self.kx), self.idx, self.idx.shape[0], csa2.IDXK_E4M3, self.rope, 64, csa2.IDX_NORM_LAYER,
                                   self.kw.cuda(), self.kb.cuda())
        cb = prefill.ChunkBuffers(self.dims, B, self.rope, self.codes, self.scales, self.kr, self.d_table, ctx, start,
                                  part(self.q), part(self.x), pos, rows, SCALE, norm_w=self.w.cuda(), exact=exact, keys=keys)
        cb.entry = torch.empty((cb.x.shape[0], 576), dtype=torch.bfloat16, device="cuda")
        return cb.allocate_outputs()

    def ran(self, cb, take):
        """Checks a chunk that has run, and counts its tokens as done."""
        torch.cuda.synchronize()
        assert csa2.get_device_status(cb.ws) == 0 and csa2.get_device_status(cb.exact.ws) == 0
        codes, scales = self.codes.cpu().numpy(), self.scales.cpu().numpy()
        f = lambda t: t.double().cpu().numpy()
        kr, kv, swa, entry = f(self.kr), f(self.kv), f(self.swa), f(cb.entry)
        o, l, qd = f(cb.out), f(cb.lse), f(cb.q)
        at = 0
        for b in range(len(self.lens)):
            n, N = take[b], self.done[b] + take[b]
            row = lambda table, t: table[b, t // 64].astype(np.int64) * 64 + t % 64
            new = np.arange(N - n, N)
            self.rows[b] = np.concatenate([self.rows[b], entry[at:at + n]])
            # the exact rows, wherever they go: bit for bit the append's
            np.testing.assert_array_equal(kv[row(self.win_table, new)], entry[at:at + n])
            held = np.arange(max(0, N - SWA), N)
            np.testing.assert_array_equal(swa[b, held % SWA], self.rows[b][held])
            np.testing.assert_array_equal(kr[row(self.table, new)], entry[at:at + n, 512:])
            if n:
                tok = np.unique(np.linspace(0, n - 1, min(n, 12)).astype(int))
                fp4 = row(self.table, np.arange(N))
                lat = ocodec.dequantize_rows(codes[fp4], scales[fp4])
                po, pl, spread, mass = op.dense_attention(qd[at + tok], lat, kr[fp4], N - n + tok, SCALE)
                ds, acc = 576 * 2.0 ** -22 * mass, (-(-N // 64) + 20) * 2.0 ** -22
                ptol = 2.0 ** -8 * np.abs(po) + (2.0 ** -11 + 2 * ds[..., None] + acc) * spread + N * 2.0 ** -31 * np.abs(lat).max()
                pltol = ds + acc + 2.0 ** -22 * np.abs(pl)
                eo, el, spread, mass = ow.window_attention(qd[at + tok], self.rows[b], N - n + tok, SCALE, self.window, self.sinks)
                ds, acc = 576 * 2.0 ** -22 * mass, (-(-N // 128) + 20) * 2.0 ** -22
                etol = (2.0 ** -8 + 2 * ds[..., None] + acc) * spread
                jo, jl, we, wp = ow.join(eo, el, po, pl)
                off = (2 * (ds + acc + pltol) + 2.0 ** -20)[..., None] * (we[..., None] * np.abs(eo) + wp[..., None] * np.abs(po))
                tol = 2.0 ** -8 * np.abs(jo) + we[..., None] * etol + wp[..., None] * ptol + off
                assert np.all(np.abs(o[at + tok] - jo) <= tol)
                assert np.all(np.abs(l[at + tok] - jl) <= ds + acc + pltol + 2.0 ** -22 * (4 + np.abs(jl)))
            at += n
        self.done = [d + t for d, t in zip(self.done, take)]


@pytest.mark.parametrize("H,window,sinks,ring", [(16, 128, 0, 0), (64, 100, 3, 0), (64, 128, 0, 6), (16, 150, 70, 0)])
def test_chunks_with_a_window(H, window, sinks, ring):
    """Prompts in unequal chunks, a sequence with none in the middle, then single tokens."""
    lens = [200, 65, 333]
    lay = Layer(lens, H, H + window, window, sinks, ring)
    for take in ([130, 63, 1], [0, 1, 200], [69, 0, 131], [1, 1, 1]):
        cb = lay.chunk(take)
        prefill.run_chunk(cb)
        lay.ran(cb, take)
    assert lay.done == lens


@pytest.mark.parametrize("H", [16, 64])
def test_decode_step_after_chunks(H):
    """What the chunks left is what a decode step reads: keys, FP4 rows, the window.  With every position
    in its Top-K set its attention is the chunk's of the same token."""
    lens = [300, 77, 512]
    lay = Layer(lens, H, 5)
    for take in ([299, 70, 400], [0, 6, 111], [1, 1, 1]):
        cb = lay.chunk(take)
        prefill.run_chunk(cb)
        lay.ran(cb, take)
    B = len(lens)
    r = np.random.default_rng(8)
    for topk in (512, 64):
        d = csa2.Dims(heads=H, swa=SWA, pool_blocks=16 if topk == 64 else 64, topk=topk, max_ctx=lay.dims.max_ctx,
                      max_pages=lay.dims.max_pages, num_pages=lay.dims.num_pages)
        iq, iw = op.to_bf16(r.standard_normal((2, B, 16, 128))), r.random((2, B, 16)).astype(np.float32)
        sb = step.StepBuffers(
            d, B, ["F", "Ru"], lay.codes, lay.scales, lay.kr, lay.idx, lay.d_table, cb.ctx_len,
            q=torch.stack([cb.q, cb.q]), swa=torch.stack([lay.swa, lay.swa]),
            swa_len=torch.tensor([[min(SWA, n) for n in lens]] * 2, dtype=torch.int32).cuda(),
            idx_q=torch.from_numpy(iq).to(torch.bfloat16).cuda(), idx_w=torch.from_numpy(iw).cuda(), scale=SCALE).allocate_outputs()
        step.run_step(sb)
        torch.cuda.synchronize()
        assert csa2.get_device_status(sb.ws) == 0
        codes, scales, keys = lay.codes.cpu().numpy(), lay.scales.cpu().numpy(), lay.idx.cpu().numpy()
        kr, swa, qd = lay.kr.double().cpu().numpy(), lay.swa.double().cpu().numpy(), cb.q.double().cpu().numpy()
        for b, N in enumerate(lens):
            fp4 = lay.table[b, np.arange(N) // 64].astype(np.int64) * 64 + np.arange(N) % 64
            want = oix.full_topk(iq[0, b], iw[0, b].astype(np.float64), ocodec.e4m3_decode(keys[fp4]), d.pool_blocks, topk)["topk"]
            np.testing.assert_array_equal(sb.topk[0, b].cpu().numpy(), want)
            lat = ocodec.dequantize_rows(codes[fp4], scales[fp4])
            for layer in (0, 1):
                o, l = oat.sparse_attn_decode(qd[b], lat, kr[fp4], want, swa[b], min(SWA, N), SCALE)
                got, gl = sb.out[layer, b].double().cpu().numpy(), sb.lse[layer, b].double().cpu().numpy()
                assert np.all(np.abs(got - o) <= 2e-3 * np.abs(o).max(-1, keepdims=True)) and np.all(np.abs(gl - l) <= 2e-3)
        if topk == 512:                                      # the chunk's own: a bf16 step, and bf16 parts and weights
            big = sb.out[0].abs().amax(-1, keepdim=True)
            assert ((cb.out.float() - sb.out[0]).abs() <= 2.0 ** -8 * sb.out[0].abs() + (2e-3 + 2.0 ** -7) * big).all()
            assert ((cb.lse - sb.lse[0]).abs() <= 2e-3 + 1e-4).all()


def test_captured_chunk_replays():
    """A captured single-token chunk, replayed for token after token with new inputs copied in."""
    lens = [140, 70]
    lay = Layer(lens, 16, 3)
    cb = lay.chunk([130, 60])
    prefill.run_chunk(cb)
    lay.ran(cb, [130, 60])
    cb = lay.chunk([1, 1])
    prefill.run_chunk(cb)                             # the first call on a device, before any capture
    lay.ran(cb, [1, 1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prefill.run_chunk(cb)
    for _ in range(5):
        nx = lay.chunk([1, 1])
        for name in ("q", "x", "pos", "dst_rows", "ctx_len"):
            getattr(cb, name).copy_(getattr(nx, name))
        cb.exact.dst_rows.copy_(nx.exact.dst_rows)
        cb.exact.swa_rows.copy_(nx.exact.swa_rows)
        cb.keys.x.copy_(nx.keys.x)
        g.replay()
        lay.ran(cb, [1, 1])


def test_two_layers_on_two_streams():
    lens = [200, 90]
    work = [Layer(lens, 64, seed) for seed in (50, 51)]
    chunks = [lay.chunk(lens) for lay in work]
    torch.cuda.synchronize()
    for cb in chunks:
        prefill.run_chunk(cb, stream=torch.cuda.Stream())
    for lay, cb in zip(work, chunks):
        lay.ran(cb, lens)
