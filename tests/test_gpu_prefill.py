"""The prompt-side operators as they are used together: rotary queries, the cache append
and the chunk's attention, in one call after another, over several chunks.

The cache's bytes are compared exactly; the attention is compared with the oracle on the
rotated queries and rope keys as the kernels left them (their own roundings are tested
on their own), with the tolerance of the dense attention's tests.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2, prefill
from oracle import codec as ocodec
from oracle import prompt as op

pytestmark = pytest.mark.gpu

SCALE = 1 / 24.0


def make(lens, H, seed):
    """A paged cache for sequences of the given final lengths; every token's projections and queries."""
    r = np.random.default_rng(seed)
    B = len(lens)
    need = [-(-c // 64) for c in lens]
    pages = sum(need) + 2
    order = r.permutation(pages)
    table = np.zeros((B, max(need)), np.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    dims = csa2.Dims(heads=H, max_ctx=max(need) * 64, max_pages=max(need), num_pages=pages)
    planes = dict(kv_codes=torch.full((pages * 64, 256), 0x77, dtype=torch.uint8).cuda(),
                  kv_scales=torch.full((pages * 64, 32), 0x7F, dtype=torch.uint8).cuda(),
                  kv_rope=torch.full((pages * 64, 64), float("nan"), dtype=torch.bfloat16).cuda(),
                  page_table=torch.from_numpy(table).cuda())
    x = [torch.from_numpy(op.to_bf16(r.standard_normal((n, 576)))).to(torch.bfloat16) for n in lens]
    q = [torch.from_numpy(op.to_bf16(r.standard_normal((n, H, 576)))).to(torch.bfloat16) for n in lens]
    w = torch.from_numpy(op.to_bf16(1 + 0.1 * r.standard_normal(512))).to(torch.bfloat16)
    return dims, planes, x, q, w, table


def chunk(dims, planes, x, q, w, done, take, rope):
    """The next take[b] tokens of every sequence after done[b]."""
    B = len(x)
    start = torch.tensor(np.concatenate([[0], np.cumsum(take)]), dtype=torch.int32).cuda()
    ctx = torch.tensor([d + t for d, t in zip(done, take)], dtype=torch.int32).cuda()
    pos, rows = prefill.cache_rows(ctx, start, planes["page_table"])
    cb = prefill.ChunkBuffers(
        dims=dims, batch=B, rope=rope, ctx_len=ctx, q_start=start, pos=pos, dst_rows=rows, scale=SCALE, norm_w=w.cuda(),
        q=torch.cat([q[b][done[b]:done[b] + take[b]] for b in range(B)]).cuda(),
        x=torch.cat([x[b][done[b]:done[b] + take[b]] for b in range(B)]).cuda(), **planes)
    cb.entry = torch.empty((cb.x.shape[0], 576), dtype=torch.bfloat16, device="cuda")
    return cb.allocate_outputs()


def rows_of(table, b, n):
    t = np.arange(n)
    return table[b, t // 64].astype(np.int64) * 64 + t % 64


def check(cb, planes, x, w, table, done, take, H):
    torch.cuda.synchronize()
    assert csa2.get_device_status(cb.ws) == 0
    codes, scales = planes["kv_codes"].cpu().numpy(), planes["kv_scales"].cpu().numpy()
    kr = planes["kv_rope"].double().cpu().numpy()
    o, l, qd = cb.out.double().cpu().numpy(), cb.lse.double().cpu().numpy(), cb.q.double().cpu().numpy()
    at = 0
    for b in range(len(x)):
        n, N = take[b], done[b] + take[b]
        rows = rows_of(table, b, N)
        _, oc, osc = op.append_row_values(x[b][:N].double().numpy(), w.double().numpy(), np.float64(np.float32(1e-6)))
        np.testing.assert_array_equal(codes[rows], oc)
        np.testing.assert_array_equal(scales[rows], osc)
        if n:
            tok = np.unique(np.linspace(0, n - 1, min(n, 16)).astype(int))
            lat = ocodec.dequantize_rows(oc, osc)
            ro, rl, spread, mass = op.dense_attention(qd[at + tok], lat, kr[rows], N - n + tok, SCALE)
            ds, acc = 576 * 2.0 ** -22 * mass, (-(-N // 64) + 20) * 2.0 ** -22
            tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2 * ds[..., None] + acc) * spread + N * 2.0 ** -31 * np.abs(lat).max()
            assert np.all(np.abs(o[at + tok] - ro) <= tol)
            assert np.all(np.abs(l[at + tok] - rl) <= ds + acc + 2.0 ** -22 * np.abs(rl))
        at += n


@pytest.mark.parametrize("H", [16, 64])
def test_chunks_of_a_ragged_batch(H):
    """Prompts in unequal chunks, a sequence with none in the middle, then single tokens."""
    lens = [200, 65, 333]
    dims, planes, x, q, w, table = make(lens, H, H)
    rope = csa2.Rope(layout=csa2.ROPE_HALF, scaling=csa2.ROPE_LINEAR, factor=4.0)
    done = [0, 0, 0]
    for take in ([130, 63, 1], [0, 1, 200], [69, 0, 131], [1, 1, 1]):
        cb = chunk(dims, planes, x, q, w, done, take, rope)
        prefill.run_chunk(cb)
        check(cb, planes, x, w, table, done, take, H)
        # the exact rows are those that a codec write would give the cache's bytes for
        c2, s2 = csa2.fp4_kv_quantize(cb.entry[:, :512].contiguous())
        keep = cb.dst_rows >= 0
        assert torch.equal(planes["kv_codes"][cb.dst_rows[keep]], c2[keep])
        assert torch.equal(planes["kv_scales"][cb.dst_rows[keep]], s2[keep])
        done = [d + t for d, t in zip(done, take)]
    assert done == lens


def test_captured_chunk_replays():
    """One captured single-token chunk, replayed for token after token with new inputs copied in."""
    lens = [90, 70]
    dims, planes, x, q, w, table = make(lens, 16, 3)
    rope = csa2.Rope()
    done = [80, 60]
    first = chunk(dims, planes, x, q, w, [0, 0], done, rope)
    prefill.run_chunk(first)
    cb = chunk(dims, planes, x, q, w, done, [1, 1], rope)
    prefill.run_chunk(cb)                             # the first call on a device, before any capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        prefill.run_chunk(cb)
    for step in range(1, 6):
        now = [d + step for d in done]
        nx = chunk(dims, planes, x, q, w, now, [1, 1], rope)
        for name in ("q", "x", "pos", "dst_rows", "ctx_len"):
            getattr(cb, name).copy_(getattr(nx, name))
        g.replay()
        check(cb, planes, x, w, table, now, [1, 1], 16)


def test_same_logits_as_the_sparse_decode_over_the_same_positions():
    """With every position in the Top-K set and no window, the decode call's attention is this one."""
    lens = [300]
    dims, planes, x, q, w, table = make(lens, 64, 9)
    rope = csa2.Rope()
    prefill.run_chunk(chunk(dims, planes, x, q, w, [0], [299], rope))
    cb = chunk(dims, planes, x, q, w, [299], [1], rope)
    prefill.run_chunk(cb)
    d = csa2.Dims(heads=64, topk=300, swa=0, max_ctx=dims.max_ctx, max_pages=dims.max_pages, num_pages=dims.num_pages)
    ws = csa2.alloc_workspace(d, 1)
    out = torch.empty(1, 64, 512, device="cuda")
    lse = torch.empty(1, 64, device="cuda")
    tk = torch.arange(300, dtype=torch.int32, device="cuda").view(1, 300)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    csa2.csa2_sparse_attn_decode(d, 1, csa2.MODE_FULL, cb.q, planes["kv_codes"], planes["kv_scales"], planes["kv_rope"],
                                 planes["page_table"], cb.ctx_len, tk, None, zero, SCALE, out, lse, ws)
    torch.cuda.synchronize()
    # the decode call is within 2e-3 of a row's largest value, this one within a bf16 step and 2^-11 of the spread
    big = out.abs().amax(-1, keepdim=True)
    assert ((cb.out.float() - out).abs() <= 2.0 ** -8 * out.abs() + 4e-3 * big).all()
    assert ((cb.lse - lse).abs() <= 1e-4).all()


@pytest.mark.parametrize("H,take", [(16, [1, 1, 0]), (64, [70, 3, 20])])
def test_padded_batch(H, take):
    """Padding tokens that hold NaN, before and behind the sequences: no cache row, no output, the same results."""
    lens = [150, 65, 40]
    rope = csa2.Rope()
    done = [n - t for n, t in zip(lens, take)]
    got = []
    for pad in (False, True):
        dims, planes, x, q, w, table = make(lens, H, 40)
        prefill.run_chunk(chunk(dims, planes, x, q, w, [0, 0, 0], done, rope))
        cb = chunk(dims, planes, x, q, w, done, take, rope)
        n = cb.q.shape[0]
        if pad:
            wide = lambda t: torch.cat([torch.full_like(t[:1], float("nan")).expand(2, *t.shape[1:]), t,
                                        torch.full_like(t[:1], float("nan")).expand(3, *t.shape[1:])]).contiguous()
            cb.q, cb.x, cb.entry = wide(cb.q), wide(cb.x), wide(cb.entry)
            cb.q_start = cb.q_start + 2
            cb.pos, cb.dst_rows = prefill.cache_rows(cb.ctx_len, cb.q_start, planes["page_table"], total=n + 5)
            cb.allocate_outputs()
            cb.out.fill_(9.0)
            cb.lse.fill_(9.0)
        prefill.run_chunk(cb)
        torch.cuda.synchronize()
        assert csa2.get_device_status(cb.ws) == 0
        if pad:
            for t in (cb.out, cb.lse):
                assert torch.all(t[:2] == 9.0) and torch.all(t[n + 2:] == 9.0)
        s = slice(2, n + 2) if pad else slice(0, n)
        got.append((cb.out[s], cb.lse[s], cb.entry[s], *(planes[k].view(torch.uint8) for k in ("kv_codes", "kv_scales", "kv_rope"))))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_chunks_of_two_layers_on_two_streams():
    lens = [200, 90]
    rope = csa2.Rope()
    work = []
    for seed in (50, 51):
        dims, planes, x, q, w, table = make(lens, 64, seed)
        work.append((chunk(dims, planes, x, q, w, [0, 0], lens, rope), planes, x, w, table))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for (cb, *_), s in zip(work, streams):
        prefill.run_chunk(cb, stream=s)
    for cb, planes, x, w, table in work:
        check(cb, planes, x, w, table, [0, 0], lens, 64)
