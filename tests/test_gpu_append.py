"""GPU cache append (norm, rotary, FP4 write) against the float64 oracle.

Latent bf16 values, FP4 codes and scales are byte-exact (the norm is rounded
once from the exact value); the rotary part is within 2^-20 (|u| + |v|) m plus
half a bf16 step, as derived in the rotary tests.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import prompt as op
from tests.helpers import bf16_f64

pytestmark = pytest.mark.gpu

PARTS = dict(scaling=csa2.ROPE_PARTS, factor=16.0, orig_ctx=4096.0, mscale=1.25)


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def run(x, w, pos, dst, rows, cfg, eps=1e-6, entry=True, fill=0xA5):
    codes = torch.full((rows, 256), fill, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 32), fill, dtype=torch.uint8, device="cuda")
    rope = torch.full((rows, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    ent = torch.full((x.shape[0], 576), 7.0, dtype=torch.bfloat16, device="cuda") if entry else None
    csa2.csa2_kv_append(cfg, x, pos, dst, codes, scales, rope, norm_w=w, eps=eps, entry=ent)
    torch.cuda.synchronize()
    return codes, scales, rope, ent


def check(x, w, pos, dst, rows, cfg, eps, got):
    codes, scales, rope, ent = got
    x64 = x.double().cpu().numpy()
    lat, oc, osc = op.append_row_values(x64, None if w is None else w.double().cpu().numpy(), np.float64(np.float32(eps)))
    f = op.rope_frequencies(64, cfg.theta, "parts" if cfg.scaling == csa2.ROPE_PARTS else "plain", cfg.factor, cfg.orig_ctx,
                            cfg.turns_lo, cfg.turns_hi)
    half = cfg.layout == csa2.ROPE_HALF
    xr = x64[:, None, 512:]
    ref = op.rope(xr, pos.cpu().numpy(), f, half, cfg.mscale)[:, 0]
    u, v = (xr[:, 0, :32], xr[:, 0, 32:]) if half else (xr[:, 0, 0::2], xr[:, 0, 1::2])
    size = (np.abs(u) + np.abs(v)) * cfg.mscale
    size = np.concatenate([size, size], -1) if half else np.repeat(size, 2, -1)
    tol = 2.0 ** -20 * size + 2.0 ** -8 * np.abs(ref)
    d = dst.cpu().numpy()
    keep = (d >= 0) & (d < rows)
    np.testing.assert_array_equal(codes.cpu().numpy()[d[keep]], oc[keep])
    np.testing.assert_array_equal(scales.cpu().numpy()[d[keep]], osc[keep])
    assert np.all(np.abs(rope.double().cpu().numpy()[d[keep]] - ref[keep]) <= tol[keep])
    rest = np.setdiff1d(np.arange(rows), d[keep])          # other rows as they were
    assert np.all(codes.cpu().numpy()[rest] == 0xA5) and np.all(scales.cpu().numpy()[rest] == 0xA5)
    assert np.all(rope.double().cpu().numpy()[rest] == 3.0)
    if ent is not None:
        np.testing.assert_array_equal(bf16_f64(bits(ent))[:, :512], lat)
        assert np.all(np.abs(ent.double().cpu().numpy()[:, 512:] - ref) <= tol)


def inputs(n, rows, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, 576, generator=g) * torch.exp(spread * torch.randn(n, 1, generator=g))
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda()
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
    dst = torch.randperm(rows, generator=g)[:n].cuda()
    return x.to(torch.bfloat16).cuda(), w, pos, dst


@pytest.mark.parametrize("n,rows", [(1, 64), (7, 64), (64, 4096), (1237, 1280), (5000, 5056)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_against_oracle(n, rows, half, norm):
    x, w, pos, dst = inputs(n, rows, 10 + n)
    if n > 5:
        dst[2], dst[4] = -1, rows                          # no cache row: skipped
    cfg = csa2.Rope(layout=csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED, **PARTS)
    w = w if norm else None
    check(x, w, pos, dst, rows, cfg, 1e-6, run(x, w, pos, dst, rows, cfg))


def test_rows_of_every_size_and_special_rows():
    """Rows from 2^-60 to 2^60, one large channel among small ones, zeros, an eps that matters."""
    x, w, pos, dst = inputs(600, 640, 77)
    s = torch.exp2(torch.linspace(-60, 60, 600)).cuda()[:, None]
    x = (x.float() * s).to(torch.bfloat16)
    x[10, :512] = 0
    x[11, :512] = 0
    x[11, 5] = 1.5
    x[12, 3] = x[12, 3] * 2 ** 12
    cfg = csa2.Rope()
    for eps in (1e-6, 1e-3, 3e-12):
        check(x, w, pos, dst, 640, cfg, eps, run(x, w, pos, dst, 640, cfg, eps=eps))


def test_many_rows_are_exact():
    """60,000 rows: some values stand next to a bf16 midpoint (about one in 10^7 within 1e-9 of it)."""
    x, w, pos, dst = inputs(60000, 60032, 5)
    cfg = csa2.Rope()
    check(x, w, pos, dst, 60032, cfg, 1e-6, run(x, w, pos, dst, 60032, cfg))


def test_exact_ties_round_to_even():
    """mean(x^2) + eps = 1 exactly in binary: products w x land on bf16 midpoints."""
    x = torch.zeros(2, 576)
    x[:, :512] = torch.tensor([0.5, -0.5]).repeat(256)
    eps = 0.75
    w = torch.full((512,), 1.0)
    w[0::4], w[1::4], w[2::4] = 1 + 2.0 ** -7, 1 + 3 * 2.0 ** -7, 1.5 + 2.0 ** -7
    x[1, :512] *= 1 + 2.0 ** -7                            # products of 16 bits, not a unit norm
    xb, wb = x.to(torch.bfloat16).cuda(), w.to(torch.bfloat16).cuda()
    pos = torch.zeros(2, dtype=torch.int32).cuda()
    dst = torch.tensor([3, 1]).cuda()
    cfg = csa2.Rope()
    check(xb, wb, pos, dst, 64, cfg, eps, run(xb, wb, pos, dst, 64, cfg, eps=eps))


def test_strided_rows_without_entry():
    g = torch.Generator().manual_seed(4)
    fused = torch.randn(130, 576 + 200, generator=g).to(torch.bfloat16).cuda()
    x = fused[:, 64:640]
    _, w, pos, dst = inputs(130, 192, 8)
    cfg = csa2.Rope()
    check(x, w, pos, dst, 192, cfg, 1e-5, run(x, w, pos, dst, 192, cfg, eps=1e-5, entry=False))


def test_same_bytes_as_the_codec_write():
    x, w, pos, dst = inputs(300, 320, 21)
    cfg = csa2.Rope()
    codes, scales, _, ent = run(x, w, pos, dst, 320, cfg)
    c2, s2 = csa2.fp4_kv_quantize(ent[:, :512].contiguous())
    assert torch.equal(codes[dst], c2) and torch.equal(scales[dst], s2)


def test_rows_with_infinities_and_nan():
    """As the formula has it: the root is infinite or NaN, so the row is 0 where finite, NaN else; other rows are alone."""
    x, w, pos, dst = inputs(9, 64, 31)
    cfg = csa2.Rope()
    clean = run(x, w, pos, dst, 64, cfg)
    x[1, 7] = float("inf")
    x[2, 100] = float("nan")
    x[3, 3], x[3, 500] = -float("inf"), float("nan")
    codes, scales, rope, ent = run(x, w, pos, dst, 64, cfg)
    e = ent[:, :512].float()
    assert torch.isnan(e[1, 7]) and torch.all(e[1, torch.arange(512) != 7] == 0)
    assert torch.isnan(e[2]).all() and torch.isnan(e[3]).all()
    rest = [0, 4, 5, 6, 7, 8]
    assert torch.equal(ent[rest], clean[3][rest])
    for got, want in ((codes, clean[0]), (scales, clean[1]), (rope, clean[2])):
        assert torch.equal(got[dst[rest]], want[dst[rest]])
    assert torch.equal(rope[dst], clean[2][dst])
    c2, s2 = csa2.fp4_kv_quantize(ent[:, :512].contiguous())
    assert torch.equal(codes[dst], c2) and torch.equal(scales[dst], s2)


def test_graph_replay_and_other_stream():
    x, w, pos, dst = inputs(20, 64, 32)
    cfg = csa2.Rope()
    want = run(x, w, pos, dst, 64, cfg)
    planes = [torch.full_like(t, 1) for t in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        csa2.csa2_kv_append(cfg, x, pos, dst, *planes[:3], norm_w=w, entry=planes[3])
    s.synchronize()
    for a, b in zip(planes[:3], want[:3]):
        assert torch.equal(a[dst], b[dst])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        csa2.csa2_kv_append(cfg, x, pos, dst, *planes[:3], norm_w=w, entry=planes[3])
    x2, _, pos2, dst2 = inputs(20, 64, 33)
    x.copy_(x2), pos.copy_(pos2), dst.copy_(dst2)
    g.replay()
    check(x2, w, pos2, dst2, 64, cfg, 1e-6, (*run(x2, w, pos2, dst2, 64, cfg)[:3], planes[3]))
    torch.cuda.synchronize()
    want = run(x2, w, pos2, dst2, 64, cfg)
    for a, b in zip(planes[:3], want[:3]):
        assert torch.equal(a[dst2], b[dst2])
    with pytest.raises(csa2.Csa2Error):                      # the bf16 rows over their own input
        csa2.csa2_kv_append(cfg, x, pos, dst, *planes[:3], norm_w=w, entry=x)


@pytest.mark.parametrize("eps", [1e-24, 2e-27, 1e-30, 1e-33, 1e-36, 1.2e-38, 1e-41, 1.4e-45])
def test_smallest_eps(eps):
    """Rows about as small as sqrt(eps), far above it and far below: every eps above 0, subnormal ones too."""
    x, w, pos, dst = inputs(400, 448, 51)
    middle = np.log2(np.float64(np.float32(eps))) / 2
    lowest = max(middle - 45, -120)                        # the results stay normal bf16 values
    s = torch.exp2(torch.linspace(lowest, middle + 40, 400)).cuda()[:, None]
    x[:, :512] = (x[:, :512].float() * s).to(torch.bfloat16)
    cfg = csa2.Rope()
    check(x, w, pos, dst, 448, cfg, eps, run(x, w, pos, dst, 448, cfg, eps=eps))
