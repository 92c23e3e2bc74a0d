"""GPU rotary positions against the float64 oracle.

Tolerance (derived): the angle is right to 2^-32 turns and then held in fp32
(2^-24 of at most pi: under 2^-22 rad), sine and cosine are good to 2 units
(2^-23), two products and a sum add 3 * 2^-24 of their size: together below
2^-20 (|u| + |v|) m.  A bf16 result adds half a step, 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import prompt as op

pytestmark = pytest.mark.gpu

SCALINGS = {"plain": dict(scaling=csa2.ROPE_PLAIN), "linear": dict(scaling=csa2.ROPE_LINEAR, factor=8.0),
            "parts": dict(scaling=csa2.ROPE_PARTS, factor=16.0, orig_ctx=4096.0, turns_lo=1.0, turns_hi=32.0, mscale=1.25),
            "base": dict(scaling=csa2.ROPE_BASE, factor=4.0)}


def freqs_of(cfg):
    name = {0: "plain", 1: "linear", 2: "parts", 3: "base"}[cfg.scaling]
    return op.rope_frequencies(cfg.rot, cfg.theta, name, cfg.factor, cfg.orig_ctx, cfg.turns_lo, cfg.turns_hi)


def check(cfg, x, pos, y, offset, inverse, before):
    """y against the oracle; channels outside the rotated part bit for bit."""
    a, b = offset, offset + cfg.rot
    xs = before.double().cpu().numpy()
    ref = op.rope(xs[..., a:b], pos.cpu().numpy(), freqs_of(cfg), cfg.layout == csa2.ROPE_HALF, cfg.mscale, inverse)
    got = y.double().cpu().numpy()
    n = cfg.rot // 2
    u, v = (xs[..., a:a + n], xs[..., a + n:b]) if cfg.layout == csa2.ROPE_HALF else (xs[..., a:b:2], xs[..., a + 1:b:2])
    size = (np.abs(u) + np.abs(v)) * cfg.mscale
    size = np.concatenate([size, size], -1) if cfg.layout == csa2.ROPE_HALF else np.repeat(size, 2, -1)
    tol = 2.0 ** -20 * size + (2.0 ** -8 * np.abs(ref) if y.dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(got[..., a:b] - ref) <= tol)
    np.testing.assert_array_equal(got[..., :a], xs[..., :a])
    np.testing.assert_array_equal(got[..., b:], xs[..., b:])


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1, 64, 0, 64), (8, 64, 576, 512, 64), (37, 5, 128, 0, 64), (9, 3, 81, 7, 26),
                                   (17, 2, 2, 0, 2), (3, 16, 256, 0, 256), (2500, 7, 40, 8, 24)])
def test_against_oracle(shape, dtype, half, scaling):
    t, h, dim, offset, rot = shape
    if scaling == "base" and rot == 2:
        rot_cfg = dict(SCALINGS["plain"])
    else:
        rot_cfg = dict(SCALINGS[scaling])
    cfg = csa2.Rope(rot=rot, layout=csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED, **rot_cfg)
    g = torch.Generator().manual_seed(t * 131 + h)
    x = torch.randn(t, h, dim, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 20, (t,), generator=g, dtype=torch.int32).cuda()
    pos[0] = 0 if t > 1 else 1048575
    for inverse in (False, True):
        y = csa2.csa2_rope_apply(cfg, x, pos, offset=offset, inverse=inverse)
        check(cfg, x, pos, y, offset, inverse, x)
        z = x.clone()
        csa2.csa2_rope_apply(cfg, z, pos, y=z, offset=offset, inverse=inverse)
        assert torch.equal(z, y)


def test_far_and_negative_positions():
    cfg = csa2.Rope(rot=64)
    x = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(3)).cuda()
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 2 ** 24 + 1, 123456789, -7], dtype=torch.int32).cuda()
    # the oracle's own 64-bit angles are off by 2^-53 of 2^31 rad (2e-7): both errors are allowed for
    y = csa2.csa2_rope_apply(cfg, x, pos).double().cpu().numpy()
    ref = op.rope(x.double().cpu().numpy(), pos.cpu().numpy(), freqs_of(cfg), False)
    u = np.abs(x.double().cpu().numpy())
    size = np.repeat(u[..., 0::2] + u[..., 1::2], 2, -1)
    assert np.all(np.abs(y - ref) <= (2.0 ** -20 + 2.0 ** -21) * size)


def test_strided_views_and_broadcast_rows():
    """A head slice of a fused projection, head-major output, and one row repeated by stride 0."""
    cfg = csa2.Rope(rot=64)
    g = torch.Generator().manual_seed(5)
    fused = torch.randn(33, 4 * 576 + 24, generator=g).to(torch.bfloat16).cuda()
    x = fused[:, 24:].view(33, 4, 576)
    keep = fused.clone()
    pos = torch.arange(33, dtype=torch.int32).cuda() * 1000
    y = torch.zeros(4, 33, 576, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    csa2.csa2_rope_apply(cfg, x, pos, y=y, offset=512)
    check(cfg, x, pos, y, 512, False, keep[:, 24:].view(33, 4, 576))
    assert torch.equal(fused, keep)
    csa2.csa2_rope_apply(cfg, x, pos, y=x, offset=512)
    assert torch.equal(fused[:, :24], keep[:, :24]) and torch.equal(x, y)
    row = torch.randn(1, 1, 128, generator=g).cuda()
    wide = row.expand(5, 3, 128)
    p5 = torch.arange(5, dtype=torch.int32).cuda()
    out = csa2.csa2_rope_apply(cfg, wide, p5)
    check(cfg, wide, p5, out, 0, False, wide)


def test_gradient_is_the_inverse_and_matches_differences():
    """<g, y(x + e d)> - <g, y(x - e d)> over 2 e equals <inverse(g), d> (y is linear in x)."""
    cfg = csa2.Rope(rot=32, layout=csa2.ROPE_HALF, **SCALINGS["parts"])
    gen = torch.Generator().manual_seed(9)
    x, g, d = (torch.randn(12, 3, 40, generator=gen).cuda() for _ in range(3))
    pos = torch.randint(0, 9000, (12,), generator=gen, dtype=torch.int32).cuda()
    f = lambda z: (csa2.csa2_rope_apply(cfg, z.contiguous(), pos, offset=4).double() * g.double()).sum()
    diff = (f(x + 0.5 * d) - f(x - 0.5 * d)).item()
    grad = csa2.csa2_rope_apply(cfg, g, pos, offset=4, inverse=True)
    dot = (grad.double() * d.double()).sum().item()
    # each of 3 * 12 * 3 * 40 terms is off by at most 2^-20 of (|u| + |v|) m |g|: below 2^-20 * 1440 * 3 * 30
    assert abs(diff - dot) <= 2.0 ** -20 * 1440 * 90


def test_replayed_graph_and_other_stream():
    cfg = csa2.Rope(rot=64)
    x = torch.randn(300, 8, 64, device="cuda")
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    want = csa2.csa2_rope_apply(cfg, x, pos)
    y = torch.zeros_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    csa2.csa2_rope_apply(cfg, x, pos, y=y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        csa2.csa2_rope_apply(cfg, x, pos, y=y)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want * 2)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_same_bits_whatever_the_strides(dtype, half):
    """Rows of odd strides and addresses, in place, and the append's rotary part: the bits of the aligned call."""
    cfg = csa2.Rope(layout=csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED, **SCALINGS["parts"])
    g = torch.Generator().manual_seed(11)
    x = torch.randn(3000, 16, 64, generator=g).to(dtype).cuda()
    pos = torch.randint(0, 1 << 20, (3000,), generator=g, dtype=torch.int32).cuda()
    for inverse in (False, True):
        want = csa2.csa2_rope_apply(cfg, x, pos, inverse=inverse)
        odd = torch.empty(3000, 16, 67, dtype=dtype, device="cuda")[..., 1:65]
        odd.copy_(x)
        assert torch.equal(csa2.csa2_rope_apply(cfg, odd, pos, inverse=inverse), want)
        csa2.csa2_rope_apply(cfg, odd, pos, y=odd, inverse=inverse)
        assert torch.equal(odd, want)
        z = x.clone()
        csa2.csa2_rope_apply(cfg, z, pos, y=z, inverse=inverse)
        assert torch.equal(z, want)
    if dtype is torch.bfloat16:
        n = 3000 * 16
        rows = torch.zeros(n, 576, dtype=dtype, device="cuda")
        rows[:, 512:] = x.view(n, 64)
        dst = torch.arange(n, device="cuda")
        codes, scales = (torch.empty(n, k, dtype=torch.uint8, device="cuda") for k in (256, 32))
        kr = torch.empty(n, 64, dtype=dtype, device="cuda")
        csa2.csa2_kv_append(cfg, rows, pos.repeat_interleave(16), dst, codes, scales, kr)
        assert torch.equal(kr.view(3000, 16, 64), csa2.csa2_rope_apply(cfg, x, pos))
