"""GPU appends of exact rows and of indexer keys against the float64 oracle.

Exact rows: the latent is byte-exact (rounded once from the exact value), the rotary part
within 2^-20 (|u| + |v|) m plus half a bf16 step, as for the FP4 append.

Indexer keys are formed in fp32: sums of 16 terms and 3 levels, products and a root of 2 units
stay within 2^-18 of a value's size (`ow.key_rows`: the row's, where a mean is taken away),
the rotation within 2^-20 of the pair's, inside of that.  Then the format's rounding: E4M3
half a step, 2^-4 of the value or 2^-10 where subnormal; FP4 (from bf16) half a step of the E2M1
grid under the stored scale, which is amax / 6 rounded to E4M3.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import codec as ocodec
from oracle import prompt as op
from oracle import window as ow

pytestmark = pytest.mark.gpu

PARTS = dict(scaling=csa2.ROPE_PARTS, factor=16.0, orig_ctx=4096.0, mscale=1.25)


def freqs_of(cfg):
    return op.rope_frequencies(cfg.rot, cfg.theta, "parts" if cfg.scaling == csa2.ROPE_PARTS else "plain", cfg.factor,
                               cfg.orig_ctx, cfg.turns_lo, cfg.turns_hi)


def places(n, rows, g):
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32).cuda()
    dst = torch.randperm(rows, generator=g)[:n].cuda()
    if n > 5:
        dst[2], dst[4] = -1, rows                          # no row: skipped
    return pos, dst


# ---------------------------------------------------------------------------
# exact rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,rows", [(1, 64), (7, 64), (64, 4096), (1237, 1280), (5000, 5056)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_exact_rows(n, rows, half, norm):
    g = torch.Generator().manual_seed(n)
    x = (torch.randn(n, 576, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).to(torch.bfloat16).cuda()
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda() if norm else None
    pos, dst = places(n, rows, g)
    cfg = csa2.Rope(layout=csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED, **PARTS)
    kv = torch.full((rows, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    csa2.csa2_window_append(cfg, x, pos, dst, kv, norm_w=w)
    x64 = x.double().cpu().numpy()
    lat = op.rms_norm_bf16(x64[:, :512], w.double().cpu().numpy(), np.float64(np.float32(1e-6))) if norm else x64[:, :512]
    ref = op.rope(x64[:, None, 512:], pos.cpu().numpy(), freqs_of(cfg), half, cfg.mscale)[:, 0]
    u, v = (x64[:, 512:544], x64[:, 544:]) if half else (x64[:, 512::2], x64[:, 513::2])
    size = (np.abs(u) + np.abs(v)) * cfg.mscale
    size = np.concatenate([size, size], -1) if half else np.repeat(size, 2, -1)
    d = dst.cpu().numpy()
    keep = (d >= 0) & (d < rows)
    got = kv.double().cpu().numpy()
    np.testing.assert_array_equal(got[d[keep], :512], lat[keep])
    assert np.all(np.abs(got[d[keep], 512:] - ref[keep]) <= (2.0 ** -20 * size + 2.0 ** -8 * np.abs(ref))[keep])
    assert np.all(got[np.setdiff1d(np.arange(rows), d[keep])] == 5.0)


def test_exact_rows_are_the_fp4_appends():
    """The same bits as that call's packed rows, for rows of every size, with infinities and NaN."""
    g = torch.Generator().manual_seed(1)
    n = 600
    x = torch.randn(n, 704, generator=g) * torch.exp2(torch.linspace(-60, 60, n))[:, None]
    x[10, 3], x[11, 8], x[12] = float("inf"), float("nan"), 0.0
    x = x.to(torch.bfloat16).cuda()[:, 64:640]              # strided rows
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(torch.bfloat16).cuda()
    pos, dst = places(n, 640, g)
    for half in (csa2.ROPE_INTERLEAVED, csa2.ROPE_HALF):
        cfg = csa2.Rope(layout=half)
        planes = [torch.zeros(640, k, dtype=torch.uint8, device="cuda") for k in (256, 32, 128)]
        entry = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
        csa2.csa2_kv_append(cfg, x, pos, dst, planes[0], planes[1], planes[2].view(torch.bfloat16), norm_w=w, entry=entry)
        kv = torch.zeros(640, 576, dtype=torch.bfloat16, device="cuda")
        csa2.csa2_window_append(cfg, x, pos, dst, kv, norm_w=w)
        keep = (dst >= 0) & (dst < 640)
        assert torch.equal(kv[dst[keep]].view(torch.int16), entry[keep].view(torch.int16))


# ---------------------------------------------------------------------------
# indexer keys
# ---------------------------------------------------------------------------
KINDS = {"e4m3": csa2.IDXK_E4M3, "fp4": csa2.IDXK_FP4, "fp32": csa2.IDXK_F32}
NORMS = {"none": csa2.IDX_NORM_NONE, "rms": csa2.IDX_NORM_RMS, "layer": csa2.IDX_NORM_LAYER}


def key_inputs(kind, n, seed, norm, mean=0.3, size=None):
    dim, dt = (64, torch.float32) if kind == "fp32" else (128, torch.bfloat16)
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, dim, generator=g) * torch.exp(0.5 * torch.randn(dim, generator=g)) + mean * torch.randn(n, 1, generator=g)
    if size is not None:
        x = x * size[:, None]
    w = (1 + 0.2 * torch.randn(dim, generator=g)).to(dt).cuda() if norm != "none" else None
    b = (0.2 * torch.randn(dim, generator=g)).to(dt).cuda() if norm == "layer" else None
    return x.to(dt).cuda(), w, b, g


def append(kind, x, pos, dst, rows, cfg, offset, norm, w, b, eps=1e-6, fill=0x33):
    size = {"e4m3": 128, "fp4": 72, "fp32": 256}[kind]
    keys = torch.full((rows * size,), fill, dtype=torch.uint8, device="cuda")
    csa2.csa2_idx_k_append(cfg, KINDS[kind], x, pos, dst, keys, rows, offset=offset, norm=NORMS[norm], norm_w=w, norm_b=b, eps=eps)
    return keys


def check_keys(kind, x, pos, dst, rows, cfg, offset, norm, w, b, keys, eps=1e-6, fill=0x33):
    f64 = lambda t: None if t is None else t.double().cpu().numpy()
    y, size = ow.key_rows(f64(x), norm, f64(w), f64(b), np.float64(np.float32(eps)), None if pos is None else pos.cpu().numpy(),
                          None if cfg is None else freqs_of(cfg), cfg is not None and cfg.layout == csa2.ROPE_HALF,
                          1.0 if cfg is None else cfg.mscale, offset)
    tol = 2.0 ** -18 * size
    if norm == "none" and cfg is None:
        tol = 0 * size
    d = dst.cpu().numpy()
    keep = (d >= 0) & (d < rows)
    raw = keys.cpu().numpy()
    rest = np.setdiff1d(np.arange(rows), d[keep])
    y, tol = y[keep], tol[keep]
    if kind == "fp32":
        got = raw.view(np.float32).reshape(rows, 64)
        assert np.all(np.abs(got[d[keep]] - y) <= tol)
        assert np.all(raw.reshape(rows, 256)[rest] == fill)
    elif kind == "e4m3":
        raw = raw.reshape(rows, 128)
        got = ocodec.e4m3_decode(raw)[d[keep]]
        near = np.clip(y, -448, 448)
        assert np.all(np.abs(got - near) <= tol + np.maximum(2.0 ** -4 * np.abs(near), 2.0 ** -10))
        assert np.all(raw[rest] == fill)
    else:
        codes, scales = raw[:rows * 64].reshape(rows, 64), raw[rows * 64:].reshape(rows, 8)
        s = np.repeat(ocodec.e4m3_decode(scales[d[keep]]), 16, 1)
        amax = np.abs(y).reshape(len(y), 8, 16).max(-1)
        wide = tol.reshape(len(y), 8, 16).max(-1) + 2.0 ** -8 * amax
        assert np.all(np.abs(s[:, ::16] - amax / 6) <= np.maximum(2.0 ** -4 * amax / 6, 2.0 ** -10) + wide / 6 * (1 + 2.0 ** -4))
        got = ocodec.dequantize_rows(codes[d[keep]], scales[d[keep]])
        off = tol + 2.0 ** -8 * np.abs(y)                    # of the bf16 row
        r = (np.abs(y) + off) / np.where(s > 0, s, 1)
        step = np.where(r < 2, 0.25, np.where(r < 4, 0.5, 1.0)) * s
        over = np.maximum(np.abs(y) - 6 * s, 0)              # saturated
        assert np.all(np.abs(got - y) <= np.maximum(step, over) + off)
        assert np.all(codes[rest] == fill) and np.all(scales[rest] == fill)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("norm", list(NORMS))
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("n,rows", [(1, 64), (3, 64), (33, 64), (1237, 1280)])
def test_keys(kind, norm, half, n, rows):
    x, w, b, g = key_inputs(kind, n, n + 7, norm)
    pos, dst = places(n, rows, g)
    dim = x.shape[1]
    for offset, rot in ((0, 64), (0, dim), (dim - 32, 32), (6, 20), (1, 2), (3, 38)):
        cfg = csa2.Rope(rot=rot, layout=csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED, **PARTS)
        keys = append(kind, x, pos, dst, rows, cfg, offset, norm, w, b)
        check_keys(kind, x, pos, dst, rows, cfg, offset, norm, w, b, keys)


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("norm", list(NORMS))
def test_keys_without_rotation(kind, norm):
    x, w, b, g = key_inputs(kind, 500, 3, norm)
    pos, dst = places(500, 512, g)
    keys = append(kind, x, None, dst, 512, None, 0, norm, w, b)
    check_keys(kind, x, None, dst, 512, None, 0, norm, w, b, keys)
    if kind == "fp4" and norm == "none":
        want = torch.full_like(keys, 0x33)
        csa2.fp4_idx_k_quantize_scatter(x, want, 512, dst)
        assert torch.equal(keys, want)


@pytest.mark.parametrize("kind", ["e4m3", "fp32"])
@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("eps", [1.0, 1e-5, 1e-12])
def test_keys_of_every_size(kind, norm, eps):
    """Rows from 2^-70 to 2^120, a row of zeros, rows with one large channel, a mean far above the spread."""
    size = torch.exp2(torch.linspace(-70, 120, 400))
    x, w, b, g = key_inputs(kind, 400, 4, norm, mean=30.0 if norm == "layer" else 0.3, size=size)
    x[5] = 0
    x[6, 1:] = 0
    pos, dst = places(400, 448, g)
    cfg = csa2.Rope(rot=32)
    keys = append(kind, x, pos, dst, 448, cfg, 0, norm, w, b, eps=eps)
    check_keys(kind, x, pos, dst, 448, cfg, 0, norm, w, b, keys, eps=eps)


def test_keys_saturate():
    x = torch.full((4, 128), 1000.0)
    x[1], x[2], x[3] = -449.0, 448.0, 2.0 ** -10
    x = x.to(torch.bfloat16).cuda()
    dst = torch.arange(4).cuda()
    keys = append("e4m3", x, None, dst, 4, None, 0, "none", None, None).view(torch.float8_e4m3fn).view(4, 128).float()
    assert torch.all(keys[0] == 448) and torch.all(keys[1] == -448) and torch.all(keys[2] == 448) and torch.all(keys[3] == 0)


def test_keys_strided_rows_and_other_rows_of_a_warp():
    """A row with an infinity leaves the other rows of its warp alone; rows strided."""
    x, w, b, g = key_inputs("e4m3", 40, 9, "layer")
    wide = torch.zeros(40, 200, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:136] = x
    pos, dst = places(40, 64, g)
    cfg = csa2.Rope(rot=64, layout=csa2.ROPE_HALF)
    a = append("e4m3", x, pos, dst, 64, cfg, 0, "layer", w, b)
    assert torch.equal(a, append("e4m3", wide[:, 8:136], pos, dst, 64, cfg, 0, "layer", w, b))
    x[9, 3], x[10, 100] = float("inf"), float("nan")
    c = append("e4m3", x, pos, dst, 64, cfg, 0, "layer", w, b).view(64, 128)
    rest = [r for r in range(64) if r not in (int(dst[9]), int(dst[10]))]
    assert torch.equal(c[rest], a.view(64, 128)[rest])


def test_many_keys():
    x, w, b, g = key_inputs("fp32", 70001, 10, "layer")
    pos, dst = places(70001, 70016, g)
    cfg = csa2.Rope(rot=64, layout=csa2.ROPE_HALF, **PARTS)
    check_keys("fp32", x, pos, dst, 70016, cfg, 0, "layer", w, b, append("fp32", x, pos, dst, 70016, cfg, 0, "layer", w, b))


def test_graph_replay_and_other_stream():
    x, w, b, g = key_inputs("e4m3", 20, 11, "layer")
    pos, dst = places(20, 64, g)
    cfg = csa2.Rope(rot=64)
    want = append("e4m3", x, pos, dst, 64, cfg, 0, "layer", w, b)
    got = torch.full_like(want, 0x33)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = lambda **kw: csa2.csa2_idx_k_append(cfg, csa2.IDXK_E4M3, x, pos, dst, got, 64, norm=csa2.IDX_NORM_LAYER, norm_w=w,
                                               norm_b=b, **kw)
    call(stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x2 = key_inputs("e4m3", 20, 12, "layer")[0]
    x.copy_(x2)
    graph.replay()
    assert torch.equal(got, append("e4m3", x, pos, dst, 64, cfg, 0, "layer", w, b))


def test_refusals():
    x, w, b, g = key_inputs("e4m3", 8, 13, "layer")
    pos, dst = places(8, 64, g)
    keys = torch.zeros(64 * 128, dtype=torch.uint8, device="cuda")
    ok = dict(cfg=csa2.Rope(rot=64), kind=csa2.IDXK_E4M3, x=x, pos=pos, dst_rows=dst, idx_k=keys, cache_rows=64,
              norm=csa2.IDX_NORM_LAYER, norm_w=w, norm_b=b)
    csa2.csa2_idx_k_append(**ok)
    for kw, code in ((dict(kind=7), 1), (dict(x=x.float()), 1), (dict(x=x[:, :64]), 1), (dict(x=x.cpu()), 1),
                     (dict(pos=pos.long()), 1), (dict(pos=None), 1), (dict(cache_rows=65), 1), (dict(norm=3), 1),
                     (dict(norm_w=w.float()), 1), (dict(norm_w=None), 1), (dict(norm=csa2.IDX_NORM_RMS), 1),
                     (dict(norm=csa2.IDX_NORM_NONE), 1), (dict(eps=0.0), 1), (dict(eps=2.0), 1), (dict(offset=65), 2),
                     (dict(cfg=csa2.Rope(rot=130)), 2), (dict(cfg=None, offset=2), 2), (dict(idx_k=x.view(torch.uint8).view(-1)[:1024], cache_rows=8), 1)):
        with pytest.raises(csa2.Csa2Error) as e:
            csa2.csa2_idx_k_append(**{**ok, **kw})
        assert e.value.code == code, kw
    xr = torch.zeros(8, 576, dtype=torch.bfloat16, device="cuda")
    for kw, code in ((dict(kv=xr), 1), (dict(cfg=csa2.Rope(rot=32)), 2), (dict(eps=0.0, norm_w=torch.ones_like(xr[0, :512])), 1),
                     (dict(kv=torch.zeros(64, 576, device="cuda")), 1), (dict(pos=None or pos[:4]), 1)):
        a = dict(cfg=csa2.Rope(), x=xr, pos=pos, dst_rows=dst, kv=torch.zeros(64, 576, dtype=torch.bfloat16, device="cuda"))
        with pytest.raises(csa2.Csa2Error) as e:
            csa2.csa2_window_append(**{**a, **kw})
        assert e.value.code == code, kw
