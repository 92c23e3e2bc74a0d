"""Host argument checks of the prompt-side calls (no GPU: every case is refused, or
is an empty call, before any CUDA call)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def mod():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300 import csa2
    return csa2


P = ctypes.c_void_p
FAKE = P(0x10000)                 # never dereferenced: validation fails first


def rope(mod, cfg=None, dtype=0, x=FAKE, y=P(0x9000000), pos=FAKE, tokens=4, heads=2, dim=128, offset=0, xs=(256, 128),
         ys=(256, 128), inverse=0):
    c = (cfg or mod.Rope()).ref()
    return mod._lib.csa2_rope_apply(c, dtype, x, y, pos, tokens, heads, dim, offset, *xs, *ys, inverse, None)


def test_rope_refusals(mod):
    R = mod.Rope
    assert rope(mod, tokens=0) == 0 and rope(mod, heads=0) == 0                  # empty calls
    for cfg in (R(rot=3), R(rot=0), R(rot=258), R(rot=-2)):
        assert rope(mod, cfg) == 2
    for cfg in (R(layout=2), R(scaling=4), R(theta=1.0), R(theta=float("inf")), R(theta=float("nan")), R(mscale=float("nan")),
                R(scaling=mod.ROPE_LINEAR, factor=0.5), R(scaling=mod.ROPE_BASE, factor=float("nan")),
                R(scaling=mod.ROPE_PARTS, factor=4.0, orig_ctx=0.0),
                R(scaling=mod.ROPE_PARTS, factor=4.0, orig_ctx=4096.0, turns_lo=32.0, turns_hi=32.0),
                R(scaling=mod.ROPE_PARTS, factor=4.0, orig_ctx=4096.0, turns_lo=-1.0)):
        assert rope(mod, cfg) == 1
    assert mod._lib.csa2_rope_apply(None, 0, FAKE, FAKE, FAKE, 1, 1, 64, 0, 64, 64, 64, 64, 0, None) == 1
    assert rope(mod, dtype=2) == 1 and rope(mod, inverse=2) == 1
    assert rope(mod, offset=65) == 2 and rope(mod, offset=-1) == 2 and rope(mod, dim=0) == 2
    assert rope(mod, tokens=-1) == 2 and rope(mod, heads=-1) == 2 and rope(mod, heads=65536, dim=64) == 2
    for kw in (dict(x=None), dict(y=None), dict(pos=None), dict(x=P(0x10001)), dict(pos=P(0x10002)), dict(dtype=1, y=P(0x9000002))):
        assert rope(mod, **kw) == 1
    # output rows that overlap, negative strides
    for kw in (dict(ys=(256, 127)), dict(ys=(255, 128)), dict(ys=(0, 128)), dict(xs=(-256, 128)), dict(xs=(256, -1))):
        assert rope(mod, **kw) == 1
    # in place with other strides; buffers that overlap
    assert rope(mod, y=FAKE, ys=(512, 128)) == 1
    assert rope(mod, y=P(0x10010)) == 1


def append(mod, cfg=None, x=FAKE, n=4, stride=576, w=FAKE, eps=1e-6, pos=FAKE, dst=FAKE, codes=FAKE, scales=FAKE, kr=FAKE,
           rows=64, entry=None):
    return mod._lib.csa2_kv_append((cfg or mod.Rope()).ref(), x, n, stride, w, eps, pos, dst, codes, scales, kr, rows, entry, None)


def test_append_refusals(mod):
    assert append(mod, n=0) == 0
    assert append(mod, mod.Rope(rot=32)) == 2
    assert append(mod, mod.Rope(theta=0.5)) == 1
    assert append(mod, n=-1) == 1 and append(mod, rows=-1) == 1
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert append(mod, eps=eps) == 1
    for k in ("x", "pos", "dst", "codes", "scales", "kr"):
        assert append(mod, **{k: None}) == 1, k
    for k, bad in (("x", 0x10008), ("pos", 0x10002), ("dst", 0x10004), ("codes", 0x10008), ("scales", 0x10001), ("kr", 0x10008),
                   ("w", 0x10008), ("entry", 0x10008)):
        assert append(mod, **{k: P(bad)}) == 1, k
    assert append(mod, stride=575) == 1 and append(mod, stride=580) == 1 and append(mod, stride=0) == 1


def dense(mod, d, batch=2, total=8, q=FAKE, start=FAKE, codes=FAKE, scales=FAKE, kr=FAKE, table=None, ctx=FAKE, scale=0.1,
          window=0, flags=0, out=FAKE, lse=FAKE, ws=P(0x100000), ws_bytes=1 << 40):
    return mod._lib.csa2_dense_attn_chunk(ctypes.byref(d.c()), batch, total, q, start, codes, scales, kr, table, ctx, scale,
                                          window, flags, out, lse, ws, ws_bytes, None)


def test_dense_refusals(mod):
    d = mod.Dims(max_ctx=1024)
    need = mod.dense_attn_workspace_size(d, 2, 8)
    assert dense(mod, d, batch=0) == 0 and dense(mod, d, total=0) == 0
    assert dense(mod, d, batch=-1) == 1 and dense(mod, d, total=-1) == 1
    for kw in (dict(heads=0), dict(heads=65), dict(max_ctx=0), dict(max_ctx=(1 << 20) + 1)):
        assert dense(mod, mod.Dims(**{"max_ctx": 1024, **kw})) == 2
        with pytest.raises(mod.Csa2Error):
            mod.dense_attn_workspace_size(mod.Dims(**{"max_ctx": 1024, **kw}), 2, 8)
    assert dense(mod, d, total=1 << 26) == 2                      # 2^32 rows
    assert dense(mod, d, batch=(1 << 20) + 1) == 2
    assert dense(mod, mod.Dims(max_ctx=1 << 20), batch=2048) == 2                # 2^31 cache rows
    assert dense(mod, d, window=-1) == 1 and dense(mod, d, flags=2) == 1
    assert dense(mod, d, window=5, flags=mod.DENSE_ALL_POSITIONS) == 1
    for s in (float("nan"), float("inf"), -float("inf")):
        assert dense(mod, d, scale=s) == 1
    for k in ("q", "start", "codes", "scales", "kr", "ctx", "out", "lse", "ws"):
        assert dense(mod, d, **{k: None}) == 1, k
    for k, bad in (("q", 0x10008), ("start", 0x10002), ("codes", 0x10008), ("scales", 0x10008), ("kr", 0x10008), ("ctx", 0x10002),
                   ("out", 0x10008), ("lse", 0x10002), ("ws", 0x100010)):
        assert dense(mod, d, **{k: P(bad)}) == 1, k
    assert dense(mod, d, ws_bytes=need - 1) == 3
    assert dense(mod, d, table=FAKE) == 1                         # a page table without pages
    assert dense(mod, mod.Dims(max_ctx=1024, max_pages=16, num_pages=16), table=P(0x10002)) == 1
    assert need < mod.dense_attn_workspace_size(d, 2, 100000) and mod.dense_attn_workspace_size(d, 0, 0) > 0


def test_binding_refuses_wrong_tensors(mod):
    """Types, shapes and devices that the C call cannot see (host tensors are refused as well)."""
    x = torch.zeros(4, 2, 64)
    pos = torch.zeros(4, dtype=torch.int32)
    for bad in (lambda: mod.csa2_rope_apply(mod.Rope(), x, pos.long()), lambda: mod.csa2_rope_apply(mod.Rope(), x.double(), pos),
                lambda: mod.csa2_rope_apply(mod.Rope(), x, pos[:3]), lambda: mod.csa2_rope_apply(mod.Rope(), x.transpose(1, 2), pos),
                lambda: mod.csa2_rope_apply(mod.Rope(), x[0], pos), lambda: mod.csa2_rope_apply(mod.Rope(), x, pos, y=x.half()),
                lambda: mod.csa2_rope_apply(mod.Rope(), x, pos)):
        with pytest.raises(mod.Csa2Error) as e:
            bad()
        assert e.value.code == 1


def test_append_limits_of_eps_and_overlap(mod):
    for eps in (1.5, 1e30):
        assert append(mod, eps=eps) == 1
    assert append(mod, n=4, entry=FAKE) == 1                      # over x itself
    assert append(mod, n=4, entry=P(FAKE.value + 3 * 1152)) == 1  # within its last row
    assert append(mod, n=4, entry=P(FAKE.value - 16 if FAKE.value > 16 else 16)) == 1
    assert append(mod, n=1 << 50, entry=P(1 << 40)) in (1, 2)


def test_rope_configurations_copy_and_pickle(mod):
    import copy
    import pickle
    r = mod.Rope(rot=32, scaling=mod.ROPE_PARTS, factor=4.0, orig_ctx=4096.0, layout=mod.ROPE_HALF)
    for c in (copy.deepcopy(r), pickle.loads(pickle.dumps(r)), copy.copy(r)):
        assert c == r and c._c.rot == 32 and c._c.orig_ctx == 4096.0 and c.ref() is not None


@pytest.mark.parametrize("paged", [False, True])
def test_cache_rows_of_padded_batches(mod, paged):
    """Every token's row by counting, with padding before, behind and empty sequences."""
    from compressed_sparse_attention_fp4_gb300 import prefill
    ctx = torch.tensor([5, 130, 0, 2, 64], dtype=torch.int32)
    start = torch.tensor([2, 5, 9, 9, 13, 14], dtype=torch.int32)      # the fourth has 4 tokens, 2 positions
    table = torch.tensor([[7, 0, 0], [3, 9, 1], [0, 0, 0], [4, 0, 0], [2, 0, 0]], dtype=torch.int32) if paged else None
    pos, rows = prefill.cache_rows(ctx, start, table, max_ctx=192, total=17)
    assert pos.dtype == torch.int32 and rows.dtype == torch.int64 and len(pos) == len(rows) == 17
    want = [-1] * 17
    for b in range(5):
        n = int(start[b + 1] - start[b])
        for i in range(n):
            p = int(ctx[b]) - n + i
            if p >= 0:
                want[int(start[b]) + i] = int(table[b, p // 64]) * 64 + p % 64 if paged else b * 192 + p
                assert int(pos[int(start[b]) + i]) == p
    assert rows.tolist() == want
    short = prefill.cache_rows(ctx, start, table, max_ctx=192)
    assert len(short[0]) == 14 and short[1].tolist() == want[:14]


def test_numbers_past_32_bits_are_refused(mod):
    """Not cut to another number that the call would take."""
    for kw in (dict(rot=2 ** 32 + 64), dict(layout=2 ** 32), dict(scaling=2 ** 32 + 1), dict(rot=-2 ** 32 + 64)):
        with pytest.raises(mod.Csa2Error):
            mod.Rope(**kw)
    for batch in (2 ** 32 + 1, -2 ** 32 + 1):
        with pytest.raises(mod.Csa2Error):
            mod.dense_attn_workspace_size(mod.Dims(max_ctx=1024), batch, 8)
