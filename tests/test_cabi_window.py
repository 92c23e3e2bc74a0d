"""Host argument checks of the window-side calls (no GPU: every case is refused, or is
an empty call, before any CUDA call)."""
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
FAR = P(0x70000000000)


def rows(mod, cfg=None, x=FAKE, n=4, stride=576, w=FAKE, eps=1e-6, pos=FAKE, dst=FAKE, kv=FAR, cache=64):
    return mod._lib.csa2_window_append((cfg or mod.Rope()).ref(), x, n, stride, w, eps, pos, dst, kv, cache, None)


def test_row_refusals(mod):
    assert rows(mod, n=0) == 0
    assert rows(mod, mod.Rope(rot=32)) == 2 and rows(mod, mod.Rope(theta=0.5)) == 1
    assert rows(mod, n=-1) == 1 and rows(mod, cache=-1) == 1
    for eps in (0.0, -1.0, 1.5, float("nan"), float("inf")):
        assert rows(mod, eps=eps) == 1
    for k in ("x", "pos", "dst", "kv"):
        assert rows(mod, **{k: None}) == 1, k
    for k, bad in (("x", 0x10008), ("pos", 0x10002), ("dst", 0x10004), ("kv", 0x70000000008), ("w", 0x10008)):
        assert rows(mod, **{k: P(bad)}) == 1, k
    assert rows(mod, stride=575) == 1 and rows(mod, stride=580) == 1 and rows(mod, stride=0) == 1
    assert rows(mod, kv=FAKE) == 1 and rows(mod, kv=P(FAKE.value + 3 * 1152)) == 1       # over x
    assert rows(mod, n=1 << 60, stride=1 << 20) == 2 and rows(mod, cache=1 << 60) == 2


def keys(mod, cfg="r", kind=0, x=FAKE, n=4, stride=128, offset=0, norm=2, w=FAKE, b=FAKE, eps=1e-6, pos=FAKE, dst=FAKE, k=FAR,
         cache=64):
    cfg = mod.Rope(rot=64) if cfg == "r" else cfg
    return mod._lib.csa2_idx_k_append(None if cfg is None else cfg.ref(), kind, x, n, stride, offset, norm, w, b, eps, pos, dst,
                                      k, cache, None)


def test_key_refusals(mod):
    assert keys(mod, n=0) == 0 and keys(mod, None, n=0, pos=None) == 0
    assert keys(mod, mod.Rope(rot=3)) == 2 and keys(mod, mod.Rope(rot=130)) == 2 and keys(mod, mod.Rope(rot=66), 1) == 2
    assert keys(mod, offset=65) == 2 and keys(mod, offset=-1) == 2 and keys(mod, None, offset=1) == 2
    assert keys(mod, mod.Rope(theta=0.5)) == 1
    assert keys(mod, kind=3) == 1 and keys(mod, kind=-1) == 1 and keys(mod, norm=3) == 1 and keys(mod, norm=-1) == 1
    assert keys(mod, n=-1) == 1 and keys(mod, cache=-1) == 1
    for eps in (0.0, 1e-13, 1.5, float("nan")):
        assert keys(mod, eps=eps) == 1
    assert keys(mod, w=None) == 1 and keys(mod, norm=0) == 1 and keys(mod, norm=0, w=None) == 1 and keys(mod, norm=1) == 1
    for k in ("x", "pos", "dst", "k"):
        assert keys(mod, **{k: None}) == 1, k
    for k, bad in (("x", 0x10008), ("pos", 0x10002), ("dst", 0x10004), ("k", 0x70000000008), ("w", 0x10008), ("b", 0x10008)):
        assert keys(mod, **{k: P(bad)}) == 1, k
    assert keys(mod, stride=127) == 1 and keys(mod, stride=132) == 1
    assert keys(mod, kind=1, stride=66) == 1 and keys(mod, kind=1, stride=63) == 1
    assert keys(mod, k=FAKE) == 1 and keys(mod, n=1 << 60, stride=1 << 20) == 2 and keys(mod, cache=1 << 60) == 2


def attend(mod, d, batch=2, total=8, q=FAKE, start=FAKE, kv=FAKE, table=None, ctx=FAKE, scale=0.1, window=128, sinks=0,
           prev=None, prev_lse=None, out=FAR, lse=FAKE, ws=P(0x100000), ws_bytes=1 << 40):
    return mod._lib.csa2_window_attn_chunk(ctypes.byref(d.c()), batch, total, q, start, kv, table, ctx, scale, window, sinks,
                                           prev, prev_lse, out, lse, ws, ws_bytes, None)


def test_attention_refusals(mod):
    d = mod.Dims(max_ctx=1024)
    need = mod.window_attn_workspace_size(d, 2, 8)
    assert attend(mod, d, batch=0) == 0 and attend(mod, d, total=0) == 0
    assert attend(mod, d, batch=-1) == 1 and attend(mod, d, total=-1) == 1
    for kw in (dict(heads=0), dict(heads=65), dict(max_ctx=0), dict(max_ctx=(1 << 20) + 1)):
        assert attend(mod, mod.Dims(**{"max_ctx": 1024, **kw})) == 2
        with pytest.raises(mod.Csa2Error):
            mod.window_attn_workspace_size(mod.Dims(**{"max_ctx": 1024, **kw}), 2, 8)
    assert attend(mod, d, total=1 << 26) == 2                      # 2^32 rows
    assert attend(mod, d, batch=(1 << 20) + 1) == 2
    assert attend(mod, mod.Dims(max_ctx=1 << 20), batch=2048) == 2                # 2^31 cache rows
    assert attend(mod, d, window=0) == 1 and attend(mod, d, window=-1) == 1 and attend(mod, d, sinks=-1) == 1
    assert attend(mod, d, window=(1 << 20) + 1) == 2 and attend(mod, d, sinks=(1 << 20) + 1) == 2
    for s in (float("nan"), float("inf"), -float("inf")):
        assert attend(mod, d, scale=s) == 1
    for k in ("q", "start", "kv", "ctx", "out", "lse", "ws"):
        assert attend(mod, d, **{k: None}) == 1, k
    for k, bad in (("q", 0x10008), ("start", 0x10002), ("kv", 0x10008), ("ctx", 0x10002), ("out", 0x70000000008), ("lse", 0x10002),
                   ("ws", 0x100010)):
        assert attend(mod, d, **{k: P(bad)}) == 1, k
    assert attend(mod, d, ws_bytes=need - 1) == 3
    assert attend(mod, d, table=FAKE) == 1                         # a page table without pages
    assert attend(mod, mod.Dims(max_ctx=1024, max_pages=16, num_pages=16), table=P(0x10002)) == 1
    assert attend(mod, d, prev=FAKE) == 1 and attend(mod, d, prev_lse=FAKE) == 1
    assert attend(mod, d, out=FAKE) == 1                           # over the queries
    assert attend(mod, d, prev=P(FAR.value + 1024), prev_lse=FAR) == 1          # over the outputs, not the same place
    assert attend(mod, d, prev=P(FAR.value + (1 << 30)), prev_lse=P(FAKE.value + 4)) == 1


def test_binding_refuses_wrong_tensors(mod):
    """Types, shapes and devices that the C call cannot see (host tensors are refused as well)."""
    x, pos, dst = torch.zeros(4, 576, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64)
    kv = torch.zeros(64, 576, dtype=torch.bfloat16)
    k, idx = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(64 * 128, dtype=torch.uint8)
    E = mod.IDXK_E4M3
    for bad in (lambda: mod.csa2_window_append(mod.Rope(), x.float(), pos, dst, kv),
                lambda: mod.csa2_window_append(mod.Rope(), x[:, :575], pos, dst, kv),
                lambda: mod.csa2_window_append(mod.Rope(), x, pos[:3], dst, kv),
                lambda: mod.csa2_window_append(mod.Rope(), x, pos, dst.int(), kv),
                lambda: mod.csa2_window_append(mod.Rope(), x, pos, dst, kv),
                lambda: mod.csa2_idx_k_append(None, E, k, None, dst, idx, 63), lambda: mod.csa2_idx_k_append(None, E, k, None, dst, idx, 64),
                lambda: mod.csa2_idx_k_append(None, mod.IDXK_F32, k, None, dst, idx, 32),
                lambda: mod.csa2_idx_k_append(None, E, k, None, dst, idx, 64, offset=1 << 32),
                lambda: mod.csa2_idx_k_append(None, E + (1 << 32), k, None, dst, idx, 64)):
        with pytest.raises(mod.Csa2Error) as e:
            bad()
        assert e.value.code == 1
    for batch in (2 ** 32 + 1, -2 ** 32 + 1):
        with pytest.raises(mod.Csa2Error):
            mod.window_attn_workspace_size(mod.Dims(max_ctx=1024), batch, 8)
