"""What the window-side calls write lies apart from everything that they read: index lists, page tables, weights and the other
attention's results, too (CPU: refused before any CUDA call)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def mod():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300 import csa2
    return csa2


def places(*names):
    return {k: (i + 1) << 40 for i, k in enumerate(names)}


def sides(at, size, mine):
    """Addresses at which a block of `mine` bytes shares its last, its first or all bytes with [at, at + size)."""
    return at + size - 256 if size > 256 else at, at - (mine - 256), at


# 8 tokens of 64 heads, 2 sequences of 17 pages of 40
BATCH, PAGES, POOL, ROWS = 2, 17, 40, 8 * 64
ATTN = places("q", "start", "kv", "table", "ctx", "prev", "prev_lse", "out", "lse", "ws")
READS = {"q": ROWS * 1152, "start": 4 * (BATCH + 1), "kv": POOL * 64 * 1152, "table": BATCH * PAGES * 4, "ctx": 4 * BATCH, "prev": ROWS * 1024,
         "prev_lse": ROWS * 4}
WRITES = {"out": ROWS * 1024, "lse": ROWS * 4}


def attend(mod, **moved):
    a = {k: ctypes.c_void_p(v) for k, v in {**ATTN, **moved}.items()}
    d = mod.Dims(heads=64, max_ctx=1024, max_pages=PAGES, num_pages=POOL)
    return mod._lib.csa2_window_attn_chunk(ctypes.byref(d.c()), BATCH, 8, a["q"], a["start"], a["kv"], a["table"], a["ctx"], 0.1, 128, 0, a["prev"],
                                           a["prev_lse"], a["out"], a["lse"], a["ws"], 1 << 40, None)


@pytest.mark.parametrize("what", ["out", "lse", "ws"])
@pytest.mark.parametrize("over", list(READS) + list(WRITES))
def test_attention_operands(mod, what, over):
    if what == over:
        return
    mine = WRITES.get(what) or mod.window_attn_workspace_size(mod.Dims(heads=64, max_ctx=1024, max_pages=PAGES, num_pages=POOL), BATCH, 8)
    same = {("out", "prev"), ("lse", "prev_lse")}            # joined in place: the whole of it is allowed
    for at in sides(ATTN[over], {**READS, **WRITES}[over], mine):
        if (what, over) in same and at == ATTN[over]:
            continue
        assert attend(mod, **{what: at}) == 1, hex(at)


def test_where_operands_end(mod):
    """A q_start of one more entry than sequences, a page table of all sequences: their last entries count."""
    assert attend(mod, start=ATTN["out"] - 4 * BATCH) == 1
    assert attend(mod, table=ATTN["lse"] - 4 * (BATCH * PAGES - 1)) == 1
    assert attend(mod, ctx=ATTN["ws"] - 4 * (BATCH - 1)) == 1


N, CACHE = 100, 64
ROW = places("x", "w", "pos", "dst", "kv")
ROW_READS = {"x": N * 1152, "w": 1024, "pos": 4 * N, "dst": 8 * N}


@pytest.mark.parametrize("over", list(ROW_READS))
def test_exact_row_operands(mod, over):
    for at in sides(ROW[over], ROW_READS[over], CACHE * 1152):
        a = {k: ctypes.c_void_p(v) for k, v in {**ROW, "kv": at}.items()}
        assert mod._lib.csa2_window_append(mod.Rope().ref(), a["x"], N, 576, a["w"], 1e-6, a["pos"], a["dst"], a["kv"], CACHE, None) == 1, hex(at)


KEY = places("x", "w", "b", "pos", "dst", "k")


@pytest.mark.parametrize("kind,dim,size,row", [(0, 128, 2, 128), (1, 64, 4, 256), (2, 128, 2, 72)])
@pytest.mark.parametrize("over", ["x", "w", "b", "pos", "dst"])
def test_key_operands(mod, kind, dim, size, row, over):
    assert (mod.IDXK_E4M3, mod.IDXK_F32, mod.IDXK_FP4) == (0, 1, 2)
    reads = {"x": N * dim * size, "w": dim * size, "b": dim * size, "pos": 4 * N, "dst": 8 * N}
    for at in sides(KEY[over], reads[over], CACHE * row):
        a = {k: ctypes.c_void_p(v) for k, v in {**KEY, "k": at}.items()}
        assert mod._lib.csa2_idx_k_append(mod.Rope(rot=64).ref(), kind, a["x"], N, dim, 0, 2, a["w"], a["b"], 1e-6, a["pos"], a["dst"], a["k"], CACHE,
                                          None) == 1, hex(at)
