"""What the prompt-side runner hands to the library's calls (CPU: the calls are recorded)."""
import pytest
import torch


@pytest.fixture
def pre(monkeypatch):
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300 import csa2, prefill
    calls = []
    for name in ("csa2_rope_apply", "csa2_window_append", "csa2_idx_k_append", "csa2_kv_append", "csa2_dense_attn_chunk",
                 "csa2_window_attn_chunk"):
        monkeypatch.setattr(csa2, name, lambda *a, _name=name, **kw: calls.append((_name, a, kw)))
    prefill.calls = calls
    return prefill


def chunk(pre, exact, tokens=4, batch=1, table=None, **kw):
    from compressed_sparse_attention_fp4_gb300 import csa2
    e, q = torch.empty(0), torch.empty(tokens, 16, 576)
    dims = csa2.Dims(heads=16, max_ctx=256, max_pages=4 if table is not None else 0, num_pages=9 if table is not None else 0)
    return pre.ChunkBuffers(dims, batch, csa2.Rope(), e, e, e, table, e, e, q, e, e, e, 1.0, exact=exact, **kw)


def attention(pre):
    (_, args, _), = [c for c in pre.calls if c[0] == "csa2_window_attn_chunk"]
    return args[0], args[5]                                  # dims, page table


def test_exact_rows_follow_the_chunks_pages(pre):
    """Without dimensions and a table of its own the window cache has the chunk's, pages included."""
    e, table = torch.empty(0), torch.zeros(1, 4, dtype=torch.int32)
    cb = chunk(pre, pre.ExactRows(e, e, 128), table=table)
    pre.run_chunk(cb)
    dims, got = attention(pre)
    assert dims is cb.dims and got is table


def test_exact_rows_of_their_own(pre):
    from compressed_sparse_attention_fp4_gb300 import csa2
    e, table, other = torch.empty(0), torch.zeros(1, 4, dtype=torch.int32), torch.ones(1, 4, dtype=torch.int32)
    own = csa2.Dims(heads=16, max_ctx=256)
    for exact, want in ((pre.ExactRows(e, e, 128, page_table=other), (None, other)), (pre.ExactRows(e, e, 128, dims=own), (own, None)),
                        (pre.ExactRows(e, e, 128, dims=own, page_table=other), (own, other))):
        pre.calls.clear()
        cb = chunk(pre, exact, table=table)
        pre.run_chunk(cb)
        dims, got = attention(pre)
        assert dims is (want[0] or cb.dims) and got is want[1]


def test_a_cache_without_pages(pre):
    e = torch.empty(0)
    cb = chunk(pre, pre.ExactRows(e, e, 128))
    pre.run_chunk(cb)
    assert attention(pre) == (cb.dims, None)


@pytest.mark.parametrize("window,ring,tokens,longest,fits", [
    (128, 128, 1, 0, True), (128, 128, 2, 0, False), (128, 192, 65, 0, True), (128, 192, 66, 0, False), (1, 64, 64, 0, True),
    (1, 64, 65, 0, False), (100, 192, 500, 93, True), (100, 192, 500, 94, False), (128, 6 * 64, 256, 256, True), (128, 0, 5000, 0, True),
    (128, 200, 4, 0, False), (128, -64, 4, 0, False)])
def test_a_chunk_that_its_ring_does_not_hold_is_refused(pre, window, ring, tokens, longest, fits):
    """Before anything is enqueued: its first tokens would read rows that its last ones have taken."""
    from compressed_sparse_attention_fp4_gb300 import csa2
    e = torch.empty(0)
    cb = chunk(pre, pre.ExactRows(e, e, window, ring=ring), tokens=tokens, longest=longest, batch=8 if longest else 1)
    if fits:
        pre.run_chunk(cb)
        assert "csa2_window_attn_chunk" in [c[0] for c in pre.calls]
    else:
        with pytest.raises(csa2.Csa2Error, match="run_chunk"):
            pre.run_chunk(cb)
        assert not pre.calls


@pytest.mark.parametrize("window,ring", [(1, 64), (37, 128), (128, 192)])
def test_the_longest_chunk_of_a_ring_is_just_that(window, ring):
    """Positions that the chunk writes and those that its tokens see keep places of their own up to it, and not beyond."""
    for n, fits in ((ring - window + 1, True), (ring - window + 2, False)):
        c = 1000
        live = set(range(c - n - window + 1, c))              # seen by some new token, or new
        assert (len({t % ring for t in live}) == len(live)) == fits
