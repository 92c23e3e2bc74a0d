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
