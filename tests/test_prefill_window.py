"""Rows of a decode step's window for a chunk's tokens (CPU), and the runner's check of them."""
import pytest
import torch


@pytest.fixture(scope="module")
def pre():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300 import prefill
    return prefill


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def test_newest_tokens_stay(pre):
    # positions 3 .. 9 and 0 .. 1: of the first the newest four
    rows = pre.window_rows(i32([10, 2]), i32([0, 7, 9]), 4)
    assert rows.dtype == torch.int64
    assert rows.tolist() == [-1, -1, -1, 2, 3, 0, 1, 4, 5]


def test_padding_and_more_tokens_than_context(pre):
    rows = pre.window_rows(i32([5, 2]), i32([1, 2, 5]), 3, total=7)
    assert rows.tolist() == [-1, 4 % 3, -1, 3, 4, -1, -1]


def test_no_sequences(pre):
    assert pre.window_rows(i32([]), i32([0]), 4, total=2).tolist() == [-1, -1]


def test_rows_differ(pre):
    ctx, start = i32([1000, 3, 0, 129]), i32([0, 900, 903, 903, 1032])
    rows = pre.window_rows(ctx, start, 128)
    rows = rows[rows >= 0]
    assert len(set(rows.tolist())) == len(rows) == 128 + 3 + 128
    assert rows.max() < 4 * 128


def test_window_of_nothing_is_refused(pre):
    from compressed_sparse_attention_fp4_gb300 import csa2
    with pytest.raises(csa2.Csa2Error):
        pre.window_rows(i32([5]), i32([0, 1]), 0)


def test_a_decode_window_needs_its_rows(pre):
    from compressed_sparse_attention_fp4_gb300 import csa2
    e = torch.empty(0)
    cb = pre.ChunkBuffers(csa2.Dims(), 0, csa2.Rope(), e, e, e, None, e, e, e, e, e, e, 1.0,
                          exact=pre.ExactRows(e, e, 128, swa=e))
    with pytest.raises(csa2.Csa2Error, match="run_chunk"):
        pre.run_chunk(cb)
