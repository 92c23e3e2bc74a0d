"""Cache rows of a chunk's tokens (CPU): lengths past a sequence's rows, empty batches, padding, bad starts."""
import pytest
import torch


@pytest.fixture(scope="module")
def rows_of():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300.prefill import cache_rows
    return cache_rows


def i32(v):
    return torch.tensor(v, dtype=torch.int32)


def test_positions_behind_the_pages_have_no_row(rows_of):
    table = i32([[3, 1], [2, 0]])
    pos, rows = rows_of(i32([130, 128]), i32([0, 4, 6]), table)
    assert pos.tolist() == [126, 127, 128, 129, 126, 127]
    assert rows.tolist() == [64 + 62, 64 + 63, -1, -1, 62, 63]


def test_positions_behind_max_ctx_are_not_the_next_sequences_rows(rows_of):
    pos, rows = rows_of(i32([101, 3]), i32([0, 3, 6]), max_ctx=100)
    assert pos.tolist() == [98, 99, 100, 0, 1, 2]
    assert rows.tolist() == [98, 99, -1, 100, 101, 102]


def test_sequences_without_a_table_need_max_ctx(rows_of):
    from compressed_sparse_attention_fp4_gb300 import csa2
    with pytest.raises(csa2.Csa2Error):
        rows_of(i32([5, 5]), i32([0, 1, 2]))
    pos, rows = rows_of(i32([5]), i32([0, 2]))                      # one sequence: its rows are the cache's
    assert rows.tolist() == [3, 4]
    with pytest.raises(csa2.Csa2Error):
        rows_of(i32([5, 5]), i32([0, 1]), max_ctx=64)


def test_empty_batches_and_tables(rows_of):
    for table in (None, torch.zeros(0, 4, dtype=torch.int32)):
        pos, rows = rows_of(i32([]), i32([0]), table, total=3)
        assert pos.tolist() == [0, 0, 0] and rows.tolist() == [-1, -1, -1]
        assert pos.dtype is torch.int32 and rows.dtype is torch.int64
    assert rows_of(i32([2]), i32([0, 2]), torch.zeros(1, 0, dtype=torch.int32))[1].tolist() == [-1, -1]


def test_starts_that_fall_back_and_padding_have_no_row(rows_of):
    table = i32([[0, 1], [2, 3], [4, 5]])
    _, rows = rows_of(i32([10, 10, 10]), i32([0, 3, 1, 4]), table, total=6)
    own = {0: range(7, 10), 2: range(256 + 7, 256 + 10)}            # sequence 0's tokens, or sequence 2's; never another position
    assert all(r == -1 or r in own[0] or r in own[2] for r in rows.tolist())
    assert rows.tolist()[4:] == [-1, -1]
    pos, rows = rows_of(i32([1, 0, 2]), i32([2, 3, 3, 5]), table, total=7)
    assert pos.tolist() == [0, 0, 0, 0, 1, 0, 0]
    assert rows.tolist() == [-1, -1, 0, 256, 257, -1, -1]
