"""Planes of an FP4 indexer-K buffer: views of its elements, however the buffer lies in memory (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def mod():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300 import csa2
    return csa2


ROWS = 5


def buffers():
    wide = torch.arange(3 * ROWS * 72, dtype=torch.int32)
    return {"whole": wide[:ROWS * 72], "behind an offset": wide[11:11 + ROWS * 72], "every second byte": wide[1::2][:ROWS * 72],
            "a column": wide.view(ROWS * 72, 3)[:, 1], "rows of a wider buffer": wide.view(3, ROWS * 72)[1].view(ROWS, 72),
            "two dimensions, strided": wide[::3].view(ROWS, 72), "longer than its rows": wide}


@pytest.mark.parametrize("name", list(buffers()))
def test_planes_are_the_buffers_elements(mod, name):
    buf = buffers()[name]
    codes, scales = mod.fp4_idx_k_planes(buf, ROWS)
    flat = buf.reshape(-1)
    assert torch.equal(codes, flat[:ROWS * 64].view(ROWS, 64))
    assert torch.equal(scales, flat[ROWS * 64:ROWS * 72].view(ROWS, 8))
    codes[1, 2], scales[3, 4] = -7, -8                 # views, not copies
    assert flat[64 + 2] == -7 and flat[ROWS * 64 + 3 * 8 + 4] == -8


def test_no_rows_and_short_buffers(mod):
    codes, scales = mod.fp4_idx_k_planes(torch.empty(0, dtype=torch.uint8), 0)
    assert codes.shape == (0, 64) and scales.shape == (0, 8)
    with pytest.raises(mod.Csa2Error):
        mod.fp4_idx_k_planes(torch.zeros(ROWS * 72 - 1, dtype=torch.uint8), ROWS)
