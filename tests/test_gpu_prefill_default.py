"""A window cache that has the chunk's own pages (GPU): the same bits as with its dimensions and table written out."""
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2, prefill
from tests.test_gpu_prefill_window import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [16, 64])
def test_the_chunks_pages_are_the_windows(H):
    lens, results = [200, 333], []
    for own in (False, True):
        lay = Layer(lens, H, 7)
        for take in ([150, 300], [50, 33]):
            cb = lay.chunk(take)
            cb.exact = prefill.ExactRows(lay.kv, cb.dst_rows, 128, dims=lay.dims if own else None,
                                         page_table=lay.d_table if own else None)
            cb.allocate_outputs()
            prefill.run_chunk(cb)
            torch.cuda.synchronize()
            assert csa2.get_device_status(cb.ws) == 0 and csa2.get_device_status(cb.exact.ws) == 0
            assert bool(torch.isfinite(cb.out).all())         # rows that were not written hold NaN
            results.append((cb.out.clone(), cb.lse.clone()))
            lay.done = [d + t for d, t in zip(lay.done, take)]
    for a, b in zip(results[:2], results[2:]):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
