"""New outputs of calls on another stream than the current one come from that stream's memory."""
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2

pytestmark = pytest.mark.gpu


def calls():
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    n = 1000
    x = torch.randn(n, 3, 128, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    rows = torch.randn(n, 512, generator=g, device="cuda").to(torch.bfloat16)
    codes, scales = csa2.fp4_kv_quantize(rows)
    cfg = csa2.Rope()
    return {"rope": lambda s: (csa2.csa2_rope_apply(cfg, x, pos, stream=s),),
            "quantize": lambda s: csa2.fp4_kv_quantize(rows, stream=s),
            "dequantize": lambda s: (csa2.fp4_kv_dequantize(codes, scales, stream=s),)}


@pytest.mark.parametrize("name", ["rope", "quantize", "dequantize"])
def test_new_outputs_are_not_blocks_of_the_current_stream(name):
    f = calls()[name]
    want = f(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    # blocks of the outputs' sizes that work on the current stream might still use: freed, so the next to be given out there
    old = [torch.empty_like(t) for t in want]
    taken = {t.data_ptr() for t in old}
    del old
    got = f(s)
    mine = {t.data_ptr() for t in got}
    assert not taken & mine
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # and freed, they are not given to the current stream while the other may still write them
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    assert not mine & {torch.empty(sh, dtype=dt, device="cuda").data_ptr() for sh, dt in shapes}
