"""The window attention's outputs lie apart from what the call reads, its workspace and each other (CPU: refused before any
CUDA call); joined in place, out and lse are the other attention's own."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def mod():
    from compressed_sparse_attention_fp4_gb300 import build
    build.build()
    from compressed_sparse_attention_fp4_gb300 import csa2
    return csa2


AT = {k: (i + 1) << 36 for i, k in enumerate(("q", "start", "kv", "ctx", "out", "lse", "prev", "prev_lse", "ws"))}
# bytes of each: 8 tokens of 64 heads, 2 sequences of 1,024 rows
SIZE = {"q": 8 * 64 * 1152, "kv": 2 * 1024 * 1152, "out": 8 * 64 * 1024, "lse": 8 * 64 * 4, "prev": 8 * 64 * 1024, "prev_lse": 8 * 64 * 4}


def attend(mod, **moved):
    a = {k: ctypes.c_void_p(v) for k, v in {**AT, **moved}.items()}
    d = mod.Dims(heads=64, max_ctx=1024)
    return mod._lib.csa2_window_attn_chunk(ctypes.byref(d.c()), 2, 8, a["q"], a["start"], a["kv"], None, a["ctx"], 0.1, 128, 0, a["prev"],
                                           a["prev_lse"], a["out"], a["lse"], a["ws"], 1 << 40, None)


@pytest.mark.parametrize("what,over", [("out", "q"), ("out", "kv"), ("out", "lse"), ("lse", "q"), ("lse", "kv"), ("lse", "out"),
                                       ("lse", "prev"), ("out", "prev_lse"), ("prev", "out"), ("prev_lse", "lse"), ("out", "ws"),
                                       ("lse", "ws")])
def test_overlaps_are_refused(mod, what, over):
    size = SIZE.get(over, mod.window_attn_workspace_size(mod.Dims(heads=64, max_ctx=1024), 2, 8))
    for at in (AT[over] + size - 16, AT[over] - SIZE[what] + 16) + (() if {what, over} in ({"prev", "out"}, {"prev_lse", "lse"}) else (AT[over],)):
        assert attend(mod, **{what: at}) == 1, at
