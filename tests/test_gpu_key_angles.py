"""Indexer keys turned by angles next to a multiple of a quarter turn (GPU).

There a sine or cosine is small and a large channel times it is an ordinary key, so that the key shows the
sine's relative error.  The angle itself is exact to 2^-32 + 2^-34 turns, 2^-29 in radians; from it the sine
passes six roundings of 2^-24 (the angle to fp32, its unit twice, the series, mscale, the product), less than
2^-21 of it.  A key is then the format's rounding of a value within 2^-28 |v| + 2^-21 |y| of y.
"""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import codec as ocodec
from oracle import prompt as op

pytestmark = pytest.mark.gpu

# positions p with p radians next to a whole number of half turns, or of quarter turns
NEAR = {"half turns": (22, 355, 710, 103993, 104348, 208341, 312689, 833719, 2 * 833719, 5 * 312689),
        "quarter turns": (11, 33, 322, 344, 366, 51819, 52174, 260515)}


def e4m3(v):
    return np.sign(v) * ocodec.e4m3_decode(ocodec.e4m3_encode_rne_sat(np.abs(v)))


def inputs(near):
    """Rows of one large channel v, so that v times the small one of sine and cosine is 2 .. 32."""
    pos = np.repeat(np.array(NEAR[near]), 256)
    small = np.where(np.abs(np.sin(pos)) < np.abs(np.cos(pos)), np.abs(np.sin(pos)), np.abs(np.cos(pos)))
    m = np.tile(np.arange(256), len(NEAR[near]))
    v = (1 + (m & 127) / 128) * np.exp2(np.floor(np.log2(8 / small))) * np.where(m < 128, 1, -1)
    return pos, v


@pytest.mark.parametrize("near", list(NEAR))
@pytest.mark.parametrize("kind,half", [("e4m3", False), ("e4m3", True), ("fp4", True)])   # (FP4 pairs side by side share a scale)
def test_keys_next_to_quarter_turns(near, kind, half):
    pos, v = inputs(near)
    n = len(pos)
    rows = -(-n // 64) * 64
    first, second = (0, 32) if half else (0, 1)
    by_sine = near == "half turns"
    x = torch.zeros(n, 128, dtype=torch.bfloat16)
    x[:, second if by_sine else first] = torch.from_numpy(v).to(torch.bfloat16)
    assert np.array_equal(x.double().numpy().sum(1), v)                  # exact in bf16
    y = -v * np.sin(pos) if by_sine else v * np.cos(pos)                 # the first channel's key
    assert np.all((np.abs(y) > 2) & (np.abs(y) < 64))
    cfg = csa2.Rope(rot=64, layout=csa2.ROPE_HALF if half else csa2.ROPE_INTERLEAVED)
    keys = torch.zeros(rows * (72 if kind == "fp4" else 128), dtype=torch.uint8, device="cuda")
    csa2.csa2_idx_k_append(cfg, csa2.IDXK_FP4 if kind == "fp4" else csa2.IDXK_E4M3, x.cuda(),
                           torch.from_numpy(pos.astype(np.int32)).cuda(), torch.arange(n).cuda(), keys, rows)
    off = 2.0 ** -28 * np.abs(v) + 2.0 ** -21 * np.abs(y)
    lo, hi = y - off, y + off
    if kind == "e4m3":
        got = ocodec.e4m3_decode(keys.cpu().numpy().reshape(rows, 128)[:n, 0])
        lo, hi = e4m3(lo), e4m3(hi)
    else:                                                                # alone in its group: 6 scales
        codes, scales = csa2.fp4_idx_k_planes(keys.cpu(), rows)
        got = ocodec.dequantize_rows(codes.numpy(), scales.numpy())[:n, 0]
        lo, hi = (6 * e4m3(op.to_bf16(t) / 6 * (1 + s * 2.0 ** -22 * np.sign(t))) for t, s in ((lo, -1), (hi, 1)))
    assert np.all((got >= np.minimum(lo, hi)) & (got <= np.maximum(lo, hi)))
    assert np.mean(lo != hi) < 0.1                                       # (the bound is narrow)
