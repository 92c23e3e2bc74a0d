"""Caches past 2^31 bytes, and references that rise from block to block, for the calls of the window side."""
import numpy as np
import pytest
import torch

from compressed_sparse_attention_fp4_gb300 import csa2
from oracle import prompt as op
from tests.test_gpu_newrows import KINDS, NORMS, PARTS, key_inputs
from tests.test_gpu_window import Problem

pytestmark = pytest.mark.gpu


def moved(p, far):
    """The problem's pages `far` pages on, in a cache of so many more."""
    kv = torch.empty((far + p.pages) * 64, 576, dtype=torch.bfloat16, device="cuda")
    kv[far * 64:] = p.kv
    p.kv = kv
    p.d_table = torch.where(p.d_table >= 0, p.d_table + far, p.d_table)
    p.dims.num_pages = far + p.pages
    return p


@pytest.mark.parametrize("lens,ctx,window", [([200, 60], [900, 700], 300), ([300, 5], [300, 900], 128), ([2] * 5, [3000] * 5, 64)])
def test_attention_far_in_a_cache(lens, ctx, window):
    moved(Problem(lens, ctx, heads=64, window=window, sinks=3, seed=31), (1 << 32) // (64 * 1152) + 77).run().check(some=8)


def test_exact_rows_far_in_a_cache():
    far = (1 << 32) // 1152 + 5
    g = torch.Generator().manual_seed(1)
    x = torch.randn(70, 576, generator=g).to(torch.bfloat16).cuda()
    pos, dst = torch.arange(70, dtype=torch.int32).cuda(), torch.randperm(128, generator=g)[:70].cuda()
    near = torch.zeros(128, 576, dtype=torch.bfloat16, device="cuda")
    csa2.csa2_window_append(csa2.Rope(**PARTS), x, pos, dst, near)
    kv = torch.zeros(far + 128, 576, dtype=torch.bfloat16, device="cuda")
    csa2.csa2_window_append(csa2.Rope(**PARTS), x, pos, dst + far, kv)
    assert torch.equal(kv[far:], near) and not kv[:far].any()


@pytest.mark.parametrize("kind", list(KINDS))
def test_keys_far_in_a_cache(kind):
    far = (1 << 32) // {"e4m3": 128, "fp4": 64, "fp32": 256}[kind] + 3
    size = {"e4m3": 128, "fp4": 72, "fp32": 256}[kind]
    x, w, b = key_inputs(kind, 70, 1, "rms")[:3]
    pos, dst = torch.arange(70, dtype=torch.int32).cuda(), torch.randperm(128, generator=torch.Generator().manual_seed(2))[:70].cuda()
    cfg = csa2.Rope(rot=32, layout=csa2.ROPE_HALF)
    out = []
    for off in (0, far):
        keys = torch.zeros((off + 128) * size, dtype=torch.uint8, device="cuda")
        csa2.csa2_idx_k_append(cfg, KINDS[kind], x, pos, dst + off, keys, off + 128, norm=NORMS["rms"], norm_w=w, norm_b=b)
        if kind == "fp4":
            codes, scales = csa2.fp4_idx_k_planes(keys, off + 128)
            out.append((codes[off:].clone(), scales[off:].clone()))
            assert not codes[:off].any() and not scales[:off].any()
        else:
            out.append((keys.view(off + 128, size)[off:].clone(),))
            assert not keys[:off * size].any()
    for u, v in zip(*out):
        assert torch.equal(u, v) and u.any()


@pytest.mark.parametrize("s", [16.0, -16.0, 4.0])
def test_long_form_rising_and_falling_logits(s):
    """Keys grow along the window, so that blocks pass the reference by more than the slack; then they fall."""
    n = 64 * 12
    p = Problem([160], [n], heads=64, window=n, paged=False, seed=33)
    v = op.to_bf16(np.repeat(np.arange(12), 64)[:, None] * np.ones((1, 64)))
    p.key[0][:, 512:] = v
    p.kv[:, 512:] = torch.from_numpy(v).to(torch.bfloat16).cuda()
    p.q64[:, :, 512:] = s
    p.q[:, :, 512:] = s
    p.run().check(some=6)
