"""The build's check of the dense attention's registers (CPU)."""
import os

import pytest

from compressed_sparse_attention_fp4_gb300 import build

PTXAS = """ptxas info    : Compiling entry function '_ZN4csa240_GLOBAL__N__50e6eb5d_8_dense_cu_c29227cf17dense_plan_kernelENS_9DenseArgsE' for 'sm_103a'
ptxas info    : Used 46 registers, used 1 barriers, 21504 bytes smem
ptxas info    : Compiling entry function '_ZN4csa240_GLOBAL__N__50e6eb5d_8_dense_cu_c29227cf17dense_pair_kernelENS_9DenseArgsENS0_9DenseMapsE' for 'sm_103a'
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 16 barriers, 8192 bytes smem
ptxas info    : Compiling entry function '_ZN4csa240_GLOBAL__N__50e6eb5d_8_dense_cu_c29227cf12dense_kernelENS_9DenseArgsENS0_9DenseMapsE' for 'sm_103a'
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 16 barriers, 8192 bytes smem
"""


def test_registers_of_the_dense_kernels():
    with open(os.path.join(build.CSRC, "dense.cu")) as f:
        source = f.read()
    build.check_registers(source, PTXAS % (72, 72))
    build.check_registers(source, "")                       # nothing said, nothing to check
    for pair, one in ((70, 72), (72, 64), (80, 80)):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(source, PTXAS % (pair, one))
