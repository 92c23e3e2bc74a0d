"""The build's check of the window attention's registers (CPU)."""
import os

import pytest

from compressed_sparse_attention_fp4_gb300 import build

PTXAS = """ptxas info    : Compiling entry function '_ZN4csa241_GLOBAL__N__1f1a5b41_9_window_cu_75e8371519window_merge_kernelENS_10WindowArgsE' for 'sm_103a'
ptxas info    : Used 48 registers, used 1 barriers, 2432 bytes smem
ptxas info    : Compiling entry function '_ZN4csa241_GLOBAL__N__1f1a5b41_9_window_cu_75e8371513window_kernelILb1EEEvNS_10WindowArgsENS0_10WindowMapsE' for 'sm_103a'
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 2 barriers, 4096 bytes smem
ptxas info    : Compiling entry function '_ZN4csa241_GLOBAL__N__1f1a5b41_9_window_cu_75e8371513window_kernelILb0EEEvNS_10WindowArgsENS0_10WindowMapsE' for 'sm_103a'
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 2 barriers, 4096 bytes smem
"""


def test_registers_of_the_window_kernels():
    with open(os.path.join(build.CSRC, "window.cu")) as f:
        source = f.read()
    build.check_registers(source, PTXAS % (80, 80), "window.cu")
    build.check_registers(source, "", "window.cu")           # nothing said, nothing to check
    for join, alone in ((78, 80), (80, 64), (85, 85)):
        with pytest.raises(RuntimeError, match="registers"):
            build.check_registers(source, PTXAS % (join, alone), "window.cu")
