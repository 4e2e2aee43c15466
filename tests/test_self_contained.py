"""libcgdr.so carries its CUDA runtime: it loads by itself and shares no error state with its process."""
import ctypes
import subprocess
import sys

import pytest

from gated_delta_rule_channelwise_gb300 import build as cbuild

LOAD = """
import ctypes, sys
ctypes.CDLL(sys.argv[1])
print("\\n".join({line.split()[-1] for line in open("/proc/self/maps") if "cuda" in line.split()[-1]}))
"""


@pytest.mark.parametrize("debug", [False, True])
def test_loads_without_another_cuda_library(debug):
    lib = cbuild.build(debug=debug)
    r = subprocess.run([sys.executable, "-c", LOAD, lib], capture_output=True, text=True, check=True)
    assert "libcudart" not in r.stdout


@pytest.mark.gpu
def test_an_error_left_in_the_process_is_not_taken_for_one_of_a_launch():
    """An invalid device number leaves an error in the runtime that torch has loaded; it is still there afterwards."""
    import torch

    import gated_delta_rule_channelwise_gb300 as cg
    cbuild.build()
    x, w, o = torch.ones(1, 8, device="cuda"), torch.ones(8, 4, device="cuda"), torch.empty(1, 8, device="cuda")
    state = torch.zeros(1, 3, 8, device="cuda")
    cg.conv_decode(x, w, state, o, silu=False)
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libcudart" in line}
    if not paths:
        pytest.skip("torch has loaded no shared CUDA runtime")
    runtime = ctypes.CDLL(paths.pop())
    wrong = runtime.cudaSetDevice(9999)
    assert wrong != 0
    try:
        cg.conv_decode(x, w, state, o, silu=False)
    finally:
        left = runtime.cudaGetLastError()
    assert left == wrong
    assert o.tolist() == [[2.0] * 8]
