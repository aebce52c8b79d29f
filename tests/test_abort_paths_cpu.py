"""Kernels of the tensor cores that give up after a bounded wait leave time for
their copies in flight before they end.  (The wait itself is never made to run
out on a GPU; this reads the sources.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "static_graph_nn_gb300", "csrc")


@pytest.mark.parametrize("name", ["gemm_group_narrow.cu", "gemm_group_tc.cu", "gemm_tc.cu", "gemm_tc2.cu", "attention_tc.cu"])
def test_copies_in_flight_end_before_the_kernel(name):
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    kernels = [k for k in re.findall(r"__global__.*?^\}", code, flags=re.S | re.M) if "dealloc" in k]
    assert kernels
    for k in kernels:
        drain, last = k.index("if (*abort_flag) drain_in_flight();"), k.rindex("__syncthreads();")
        assert drain < last < k.index("dealloc")
        assert "mbar_wait" not in k[drain:] and "tma_" not in k[drain:]
