"""Kernels that may start while the one before them still writes (programmatic
dependents) read what it writes with ordinary loads: the read-only path asks for
data that does not change while the kernel is resident, and a compiler may
move such a load over the wait."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "static_graph_nn_gb300", "csrc")


def _functions(text):
    """The top-level functions' texts (from the signature to the closing brace in column 0)."""
    return re.findall(r"^(?:template|__global__|static|cudaError_t|__device__)[^;{]*\{.*?^\}", text, flags=re.S | re.M)


def test_no_read_only_loads_behind_a_dependency_wait():
    kernels = 0
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith(".cu"):
            continue
        for body in _functions(open(os.path.join(CSRC, f)).read()):
            code = re.sub(r"//[^\n]*", "", body)
            if "__global__" in code and "dependency_wait()" in code:
                kernels += 1
                for word in ("__ldg", "ld.global.nc", "__restrict__"):
                    assert word not in code, (f, word, body.split("{")[0])
    assert kernels >= 4        # the scan finds them: sums and their join, clipping's scaling, the products' join
