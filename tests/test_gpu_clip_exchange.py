"""The one-launch form of clipping: blocks exchange their sums, marked with the
call's number, in global memory.  Tolerances as in test_gpu_grad_clip."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from test_gpu_grad_clip import NORM_TOL, U32, _make, _want   # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("sizes", [[10], [8192] * 40 + [77], [8192 * 450]])
def test_calls_back_to_back(sizes):
    """Hundreds of calls of one list without a wait between them, each on other
    values: no call takes a sum of the one before."""
    grads = _make(sizes, ["f32"], 1)
    outs = [torch.empty_like(x) for x in grads]
    n = 400
    stats = torch.empty(n, 2, device="cuda")
    lst = mg.GradList(grads, outs)
    norm, _ = _want(grads, 1.0)
    for i in range(n):
        lst.clip(norm * 1.5, stats[i])           # norms 1, 2, 1, 2, ...: clipped every second time
        for x in grads:
            x.mul_(2.0 if i % 2 == 0 else 0.5)
    got = stats.cpu().double()
    for i in range(n):
        want = norm * (1 + i % 2)
        c = 0.75 if i % 2 else 1.0
        assert abs(float(got[i, 0]) - want) <= NORM_TOL * want
        assert abs(float(got[i, 1]) - c) <= (NORM_TOL + 2 * U32) * c      # the factor's rounding and max_norm's
    lst.close()
