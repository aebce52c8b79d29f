"""The one-launch form of clipping: blocks exchange their sums, marked with the
call's number, in global memory.  Tolerances as in test_gpu_grad_clip."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from test_gpu_grad_clip import NORM_TOL, U32, _check, _make, _want   # noqa: E402


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


def test_a_wait_that_gives_up_is_reported(monkeypatch):
    """With one try a wait, blocks give up as they find sums missing.  Whatever each
    of them met, statistics that are numbers mean that every chunk was written."""
    grads = _make([8192] * 300, ["f32"], 2)
    norm, c = _want(grads, 1.0)
    lst = {}
    for tries in ("1", ""):
        monkeypatch.setenv("MG_CLIP_WAIT", tries)
        outs = [torch.empty_like(x) for x in grads]
        lst[tries] = (mg.GradList(grads, outs), outs)
    stats = torch.empty(2, device="cuda")
    gave_up = 0
    for _ in range(60):
        gl, outs = lst["1"]
        for o in outs:
            o.fill_(float("nan"))
        gl.clip(1.0, stats)
        nan = torch.isnan(stats)
        assert bool(nan[0]) == bool(nan[1])
        if bool(nan[0]):
            gave_up += 1
        elif gave_up:
            raise AssertionError("numbers from a list whose exchange has failed before")
        else:
            assert abs(float(stats[0]) - norm) <= NORM_TOL * norm
            assert not any(torch.isnan(o).any() for o in outs)
        # another list is not touched
        gl, outs = lst[""]
        gl.clip(1.0, stats)
        _check(grads, outs, stats, 1.0)
    assert gave_up
    for gl, _ in lst.values():
        gl.close()
