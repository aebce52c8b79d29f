"""Products grouped by expert where NaN and infinities lie in everything that no
result may depend on: rows before the first and behind the last group, the rows
of other groups, the weights of groups without rows.

Every comparison is in the form |got - want| <= bound, which a NaN fails.  The
bound is derived as in test_gpu_grouped_linear: one step (2^-23) of the running
sum per addition, and half a bf16 step of the result where it is stored in
bf16."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from test_gpu_grouped_linear import DT, SHAPES, U16, _data, _offsets   # noqa: E402

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _within(got, want, mag, k, t):
    bound = 1.01 * k * 2.0 ** -23 * mag + 1e-40
    if t == "bf16":
        bound = bound + 1.01 * U16 * want.abs()
    assert ((got.double() - want).abs() <= bound).all()


def _run(x, dy, w, off, ws, t):
    e, k, n = w.shape
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    y = torch.full((x.shape[0], n), 77.0, dtype=DT[t], device="cuda")
    dx = torch.full((x.shape[0], k), 77.0, dtype=DT[t], device="cuda")
    dw = torch.full((e, k, n), 77.0, device="cuda")
    mg.grouped_linear_forward(x, offs, w, y, ws)
    mg.grouped_linear_backward_input(dy, offs, w, dx, ws)
    mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
    assert int(ws[:4].view(torch.int32)) == 0
    return y, dx, dw


def _check(x, dy, w, off, y, dx, dw, t, groups):
    k, n = w.shape[1:]
    for g in groups:
        a, b = off[g], off[g + 1]
        xs, ds, we = x[a:b].double(), dy[a:b].double(), w[g].double()
        if a < b:
            _within(y[a:b], xs @ we, xs.abs() @ we.abs(), k, t)
            _within(dx[a:b], ds @ we.t(), ds.abs() @ we.abs().t(), n, t)
        _within(dw[g], xs.t() @ ds, xs.abs().t() @ ds.abs(), b - a, "f32")


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,e,k,n", SHAPES)
def test_outside_rows_and_idle_weights(rows, e, k, n, t):
    first, last = rows // 5, rows - rows // 4
    x, dy, w, ws = _data(rows, e, k, n, t)
    off = _offsets(rows, e, 7, first, last)
    x[:first], dy[:first], x[last:], dy[last:] = NAN, INF, INF, NAN
    for g in range(e):
        if off[g] == off[g + 1]:
            w[g] = NAN
    y, dx, dw = _run(x, dy, w, off, ws, t)
    _check(x, dy, w, off, y, dx, dw, t, range(e))
    for a in (y, dx):
        assert (a[:first] == 77.0).all() and (a[last:] == 77.0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,e,k,n", [s for s in SHAPES if s[1] > 1])
def test_other_groups(rows, e, k, n, t):
    """Every second group holds NaN in rows and weights; the others are as without."""
    x, dy, w, ws = _data(rows, e, k, n, t)
    off = _offsets(rows, e, 11)
    for g in range(0, e, 2):
        x[off[g]:off[g + 1]], dy[off[g]:off[g + 1]], w[g] = NAN, INF, NAN
    y, dx, dw = _run(x, dy, w, off, ws, t)
    _check(x, dy, w, off, y, dx, dw, t, range(1, e, 2))
    for g in range(0, e, 2):
        if off[g] < off[g + 1]:
            assert torch.isnan(y[off[g]:off[g + 1]]).all() and torch.isnan(dx[off[g]:off[g + 1]]).all()
            assert torch.isnan(dw[g]).all()
        else:
            assert (dw[g] == 0).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,e,k,n", SHAPES)
def test_all_groups(rows, e, k, n, t):
    x, dy, w, ws = _data(rows, e, k, n, t)
    off = _offsets(rows, e, 13)
    y, dx, dw = _run(x, dy, w, off, ws, t)
    _check(x, dy, w, off, y, dx, dw, t, range(e))
