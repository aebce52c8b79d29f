"""Matrix products grouped by expert (forward, input gradient, weight gradient)
against per-group products in 64 bits, element by element.

Tolerance of one output with a sum of K products: the products of bf16 values
are exact in fp32; each fp32 addition is off by at most one step (2^-23, the
tensor cores may truncate) of the running sum, which sum|a b| bounds; fp32
inputs add a rounding per product (inside the same allowance: FFMA rounds
once).  So K 2^-23 sum|a b|, plus half a bf16 step of the result where it is
stored in bf16."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U16 = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _randn(shape, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[t])


def _data(rows, e, k, n, t, seed=1):
    return (_randn((rows, k), t, seed), _randn((rows, n), t, seed + 1), _randn((e, k, n), t, seed + 2),
            torch.zeros(mg.grouped_linear_workspace_bytes(rows, e, k, n), dtype=torch.uint8, device="cuda"))


def _close(got, want, mag, k, t):
    bound = 1.01 * k * 2.0 ** -23 * mag
    if t == "bf16":
        bound = bound + 1.01 * U16 * want.abs()
    bad = (got.double() - want).abs() > bound + 1e-40
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(),
                           float((got.double() - want).abs().max()))


def _check_all(off, rows, e, k, n, t, x, dy, w, ws, clamped=None):
    """The three calls; off: list of e + 1 offsets (clamped: what they mean)."""
    o = clamped or off
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    mark = 77.0
    y = torch.full((rows + 1, n), mark, dtype=DT[t], device="cuda")
    dx = torch.full((rows + 1, k), mark, dtype=DT[t], device="cuda")
    dw = torch.full((e + 1, k, n), mark, device="cuda")
    mg.grouped_linear_forward(x, offs, w, y[:rows], ws)
    mg.grouped_linear_backward_input(dy, offs, w, dx[:rows], ws)
    mg.grouped_linear_backward_weight(x, dy, offs, dw[:e], ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    assert (y[rows] == mark).all() and (dx[rows] == mark).all() and (dw[e] == mark).all()
    inside = torch.zeros(rows, dtype=torch.bool)
    for g in range(e):
        a, b = o[g], o[g + 1]
        inside[a:b] = True
        xs, ds, we = x[a:b].double(), dy[a:b].double(), w[g].double()
        _close(y[a:b], xs @ we, xs.abs() @ we.abs(), k, t)
        _close(dx[a:b], ds @ we.t(), ds.abs() @ we.abs().t(), n, t)
        _close(dw[g], xs.t() @ ds, xs.abs().t() @ ds.abs(), b - a, "f32")
        if a == b:
            assert (dw[g] == 0).all()
    assert (y[:rows][~inside.cuda()] == mark).all() and (dx[:rows][~inside.cuda()] == mark).all()


def _offsets(rows, e, seed, first=0, last=None):
    g = torch.Generator().manual_seed(seed)
    cut = torch.randint(first, (rows if last is None else last) + 1, (e - 1,), generator=g).sort().values.tolist()
    return [first] + cut + [rows if last is None else last]


SHAPES = [
    # rows, groups, d_in, d_out
    (1, 1, 8, 8), (1, 3, 64, 256), (5, 4, 72, 136), (24, 8, 512, 1024), (63, 2, 8, 264), (64, 1, 64, 64),
    (300, 7, 200, 328), (1000, 16, 520, 1032), (129, 5, 256, 128), (2049, 3, 136, 264), (700, 64, 264, 72),
    # few tiles and a long sum: two or four blocks share one
    (20, 3, 2048, 200), (7, 1, 4104, 72), (30, 2, 200, 1160), (16, 1, 1088, 2304),
    # few tiles and long sums over d_in, d_out and the rows: split over blocks and joined
    (300, 2, 1032, 136), (200, 3, 136, 2056), (5000, 2, 200, 72), (4000, 3, 72, 264), (700, 1, 2056, 1032),
    # widths that rows of 16 bytes do not divide
    (111, 1, 404, 1003), (130, 2, 1003, 70), (3000, 2, 65, 33), (700, 3, 601, 1003), (640, 2, 1001, 520), (1500, 4, 520, 999), (20, 4, 1501, 999), (30, 3, 1000, 2003),
    (77, 3, 33, 17), (300, 5, 1, 1), (50, 2, 100, 65),
]


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,e,k,n", SHAPES)
def test_products(rows, e, k, n, t):
    x, dy, w, ws = _data(rows, e, k, n, t)
    _check_all(_offsets(rows, e, 5), rows, e, k, n, t, x, dy, w, ws)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_one_workspace_for_fewer_rows(t):
    """A workspace of the size for many rows, filled to its end by earlier calls,
    serves calls of fewer (which split more)."""
    e, k, n = 2, 1032, 1003
    ws = torch.zeros(mg.grouped_linear_workspace_bytes(3001, e, k, n), dtype=torch.uint8, device="cuda")
    for rows in (3001, 700, 130, 17, 1):
        x, dy, w, _ = _data(rows, e, k, n, t)
        _check_all(_offsets(rows, e, rows), rows, e, k, n, t, x, dy, w, ws)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,e,k,n", [(300, 4, 136, 264), (40, 6, 256, 512), (65, 2, 72, 40), (9, 3, 33, 17),
                                          (300, 2, 1032, 136), (4000, 3, 72, 264), (900, 3, 601, 1003),
                                          (25, 4, 1501, 999)])
def test_rows_of_no_group(rows, e, k, n, t):
    """Rows before the first and behind the last group hold NaN: neither read nor
    written, and the gradients stay finite."""
    first, last = rows // 5, rows - rows // 4
    x, dy, w, ws = _data(rows, e, k, n, t)
    for a in (x, dy):
        a[:first] = float("nan")
        a[last:] = float("inf")
    _check_all(_offsets(rows, e, 6, first, last), rows, e, k, n, t, x, dy, w, ws)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_neighbours_do_not_leak(t):
    """A group of NaN rows between two others, at boundaries inside a tile."""
    rows, e, k, n = 200, 3, 128, 256
    x, dy, w, ws = _data(rows, e, k, n, t)
    off = [0, 61, 133, 200]
    x[61:133] = float("nan")
    dy[61:133] = float("nan")
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    dw = torch.empty(e, k, n, device="cuda")
    mg.grouped_linear_forward(x, offs, w, y, ws)
    mg.grouped_linear_backward_input(dy, offs, w, dx, ws)
    mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
    for a in (y, dx):
        assert torch.isfinite(a[:61]).all() and torch.isfinite(a[133:]).all() and torch.isnan(a[61:133]).all()
    assert torch.isfinite(dw[0]).all() and torch.isfinite(dw[2]).all() and torch.isnan(dw[1]).all()


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("off", [[0, 0, 0, 40], [40, 40, 40, 40], [0, 40, 40, 40], [0, 0, 0, 0], [0, 1, 39, 40]])
def test_empty_and_full_groups(t, off):
    x, dy, w, ws = _data(40, 3, 64, 136, t)
    _check_all(off, 40, 3, 64, 136, t, x, dy, w, ws)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("off,means", [([-5, 10, 20, 99], [0, 10, 20, 40]), ([0, 30, 10, 40], [0, 30, 30, 40]),
                                       ([2**31 - 1, 0, 0, 0], [40, 40, 40, 40]), ([-2**31, -1, -7, 3], [0, 0, 0, 3])])
def test_bad_offsets_are_clamped(t, off, means):
    x, dy, w, ws = _data(40, 3, 64, 136, t)
    _check_all(off, 40, 3, 64, 136, t, x, dy, w, ws, clamped=means)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_no_rows(t):
    """rows = 0: nothing to do forward, all-zero weight gradients."""
    w = _randn((3, 64, 32), t, 1)
    ws = torch.zeros(mg.grouped_linear_workspace_bytes(0, 3, 64, 32), dtype=torch.uint8, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x, dy = torch.empty(0, 64, dtype=DT[t], device="cuda"), torch.empty(0, 32, dtype=DT[t], device="cuda")
    dw = torch.full((3, 64, 32), 5.0, device="cuda")
    mg.grouped_linear_forward(x, off, w, dy, ws)
    mg.grouped_linear_backward_input(dy, off, w, x, ws)
    mg.grouped_linear_backward_weight(x, dy, off, dw, ws)
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_many_groups():
    """More groups than rows, up to the limit of 1024."""
    rows, e, k, n = 500, 1024, 24, 16
    x, dy, w, ws = _data(rows, e, k, n, "bf16")
    _check_all(_offsets(rows, e, 8), rows, e, k, n, "bf16", x, dy, w, ws)


def test_same_bits_again():
    rows, e, k, n = 3000, 4, 256, 384
    x, dy, w, ws = _data(rows, e, k, n, "bf16")
    offs = torch.tensor(_offsets(rows, e, 9), dtype=torch.int32, device="cuda")
    res = []
    for _ in range(2):
        y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty(e, k, n, device="cuda")
        mg.grouped_linear_forward(x, offs, w, y, ws)
        mg.grouped_linear_backward_input(dy, offs, w, dx, ws)
        mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
        res.append((y, dx, dw))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_weight_gradient_matches_differences():
    """d/dw of sum(dy * y) by central differences of the forward call (linear in
    w, so any step is exact up to rounding)."""
    rows, e, k, n = 37, 3, 24, 16
    x, dy, w, ws = _data(rows, e, k, n, "f32")
    offs = torch.tensor([0, 11, 11, 37], dtype=torch.int32, device="cuda")
    dw = torch.empty(e, k, n, device="cuda")
    mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
    y = torch.empty(rows, n, device="cuda")

    def loss(wt):
        mg.grouped_linear_forward(x, offs, wt, y, ws)
        return float((y.double() * dy.double()).sum())

    h = 0.5
    for g, r, c in ((0, 0, 0), (1, 3, 3), (2, 23, 15)):
        a, b = w.clone(), w.clone()
        a[g, r, c] += h
        b[g, r, c] -= h
        mag = float((x.abs().double() @ (w.abs().double().sum(0) + h) * dy.abs()).sum())
        assert abs((loss(a) - loss(b)) / (2 * h) - float(dw[g, r, c])) <= 2 * k * 2.0 ** -23 * mag / h


def test_streams_and_graph_replay():
    """Captured once, replayed with other offsets and data."""
    rows, e, k, n = 600, 5, 128, 264
    x, dy, w, ws = _data(rows, e, k, n, "bf16")
    offs = torch.tensor(_offsets(rows, e, 1), dtype=torch.int32, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty(e, k, n, device="cuda")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mg.grouped_linear_forward(x, offs, w, y, ws, stream=s)
        mg.grouped_linear_backward_input(dy, offs, w, dx, ws, stream=s)
        mg.grouped_linear_backward_weight(x, dy, offs, dw, ws, stream=s)
    for seed in (11, 12, 13):
        off = _offsets(rows, e, seed)
        offs.copy_(torch.tensor(off, dtype=torch.int32))
        x.copy_(_randn((rows, k), "bf16", seed))
        g.replay()
        torch.cuda.synchronize()
        for q in range(e):
            a, b = off[q], off[q + 1]
            xs, ds, we = x[a:b].double(), dy[a:b].double(), w[q].double()
            _close(y[a:b], xs @ we, xs.abs() @ we.abs(), k, "bf16")
            _close(dx[a:b], ds @ we.t(), ds.abs() @ we.abs().t(), n, "bf16")
            _close(dw[q], xs.t() @ ds, xs.abs().t() @ ds.abs(), b - a, "f32")


def test_mixed_types_are_refused():
    x, dy, w, ws = _data(8, 2, 16, 8, "bf16")
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for call in (lambda: mg.grouped_linear_forward(x, off, w.float(), dy, ws),
                 lambda: mg.grouped_linear_forward(x, off.long(), w, dy, ws),
                 lambda: mg.grouped_linear_forward(x, off[:2], w, dy, ws),
                 lambda: mg.grouped_linear_backward_weight(x, dy.float(), off, torch.empty(2, 16, 8, device="cuda"), ws),
                 lambda: mg.grouped_linear_forward(x, off, w, dy, ws[:2])):
        with pytest.raises(binding.MGError):
            call()
