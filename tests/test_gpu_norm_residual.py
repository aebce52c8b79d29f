"""The residual stream's norms with gate and scale, and their gradients, against the
definitions in 64 bits.

Tolerances.  Every result is a sum of products of inputs (and of 1 / sqrt of a
mean).  An operation rounds by u = 2^-24 of its result, so a result that goes
through D operations is off by at most D u times the same expression with every
term taken at its absolute value.  A row's sum goes through at most dim / 32 + 10
additions (a warp's lanes or more, then a tree), a column's sum through at most as
many as it has rows plus 10.  Then half a step of the stored type."""
import math
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _inputs(rows, dim, t, gates, post, pre, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return {"y": rnd(rows, dim).to(DT[t]), "x": (2 * rnd(rows, dim)).to(DT[t]),
            "g1": 1 + 0.3 * rnd(dim) if post else None, "gate": 0.5 + rnd(gates, dim) if gates else None,
            "g2": 1 + 0.3 * rnd(dim) if pre else None, "dxo": rnd(rows, dim).to(DT[t]),
            "dh": rnd(rows, dim).to(DT[t]) if pre else None}


def _row_gate(i):
    x = i["x"]
    if i["gate"] is None:
        return 1.0
    return i["gate"].double().repeat_interleave(max(1, x.shape[0] // i["gate"].shape[0]), 0)


def _forward(i, scale, stream=None, inplace=False):
    x = i["x"]
    xo = x if inplace else torch.full_like(x, 77.0)
    h = None if i["g2"] is None else i["y"] if inplace else torch.full_like(x, 77.0)
    rstd = torch.full((x.shape[0], 2), 77.0, device="cuda")
    mg.norm_residual_forward(i["y"], x, xo, h, gamma_post=i["g1"], gate=i["gate"], gamma_pre=i["g2"], scale=scale,
                             eps=EPS, rstd=rstd, stream=stream)
    return xo, h, rstd


def _forward_check(i, scale, out, t):
    xo, h, rstd = out
    y, x = i["y"].double(), i["x"].double()
    d = x.shape[1]
    depth = d / 32 + 10
    one = torch.ones(x.shape[0], 1, dtype=torch.float64, device="cuda")
    gate = _row_gate(i)
    r1 = (y.square().mean(1, keepdim=True) + EPS).rsqrt() if i["g1"] is not None else one
    # the root halves the mean's error (a square, the sum, the division, eps), and rounds with the division: 4
    e1 = (0.5 * (depth + 3) + 4) * U if i["g1"] is not None else 0.0
    u = y * r1 * (i["g1"].double() if i["g1"] is not None else 1.0) * gate
    want = scale * x + u
    err = (e1 + 5 * U) * u.abs() + 3 * U * (scale * x).abs()
    assert ((xo.double() - want).abs() <= err + HALF[t] * (want.abs() + err)).all()
    assert ((rstd[:, :1].double() - r1).abs() <= e1 * r1).all()
    if i["g2"] is None:
        assert h is None and (rstd[:, 1] == 1).all()
        return
    r2 = (want.square().mean(1, keepdim=True) + EPS).rsqrt()
    # x_out's own error moves the mean of squares by at most 2 mean(|x_out| err)
    e2 = r2.square() * (want.abs() * err).mean(1, keepdim=True) + (0.5 * (depth + 3) + 4) * U
    assert ((rstd[:, 1:].double() - r2).abs() <= e2 * r2).all()
    g2 = i["g2"].double()
    wh = want * r2 * g2
    eh = err * r2 * g2.abs() + (e2 + 3 * U) * wh.abs()
    assert ((h.double() - wh).abs() <= eh + HALF[t] * (wh.abs() + eh)).all()


def _formula(i, rstd, scale, minus):
    """The gradients in 64 bits (minus = -1), or with minus = 1 and everything at its absolute value their
    expressions' magnitudes."""
    f = (lambda v: v.double()) if minus < 0 else (lambda v: v.double().abs())
    y, x = f(i["y"]), f(i["x"])
    scale = scale if minus < 0 else abs(scale)
    r1, r2 = rstd[:, :1].double(), rstd[:, 1:].double()
    g1 = f(i["g1"]) if i["g1"] is not None else None
    gate = _row_gate(i)
    gate = gate if minus < 0 or i["gate"] is None else gate.abs()
    u = y * r1 * g1 if g1 is not None else y
    t = f(i["dxo"]) if i["dxo"] is not None else torch.zeros_like(x)
    out = {}
    if i["dh"] is not None:
        xo, dh = scale * x + gate * u, f(i["dh"])
        a = dh * f(i["g2"])
        t = t + r2 * a + minus * xo * r2 ** 3 * (a * xo).mean(1, keepdim=True)
        out["g2"] = (dh * xo * r2).sum(0)
    if i["gate"] is not None:
        out["gate"] = (t * u).view(i["gate"].shape[0], -1, x.shape[1]).sum(1)
    w = gate * t
    if g1 is not None:
        out["g1"] = (w * y * r1).sum(0)
        out["dy"] = r1 * w * g1 + minus * y * r1 ** 3 * (w * g1 * y).mean(1, keepdim=True)
    else:
        out["dy"] = w
    out["dx"] = scale * t
    return out


def _backward(i, rstd, scale, stream=None, inplace=False, ws=None):
    x = i["x"]
    r, d = x.shape
    n = 0 if i["gate"] is None else i["gate"].shape[0]
    o = {"dy": torch.full_like(x, 77.0) if not inplace else i["y"], "dx": torch.full_like(x, 77.0) if not inplace else i["dxo"]}
    for k in ("g1", "g2", "gate"):
        if i[k] is not None and (k != "g2" or i["dh"] is not None):
            o[k] = torch.full_like(i[k], 77.0)
    if ws is None:
        ws = torch.full((mg.norm_residual_workspace_bytes(r, d, n),), 255, dtype=torch.uint8, device="cuda")
    mg.norm_residual_backward(i["dxo"], i["dh"], i["y"], x, rstd, o["dy"], o["dx"], ws, gamma_post=i["g1"],
                              gate=i["gate"], gamma_pre=i["g2"], dgamma_post=o.get("g1"), dgate=o.get("gate"),
                              dgamma_pre=o.get("g2"), scale=scale, stream=stream)
    return o


def _backward_check(i, rstd, scale, o, t):
    r, d = i["x"].shape
    per = r // (i["gate"].shape[0] if i["gate"] is not None else 1)
    want, mag = _formula(i, rstd, scale, -1), _formula(i, rstd, scale, 1)
    ops = 30 + 2 * (d / 32 + 10)
    assert set(o) == set(want)
    for k in ("dy", "dx"):
        e = ops * U * mag[k]
        assert ((o[k].double() - want[k]).abs() <= e + HALF[t] * (want[k].abs() + e)).all(), k
    for k in set(want) - {"dy", "dx"}:
        n = per if k == "gate" else r
        assert ((o[k].double() - want[k]).abs() <= (ops + n + 10) * U * mag[k]).all(), k


SHAPES = [(1, 1, 1), (3, 2, 0), (5, 8, 1), (4, 100, 2), (7, 777, 7), (33, 1024, 1), (64, 2048, 4), (130, 520, 0),
          (19, 4096, 1), (5, 4100, 1), (6, 8192, 2), (3, 16384, 1), (2, 16392, 1), (2, 40001, 2), (1000, 64, 1),
          (2500, 264, 50), (300, 2056, 300), (9, 6000, 9), (400, 256, 1), (77, 250, 7), (40, 12288, 2), (30, 9001, 1),
          (6, 32768, 3), (3, 65536, 1), (2, 70001, 1), (4, 70000, 2)]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,gates", SHAPES)
def test_forward_and_backward(rows, dim, gates, t):
    i = _inputs(rows, dim, t, gates, True, True, rows + dim)
    out = _forward(i, 0.7)
    _forward_check(i, 0.7, out, t)
    o = _backward(i, out[2], 0.7)
    _backward_check(i, out[2], 0.7, o, t)
    again = _backward(i, out[2], 0.7)
    assert all(torch.equal(o[k], again[k]) for k in o)
    # in place: x_out over x and h over y; dy over y and dx over dx_out
    o2 = _backward(i, out[2], 0.7, inplace=True)
    assert all(torch.equal(o[k], o2[k]) for k in o)
    i = _inputs(rows, dim, t, gates, True, True, rows + dim)
    xo, h, rstd = _forward(i, 0.7, inplace=True)
    assert torch.equal(xo, out[0]) and torch.equal(h, out[1]) and torch.equal(rstd, out[2])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gates", [0, 1, 6])
@pytest.mark.parametrize("dim", [200, 333, 2048])
def test_parts_left_out(dim, gates, pre, post, t):
    i = _inputs(12, dim, t, gates, post, pre, dim + gates)
    out = _forward(i, -1.25)
    _forward_check(i, -1.25, out, t)
    _backward_check(i, out[2], -1.25, _backward(i, out[2], -1.25), t)
    if pre:
        i["dxo"] = None
        _backward_check(i, out[2], -1.25, _backward(i, out[2], -1.25), t)
    i = _inputs(12, dim, t, gates, post, pre, dim + gates)
    i["dh"] = None
    _backward_check(i, out[2], -1.25, _backward(i, out[2], -1.25), t)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,gates", [(60000, 64, 60000), (60000, 64, 30000), (50001, 50, 50001), (12000, 1024, 12000),
                                            (9000, 777, 9000), (5000, 16384, 5000), (30000, 40, 15000)])
def test_many_gates(rows, dim, gates, t):
    """More gates than blocks: a block has several whole gates."""
    i = _inputs(rows, dim, t, gates, True, True, gates)
    out = _forward(i, 0.7)
    _forward_check(i, 0.7, out, t)
    o = _backward(i, out[2], 0.7)
    _backward_check(i, out[2], 0.7, o, t)
    again = _backward(i, out[2], 0.7)
    assert all(torch.equal(o[k], again[k]) for k in o)


def test_a_workspace_for_more_rows_serves_fewer():
    ws = torch.full((mg.norm_residual_workspace_bytes(9000, 520, 3),), 255, dtype=torch.uint8, device="cuda")
    for rows in (9000, 2001, 30, 3):
        for t in ("f32", "bf16"):
            i = _inputs(rows, 520, t, 3, True, True, rows)
            out = _forward(i, 1.1)
            _backward_check(i, out[2], 1.1, _backward(i, out[2], 1.1, ws=ws), t)


# around a warp's words, a unit, one block's rows, a cluster's parts; odd, even and aligned rows
EDGES = [1, 2, 3, 7, 9, 63, 65, 127, 130, 255, 257, 258, 511, 513, 514, 1023, 1025, 1026, 1537, 2047, 2050, 4095, 4097, 6145,
         8191, 8193, 8194, 9601, 12289, 16383, 16385]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("dim", EDGES)
def test_any_offset(dim, t):
    i = _inputs(13, dim, t, 1, True, True, dim)
    out = _forward(i, 0.7)
    _forward_check(i, 0.7, out, t)
    _backward_check(i, out[2], 0.7, _backward(i, out[2], 0.7), t)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [50, 777, 778, 2045, 2124, 4097, 9011, 16385])
def test_neighbours_of_other_kinds(dim, t):
    """Rows and elements beside a matrix that are no numbers reach no other row; what lies around the outputs stays."""
    rows, before, after = 9, 16, 64
    n = rows * dim

    def placed(v, fill):
        big = torch.full((before + n + after,), fill, dtype=DT[t], device="cuda")
        at = big[before:before + n].view(rows, dim)
        at.copy_(v)
        return big, at

    i = _inputs(rows, dim, t, 1, True, True, dim + 1)
    keep = [r for r in range(rows) if r not in (0, 4, 8)]
    small = {k: v[keep].contiguous() if k in ("y", "x", "dxo", "dh") else v for k, v in i.items()}
    for k in ("y", "x", "dxo", "dh"):
        i[k][[0, 4, 8]] = float("nan")
        i[k] = placed(i[k], float("inf"))[1]
    rstd = torch.full((rows, 2), 77.0, device="cuda")
    outs = [placed(torch.zeros(rows, dim, device="cuda"), 77.0) for _ in range(4)]
    mg.norm_residual_forward(i["y"], i["x"], outs[0][1], outs[1][1], gamma_post=i["g1"], gate=i["gate"], gamma_pre=i["g2"],
                             scale=0.7, eps=EPS, rstd=rstd)
    ws = torch.full((mg.norm_residual_workspace_bytes(rows, dim, 1),), 255, dtype=torch.uint8, device="cuda")
    mg.norm_residual_backward(i["dxo"], i["dh"], i["y"], i["x"], rstd, outs[2][1], outs[3][1], ws, gamma_post=i["g1"],
                              gate=i["gate"], gamma_pre=i["g2"], scale=0.7)
    for big, at in outs:
        assert (big[:before] == 77).all() and (big[before + n:] == 77).all()
        assert at[[0, 4, 8]].isnan().all()
    _forward_check(small, 0.7, (outs[0][1][keep], outs[1][1][keep], rstd[keep]), t)
    want, mag = _formula(small, rstd[keep], 0.7, -1), _formula(small, rstd[keep], 0.7, 1)
    for k, o in (("dy", outs[2][1]), ("dx", outs[3][1])):
        e = (30 + 2 * (dim / 32 + 10)) * U * mag[k]
        assert ((o[keep].double() - want[k]).abs() <= e + HALF[t] * (want[k].abs() + e)).all(), k


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [9600, 9011, 16384, 8192])
@pytest.mark.parametrize("gates", [4, 9, 10, 13, 18, 19, 28, 38, 76, 150])
def test_gates_of_wide_rows_stay_in_the_workspace(gates, dim, t):
    need = mg.norm_residual_workspace_bytes(3 * gates, dim, gates)
    ws = torch.full((need + 4096 * 64,), 255, dtype=torch.uint8, device="cuda")
    i = _inputs(3 * gates, dim, t, gates, True, True, gates)
    out = _forward(i, 0.7)
    _backward_check(i, out[2], 0.7, _backward(i, out[2], 0.7, ws=ws[:need]), t)
    assert (ws[need:] == 255).all()


def test_against_differences():
    """Central differences of the definition in 64 bits (step 1e-5: truncation below 1e-8 of third derivatives under
    100, rounding 1e-10) beside the kernel's own bound; rstd is the forward's, within its bound of the exact one, and
    changes the gradients by no more than four times its relative error of their magnitudes."""
    i = _inputs(3, 11, "f32", 3, True, True, 5)
    out = _forward(i, 0.7)
    o = _backward(i, out[2], 0.7)
    mag = _formula(i, out[2], 0.7, 1)
    names = {"y": "dy", "x": "dx", "g1": "g1", "gate": "gate", "g2": "g2"}
    base = {k: i[k].double() for k in names}

    def f(v):
        u = v["y"] * (v["y"].square().mean(1, keepdim=True) + EPS).rsqrt() * v["g1"]
        xo = 0.7 * v["x"] + v["gate"] * u
        h = xo * (xo.square().mean(1, keepdim=True) + EPS).rsqrt() * v["g2"]
        return float((i["dxo"].double() * xo + i["dh"].double() * h).sum())

    for k, n in names.items():
        flat = o[n].double().flatten()
        for c in range(flat.numel()):
            d = torch.zeros(flat.numel(), dtype=torch.float64, device="cuda")
            d[c] = 1e-5
            d = d.view_as(base[k])
            diff = (f(base | {k: base[k] + d}) - f(base | {k: base[k] - d})) / 2e-5
            assert abs(diff - float(flat[c])) <= (30 + 2 * 11 + 13 + 4 * 20) * U * float(mag[n].flatten()[c]) + 1e-7


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_rows_of_zeros_and_not_finite(t):
    """A row of zeros has the norm's eps alone; what is not finite stays in its row (and in the columns' sums)."""
    i = _inputs(9, 300, t, 1, True, True, 8)
    i["y"][2] = 0
    i["x"][2] = 0
    clean = {k: None if v is None else v.clone() for k, v in i.items()}
    out = _forward(i, 1.0)
    _forward_check(i, 1.0, out, t)
    assert (out[0][2] == 0).all() and (out[1][2] == 0).all()
    _backward_check(i, out[2], 1.0, _backward(i, out[2], 1.0), t)
    i["y"][4, 7] = math.nan
    i["x"][6, 299] = math.inf
    bad = _forward(i, 1.0)
    rest = [0, 1, 2, 3, 5, 7, 8]
    for a, b in zip(out, bad):
        assert torch.equal(a[rest], b[rest])
    assert torch.isnan(bad[1][4]).all()
    assert torch.isinf(bad[0][6, 299]) and torch.equal(bad[0][6, :299], out[0][6, :299])
    o, w = _backward(i, bad[2], 1.0), _backward(clean, out[2], 1.0)
    for k in ("dy", "dx"):
        assert torch.equal(o[k][rest], w[k][rest])


def test_no_rows():
    i = _inputs(0, 64, "bf16", 0, True, True, 1)
    out = _forward(i, 1.0)
    o = _backward(i, out[2], 1.0)
    assert (o["g1"] == 0).all() and (o["g2"] == 0).all()
    i["gate"] = torch.ones(3, 64, device="cuda")
    o = _backward(i, out[2], 1.0)
    assert (o["gate"] == 0).all()


def test_views_of_more_dimensions():
    i = _inputs(12, 136, "bf16", 4, True, True, 2)
    out = _forward(i, 0.5)
    o = _backward(i, out[2], 0.5)
    j = {k: v if v is None or v.shape[0] != 12 else v.view(4, 3, 136) for k, v in i.items()}
    xo, h = torch.zeros_like(j["x"]), torch.zeros_like(j["x"])
    rstd = torch.zeros(4, 3, 2, device="cuda")
    mg.norm_residual_forward(j["y"], j["x"], xo, h, gamma_post=i["g1"], gate=i["gate"], gamma_pre=i["g2"], scale=0.5, rstd=rstd)
    assert torch.equal(xo.view(12, 136), out[0]) and torch.equal(rstd.view(12, 2), out[2])
    dy, dx = torch.zeros_like(xo), torch.zeros_like(xo)
    ws = torch.zeros(mg.norm_residual_workspace_bytes(12, 136, 4), dtype=torch.uint8, device="cuda")
    mg.norm_residual_backward(j["dxo"], j["dh"], j["y"], j["x"], rstd, dy, dx, ws, gamma_post=i["g1"], gate=i["gate"],
                              gamma_pre=i["g2"], scale=0.5)
    assert torch.equal(dy.view(12, 136), o["dy"]) and torch.equal(dx.view(12, 136), o["dx"])
    # a one-dimensional gate
    mg.norm_residual_forward(i["y"], i["x"], xo.view(12, 136), gate=i["gate"][0])


def test_overlaps_are_refused():
    b = torch.zeros(40, 64, device="cuda")
    y, x = torch.zeros(8, 64, device="cuda"), b[:8]
    for xo in (b[4:12], b[7:15]):
        with pytest.raises(binding.MGError):
            mg.norm_residual_forward(y, x, xo)
    g = torch.ones(64, device="cuda")
    with pytest.raises(binding.MGError):
        mg.norm_residual_forward(y, x, b[20:28], b[20:28], gamma_pre=g)
    rstd = torch.ones(8, 2, device="cuda")
    ws = torch.zeros(mg.norm_residual_workspace_bytes(8, 64, 0), dtype=torch.uint8, device="cuda")
    for dy, dx in ((b[20:28], b[20:28]), (b[20:28], b[24:32]), (b[4:12], b[20:28])):
        with pytest.raises(binding.MGError):
            mg.norm_residual_backward(b[12:20], None, y, x, rstd, dy, dx, ws)
    with pytest.raises(binding.MGError):
        mg.norm_residual_backward(b[12:20], None, y, x, rstd, b[20:28], b[28:36], ws[:-8])


def test_rows_past_2_31_elements():
    rows, d = 1_100_000, 2048
    y = torch.zeros(rows, d, device="cuda", dtype=torch.bfloat16)
    x = torch.zeros_like(y)
    at = [0, 1, 1_048_575, 1_048_576, 1_048_577, rows - 1]
    j = _inputs(len(at), d, "bf16", 1, True, True, 3)
    y[at], x[at] = j["y"], j["x"]
    i = j | {"y": y, "x": x}
    out = _forward(i, 0.5)
    _forward_check(j, 0.5, tuple(o[at] for o in out), "bf16")
    dxo, dh = torch.zeros_like(y), torch.zeros_like(y)
    dxo[at], dh[at] = j["dxo"], j["dh"]
    o = _backward(i | {"dxo": dxo, "dh": dh}, out[2], 0.5)
    o["dy"], o["dx"] = o["dy"][at], o["dx"][at]
    _backward_check(j, out[2][at], 0.5, o, "bf16")       # the other rows add zeros


@pytest.mark.parametrize("rows,dim,gates,t", [(50, 2048, 1, "bf16"), (21, 777, 3, "f32")])
def test_stream_and_graph(rows, dim, gates, t):
    i = _inputs(rows, dim, t, gates, True, True, 50)
    s = torch.cuda.Stream()
    ws = torch.zeros(mg.norm_residual_workspace_bytes(rows, dim, gates), dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = _forward(i, 0.9, stream=s)
        o = _backward(i, out[2], 0.9, stream=s, ws=ws)
    for seed in (51, 52):
        for k, v in _inputs(rows, dim, t, gates, True, True, seed).items():
            i[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        _forward_check(i, 0.9, out, t)
        _backward_check(i, out[2], 0.9, o, t)


@pytest.mark.parametrize("rows,dim,gates,t", [(40, 12288, 2, "bf16"), (40, 12291, 1, "bf16"), (20, 20000, 1, "f32"), (9, 16385, 3, "f32")])
def test_stream_and_graph_of_wide_rows(rows, dim, gates, t):
    test_stream_and_graph(rows, dim, gates, t)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_host_threads(t):
    """Calls of six host threads at once, each with its own tensors, workspace and stream, of widths that take the same
    kernel with different amounts of shared memory: none fails, and each computes its own."""
    dims = (6144, 8192) if t == "bf16" else (2560, 4096)
    lib, work = binding.load(), []
    for n in range(6):
        i = _inputs(1, dims[n % 2], t, 0, True, True, 90 + n)
        rstd = _forward(i, 0.7)[2]
        ws = torch.zeros(mg.norm_residual_workspace_bytes(1, dims[n % 2], 0), dtype=torch.uint8, device="cuda")
        s, o = torch.cuda.Stream(), _backward(i, rstd, 0.7, ws=ws)
        # (the C call: most of the thread's time passes inside of it, where threads run at once)
        args = (int(t == "bf16"), *(i[k].data_ptr() for k in ("dxo", "dh", "y", "x")), rstd.data_ptr(), 1, dims[n % 2],
                i["g1"].data_ptr(), None, 0, 0.7, i["g2"].data_ptr(), o["dy"].data_ptr(), o["dx"].data_ptr(), None, None, None,
                ws.data_ptr(), ws.nbytes, s.cuda_stream)
        work.append((i, rstd, o, args, s, ws))
    torch.cuda.synchronize()
    for _, _, o, *_ in work:
        o["dy"].fill_(77.0)
        o["dx"].fill_(77.0)
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(work)), []

    def calls(args):
        start.wait()
        failed.append(sum(lib.mg_norm_residual_backward(*args) != 0 for _ in range(4000)))

    threads = [threading.Thread(target=calls, args=(w[3],)) for w in work]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert failed == [0] * len(work)
    for i, rstd, o, *_ in work:
        _backward_check(i, rstd, 0.7, o, t)


def test_two_widths_of_a_kernel_in_one_graph():
    work = []
    for n, dim in enumerate((8192, 6144, 8192)):
        i = _inputs(4, dim, "bf16", 1, True, True, 95 + n)
        work.append((i, torch.zeros(mg.norm_residual_workspace_bytes(4, dim, 1), dtype=torch.uint8, device="cuda")))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph, outs = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph, stream=s):
        for i, ws in work:
            out = _forward(i, 0.7, stream=s)
            outs.append((out, _backward(i, out[2], 0.7, stream=s, ws=ws)))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for (i, _), (out, o) in zip(work, outs):
        _forward_check(i, 0.7, out, "bf16")
        _backward_check(i, out[2], 0.7, o, "bf16")


def test_the_widest_row():
    """A row of 2^30 columns: every column's sum is its own, whatever the workspace held.  Small whole numbers, so that
    all sums are exact: y is 0, 1, 0, 1, ..., t = dx_out = 1, 1 / sqrt of the mean is given as 1."""
    d = 1 << 30
    y = torch.ones(1, d, dtype=torch.bfloat16, device="cuda")
    y[:, ::2] = 0
    dxo = torch.ones_like(y)
    g1 = torch.ones(d, device="cuda")
    rstd = torch.ones(1, 2, device="cuda")
    dy, dx, dg1 = torch.full_like(y, 77.0), torch.full_like(y, 77.0), torch.full_like(g1, 77.0)
    ws = torch.full((mg.norm_residual_workspace_bytes(1, d, 0),), 255, dtype=torch.uint8, device="cuda")
    mg.norm_residual_backward(dxo, None, y, y, rstd, dy, dx, ws, gamma_post=g1, dgamma_post=dg1)
    del ws
    assert (dx == 1).all()
    assert (dg1[::2] == 0).all() and (dg1[1::2] == 1).all()
    assert (dy[0, ::2] == 1).all() and (dy[0, 1::2] == 0.5).all()        # t - y mean(t y)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [200, 777, 2048, 9011, 70001])
@pytest.mark.parametrize("ymag,xmag,eps", [(1e14, 1.0, 1e-6), (1e15, 1e15, 1e-6), (1e16, 1e-3, 1e-6), (1.0, 1e15, 1e-6),
                                           (1e-14, 1e-14, 1e-30), (1.0, 1.0, 1e-30)])
@pytest.mark.parametrize("post", [True, False])
def test_magnitudes(ymag, xmag, eps, dim, post, t, monkeypatch):
    """Rows far from 1 and rows of zeros under a small eps: the cube of 1 / sqrt of the mean leaves fp32's range, the
    gradients do not."""
    monkeypatch.setattr(sys.modules[__name__], "EPS", eps)
    i = _inputs(6, dim, t, 2, post, True, dim)
    i["y"] *= ymag
    i["x"] *= xmag
    i["y"][2] = 0
    i["x"][2] = 0
    i["y"][4] = 0
    out = _forward(i, 0.7)
    _forward_check(i, 0.7, out, t)
    assert torch.isfinite(out[2]).all()
    _backward_check(i, out[2], 0.7, _backward(i, out[2], 0.7), t)
    i["dxo"] = None
    _backward_check(i, out[2], 0.7, _backward(i, out[2], 0.7), t)


# Wider than eight blocks hold: 220 KB of shared memory for two rows of two arrays (fp32: 112640), 512 threads of 32
# elements (131072); the gradients' rows leave the blocks at half of it.
@pytest.mark.parametrize("rows,dim,gates,t", [(3, 112648, 1, "f32"), (2, 131073, 2, "f32"), (2, 131080, 2, "bf16"),
                                              (3, 131073, 1, "bf16"), (2, 200003, 0, "bf16")])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
def test_rows_wider_than_a_cluster(rows, dim, gates, t, post, pre):
    i = _inputs(rows, dim, t, gates, post, pre, dim)
    out = _forward(i, -0.7)
    _forward_check(i, -0.7, out, t)
    o = _backward(i, out[2], -0.7)
    _backward_check(i, out[2], -0.7, o, t)
    o2 = _backward(i, out[2], -0.7, inplace=True)
    assert all(torch.equal(o[k], o2[k]) for k in o)
    i = _inputs(rows, dim, t, gates, post, pre, dim)
    xo, h, rstd = _forward(i, -0.7, inplace=True)
    assert torch.equal(xo, out[0]) and torch.equal(rstd, out[2]) and (h is None or torch.equal(h, out[1]))
