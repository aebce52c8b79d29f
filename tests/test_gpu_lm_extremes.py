"""Calls of the language-model operators at the ends of what they allow: operands
of more than 2^31 elements, as many groups as there may be beside many rows,
buffers aligned to 16 bytes and no more, plans of a single such layer.

Bounds as in the operators' own tests (one 2^-23 step of the running sum per
addition, half a step of the stored type)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import Plan   # noqa: E402
from static_graph_nn_gb300 import workloads as W  # noqa: E402
from test_gpu_embedding import _bwd_check, _ids   # noqa: E402
from test_gpu_grouped_finite import _check, _within   # noqa: E402

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _randn(shape, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=DT[t])


def _ws(rows, e, k, n):
    return torch.zeros(mg.grouped_linear_workspace_bytes(rows, e, k, n), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("t,n", [("bf16", 8192), ("bf16", 8191), ("f32", 8191)])
def test_rows_past_2_31_elements(t, n):
    """rows * d_out beyond 2^31: the ends of the last group and of the one before."""
    rows, k = 265000, 64
    x, w = _randn((rows, k), t, 1), _randn((2, k, n), t, 2)
    off = [0, 264000, rows]
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    ws = _ws(rows, 2, k, n)
    y = torch.full((rows, n), 77.0, dtype=DT[t], device="cuda")
    mg.grouped_linear_forward(x, offs, w, y, ws)
    for a, b, g in ((0, 200, 0), (263800, 264000, 0), (264000, 264200, 1), (264800, rows, 1)):
        xs, we = x[a:b].double(), w[g].double()
        _within(y[a:b], xs @ we, xs.abs() @ we.abs(), k, t)
    # y as the gradient of itself
    dx = torch.full((rows, k), 77.0, dtype=DT[t], device="cuda")
    mg.grouped_linear_backward_input(y, offs, w, dx, ws)
    for a, b, g in ((0, 200, 0), (263800, 264000, 0), (264000, 264200, 1), (264800, rows, 1)):
        ds, we = y[a:b].double(), w[g].double()
        _within(dx[a:b], ds @ we.t(), ds.abs() @ we.abs().t(), n, t)
    dw = torch.full((2, k, n), 77.0, device="cuda")
    mg.grouped_linear_backward_weight(x, y, offs, dw, ws)
    xs, ds = x[264000:].double(), y[264000:].double()
    _within(dw[1], xs.t() @ ds, xs.abs().t() @ ds.abs(), 1000, "f32")
    want, mag = torch.zeros(k, n, dtype=torch.float64, device="cuda"), torch.zeros(k, n, dtype=torch.float64, device="cuda")
    for a in range(0, 264000, 8000):
        xs, ds = x[a:a + 8000].double(), y[a:a + 8000].double()
        want += xs.t() @ ds
        mag += xs.abs().t() @ ds.abs()
    _within(dw[0], want, mag, 264000, "f32")
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("t,n", [("bf16", 8192), ("bf16", 8191), ("f32", 8192)])
def test_weights_past_2_31_elements(t, n):
    rows, e, k = 50, 34, 8192
    w = _randn((e, k, n), t, 1)
    x, dy = _randn((rows, k), t, 2), _randn((rows, n), t, 3)
    off = [0] * 32 + [10, 10, rows]
    ws = _ws(rows, e, k, n)
    y, dx = torch.empty_like(dy), torch.empty_like(x)
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    mg.grouped_linear_forward(x, offs, w, y, ws)
    mg.grouped_linear_backward_input(dy, offs, w, dx, ws)
    for g in (31, 33):
        a, b = off[g], off[g + 1]
        xs, ds, we = x[a:b].double(), dy[a:b].double(), w[g].double()
        _within(y[a:b], xs @ we, xs.abs() @ we.abs(), k, t)
        _within(dx[a:b], ds @ we.t(), ds.abs() @ we.abs().t(), n, t)
    del w
    dw = torch.full((e, k, n), 77.0, device="cuda")
    mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
    for g in (31, 33):
        a, b = off[g], off[g + 1]
        xs, ds = x[a:b].double(), dy[a:b].double()
        _within(dw[g], xs.t() @ ds, xs.abs().t() @ ds.abs(), b - a, "f32")
    assert int(torch.count_nonzero(dw[:31])) == 0 and int(torch.count_nonzero(dw[32])) == 0
    assert int(ws[:4].view(torch.int32)) == 0


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("k,n", [(72, 136), (65, 131)])
def test_1024_groups_of_many_rows(t, k, n):
    rows, e = 17500, 1024
    g = torch.Generator().manual_seed(1)
    off = [0] + torch.randint(0, rows + 1, (e - 1,), generator=g).sort().values.tolist() + [rows]
    x, dy, w = _randn((rows, k), t, 1), _randn((rows, n), t, 2), _randn((e, k, n), t, 3)
    ws = _ws(rows, e, k, n)
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty(e, k, n, device="cuda")
    mg.grouped_linear_forward(x, offs, w, y, ws)
    mg.grouped_linear_backward_input(dy, offs, w, dx, ws)
    mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
    _check(x, dy, w, off, y, dx, dw, t, list(range(0, e, 37)) + [1, e - 2, e - 1])


def _off16(shape, t, fill=None):
    """A dense tensor 16 bytes, not 32, beyond a 256-byte boundary."""
    n = 1
    for s in shape:
        n *= s
    step = 16 // torch.empty(0, dtype=DT[t]).element_size()
    return torch.zeros(n + 2 * step, dtype=DT[t], device="cuda")[step:step + n].view(shape)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("rows,e,k,n", [(700, 3, 128, 256), (24, 8, 512, 1024), (700, 3, 65, 131), (300, 2, 1032, 136)])
def test_buffers_on_16_byte_boundaries(t, rows, e, k, n):
    x, dy, w = _off16((rows, k), t), _off16((rows, n), t), _off16((e, k, n), t)
    for i, a in enumerate((x, dy, w)):
        a.copy_(_randn(a.shape, t, i))
    off = [0] + [rows * (i + 1) // e - i % 2 for i in range(e - 1)] + [rows]
    raw = torch.zeros(mg.grouped_linear_workspace_bytes(rows, e, k, n) + 32, dtype=torch.uint8, device="cuda")
    ws = raw[16:-16]
    offs = torch.zeros(e + 2, dtype=torch.int32, device="cuda")[1:]
    offs.copy_(torch.tensor(off, dtype=torch.int32))
    y, dx, dw = _off16((rows, n), t), _off16((rows, k), t), _off16((e, k, n), "f32")
    mg.grouped_linear_forward(x, offs, w, y, ws)
    mg.grouped_linear_backward_input(dy, offs, w, dx, ws)
    mg.grouped_linear_backward_weight(x, dy, offs, dw, ws)
    _check(x, dy, w, off, y, dx, dw, t, range(e))
    assert int(raw[-16:].count_nonzero()) == 0


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,v,d", [(3000, 500, 64), (3000, 500, 33), (70001, 513, 40), (20, 9, 2048)])
def test_embedding_on_16_byte_boundaries(t, n, v, d):
    table, dout, dtable = _off16((v, d), t), _off16((n, d), t), _off16((v, d), "f32")
    out = _off16((n, d), t)
    table.copy_(_randn((v, d), t, 1))
    dout.copy_(_randn((n, d), t, 2))
    ids = _ids(n, v, "i64", 3, hot=0.2)
    raw = torch.full((mg.embedding_workspace_bytes(n, v, d) + 32,), 7, dtype=torch.uint8, device="cuda")
    mg.embedding_forward(table, ids, out)
    ok = (ids >= 0) & (ids < v)
    assert torch.equal(out[ok], table[ids[ok]]) and int(out[~ok].count_nonzero()) == 0
    mg.embedding_backward(dout, ids, dtable, raw[16:-16], scale=0.5)
    _bwd_check(dout, ids, v, 0.5, dtable)
    assert (raw[-16:] == 7).all() and (raw[:16] == 7).all()


def test_gradient_rows_past_2_31_elements():
    n, v, d = 265000, 7, 8192
    dout = torch.ones(n, d, dtype=torch.bfloat16, device="cuda")
    ids = (torch.arange(n, device="cuda") % 8).to(torch.int32)        # 7: padding
    ids[-1], ids[-2] = 6, 6
    dout[-1] = 3.0
    dt = torch.empty(v, d, device="cuda")
    ws = torch.empty(mg.embedding_workspace_bytes(n, v, d), dtype=torch.uint8, device="cuda")
    mg.embedding_backward(dout, ids, dt, ws)
    for i in range(v):      # whole numbers below 2^24: exact in fp32
        want = float((ids == i).sum()) + (2.0 if i == 6 else 0.0)
        assert (dt[i] == want).all()
    out = torch.empty(n, d, dtype=torch.bfloat16, device="cuda")
    mg.embedding_forward(dout[:7], ids, out, scale=2.0)
    assert (out[-3:-1] == 2.0).all() and (out[-9] == 0).all() == bool(ids[-9] == 7)


@pytest.mark.parametrize("precision", ["strict", "bf16"])
@pytest.mark.parametrize("loss", ["mse", "ce_index"])
def test_plans_of_one_layer(precision, loss):
    """An embedding, or a grouped layer, as a plan's only parameters; a batch of one row."""
    t = torch.float32 if precision == "strict" else torch.bfloat16
    for batch in (1, 77):
        y_ids = torch.randint(0, 16, (batch,), generator=torch.Generator().manual_seed(1), dtype=torch.int32).cuda()
        y = y_ids if loss == "ce_index" else _randn((batch, 16), "f32", 2).to(t)
        for layers in ([W.embedding(9, 16, 0.5)], [W.grouped_linear(3, 24, 16)]):
            plan = Plan(layers, batch, loss, precision, "sgd")
            p = _randn((plan.param_count,), "f32", 3)
            grads, m, v = (torch.zeros_like(p) for _ in range(3))
            o, r, c = plan.param_info()[0]
            w = p[o:o + r * c].view(r, c).clone()
            if precision == "bf16":
                w = w.bfloat16().float()
            w = w.double().requires_grad_()
            if layers[0]["op"] == "embedding":
                x = torch.randint(-1, 9, (batch,), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
                z = w[x.long().clamp_min(0)] * (x >= 0)[:, None] * 0.5
            else:
                x = _randn((batch, 24), "f32", 5).to(t)
                cut = [0, batch // 3, batch // 3, batch]
                plan.set_row_groups(torch.tensor(cut, dtype=torch.int32, device="cuda"))
                z = torch.cat([x[a:b].double() @ w[24 * g:24 * g + 24] for g, (a, b) in enumerate(zip(cut, cut[1:]))])
            if loss == "mse":
                want = ((z - y.double()) ** 2).mean()
            else:
                want = torch.nn.functional.cross_entropy(z, y.long())
            want.backward()
            for step in (1, 2):           # the second call replays a captured graph
                plan.train_step(p.clone() if step == 1 else p, grads, m, v, x, y, 0.0, step)
            got = grads[o:o + r * c].double().view(r, c)
            # bf16: output, loss gradient and its rows each rounded once (2^-8), of cancelling terms
            rel = 1e-4 if precision == "strict" else 2e-2
            want = float(want.detach())
            assert abs(plan.loss() - want) <= rel * abs(want)
            assert float((got - w.grad).abs().max()) <= rel * float(w.grad.abs().max())
            plan.close()
