"""The embedding and grouped-linear layers and gradient clipping inside a training
step: a small language model (ids -> embedding -> residual expert block -> head
-> cross-entropy) against PyTorch autograd in float64, with the parity gates of
the other training-step tests (strict f32: max|a-b|/max|b| <= 1e-4 per gradient
tensor; bf16: gradient cosine >= 0.999, loss within 1e-2)."""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from static_graph_nn_gb300 import Plan, binding   # noqa: E402
from static_graph_nn_gb300 import workloads as W  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


V, D, H, E, B, SCALE = 97, 64, 136, 5, 300, 8.0
LAYERS = [W.embedding(V, D, SCALE), W.residual_begin(), W.rmsnorm(D, 1e-6), W.grouped_linear(E, D, H),
          W.gelu_tanh(), W.grouped_linear(E, H, D), W.residual_end(), W.linear(D, V, True)]


def _params(layers, seed):
    rng = np.random.default_rng(seed)
    out = []
    for name, shape in W.param_shapes(layers):
        if name.endswith("gamma"):
            a = 1.0 + 0.1 * rng.standard_normal(shape)
        elif name.endswith("table"):
            a = 0.1 * rng.standard_normal(shape)
        else:
            a = rng.standard_normal(shape) / math.sqrt(shape[-2] if len(shape) > 1 else 10.0)
        out.append(a.astype(np.float32))
    return out


def _batch(seed, pad=True):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    ids[ids > 60] = 7
    if pad:
        ids[5], ids[B - 1], ids[100] = -1, V, 2 ** 31 - 1
    y = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    return ids.cuda(), y.cuda()


def _reference(layers, params, ids, y, off):
    """Loss and gradients in float64 (torch autograd); rows of no group are zero."""
    ps = [torch.tensor(p, dtype=torch.float64, device="cuda", requires_grad=True) for p in params]
    it = iter(ps)
    x, skip = None, None

    def gelu(z):
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))

    for l in layers:
        op = l["op"]
        if op == "embedding":
            t, i = next(it), ids.long()
            ok = (i >= 0) & (i < l["vocab"])
            x = t[torch.where(ok, i, 0)] * ok[:, None] * l["scale"]
        elif op == "rmsnorm":
            x = x / torch.sqrt((x * x).mean(1, keepdim=True) + l["eps"]) * next(it)
        elif op == "grouped_linear":
            w = next(it)
            out = torch.zeros(x.shape[0], l["d_out"], dtype=torch.float64, device="cuda")
            parts = [(a, b, x[a:b] @ w[e]) for e, (a, b) in enumerate(zip(off, off[1:])) if b > a]
            out = torch.cat([torch.zeros(off[0], l["d_out"], dtype=torch.float64, device="cuda")]
                            + [q for _, _, q in parts]
                            + [torch.zeros(x.shape[0] - off[-1], l["d_out"], dtype=torch.float64, device="cuda")])
            x = out
        elif op == "linear":
            x = x @ next(it)
            if l["bias"]:
                x = x + next(it)
        elif op == "gelu_tanh":
            x = gelu(x)
        elif op == "relu":
            x = torch.relu(x)
        elif op == "residual_begin":
            skip = x
        elif op == "residual_end":
            x = x + skip
    loss = torch.nn.functional.cross_entropy(x, y.long())
    loss.backward()
    return float(loss.detach()), [p.grad.cpu().numpy() for p in ps]


class Run:
    def __init__(self, layers, precision, optimizer, params, batch=B):
        self.plan = Plan(layers, batch, "ce_index", precision, optimizer)
        flat = torch.full((self.plan.param_count,), float("nan"))     # gaps are never touched
        self.info = self.plan.param_info()
        for (o, r, c), t in zip(self.info, params):
            assert r * c == t.size
            flat[o:o + r * c] = torch.from_numpy(t.reshape(-1))
        self.params = flat.cuda()
        self.grads, self.m, self.v = (torch.zeros_like(self.params) for _ in range(3))

    def step(self, ids, y, t, lr=1e-2, stream=None):
        self.plan.train_step(self.params, self.grads, self.m, self.v, ids, y, lr, t, stream)

    def tensors(self, flat):
        f = flat.cpu().numpy()
        return [f[o:o + r * c] for o, r, c in self.info]


def _compare(got, want, precision):
    for i, (g, w) in enumerate(zip(got, want)):
        w = w.reshape(-1)
        g = g.astype(np.float64)
        if precision == "strict":
            assert np.abs(g - w).max() <= 1e-4 * np.abs(w).max(), i
        else:
            assert g @ w >= 0.999 * np.linalg.norm(g) * np.linalg.norm(w), i


OFFS = {"ragged": [0, 41, 41, 150, 291, 300], "gaps": [20, 21, 100, 100, 180, 270],
        "one": [0, 0, 0, 300, 300, 300]}


@pytest.mark.parametrize("off", sorted(OFFS))
@pytest.mark.parametrize("precision", ["strict", "bf16"])
def test_gradients(precision, off):
    off = OFFS[off]
    params = _params(LAYERS, 1)
    run = Run(LAYERS, precision, "sgd", params)
    run.plan.set_row_groups(torch.tensor(off, dtype=torch.int32, device="cuda"))
    ids, y = _batch(2)
    want_loss, want = _reference(LAYERS, params, ids, y, off)
    run.step(ids, y, 1)
    assert abs(run.plan.loss() - want_loss) <= (1e-4 if precision == "strict" else 1e-2) * want_loss
    _compare(run.tensors(run.grads), want, precision)
    # forward on its own, from the starting parameters
    run2 = Run(LAYERS, precision, "sgd", params)
    run2.plan.set_row_groups(torch.tensor(off, dtype=torch.int32, device="cuda"))
    out = torch.empty(B, V, device="cuda")
    run2.plan.forward(run2.params, ids, out)
    loss = float(torch.nn.functional.cross_entropy(out.double(), y.long()))
    assert abs(loss - want_loss) <= (1e-4 if precision == "strict" else 1e-2) * want_loss


@pytest.mark.parametrize("precision", ["strict", "bf16"])
def test_small_batch_and_odd_widths(precision):
    """A few rows per group (the weight-streaming kernel in bf16), widths that are
    no multiples of 8, ReLU, an embedding straight into a grouped layer."""
    for d, h, batch, off in ((64, 136, 9, [0, 2, 2, 3, 8, 8]), (33, 50, 21, [1, 2, 9, 9, 9, 20])):
        layers = [W.embedding(V, d, 0.5), W.grouped_linear(E, d, h), W.relu(), W.grouped_linear(E, h, d),
                  W.linear(d, V, False)]
        params = _params(layers, 3)
        run = Run(layers, precision, "sgd", params, batch=batch)
        run.plan.set_row_groups(torch.tensor(off, dtype=torch.int32, device="cuda"))
        ids, y = _batch(4, pad=False)
        ids, y = ids[:batch].clone(), y[:batch].clone()
        want_loss, want = _reference(layers, params, ids, y, off)
        run.step(ids, y, 1)
        assert abs(run.plan.loss() - want_loss) <= (1e-4 if precision == "strict" else 1e-2) * want_loss
        _compare(run.tensors(run.grads), want, precision)


@pytest.mark.parametrize("optimizer", ["sgd", "adam", "laprop", "sgd_momentum"])
@pytest.mark.parametrize("precision", ["strict", "bf16"])
def test_clipping(precision, optimizer):
    """With clipping on, the optimizer sees factor * gradient: the same step of an
    unclipped plan with a scaled loss does not exist, so the update is repeated on
    the host in float64 from the step's own gradients."""
    off = OFFS["ragged"]
    offs = torch.tensor(off, dtype=torch.int32, device="cuda")
    params = _params(LAYERS, 5)
    run, free = (Run(LAYERS, precision, optimizer, params) for _ in range(2))
    run.plan.set_row_groups(offs)
    free.plan.set_row_groups(offs)
    ids, y = _batch(6)
    free.step(ids, y, 1)
    norm = math.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in free.tensors(free.grads)))
    run.plan.set_grad_clip(norm / 3)
    lr, b1, b2, eps = 1e-2, 0.9, 0.999, 1e-8
    p = [a.astype(np.float64).reshape(-1) for a in params]
    m, v = [np.zeros_like(a) for a in p], [np.zeros_like(a) for a in p]
    for t in (1, 2, 3, 4):                       # the second call on replays a graph
        run.step(ids, y, t, lr)
        g = [a.astype(np.float64) for a in run.tensors(run.grads)]
        want_norm = math.sqrt(sum(float((a ** 2).sum()) for a in g))
        c = min(1.0, norm / 3 / want_norm)
        got_norm, got_c = run.plan.grad_norm()
        assert abs(got_norm - want_norm) <= 1e-6 * want_norm and abs(got_c - c) <= 1e-6 * c
        if t == 1:
            # unclipped gradients: as the plan without clipping leaves them
            assert all(np.array_equal(a, b) for a, b in zip(run.tensors(run.grads), free.tensors(free.grads)))
            assert c < 0.34
        for i in range(len(p)):
            gi = g[i] * c
            if optimizer == "sgd":
                p[i] -= lr * gi
            elif optimizer == "sgd_momentum":
                m[i] = b1 * m[i] + gi
                p[i] -= lr * m[i]
            else:
                v[i] = b2 * v[i] + (1 - b2) * gi * gi
                root = np.sqrt(v[i] / (1 - b2 ** t)) + eps
                m[i] = b1 * m[i] + (1 - b1) * (gi if optimizer == "adam" else gi / root)
                p[i] -= lr / (1 - b1 ** t) * (m[i] / root if optimizer == "adam" else m[i])
        for i, (a, w) in enumerate(zip(run.tensors(run.params), p)):
            # fp32 arithmetic of the update: some 2^-24 steps of the parameter and of
            # the movement, amplified where a normalised update divides tiny numbers
            assert np.abs(a - w).max() <= 2e-5 * max(np.abs(w).max(), lr), (t, i)
            p[i] = a.astype(np.float64)          # teacher-forced
        for buf, mine in ((run.m, m), (run.v, v)):
            for i, a in enumerate(run.tensors(buf)):
                if optimizer != "sgd" and (buf is run.m or optimizer in ("adam", "laprop")):
                    mine[i] = a.astype(np.float64)
    assert run.plan.graph_replays() > 0


def test_clipping_on_and_off():
    """Measuring only (infinity) and off again leave the updates bitwise as without."""
    offs = torch.tensor(OFFS["ragged"], dtype=torch.int32, device="cuda")
    params = _params(LAYERS, 7)
    a, b = (Run(LAYERS, "bf16", "adam", params) for _ in range(2))
    a.plan.set_row_groups(offs)
    b.plan.set_row_groups(offs)
    assert b.plan.grad_norm_device_ptr() is None
    with pytest.raises(binding.MGError):
        b.plan.grad_norm()
    ids, y = _batch(8)
    for t in range(1, 9):
        if t == 3:
            b.plan.set_grad_clip(math.inf)
        if t == 6:
            b.plan.set_grad_clip(0.0)
        a.step(ids, y, t)
        b.step(ids, y, t)
        assert torch.equal(a.params[~torch.isnan(a.params)], b.params[~torch.isnan(b.params)])
    assert b.plan.grad_norm()[1] == 1.0
    for bad in (-1.0, float("nan")):
        with pytest.raises(binding.MGError):
            b.plan.set_grad_clip(bad)


def test_clipping_keeps_nan_visible():
    layers = [W.linear(16, 24, True), W.relu(), W.linear(24, 10, False)]
    params = _params(layers, 9)
    run = Run(layers, "strict", "sgd", params, batch=32)
    run.plan.set_grad_clip(1.0)
    x = torch.randn(32, 16, device="cuda")
    x[3, 3] = float("nan")
    y = torch.zeros(32, dtype=torch.int32, device="cuda")
    run.step(x, y, 1)
    norm, c = run.plan.grad_norm()
    assert math.isnan(norm) and c == 1.0


def test_row_groups_change_between_steps():
    """New offset values in the same buffer reach replayed steps; a new buffer too."""
    params = _params(LAYERS, 10)
    run = Run(LAYERS, "strict", "sgd", params)
    ids, y = _batch(11)
    with pytest.raises(binding.MGError):
        run.step(ids, y, 1)                      # not set yet
    offs = torch.tensor(OFFS["ragged"], dtype=torch.int32, device="cuda")
    run.plan.set_row_groups(offs)
    for t, name in enumerate(["ragged", "gaps", "one", "gaps", "ragged"], 1):
        if t == 4:
            offs = torch.empty(E + 1, dtype=torch.int32, device="cuda")
            run.plan.set_row_groups(offs)
        offs.copy_(torch.tensor(OFFS[name], dtype=torch.int32))
        cur = [a.copy() for a in run.tensors(run.params)]
        shaped = [a.reshape(s) for a, (_, s) in zip(cur, W.param_shapes(LAYERS))]
        _, want = _reference(LAYERS, shaped, ids, y, OFFS[name])
        run.step(ids, y, t, lr=0.1)
        _compare(run.tensors(run.grads), want, "strict")


def test_recompute_and_checkpoint():
    """GELU recomputation leaves grouped layers' results alone, and a checkpoint of
    the model restores bit for bit."""
    import os
    offs = torch.tensor(OFFS["gaps"], dtype=torch.int32, device="cuda")
    layers = LAYERS[:-1] + [W.linear(D, H, False), W.gelu_tanh(), W.linear(H, V, True)]
    params = _params(layers, 12)
    ids, y = _batch(13)
    plain = Run(layers, "strict", "adam", params)
    os.environ["MG_RECOMPUTE_GELU"] = "1"
    try:
        again = Run(layers, "strict", "adam", params)
    finally:
        del os.environ["MG_RECOMPUTE_GELU"]
    for r in (plain, again):
        r.plan.set_row_groups(offs)
        for t in (1, 2, 3):
            r.step(ids, y, t)
    assert all(np.array_equal(a, b) for a, b in zip(plain.tensors(plain.params), again.tensors(again.params)))
    img = plain.plan.checkpoint_save(plain.params, plain.m, plain.v)
    other = Run(layers, "strict", "adam", _params(layers, 99))
    other.plan.set_row_groups(offs)
    other.plan.checkpoint_load(img, other.params, other.m, other.v)
    for r in (plain, other):
        r.step(ids, y, 4)
    assert all(np.array_equal(a, b) for a, b in zip(plain.tensors(plain.params), other.tensors(other.params)))


def test_operators_together_without_a_plan():
    """Routing by hand: rows gathered by expert with the embedding lookup, expert
    products, rows summed back with its gradient, all gradients clipped as one
    list -- against float64 autograd."""
    import static_graph_nn_gb300 as mg
    n, d, h, e, k = 200, 64, 96, 4, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, d, generator=g, device="cuda")
    w1 = torch.randn(e, d, h, generator=g, device="cuda") / 8
    dy = torch.randn(n * k, h, generator=g, device="cuda")
    expert = torch.randint(0, e, (n * k,), generator=g, device="cuda")
    order = torch.argsort(expert, stable=True)
    token = (order // k).to(torch.int32)
    off = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.cumsum(torch.bincount(expert, minlength=e), 0)
    xs, y = torch.empty(n * k, d, device="cuda"), torch.empty(n * k, h, device="cuda")
    dxs, dx, dw = torch.empty(n * k, d, device="cuda"), torch.empty(n, d, device="cuda"), torch.empty_like(w1)
    ws = torch.zeros(mg.grouped_linear_workspace_bytes(n * k, e, d, h), dtype=torch.uint8, device="cuda")
    ews = torch.empty(mg.embedding_workspace_bytes(n * k, n, d), dtype=torch.uint8, device="cuda")
    mg.embedding_forward(x, token, xs)
    mg.grouped_linear_forward(xs, off, w1, y, ws)
    mg.grouped_linear_backward_weight(xs, dy, off, dw, ws)
    mg.grouped_linear_backward_input(dy, off, w1, dxs, ws)
    mg.embedding_backward(dxs, token, dx, ews)
    stats = torch.empty(2, device="cuda")
    raw = [dx.clone(), dw.clone()]
    lst = mg.GradList([dx, dw])
    lst.clip(1.0, stats)
    xr, wr = x.double().requires_grad_(), w1.double().requires_grad_()
    yr = torch.einsum("td,tdh->th", xr[token.long()], wr[expert[order]])
    yr.backward(dy.double())
    assert (y.double() - yr).abs().max() <= 1e-4 * yr.abs().max()
    norm = math.sqrt(float(xr.grad.square().sum() + wr.grad.square().sum()))
    assert abs(float(stats[0]) - norm) <= 1e-4 * norm
    for got, full, want in zip((dx, dw), raw, (xr.grad, wr.grad)):
        assert (full.double() - want).abs().max() <= 1e-4 * want.abs().max()
        assert (got.double() - want / norm).abs().max() <= 1e-4 * want.abs().max() / norm
    lst.close()


def test_plan_refuses_wrong_ids_and_offsets():
    run = Run(LAYERS, "strict", "sgd", _params(LAYERS, 20))
    ids, y = _batch(21)
    with pytest.raises(binding.MGError):
        run.plan.set_row_groups(torch.zeros(E, dtype=torch.int32, device="cuda"))
    with pytest.raises(binding.MGError):
        run.plan.set_row_groups(torch.zeros(E + 1, dtype=torch.int32))        # host memory
    run.plan.set_row_groups(torch.tensor(OFFS["ragged"], dtype=torch.int32, device="cuda"))
    for bad in (ids.long(), ids[:-1], ids.float()):
        with pytest.raises(binding.MGError):
            run.step(bad, y, 1)
    linear = Run([W.linear(16, 4, False)], "strict", "sgd", _params([W.linear(16, 4, False)], 1), batch=8)
    with pytest.raises(binding.MGError):
        linear.plan.set_row_groups(torch.zeros(3, dtype=torch.int32, device="cuda"))


def test_step_on_a_side_stream_inside_a_capture():
    """A whole clipped step with embedding and grouped layers captured by the caller
    gives what an eager one gives."""
    params = _params(LAYERS, 22)
    offs = torch.tensor(OFFS["gaps"], dtype=torch.int32, device="cuda")
    ids, y = _batch(23)
    a, b = (Run(LAYERS, "bf16", "sgd", params) for _ in range(2))
    for r in (a, b):
        r.plan.set_row_groups(offs)
        r.plan.set_grad_clip(0.1)
        r.step(ids, y, 1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.step(ids, y, 2, stream=s)
    for t in (2, 3):
        a.step(ids, y, t)
        g.replay()
    torch.cuda.synchronize()
    assert all(np.array_equal(u, v) for u, v in zip(a.tensors(a.params), b.tensors(b.params)))
    assert a.plan.grad_norm() == b.plan.grad_norm()
