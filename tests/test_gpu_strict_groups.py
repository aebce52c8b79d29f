"""Strict plans: a grouped layer's forward follows the rule of the dense ones, sums
that carry their rounding errors, so that the stored value is the correctly
rounded one and a ReLU decides on the sign of the exact pre-activation.

Tolerance of such a sum of K products: half a step of the exact value, and (K
2^-24)^2 of the sum of the magnitudes (the errors of the error terms)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from static_graph_nn_gb300 import Plan   # noqa: E402
from static_graph_nn_gb300 import workloads as W  # noqa: E402

U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _flat(plan, tensors):
    flat = torch.zeros(plan.param_count, device="cuda")
    for (o, r, c), t in zip(plan.param_info(), tensors):
        flat[o:o + r * c] = t.reshape(-1)
    return flat


def _randn(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


# rows, groups, d_in, d_out, offsets' ends: one launch; sums split over blocks
# (few tiles, long sums); odd widths; a few rows
@pytest.mark.parametrize("rows,e,k,n,first,last", [
    (5000, 5, 200, 328, 0, 5000), (700, 3, 601, 1003, 20, 650), (1, 1, 8, 8, 0, 1), (24, 8, 512, 72, 0, 24),
    (20, 3, 2048, 200, 1, 19), (300, 2, 1032, 136, 0, 300), (77, 3, 33, 17, 10, 70), (40, 3, 64, 136, 40, 40)])
def test_forward_is_correctly_rounded(rows, e, k, n, first, last):
    x, w = _randn((rows, k), 1), _randn((e, k, n), 2)
    cut = torch.randint(first, last + 1, (e - 1,), generator=torch.Generator().manual_seed(3)).sort().values.tolist()
    off = [first] + cut + [last]
    plan = Plan([W.grouped_linear(e, k, n)], rows, "mse", "strict", "sgd")
    plan.set_row_groups(torch.tensor(off, dtype=torch.int32, device="cuda"))
    out = torch.full((rows, n), 7.0, device="cuda")
    plan.forward(_flat(plan, [w]), x, out)
    assert (out[:first] == 0).all() and (out[last:] == 0).all()
    for g in range(e):
        a, b = off[g], off[g + 1]
        xs, ws = x[a:b].double(), w[g].double()
        want, mag = xs @ ws, xs.abs() @ ws.abs()
        assert ((out[a:b].double() - want).abs() <= 1.001 * U32 * want.abs() + (k * U32) ** 2 * mag).all()
    plan.close()


def test_infinities_stay_infinite():
    """A sum that is infinite has no error term; it stays what it is."""
    x, w = torch.ones(70, 64, device="cuda"), torch.ones(1, 64, 65, device="cuda")
    x[3, 5], x[9, 7], w[0, 2, 64] = float("inf"), 3e38, -3e38
    x[9, 2] = -3.0
    plan = Plan([W.grouped_linear(1, 64, 65)], 70, "mse", "strict", "sgd")
    plan.set_row_groups(torch.tensor([0, 70], dtype=torch.int32, device="cuda"))
    out = torch.empty(70, 65, device="cuda")
    plan.forward(_flat(plan, [w]), x, out)
    assert torch.isinf(out[3, :64]).all() and (out[3, :64] > 0).all()
    assert float(out[9, 64]) == float("inf")       # 3e38 + 9e38
    assert not torch.isnan(out).any()
    plan.close()


def test_relu_decides_on_the_exact_sign():
    """Pre-activations near 0 beside large terms: x = [u, -u], W = [V; V + small].  A
    sum off by a rounding takes the other side of the ReLU and moves a weight gradient
    far past the gate (max|a - b| <= 1e-4 max|b|)."""
    rows, e, half, h, c = 4000, 4, 300, 256, 10
    u, v = _randn((rows, half), 1), _randn((e, half, h), 2)
    x = torch.cat([u, -u], 1)
    w1 = torch.cat([v, v * (1 + 2.0 ** -18 * _randn((e, half, h), 3))], 1)
    w2 = _randn((h, c), 4) / 16
    off = [0, 900, 900, 2500, 4000]
    y = torch.randint(0, c, (rows,), generator=torch.Generator().manual_seed(5), dtype=torch.int32).cuda()
    layers = [W.grouped_linear(e, 2 * half, h), W.relu(), W.linear(h, c, False)]
    plan = Plan(layers, rows, "ce_index", "strict", "sgd")
    plan.set_row_groups(torch.tensor(off, dtype=torch.int32, device="cuda"))
    scale = 4096.0          # the pre-activations to about 0.3
    params = _flat(plan, [w1 * scale, w2])
    grads, m, vv = (torch.zeros_like(params) for _ in range(3))
    plan.train_step(params.clone(), grads, m, vv, x, y, 0.1, 1)
    p1, p2 = (w1 * scale).double().requires_grad_(), w2.double().requires_grad_()
    z = torch.cat([x[a:b].double() @ p1[i] for i, (a, b) in enumerate(zip(off, off[1:]))])
    torch.nn.functional.cross_entropy(torch.relu(z) @ p2, y.long()).backward()
    for (o, r, cc), want in zip(plan.param_info(), (p1.grad, p2.grad)):
        got = grads[o:o + r * cc].double()
        want = want.reshape(-1)
        assert float((got - want).abs().max()) <= 1e-4 * float(want.abs().max())
    plan.close()


def test_steps_repeat_and_replay():
    """Replayed steps of a plan whose forward is split give the bits of launched ones."""
    rows, e, k, n = 300, 2, 1032, 136
    layers = [W.grouped_linear(e, k, n), W.relu(), W.linear(n, 10, True)]
    off = torch.tensor([7, 100, 290], dtype=torch.int32, device="cuda")
    x = _randn((rows, k), 1)
    y = torch.zeros(rows, dtype=torch.int32, device="cuda")
    res = []
    for _ in range(2):
        plan = Plan(layers, rows, "ce_index", "strict", "adam")
        plan.set_row_groups(off)
        g = np.random.default_rng(3)
        p = _flat(plan, [torch.from_numpy(g.standard_normal(s).astype(np.float32) / 30).cuda()
                         for _, s in W.param_shapes(layers)])
        grads, m, v = (torch.zeros_like(p) for _ in range(3))
        for t in range(1, 5):
            plan.train_step(p, grads, m, v, x, y, 1e-3, t)
        res.append(p.clone())
        plan.close()
    assert torch.equal(*res)
