"""Limits of a plan's clipping that fp32 cannot hold, and statistics that would be
written into the gradients."""
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


def test_a_limit_too_small_for_fp32_does_not_turn_clipping_off():
    plan = Plan([W.linear(16, 8, False)], 32, "ce_index", "strict", "sgd")
    p = torch.randn(plan.param_count, device="cuda")
    g, m, v = (torch.zeros_like(p) for _ in range(3))
    x, y = torch.randn(32, 16, device="cuda"), torch.zeros(32, dtype=torch.int32, device="cuda")
    plan.set_grad_clip(0.5)
    with pytest.raises(binding.MGError) as e:
        plan.set_grad_clip(1e-50)
    assert e.value.status == binding.MG_ERR_INVALID_ARG
    plan.train_step(p, g, m, v, x, y, 0.1, 1)          # the limit before still holds
    norm, c = plan.grad_norm()
    assert norm > 0.5 and abs(c * norm - 0.5) <= 1e-6
    plan.set_grad_clip(1e-45)                          # the smallest that fp32 holds
    keep = p.clone()
    plan.train_step(p, g, m, v, x, y, 0.1, 2)
    assert plan.grad_norm()[1] < 1e-44 and torch.equal(p, keep)
    plan.close()


def test_statistics_inside_the_list_are_refused():
    """Blocks would read and write them while others write the norm there."""
    import static_graph_nn_gb300 as mg
    buf = torch.ones(40000, device="cuda")
    out = torch.zeros(3000, device="cuda")
    a, b = buf[64:20000], buf[30000:33000]
    lst = mg.GradList([a, b, buf[0:0]], [a, out, buf[0:0]])
    for stats in (buf[64:66], buf[19998:20000], buf[30000:30002], buf[32998:33000], out[2998:], a[100:102]):
        with pytest.raises(binding.MGError) as e:
            lst.clip(1.0, stats)
        assert e.value.status == binding.MG_ERR_INVALID_ARG
    for stats in (buf[62:64], buf[20000:20002], buf[29998:30000], buf[33000:33002], torch.zeros(2, device="cuda")):
        lst.clip(float("inf"), stats)
        assert abs(float(stats[0]) - 22936 ** 0.5) <= 1e-4
    assert (a == 1).all() and (b == 1).all() and (out == 1).all()
    lst.close()
