"""Limits of a plan's clipping that fp32 cannot hold."""
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
