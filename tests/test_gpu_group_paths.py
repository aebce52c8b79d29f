"""Which kernels a plan's grouped layers run on, and that the plan says so."""
import re

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from static_graph_nn_gb300 import Plan   # noqa: E402
from static_graph_nn_gb300 import workloads as W  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _sites(plan):
    """{kernel's role: the path it is said to take} of the grouped products."""
    return {m[1]: m[2] for m in re.finditer(r"kernel \d+: (grouped_\w+)\[l\d+\] .* (\S+)  \(", plan.dump())}


def _step(layers, batch, off, monkeypatch=None):
    if monkeypatch:
        monkeypatch.setenv("MG_GEMM", "simt")
    plan = Plan(layers, batch, "ce_index", "bf16", "sgd")
    plan.set_row_groups(torch.tensor(off, dtype=torch.int32, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(1)
    p = torch.randn(plan.param_count, generator=g, device="cuda") / 16
    x = torch.randn(batch, layers[0]["d_in"], generator=g, device="cuda").bfloat16()
    y = torch.randint(0, layers[-1]["d_out"], (batch,), generator=g, device="cuda", dtype=torch.int32)
    grads, m, v = (torch.zeros_like(p) for _ in range(3))
    plan.train_step(p, grads, m, v, x, y, 0.1, 1)
    return plan, grads


@pytest.mark.parametrize("rows,k,h", [(600, 256, 512), (20, 512, 264), (600, 264, 1003)])
def test_simt_switch(rows, k, h, monkeypatch):
    """MG_GEMM=simt: CUDA-core products only, grouped ones too; the gradients are
    the tensor cores' within the rounding of bf16 values."""
    layers = [W.linear(k, k, False), W.grouped_linear(4, k, h), W.gelu_tanh(), W.linear(h, 16, False)]
    off = [0, rows // 3, rows // 3, rows // 2, rows - 1]
    tc, want = _step(layers, rows, off)
    assert "tcgen05" in tc.dump()
    simt, got = _step(layers, rows, off, monkeypatch)
    assert "tcgen05" not in simt.dump()
    assert set(_sites(simt)) == {"grouped_fwd", "grouped_dW", "grouped_dX"}
    for o, r, c in tc.param_info():
        a, b = got[o:o + r * c].double(), want[o:o + r * c].double()
        assert float(a @ b) >= 0.999 * float(a.norm() * b.norm())
    tc.close()
    simt.close()


def test_each_product_is_named_by_its_own_path():
    """Odd widths, a few rows: the forward is worth the tensor cores, the weight
    gradient is not, nor is an input gradient of a short sum."""
    layers = [W.linear(128, 128, False), W.grouped_linear(8, 128, 65), W.linear(65, 16, False)]
    plan, _ = _step(layers, 24, [0, 3, 3, 9, 12, 13, 20, 22, 24])
    assert _sites(plan) == {"grouped_fwd": "bf16-tcgen05", "grouped_dW": "bf16-simt", "grouped_dX": "bf16-simt"}
    plan.close()
    layers = [W.linear(128, 128, False), W.grouped_linear(4, 128, 256), W.linear(256, 16, False)]
    plan, _ = _step(layers, 600, [0, 100, 200, 200, 600])
    assert set(_sites(plan).values()) == {"bf16-tcgen05"}
    plan.close()
