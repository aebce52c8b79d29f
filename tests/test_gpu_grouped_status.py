"""A device-side wait that gave up reaches the callers of the grouped products: the
workspace's first int, as the kernels leave it, becomes an error."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float32])
def test_status(t):
    rows, e, k, n = 300, 3, 64, 136
    x, w = torch.randn(rows, k, device="cuda").to(t), torch.randn(e, k, n, device="cuda").to(t)
    off = torch.tensor([0, 10, 200, 300], dtype=torch.int32, device="cuda")
    y = torch.empty(rows, n, dtype=t, device="cuda")
    ws = torch.zeros(mg.grouped_linear_workspace_bytes(rows, e, k, n), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mg.grouped_linear_forward(x, off, w, y, ws, stream=s)
    mg.grouped_linear_status(ws, stream=s)                  # waits: y is there
    assert torch.isfinite(y).all()
    ws[:4].view(torch.int32).fill_(1)                       # as a kernel that gave up leaves it
    mg.grouped_linear_forward(x, off, w, y, ws)             # a later call does not take it back
    with pytest.raises(binding.MGError) as err:
        mg.grouped_linear_status(ws)
    assert err.value.status == binding.MG_ERR_TIMEOUT
    ws.zero_()
    mg.grouped_linear_status(ws)


def test_refusals():
    for bad, want in ((0, binding.MG_ERR_INVALID_ARG), (torch.zeros(8, device="cuda").data_ptr() + 4, binding.MG_ERR_ALIGN)):
        assert binding.load().mg_grouped_linear_status(bad, None) == want
    with pytest.raises(binding.MGError):
        mg.grouped_linear_status(torch.zeros(64, dtype=torch.uint8))         # host memory
