"""Sizes beyond 32 bits are refused by the Python calls, not cut to their low bits
(a vocabulary of 2^32 + 5 rows would have been one of 5, and every other id
padding).  Shapes without memory (torch's meta device) stand for such tensors."""
import pytest

import __graft_entry__
from static_graph_nn_gb300 import binding
from static_graph_nn_gb300 import workloads as W

torch = pytest.importorskip("torch")

BIG = 2 ** 32 + 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    __graft_entry__.build()


def _m(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


I32 = torch.int32


@pytest.mark.parametrize("call", [
    lambda: binding.embedding_forward(_m(BIG, 8), _m(4, dtype=I32), _m(4, 8)),
    lambda: binding.embedding_forward(_m(8, BIG), _m(4, dtype=I32), _m(4, BIG)),
    lambda: binding.embedding_backward(_m(4, 8), _m(4, dtype=I32), _m(BIG, 8), _m(1 << 20, dtype=torch.uint8)),
    lambda: binding.grouped_linear_forward(_m(BIG, 8), _m(3, dtype=I32), _m(2, 8, 8), _m(BIG, 8), _m(1 << 20)),
    lambda: binding.grouped_linear_forward(_m(4, BIG), _m(3, dtype=I32), _m(2, BIG, 8), _m(4, 8), _m(1 << 20)),
    lambda: binding.grouped_linear_forward(_m(4, 8), _m(BIG + 1, dtype=I32), _m(BIG, 8, 8), _m(4, 8), _m(1 << 20)),
    lambda: binding.grouped_linear_backward_input(_m(BIG, 8), _m(3, dtype=I32), _m(2, 8, 8), _m(BIG, 8), _m(1 << 20)),
    lambda: binding.grouped_linear_backward_weight(_m(BIG, 8), _m(BIG, 8), _m(3, dtype=I32), _m(2, 8, 8), _m(1 << 20)),
    lambda: binding.grouped_linear_backward_weight(_m(4, 8), _m(4, BIG), _m(3, dtype=I32), _m(2, 8, BIG), _m(1 << 20)),
])
def test_calls_refuse_them(call):
    with pytest.raises(binding.MGError) as e:
        call()
    assert e.value.status in (binding.MG_ERR_SHAPE, binding.MG_ERR_UNSUPPORTED)


def test_workspace_sizes_are_zero():
    assert binding.embedding_workspace_bytes(4, BIG, 8) == 0
    assert binding.embedding_workspace_bytes(4, 8, BIG) == 0
    assert binding.embedding_workspace_bytes(2 ** 64 + 4, 8, 8) == 0
    for i in range(4):
        sizes = [8, 2, 8, 8]
        sizes[i] += 2 ** 32
        assert binding.grouped_linear_workspace_bytes(*sizes) == 0


@pytest.mark.parametrize("layer", [W.embedding(BIG, 8), W.embedding(10, BIG), W.grouped_linear(2, BIG, 8),
                                   W.grouped_linear(2, 8, BIG), W.grouped_linear(BIG, 8, 8)])
def test_layers_refuse_them(layer):
    with pytest.raises(binding.MGError) as e:
        binding.layer_struct(layer)
    assert e.value.status == binding.MG_ERR_SHAPE
