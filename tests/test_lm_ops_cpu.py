"""Refusals of the language-model operators, all before any device work (no GPU):
the C entry points' checks of types, sizes, pointers and workspaces, and the
Python wrappers' checks of shapes, types and layouts."""
import ctypes

import pytest

import __graft_entry__
from static_graph_nn_gb300 import binding
from static_graph_nn_gb300 import workloads as W

torch = pytest.importorskip("torch")

E, S, A, U = (binding.MG_ERR_INVALID_ARG, binding.MG_ERR_SHAPE, binding.MG_ERR_ALIGN,
              binding.MG_ERR_UNSUPPORTED)
P = 4096          # an aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load()


def _fwd(lib, tt=0, table=P, v=10, d=8, kind=0, ids=P, n=4, scale=1.0, ot=0, out=P):
    return lib.mg_embedding_forward(tt, table, v, d, kind, ids, n, scale, ot, out, None)


def _bwd(lib, t=0, dout=P, v=10, d=8, kind=0, ids=P, n=4, scale=1.0, dtable=P, ws=P, nb=1 << 30):
    return lib.mg_embedding_backward(t, dout, v, d, kind, ids, n, scale, dtable, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tt=2), E), (dict(ot=-1), E), (dict(kind=2), E), (dict(v=0), S), (dict(d=0), S),
    (dict(v=2**31 - 1), S), (dict(n=-1), S), (dict(n=2**31), S), (dict(scale=float("nan")), E),
    (dict(scale=float("inf")), E), (dict(table=None), E), (dict(ids=None), E), (dict(out=None), E),
    (dict(table=P + 8), A), (dict(out=P + 2), A), (dict(ids=P + 2), A), (dict(ids=P + 4, kind=1), A),
])
def test_embedding_forward_refusals(lib, kw, want):
    assert _fwd(lib, **kw) == want
    assert b"mg_embedding_forward" in lib.mg_last_error(None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=2), E), (dict(kind=-1), E), (dict(v=0), S), (dict(d=-3), S), (dict(n=-1), S),
    (dict(scale=float("inf")), E), (dict(dout=None), E), (dict(ids=None), E), (dict(dtable=None), E),
    (dict(ws=None), E), (dict(nb=16), E), (dict(dtable=P + 4), A), (dict(ws=P + 1), A),
])
def test_embedding_backward_refusals(lib, kw, want):
    assert _bwd(lib, **kw) == want
    assert b"mg_embedding_backward" in lib.mg_last_error(None)


def test_workspace_sizes(lib):
    assert lib.mg_embedding_workspace_bytes(-1, 10, 8) == 0
    assert lib.mg_embedding_workspace_bytes(4, 0, 8) == 0
    assert lib.mg_embedding_workspace_bytes(0, 10, 8) > 0
    assert lib.mg_embedding_workspace_bytes(1 << 20, 32000, 64) > (1 << 20) * 16
    assert lib.mg_grouped_linear_workspace_bytes(8, 0, 8, 8) == 0
    assert lib.mg_grouped_linear_workspace_bytes(8, 1025, 8, 8) == 0
    assert lib.mg_grouped_linear_workspace_bytes(0, 1, 8, 8) >= 4


@pytest.mark.parametrize("groups,k,n", [(1, 8, 8), (1, 1224, 3148), (8, 2048, 8192), (3, 601, 1003), (64, 4096, 64),
                                        (2, 64, 16384)])
def test_a_workspace_serves_fewer_rows(lib, groups, k, n):
    sizes = [lib.mg_grouped_linear_workspace_bytes(r, groups, k, n)
             for r in (0, 1, 2, 17, 64, 100, 111, 257, 300, 1000, 4099, 9000, 40000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    sizes = [lib.mg_embedding_workspace_bytes(r, n, k)
             for r in (0, 1, 8, 100, 2432, 4863, 4864, 4865, 9000, 16384, 65536, 65537, 200000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("sizes", [(2**30 + 1, 2, 8, 8), (4, 2, 2**30 + 1, 8), (4, 2, 8, 2**31 - 1)])
def test_sizes_beyond_an_int_of_tiles_are_refused(lib, sizes):
    rows, groups, k, n = sizes
    assert lib.mg_grouped_linear_workspace_bytes(rows, groups, k, n) == 0
    for which in ("forward", "backward_input", "backward_weight"):
        assert _grouped(lib, which, rows=rows, groups=groups, k=k, n=n) == S
    assert lib.mg_embedding_workspace_bytes(4, 10, 2**30 + 1) == 0
    assert _fwd(lib, d=2**30 + 1) == S
    assert _bwd(lib, d=2**31 - 1) == S
    assert _create(lib, [W.embedding(10, 2**30 + 1), W.linear(2**30 + 1, 4, False)]) == S
    assert _create(lib, [W.grouped_linear(1, 8, 2**30 + 1)]) == S


def _grouped(lib, which, dtype=1, a=P, b=P, off=P, rows=4, groups=2, k=8, n=8, out=P, ws=P, nb=1 << 30):
    if which == "backward_weight":
        return lib.mg_grouped_linear_backward_weight(dtype, a, b, off, rows, groups, k, n, out, ws, nb, None)
    f = getattr(lib, "mg_grouped_linear_" + which)
    return f(dtype, a, off, rows, groups, k, n, b, out, ws, nb, None)


@pytest.mark.parametrize("which", ["forward", "backward_input", "backward_weight"])
@pytest.mark.parametrize("kw,want", [
    (dict(dtype=2), E), (dict(rows=-1), S), (dict(groups=0), S), (dict(groups=1025), U), (dict(k=0), S),
    (dict(n=-8), S), (dict(a=None), E), (dict(b=None), E), (dict(off=None), E), (dict(out=None), E),
    (dict(ws=None), E), (dict(nb=3), E), (dict(a=P + 2), A), (dict(b=P + 4), A), (dict(off=P + 2), A),
    (dict(out=P + 8), A), (dict(ws=P + 4), A),
])
def test_grouped_linear_refusals(lib, which, kw, want):
    assert _grouped(lib, which, **kw) == want
    assert ("mg_grouped_linear_" + which).encode() in lib.mg_last_error(None)


def _list(lib, ptrs, counts, types, out=None):
    n = len(ptrs)
    h = ctypes.c_void_p()
    VP = ctypes.c_void_p
    st = lib.mg_grad_list_create(n, (VP * max(1, n))(*ptrs), (VP * max(1, n))(*out) if out else None,
                                 (ctypes.c_size_t * max(1, n))(*counts),
                                 (ctypes.c_int * max(1, n))(*types), ctypes.byref(h))
    return st, h


@pytest.mark.parametrize("args,want", [
    (([], [], []), E), (([P], [4], [2]), E), (([None], [4], [0]), E), (([P + 2], [4], [0]), A),
    (([P + 1], [4], [1]), A), (([P], [2**60], [0]), S), (([P], [2**41], [1]), S),
    (([P], [4], [0], [None]), E), (([P], [4], [0], [P + 2]), A),
])
def test_grad_list_refusals(lib, args, want):
    st, h = _list(lib, *args)
    assert st == want
    assert h.value is None


def test_grad_list_null_arguments(lib):
    assert lib.mg_grad_list_create(1, None, None, None, None, None) == E
    h = ctypes.c_void_p()
    assert lib.mg_grad_list_create(1, None, None, None, None, ctypes.byref(h)) == E
    assert lib.mg_grad_list_clip(None, 1.0, P, None) == E
    lib.mg_grad_list_destroy(None)


def _z(*shape, dtype=None):
    return torch.zeros(*shape, dtype=dtype or torch.float32)


@pytest.mark.parametrize("call", [
    lambda: binding.embedding_forward(_z(4), _z(3, dtype=torch.int32), _z(3, 4)),
    lambda: binding.embedding_forward(_z(4, 8), _z(3, dtype=torch.int32), _z(3, 8)),      # host memory
    lambda: binding.embedding_forward(_z(8, 4).t(), _z(3, dtype=torch.int32), _z(3, 8)),  # strided
    lambda: binding.embedding_backward(_z(3, 8), _z(3, dtype=torch.int32), _z(4, 8, dtype=torch.bfloat16),
                                       _z(64)),
    lambda: binding.grouped_linear_forward(_z(4, 8), _z(3, dtype=torch.int32), _z(8, 8), _z(4, 8), _z(64)),
    lambda: binding.grouped_linear_backward_weight(_z(4, 8), _z(4, 8), _z(3, dtype=torch.int32), _z(8, 8),
                                                   _z(64)),
    lambda: binding.GradList([]),
    lambda: binding.GradList([_z(4)]),
    lambda: binding.GradList([_z(4)], [_z(4), _z(4)]),
])
def test_wrappers_refuse(lib, call):
    with pytest.raises(binding.MGError):
        call()


def _create(lib, layers, batch=8, precision="strict"):
    arr = (binding.mg_layer * len(layers))(*[binding.layer_struct(l) for l in layers])
    d = binding.mg_graph_desc()
    d.batch, d.n_layers, d.layers = batch, len(layers), arr
    d.loss, d.precision, d.optimizer = 0, binding.PRECISIONS[precision], binding.OPTIMIZERS["sgd"]
    h = ctypes.c_void_p()
    st = lib.mg_step_plan_create(ctypes.byref(d), ctypes.byref(h))
    if st == 0:
        lib.mg_step_plan_destroy(h)
    return st


@pytest.mark.parametrize("layers,want", [
    ([W.linear(4, 8, False), W.embedding(10, 8), W.linear(8, 4, False)], U),
    ([W.embedding(0, 8), W.linear(8, 4, False)], S),
    ([W.embedding(10, -8), W.linear(8, 4, False)], S),
    ([W.embedding(10, 8, float("inf")), W.linear(8, 4, False)], E),
    ([W.embedding(10, 8), W.linear(9, 4, False)], S),
    ([W.embedding(10, 8), W.relu(), W.linear(8, 4, False)], U),
    ([W.grouped_linear(0, 8, 4)], S),
    ([W.grouped_linear(1025, 8, 4)], U),
    ([W.grouped_linear(2, 8, 4), W.linear(5, 4, False)], S),
    ([W.grouped_linear(2, 8, 8), W.grouped_linear(3, 8, 4)], U),
    ([W.grouped_linear(2, 8, 8), W.relu()], U),
])
def test_layer_refusals(lib, layers, want):
    assert _create(lib, layers) == want


def test_null_plan_in_the_new_calls(lib):
    f = (ctypes.c_float * 2)()
    assert lib.mg_set_row_groups(None, P) == E
    assert lib.mg_set_grad_clip(None, 1.0) == E
    assert lib.mg_grad_norm_device_ptr(None) is None
    assert lib.mg_grad_norm(None, f, None) == E
