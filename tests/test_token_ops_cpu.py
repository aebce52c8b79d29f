"""Refusals of the token log probabilities, the residual norms and AdamW, all before
any device work (no GPU): the C entry points' checks and the Python wrappers'."""
import ctypes

import pytest

import __graft_entry__
from static_graph_nn_gb300 import binding

torch = pytest.importorskip("torch")

E, S, A = binding.MG_ERR_INVALID_ARG, binding.MG_ERR_SHAPE, binding.MG_ERR_ALIGN
P = 4096          # an aligned address that no refused call touches
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    return binding.load()


def _logp(lib, t=0, x=P, rows=4, v=10, ld=10, kind=0, ids=P, temp=1.0, logp=P, stats=P, ent=P, k=2, ti=P, tl=P):
    return lib.mg_token_logprobs(t, x, rows, v, ld, kind, ids, temp, logp, stats, ent, k, ti, tl, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=2), E), (dict(kind=2), E), (dict(rows=-1), S), (dict(rows=2**31), S), (dict(v=0), S), (dict(v=2**30 + 1, ld=2**31), S),
    (dict(ld=9), S), (dict(ld=2**31 + 1), S), (dict(temp=0.0), E), (dict(temp=-1.0), E), (dict(temp=NAN), E),
    (dict(temp=INF), E), (dict(temp=1e-45), E), (dict(temp=3.5e-39), E), (dict(k=-1), S), (dict(k=11), S), (dict(v=100, ld=100, k=33), S),
    (dict(x=None), E), (dict(ids=None), E), (dict(logp=None), E), (dict(ti=None), E), (dict(tl=None), E),
    (dict(ids=None, logp=None, stats=None, ent=None, k=0), E), (dict(x=P + 2), A), (dict(t=1, x=P + 1), A),
    (dict(ids=P + 2), A), (dict(ids=P + 4, kind=1), A), (dict(logp=P + 2), A), (dict(stats=P + 4), A),
    (dict(ent=P + 1), A), (dict(ti=P + 2), A), (dict(tl=P + 3), A),
])
def test_token_logprobs_refusals(lib, kw, want):
    assert _logp(lib, **kw) == want
    assert b"mg_token_logprobs" in lib.mg_last_error(None)


def _logp_bwd(lib, t=0, x=P, rows=4, v=10, ld=10, kind=0, ids=P, temp=1.0, stats=P, ent=P, dlp=P, de=P, dx=P, ldd=10):
    return lib.mg_token_logprobs_backward(t, x, rows, v, ld, kind, ids, temp, stats, ent, dlp, de, dx, ldd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=-1), E), (dict(kind=3), E), (dict(rows=-1), S), (dict(ld=8), S), (dict(ldd=8), S), (dict(temp=0.0), E),
    (dict(x=None), E), (dict(stats=None), E), (dict(dx=None), E), (dict(dlp=None, de=None), E), (dict(ids=None), E),
    (dict(ent=None), E), (dict(x=P + 2), A), (dict(dx=P + 1), A), (dict(stats=P + 4), A), (dict(dlp=P + 2), A),
    (dict(de=P + 2), A),
])
def test_token_logprobs_backward_refusals(lib, kw, want):
    assert _logp_bwd(lib, **kw) == want
    assert b"mg_token_logprobs_backward" in lib.mg_last_error(None)


def _norm(lib, t=0, y=P, x=P, rows=4, d=8, g1=P, gate=P, gates=1, scale=1.0, g2=P, eps=1e-6, xo=P, h=P, rstd=P):
    return lib.mg_norm_residual_forward(t, y, x, rows, d, g1, gate, gates, scale, g2, eps, xo, h, rstd, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=2), E), (dict(rows=-1), S), (dict(rows=2**30 + 1), S), (dict(d=0), S), (dict(d=2**30 + 1), S),
    (dict(gates=0), S), (dict(gates=3), S), (dict(gates=8), S), (dict(gates=-1), S), (dict(gate=None), S), (dict(scale=NAN), E),
    (dict(scale=INF), E), (dict(eps=0.0), E), (dict(eps=NAN), E), (dict(eps=INF), E), (dict(y=None), E), (dict(x=None), E),
    (dict(xo=None), E), (dict(h=None), E), (dict(g2=None), E), (dict(y=P + 8), A), (dict(x=P + 2), A),
    (dict(g1=P + 4), A), (dict(gate=P + 4), A), (dict(h=P + 8), A), (dict(rstd=P + 8), A),
])
def test_norm_residual_refusals(lib, kw, want):
    assert _norm(lib, **kw) == want
    assert b"mg_norm_residual_forward" in lib.mg_last_error(None)


def _norm_bwd(lib, t=0, dxo=P, dh=P, y=P, x=P, rstd=P, rows=4, d=8, g1=P, gate=P, gates=1, scale=1.0, g2=P, dy=P, dx=P,
              dg1=P, dgate=P, dg2=P, ws=P, nb=1 << 30):
    return lib.mg_norm_residual_backward(t, dxo, dh, y, x, rstd, rows, d, g1, gate, gates, scale, g2, dy, dx, dg1, dgate,
                                         dg2, ws, nb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(t=2), E), (dict(rows=-1), S), (dict(d=0), S), (dict(gates=3), S), (dict(scale=NAN), E), (dict(y=None), E),
    (dict(x=None), E), (dict(rstd=None), E), (dict(dy=None), E), (dict(dx=None), E), (dict(dxo=None, dh=None), E),
    (dict(ws=None), E), (dict(nb=16), E), (dict(g2=None), E), (dict(g1=None), E), (dict(gate=None, gates=0), E),
    (dict(dy=P + 8), A), (dict(dgate=P + 4), A), (dict(ws=P + 4), A),
])
def test_norm_residual_backward_refusals(lib, kw, want):
    assert _norm_bwd(lib, **kw) == want
    assert b"mg_norm_residual_backward" in lib.mg_last_error(None)


def test_norm_residual_workspace(lib):
    f = lib.mg_norm_residual_workspace_bytes
    assert f(-1, 8, 0) == 0 and f(4, 0, 0) == 0 and f(4, 8, 3) == 0 and f(4, 8, -1) == 0 and f(2**30 + 1, 8, 0) == 0
    assert f(0, 8, 0) > 0 and f(4, 8, 4) > 0
    assert binding.norm_residual_workspace_bytes(2**40, 8) == 0
    assert binding.norm_residual_workspace_bytes(16384, 2048, 1) == f(16384, 2048, 1) > 0


@pytest.mark.parametrize("dim,gates", [(64, 1), (777, 7), (1000, 0), (2048, 1), (2048, 300), (8192, 4), (16384, 2), (70001, 1)])
def test_a_workspace_serves_fewer_rows(lib, dim, gates):
    g = max(1, gates)
    sizes = [lib.mg_norm_residual_workspace_bytes(r * g, dim, gates) for r in (0, 1, 2, 7, 8, 9, 100, 431, 5000, 40000, 200000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def _tensor(**kw):
    t = dict(param=P, grad=2 * P, m=3 * P, v=4 * P, m_scales=None, v_scales=None, copy=None, count=4, param_dtype=0,
             grad_dtype=0, weight_decay=0.0) | kw
    s = binding.mg_adamw_tensor()
    for k, v in t.items():
        setattr(s, k, v)
    return s


def _adamw(lib, tensors, n=None, bits=32, b1=0.9, b2=0.999, eps=1e-8):
    h = ctypes.c_void_p()
    arr = (binding.mg_adamw_tensor * max(1, len(tensors)))(*tensors)
    st = lib.mg_adamw_create(len(tensors) if n is None else n, arr, bits, b1, b2, eps, 0, ctypes.byref(h))
    if st == 0:
        lib.mg_adamw_destroy(h)
    return st


@pytest.mark.parametrize("kw,want", [
    (dict(param=None), E), (dict(grad=None), E), (dict(m=None), E), (dict(v=None), E), (dict(param_dtype=2), E),
    (dict(grad_dtype=-1), E), (dict(weight_decay=-0.1), E), (dict(weight_decay=NAN), E), (dict(weight_decay=INF), E),
    (dict(count=2**60), S), (dict(param=P + 2), A), (dict(grad=P + 1, grad_dtype=1), A), (dict(m=P + 2), A),
    (dict(copy=P + 1), A),
])
def test_adamw_tensor_refusals(lib, kw, want):
    assert _adamw(lib, [_tensor(**kw)]) == want
    assert b"mg_adamw_create" in lib.mg_last_error(None)


def test_adamw_refusals(lib):
    assert _adamw(lib, []) == E
    for kw in (dict(bits=16), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=NAN), dict(b1=1.0 - 1e-9), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=1e-60), dict(eps=1e-39), dict(eps=1e39), dict(eps=INF)):
        assert _adamw(lib, [_tensor()], **kw) == E
    assert _adamw(lib, [_tensor()], bits=8) == E            # no scales
    assert lib.mg_adamw_create(1, None, 32, 0.9, 0.999, 1e-8, 0, ctypes.byref(ctypes.c_void_p())) == E
    assert lib.mg_adamw_create(1, None, 32, 0.9, 0.999, 1e-8, 0, None) == E
    assert lib.mg_adamw_step(None, 0.1, 1, None, None, None, 1.0, None) == E
    lib.mg_adamw_destroy(None)


def _z(*shape, dtype=None):
    return torch.zeros(*shape, dtype=dtype or torch.float32)


I32, BF = torch.int32, torch.bfloat16


@pytest.mark.parametrize("call", [
    lambda: binding.token_logprobs(_z(4, 8), _z(4, dtype=I32), _z(4)),                                # host memory
    lambda: binding.token_logprobs(_z(8, 4).t(), _z(4, dtype=I32), _z(4)),                            # columns apart
    lambda: binding.token_logprobs(_z(4, 8), _z(3, dtype=I32), _z(4)),
    lambda: binding.token_logprobs(_z(4, 8), _z(4), _z(4)),
    lambda: binding.token_logprobs(_z(4, 8, dtype=torch.float16), _z(4, dtype=I32), _z(4)),
    lambda: binding.token_logprobs(_z(4, 8), stats=_z(4, 3)),
    lambda: binding.token_logprobs(_z(4, 8), entropy=_z(4, dtype=BF)),
    lambda: binding.token_logprobs(_z(4, 8), top_ids=_z(4, 2, dtype=I32)),
    lambda: binding.token_logprobs(_z(4, 8), top_ids=_z(4, 2, dtype=torch.int64), top_logp=_z(4, 2)),
    lambda: binding.token_logprobs(_z(4, 8), top_ids=_z(4, 9, dtype=I32), top_logp=_z(4, 9)),
    lambda: binding.token_logprobs(_z(2, 3, 16)[..., :8], stats=_z(2, 3, 2)),
    lambda: binding.token_logprobs_backward(_z(4, 8), _z(4, dtype=I32), _z(4, 2), _z(4), _z(4, 9)),
    lambda: binding.token_logprobs_backward(_z(4, 8), _z(4, dtype=I32), _z(4, 2), _z(4), _z(4, 8, dtype=BF)),
    lambda: binding.token_logprobs_backward(_z(4, 8), _z(4, dtype=I32), _z(4, 2), None, _z(4, 8)),
    lambda: binding.norm_residual_forward(_z(4, 8), _z(4, 8), _z(4, 8)),                              # host memory
    lambda: binding.norm_residual_forward(_z(4, 7), _z(4, 8), _z(4, 8)),
    lambda: binding.norm_residual_forward(_z(4, 8, dtype=BF), _z(4, 8), _z(4, 8)),
    lambda: binding.norm_residual_forward(_z(4, 8), _z(4, 8), _z(4, 8), gamma_post=_z(8, dtype=BF)),
    lambda: binding.norm_residual_forward(_z(4, 8), _z(4, 8), _z(4, 8), gate=_z(3, 8)),
    lambda: binding.norm_residual_forward(_z(4, 8), _z(4, 8), _z(4, 8), _z(4, 8)),                    # h, no gamma_pre
    lambda: binding.norm_residual_backward(_z(4, 8), None, _z(4, 8), _z(4, 8), _z(4, 3), _z(4, 8), _z(4, 8), _z(9)),
    lambda: binding.norm_residual_backward(_z(4, 8), None, _z(4, 8), _z(4, 8), _z(4, 2), _z(4, 8), _z(4, 8), _z(9),
                                           dgate=_z(8)),
    lambda: binding.AdamW([], [], [], []),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4)], [_z(4)]),                                        # host memory
    lambda: binding.AdamW([_z(4)], [_z(5)], [_z(4)], [_z(4)]),
    lambda: binding.AdamW([_z(4)], [None], [_z(4)], [_z(4)]),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4, dtype=BF)], [_z(4)]),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4, dtype=torch.uint8)], [_z(4)]),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4, dtype=torch.uint8)], [_z(4, dtype=torch.uint8)]),  # no scales
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4)], [_z(4)], m_scales=[_z(1)], v_scales=[_z(1)]),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4)], [_z(4)], copies=[_z(4)]),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4)], [_z(4)], weight_decay=[0.1, 0.1]),
    lambda: binding.AdamW([_z(4)], [_z(4)], [_z(4)], [_z(4)], seed=-1),
    lambda: binding.adamw_state([_z(4)], 16),
])
def test_wrappers_refuse(lib, call):
    with pytest.raises(binding.MGError):
        call()


def test_adamw_state_shapes():
    m, v, ms, vs = binding.adamw_state([_z(3, 100), _z(256), _z(0)], 8)
    assert [t.shape for t in m] == [t.shape for t in v] == [(3, 100), (256,), (0,)]
    assert all(t.dtype == torch.float8_e4m3fn for t in m + v)
    assert [t.numel() for t in ms] == [t.numel() for t in vs] == [2, 1, 0]
    m, v, ms, vs = binding.adamw_state([_z(7)])
    assert m[0].dtype == v[0].dtype == torch.float32 and ms is None and vs is None
