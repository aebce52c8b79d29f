"""Embedding lookup with scaling and its gradient against the definitions in 64
bits, element by element.

Tolerances.  Forward: one product in fp32 and one rounding to the output type,
each off by at most half a step (2^-24, and 2^-8 for bf16).  Backward: a sum of
c fp32 terms in any fixed order is off by at most c 2^-24 sum|term| to first
order, and the factor adds one rounding; 1 % covers the higher orders."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402

U32, U16 = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
IT = {"i32": torch.int32, "i64": torch.int64}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _ids(n, v, kind, seed, bad=0.1, hot=0.0):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, v, (n,), generator=g)
    if n:
        u = torch.rand(n, generator=g)
        ids[u < hot] = min(3, v - 1)
        w = torch.rand(n, generator=g)
        ids[w < bad / 2] = -1
        ids[(w >= bad / 2) & (w < bad)] = v
        if n > 5 and bad:
            ids[1], ids[2] = -2 ** 31, 2 ** 31 - 1
            if kind == "i64":
                ids[3], ids[4] = 2 ** 40, -2 ** 62
    return ids.to(IT[kind]).cuda()


def _randn(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(DT[dtype])


def _fwd_want(table, ids, scale):
    i = ids.long()
    ok = (i >= 0) & (i < table.shape[0])
    out = torch.zeros(i.numel(), table.shape[1], dtype=torch.float64, device="cuda")
    out[ok] = table[i[ok]].double() * scale
    return out


@pytest.mark.parametrize("n,v,d", [(0, 5, 8), (1, 1, 1), (1, 32000, 2048), (33, 7, 24), (257, 1000, 777),
                                   (4099, 50, 64), (3001, 211, 4104), (20000, 100, 8)])
@pytest.mark.parametrize("tt,ot,kind", [("f32", "f32", "i32"), ("bf16", "bf16", "i64"),
                                        ("f32", "bf16", "i64"), ("bf16", "f32", "i32")])
def test_forward(n, v, d, tt, ot, kind):
    table = _randn((v, d), tt, 1)
    ids = _ids(n, v, kind, 2)
    # rows behind the output stay as they were
    buf = torch.full((n + 2, d), 7.0, dtype=DT[ot], device="cuda")
    for scale in (1.0, -0.37):
        mg.embedding_forward(table, ids, buf[:n], scale=scale)
        want = _fwd_want(table, ids, float(torch.tensor(scale, dtype=torch.float32)))
        tol = (U32 + (U16 if ot == "bf16" else 0.0)) * 1.01
        assert ((buf[:n].double() - want).abs() <= tol * want.abs()).all()
        assert (buf[n:] == 7.0).all()


def test_forward_absent_rows_are_not_read():
    """NaN rows that no id names, and padding under a factor, leave no trace."""
    table = torch.full((9, 16), float("nan"), device="cuda")
    table[4] = 2.0
    ids = torch.tensor([4, -1, 9, 4], dtype=torch.int32, device="cuda")
    out = torch.empty(4, 16, device="cuda")
    mg.embedding_forward(table, ids, out, scale=-3.0)
    assert (out[0] == -6).all() and (out[3] == -6).all()
    assert (out[1:3] == 0).all()


def _bwd(dout, ids, v, scale, ws=None, stream=None):
    n, d = dout.shape
    nb = mg.embedding_workspace_bytes(n, v, d)
    if ws is None:
        ws = torch.full((nb,), 255, dtype=torch.uint8, device="cuda")     # contents do not matter
    buf = torch.full((v + 1, d), float("nan"), device="cuda")
    mg.embedding_backward(dout, ids, buf[:v], ws, scale=scale, stream=stream)
    assert torch.isnan(buf[v]).all()
    return buf[:v]


def _bwd_check(dout, ids, v, scale, got):
    i = ids.long()
    ok = (i >= 0) & (i < v)
    want = torch.zeros(v, dout.shape[1], dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    cnt = torch.zeros(v, dtype=torch.float64, device="cuda")
    want.index_add_(0, i[ok], dout[ok].double())
    mag.index_add_(0, i[ok], dout[ok].double().abs())
    cnt.index_add_(0, i[ok], torch.ones_like(i[ok], dtype=torch.float64))
    s = float(torch.tensor(scale, dtype=torch.float32))
    err = (got.double() - want * s).abs()
    bound = 1.01 * U32 * (cnt[:, None] + 1) * mag * abs(s)
    assert (err <= bound).all(), float((err - bound).max())


@pytest.mark.parametrize("n,v,d,hot", [
    (0, 5, 8, 0.0), (1, 1, 1, 0.0), (1, 70000, 16, 0.0), (33, 7, 24, 0.0), (257, 1000, 777, 0.0),
    (5000, 50, 33, 0.3), (4096, 3, 128, 0.0), (4097, 600, 2056, 0.4), (20000, 300000, 8, 0.2),
    (129, 2, 64, 1.0), (128, 2, 64, 1.0), (70001, 513, 40, 0.5), (30000, 40, 1030, 0.6)])
@pytest.mark.parametrize("t,kind", [("f32", "i32"), ("bf16", "i64")])
def test_backward(n, v, d, hot, t, kind):
    dout = _randn((n, d), t, 3)
    ids = _ids(n, v, kind, 4, hot=hot)
    got = _bwd(dout, ids, v, 0.731)
    _bwd_check(dout, ids, v, 0.731, got)
    # the same bits again
    assert torch.equal(got, _bwd(dout, ids, v, 0.731))


def test_backward_one_id_for_all():
    n, v, d = 150000, 11, 24
    dout = _randn((n, d), "bf16", 5)
    ids = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    got = _bwd(dout, ids, v, 1.0)
    _bwd_check(dout, ids, v, 1.0, got)
    assert (got[:7] == 0).all() and (got[8:] == 0).all()


def test_backward_padding_is_not_read():
    """NaN and infinities in the rows of padding ids reach no gradient."""
    dout = torch.ones(300, 40, device="cuda")
    ids = torch.arange(300, device="cuda", dtype=torch.int32) % 5
    ids[::7] = -1
    dout[::7] = float("nan")
    ids[3::7] = 5
    dout[3::7] = float("inf")
    got = _bwd(dout, ids, 5, 1.0)
    assert torch.isfinite(got).all()
    _bwd_check(torch.nan_to_num(dout, 0, 0, 0), ids, 5, 1.0, got)


def test_backward_matches_differences():
    """The gradient of sum(w * out) by central differences of the forward call."""
    v, d, n, scale = 6, 8, 40, 0.5
    table, w = _randn((v, d), "f32", 8), _randn((n, d), "f32", 9)
    ids = _ids(n, v, "i32", 10)
    got = _bwd(w, ids, v, scale)
    out = torch.empty(n, d, device="cuda")

    def loss(t):
        mg.embedding_forward(t, ids, out, scale=scale)
        return float((w.double() * out.double()).sum())

    for r, c in ((0, 0), (3, 5), (5, 7)):
        h = 2.0 ** -4          # the call is linear: no truncation error at any step
        a, b = table.clone(), table.clone()
        a[r, c] += h
        b[r, c] -= h
        # each side's elements are off by 2^-24 of their size, at most n of them here
        tol = 2 * U32 * float((w.abs().max() * (table.abs().max() + 1) * n) / h)
        assert abs((loss(a) - loss(b)) / (2 * h) - float(got[r, c])) <= tol


def test_offsets_past_32_bits():
    """A table and a gradient of more than 2^31 elements: the last rows."""
    v, d = 300000, 8192
    table = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    table[-2:] = 3.0
    ids = torch.tensor([v - 1, v - 2, v - 1], dtype=torch.int64, device="cuda")
    out = torch.empty(3, d, dtype=torch.bfloat16, device="cuda")
    mg.embedding_forward(table, ids, out, scale=2.0)
    assert (out == 6.0).all()
    del table
    got = _bwd(out, ids, v, 0.5)
    assert (got[v - 1] == 6.0).all() and (got[v - 2] == 3.0).all()
    assert int(torch.count_nonzero(got)) == 2 * d


def test_streams_and_graph_replay():
    """Both calls captured on a side stream; replays follow new ids and data."""
    v, d, n = 500, 64, 3000
    table = _randn((v, d), "f32", 11)
    ids = _ids(n, v, "i32", 12, hot=0.3)
    dout = _randn((n, d), "bf16", 13)
    out = torch.empty(n, d, device="cuda")
    dt = torch.empty(v, d, device="cuda")
    ws = torch.empty(mg.embedding_workspace_bytes(n, v, d), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mg.embedding_forward(table, ids, out, stream=s)
        mg.embedding_backward(dout, ids, dt, ws, stream=s)
    for seed in (20, 21, 22):
        ids.copy_(_ids(n, v, "i32", seed, hot=0.1 * (seed - 20)))
        dout.copy_(_randn((n, d), "bf16", seed))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.double(), _fwd_want(table, ids, 1.0))
        _bwd_check(dout, ids, v, 1.0, dt)


def test_two_calls_at_once_with_their_own_workspaces():
    v, d, n = 4000, 512, 8192
    douts = [_randn((n, d), "f32", 30 + i) for i in range(2)]
    idss = [_ids(n, v, "i32", 40 + i, hot=0.2) for i in range(2)]
    wss = [torch.empty(mg.embedding_workspace_bytes(n, v, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    dts = [torch.empty(v, d, device="cuda") for _ in range(2)]
    ss = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i in range(2):
            mg.embedding_backward(douts[i], idss[i], dts[i], wss[i], stream=ss[i])
    torch.cuda.synchronize()
    for i in range(2):
        _bwd_check(douts[i], idss[i], v, 1.0, dts[i])


def test_wrong_memory_is_refused():
    lib = binding.load()
    host = torch.zeros(64)
    dev = torch.zeros(64, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    st = lib.mg_embedding_forward(0, dev.data_ptr(), 4, 8, 0, ids.data_ptr(), 4, 1.0, 0, host.data_ptr() + 64, None)
    assert st in (binding.MG_ERR_INVALID_ARG, binding.MG_ERR_ALIGN)
    with pytest.raises(binding.MGError):
        mg.embedding_backward(dev.view(8, 8), ids, dev.view(8, 8), torch.empty(8, dtype=torch.uint8, device="cuda"))
