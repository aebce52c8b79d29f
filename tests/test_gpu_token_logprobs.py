"""Log probabilities of given tokens, entropy, alternatives and their gradient,
against the definitions in 64 bits.

Tolerances, in units of u = 2^-24.  A term's exponent t = (x - m) / T carries the
roundings of the difference, the factor (two) and the product: 4 u |t|; its
exponential 8 u.  A sum of V terms goes through at most V / 128 + 40 additions
(256 threads or more, or a warp's lanes at small V, each a sum of its own, and a
tree).  So the sum s has a relative error e_s = (4 A1 + 8 + depth) u, A1 = sum
p |t|; logp = t_id - L adds 4 |t_id| + 2 |L| + |logp|, and the entropy's sum q / s an
absolute error (4 A2 + (8 + depth) A1) u + A1 (e_s + 2 u), A2 = sum p t^2.  The
gradient, of the given statistics: log p has (4 |t| + |L| + |log p|) u, p that and
8 u, and each further operation one u of its result; then half a step of the
stored type."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _logits(rows, vocab, t, seed, stride=None, scale=2.0):
    buf = torch.randn(rows, stride or vocab, generator=_gen(seed), device="cuda") * scale
    return buf.to(DT[t])[:, :vocab]


def _ids(rows, vocab, seed, kind=torch.int32, pad=False):
    ids = torch.randint(0, vocab, (rows,), generator=_gen(seed), device="cuda")
    if pad and rows > 1:
        ids[1::5] = -1
        ids[0] = vocab
    return ids.to(kind)


def _forward(x, ids, k=0, temp=1.0, entropy=True, stream=None):
    r = x.shape[0]
    new = lambda *s, t=torch.float32: torch.full(s, 77, device="cuda", dtype=t)  # noqa: E731
    o = {"logp": new(r) if ids is not None else None, "stats": new(r, 2), "entropy": new(r) if entropy else None,
         "top_ids": new(r, k, t=torch.int32) if k else None, "top_logp": new(r, k) if k else None}
    mg.token_logprobs(x, ids, o["logp"], temperature=temp, stream=stream,
                      **{n: o[n] for n in ("stats", "entropy", "top_ids", "top_logp")})
    return o


def _check(x, ids, o, k=0, temp=1.0):
    """Rows without NaN and +inf."""
    rows, v = x.shape
    depth = v / 128 + 40
    for a in range(0, rows, 512):
        z = x[a:a + 512].double()
        n = z.shape[0]
        live = torch.ones(n, dtype=torch.bool, device="cuda") if ids is None else (ids[a:a + n] >= 0) & (ids[a:a + n] < v)
        m = z.amax(1, keepdim=True)
        none = (m == -INF)[:, 0]
        t = (z - torch.where(m == -INF, torch.zeros_like(m), m)) / temp
        e = t.exp()
        s = e.sum(1, keepdim=True)
        lse = s.log()
        p = torch.where(none[:, None], torch.zeros_like(e), e / s)
        ta = torch.where(p > 0, t.abs(), torch.zeros_like(t))
        a1, a2 = (p * ta).sum(1), (p * ta * ta).sum(1)
        es = (4 * a1 + 8 + depth) * U
        lz = torch.where(none, torch.zeros_like(s[:, 0]), lse[:, 0])
        ok = live & ~none
        got = o["stats"][a:a + n].double()
        assert torch.equal(got[live, 0], m[live, 0])
        assert ((got[ok, 1] - lz[ok]).abs() <= (es + 2 * lz.abs() * U)[ok]).all()
        assert torch.isinf(got[live & none]).all() and (got[~live] == 0).all()

        def close(g, at):
            tt, lp = t.gather(1, at), t.gather(1, at) - lse
            tol = (es + 2 * lz.abs() * U)[:, None] + (4 * tt.abs() + lp.abs()) * U
            gone = torch.isinf(lp.float())     # a probability of 0, or a logarithm beyond fp32's range (masks by the lowest value)
            assert (g[ok][gone[ok]] == -INF).all() and (g[live & none] == -INF).all() and (g[~live] == 0).all()
            keep = ~gone & ok[:, None]
            assert ((g - lp).abs()[keep] <= tol[keep]).all()

        if ids is not None:
            close(o["logp"][a:a + n, None].double(), ids[a:a + n].long().clamp(0, v - 1)[:, None])
        if o["entropy"] is not None:
            want = -torch.special.xlogy(p, p).sum(1)
            tol = es + 2 * lz.abs() * U + (4 * a2 + (8 + depth) * a1) * U + a1 * (es + 2 * U) + want.abs() * U
            got = o["entropy"][a:a + n].double()
            assert ((got - want).abs()[ok] <= tol[ok]).all()
            assert (got[live & none] == 0).all() and (got[~live] == 0).all()
        if k:
            top = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :k]
            assert torch.equal(o["top_ids"][a:a + n].long(), torch.where(live[:, None], top, -torch.ones_like(top)))
            close(o["top_logp"][a:a + n].double(), top)


SIZES = [(1, 1), (3, 2), (2, 31), (5, 33), (4, 257), (7, 1000), (33, 2048), (3, 8191), (2, 32000), (300, 4104),
         (1, 131072), (9, 50021), (700, 777), (2000, 130)]


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_forward(rows, vocab, t):
    x = _logits(rows, vocab, t, rows + vocab)
    ids = _ids(rows, vocab, 3, pad=True)
    k = min(20, vocab)
    o = _forward(x, ids, k)
    _check(x, ids, o, k)
    again = _forward(x, ids, k)
    assert all(torch.equal(o[n], again[n]) for n in o)
    _check(x, None, _forward(x, None, min(vocab, 32), 0.6), min(vocab, 32), 0.6)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("vocab,stride,shift", [(100, 107, 0), (1003, 1003, 1), (4096, 4099, 3), (32000, 32064, 5)])
def test_strides_and_alignments(vocab, stride, shift, t):
    """Rows that begin anywhere, beside memory that is not theirs."""
    buf = torch.full((8, stride + shift), NAN, device="cuda", dtype=DT[t])
    x = buf[:, shift:shift + vocab]
    x.copy_(_logits(8, vocab, t, 5))
    ids = _ids(8, vocab, 6, torch.int64)
    o = _forward(x, ids, 5, 1.3)
    _check(x, ids, o, 5, 1.3)
    out = torch.full((8, stride + shift + 2), 5.0, device="cuda", dtype=DT[t])
    _gradient(x, ids, o, t, 1.3, out[:, 2 + shift:2 + shift + vocab])
    assert (out[:, :2 + shift] == 5).all() and (out[:, 2 + shift + vocab:] == 5).all()


def _formula(x, ids, stats, g, h, ent, temp):
    """The gradient in 64 bits from the given statistics, and its error bound without the last rounding."""
    v = x.shape[1]
    z = x.double()
    m, ls = stats[:, :1].double(), stats[:, 1:].double()
    live = torch.ones(x.shape[0], dtype=torch.bool, device="cuda") if ids is None else (ids >= 0) & (ids < v)
    live &= ~torch.isinf(m[:, 0])
    zero = torch.zeros_like(z[:, 0])
    g, h = (zero if q is None else q.double() for q in (g, h))
    live &= (g != 0) | (h != 0)
    g, h = (torch.where(live, q, zero)[:, None] for q in (g, h))
    ent = zero[:, None] if ent is None else ent.double()[:, None]
    t = (z - torch.where(live[:, None], m, torch.zeros_like(m))) / temp
    lp = t - ls
    p = torch.where(live[:, None], lp.exp(), torch.zeros_like(z))
    lp = torch.where(p > 0, lp, torch.zeros_like(lp))
    ta = torch.where(p > 0, t.abs(), torch.zeros_like(t))
    one = torch.zeros_like(z)
    if ids is not None:
        one.scatter_(1, ids.long().clamp(0, v - 1)[:, None], 1.0)
    want = (g * (one - p) - h * p * (lp + ent)) / temp
    dlp = (4 * ta + torch.where(live[:, None], ls.abs(), torch.zeros_like(ls)) + lp.abs()) * U
    dp = dlp + 8 * U
    mag = lp.abs() + ent.abs()
    tol = (g.abs() * p * dp + h.abs() * p * (dp * mag + dlp)) + 8 * U * (g.abs() * (one + p) + h.abs() * p * mag)
    return want, tol / temp


def _gradient(x, ids, o, t, temp, out=None, seed=9, which="both"):
    g = torch.randn(x.shape[0], generator=_gen(seed), device="cuda")
    h = torch.randn(x.shape[0], generator=_gen(seed + 1), device="cuda")
    g = None if which == "entropy" else g
    h = None if which == "logp" else h
    if x.shape[0] > 3 and which == "both":
        g[2] = h[2] = 0.0
    out = torch.full(x.shape, 77.0, device="cuda", dtype=DT[t]) if out is None else out
    keep = x.clone()
    mg.token_logprobs_backward(x, ids, o["stats"], g, out, entropy=None if h is None else o["entropy"], dentropy=h,
                               temperature=temp)
    for a in range(0, x.shape[0], 512):
        c = slice(a, a + 512)
        want, tol = _formula(keep[c], None if ids is None else ids[c], o["stats"][c], None if g is None else g[c],
                             None if h is None else h[c], o["entropy"][c], temp)
        assert ((out[c].double() - want).abs() <= tol * (1 + HALF[t]) + HALF[t] * want.abs() + 2.0 ** -140).all()
    return g, h, out


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", SIZES)
def test_backward(rows, vocab, t):
    x = _logits(rows, vocab, t, rows + vocab)
    ids = _ids(rows, vocab, 3, pad=True)
    o = _forward(x, ids, 0, 0.8)
    _gradient(x, ids, o, t, 0.8)
    _gradient(x, ids, o, t, 0.8, which="logp")
    _gradient(x, None, _forward(x, None, 0, 0.8), t, 0.8, which="entropy")
    _gradient(x, ids, o, t, 0.8, out=x)          # in place


def test_backward_against_differences():
    """Central differences of the definition in 64 bits, step 1e-4: third derivatives of logp and entropy stay
    below 20, so 20 / 6 1e-8 of truncation, 1e-11 of rounding; beside the kernel's own bound."""
    x = _logits(3, 19, "f32", 1)
    ids = _ids(3, 19, 2)
    o = _forward(x, ids, 0, 0.9)
    g, h, out = _gradient(x, ids, o, "f32", 0.9)

    def f(z):
        lp = torch.log_softmax(z / 0.9, 1)
        ent = -(lp.exp() * lp).sum(1)
        return (g.double() * lp.gather(1, ids.long()[:, None])[:, 0] + h.double() * ent).sum(0)

    want, tol = _formula(x, ids, o["stats"], g, h, o["entropy"], 0.9)
    # the statistics are the forward's, within its own bounds of the exact ones
    slack = (g.abs() + h.abs()).double()[:, None] * 1e-4 / 10
    for r in range(3):
        for c in range(19):
            d = torch.zeros_like(x, dtype=torch.float64)
            d[r, c] = 1e-4
            diff = (f(x.double() + d) - f(x.double() - d)) / 2e-4
            assert abs(float(diff) - float(out[r, c])) <= float(tol[r, c] + U * want[r, c].abs() + slack[r, 0]) + 1e-7


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [5, 300, 32000, 131072])
def test_masks(vocab, t):
    """-inf and the type's lowest value: over most of a row, all of it, all but one."""
    low = torch.finfo(DT[t]).min
    x = _logits(9, vocab, t, 11)
    x[0] = -INF
    x[1, 1:] = -INF
    x[2, :-1] = -INF
    x[3, 2:] = low
    x[4] = low
    x[5, ::2] = -INF
    x[6] = 0.0
    x[7, : vocab // 2] = low
    x[7, vocab // 2:] = -INF
    ids = _ids(9, vocab, 12)
    ids[1], ids[2] = 0, 0
    k = min(vocab, 20)
    for temp in (1.0, 0.25, 4.0):
        o = _forward(x, ids, k, temp)
        _check(x, ids, o, k, temp)
        assert torch.isfinite(o["entropy"]).all()
        _gradient(x, ids, o, t, temp)


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_not_finite(bad, t):
    """NaN and +inf stay in their row, and in padded rows and rows without a gradient they are not read."""
    x = _logits(8, 1000, t, 13)
    clean = x.clone()
    ids = _ids(8, 1000, 14)
    ids[6] = -1
    for r in (2, 5, 6):
        x[r, 17 * r] = bad
    o = _forward(x, ids, 4)
    for n in ("logp", "entropy", "top_logp"):
        assert torch.isnan(o[n][[2, 5]]).all()
    rest = [0, 1, 3, 4, 6, 7]
    want = _forward(clean, ids, 4)
    for n in o:
        assert torch.equal(o[n][rest], want[n][rest])
    order = torch.nan_to_num(x.float(), nan=-INF, posinf=INF, neginf=-INF).sort(dim=1, descending=True, stable=True)[1]
    assert torch.equal(o["top_ids"][[2, 5]].long(), order[[2, 5], :4])
    g = torch.ones(8, device="cuda")
    g[5] = 0.0
    out, ref = torch.full_like(x, 3.0), torch.full_like(x, 3.0)
    mg.token_logprobs_backward(x, ids, o["stats"], g, out)
    mg.token_logprobs_backward(clean, ids, want["stats"], g, ref)
    assert torch.isnan(out[2]).all() and (out[[5, 6]] == 0).all()
    assert torch.equal(out[[0, 1, 3, 4, 7]], ref[[0, 1, 3, 4, 7]])


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [40, 2048, 32000, 200001])
@pytest.mark.parametrize("k", [1, 7, 32])
def test_alternatives_among_equals(vocab, k, t):
    """Rows of many equal values, rows in order, all large values in one thread's or one block's places: the
    lowest index first."""
    c = torch.arange(vocab, device="cuda")
    rows = [torch.zeros(vocab, device="cuda"), -(c % 3).float(), (c // 8 % 2).float(), c.float() / vocab, -c.float() / vocab,
            (c % 2048 < 8).float() * (1 + (c // 2048 % 5)), (c % 4096 < 16).float() * 2 + (c % 7) / 8.0, (c < vocab // 3).float(),
            (c >= vocab - 40).float(), torch.where(c % 97 == 5, 0.0, -INF), -0.0 * (c % 2), (c % 5 == 0).float() - (c % 5 == 1).float()]
    x = torch.stack([r.float() for r in rows]).to(DT[t])
    o = _forward(x, None, k)
    _check(x, None, o, k)


def test_large_vocabularies():
    """Rows of millions of logits, by one cluster each and by one block each."""
    for rows, vocab, t in ((3, 5_000_001, "bf16"), (2, 1 << 22, "f32"), (700, 300_007, "bf16")):
        x = _logits(rows, vocab, t, vocab)
        ids = _ids(rows, vocab, 4, torch.int64)
        ids[0] = vocab - 1
        o = _forward(x, ids, 32, 0.9)
        at = [0, 1, rows - 1]
        _check(x[at], ids[at], {n: v[at] for n, v in o.items()}, 32, 0.9)
        if rows < 10:
            _gradient(x, ids, o, t, 0.9)
        del x, o


def test_ids_beyond_32_bits_are_padding():
    x = _logits(6, 100, "f32", 50)
    ids = torch.tensor([2 ** 32 + 5, -2 ** 32 + 5, 2 ** 31, -1, 100, 5], device="cuda")
    o = _forward(x, ids, 3)
    assert (o["logp"][:5] == 0).all() and (o["top_ids"][:5] == -1).all() and float(o["logp"][5]) < 0
    dx = torch.full_like(x, 7.0)
    mg.token_logprobs_backward(x, ids, o["stats"], torch.ones(6, device="cuda"), dx)
    assert (dx[:5] == 0).all() and (dx[5] != 0).any()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("temp", [1e-3, 1e3])
def test_far_temperatures(temp, t):
    x = _logits(40, 3001, t, 51)
    x[::3, ::2] = -INF
    ids = _ids(40, 3001, 52, pad=True)
    o = _forward(x, ids, 10, temp)
    _check(x, ids, o, 10, temp)
    _gradient(x, ids, o, t, temp)


def test_gradient_of_the_entropy_alone_keeps_the_padding():
    x = _logits(9, 500, "bf16", 53)
    ids = _ids(9, 500, 54)
    ids[3] = -1
    o = _forward(x, ids, 0)
    _gradient(x, ids, o, "bf16", 1.0, which="entropy")


def test_empty_and_outputs_left_out():
    x = _logits(6, 100, "f32", 20)
    ids = _ids(6, 100, 21)
    full = _forward(x, ids, 3)
    lp = torch.zeros(6, device="cuda")
    mg.token_logprobs(x, ids, lp)
    assert torch.equal(lp, full["logp"])
    st = torch.zeros(6, 2, device="cuda")
    mg.token_logprobs(x, stats=st)
    assert torch.equal(st, full["stats"])
    ti, tl = torch.zeros(6, 3, dtype=torch.int32, device="cuda"), torch.zeros(6, 3, device="cuda")
    mg.token_logprobs(x, top_ids=ti, top_logp=tl)
    assert torch.equal(ti, full["top_ids"]) and torch.equal(tl, full["top_logp"])
    mg.token_logprobs(x[:0], ids[:0], lp[:0])
    mg.token_logprobs_backward(x[:0], ids[:0], st[:0], lp[:0], x[:0].clone())
    # more dimensions
    y, yi = _logits(6, 100, "f32", 20).view(2, 3, 100), ids.view(2, 3)
    lp2 = torch.zeros(2, 3, device="cuda")
    mg.token_logprobs(y, yi, lp2)
    assert torch.equal(lp2.view(-1), full["logp"])


def test_overlaps_are_refused():
    x = torch.zeros(64, 64, device="cuda")
    flat = x.view(-1)
    ids = torch.zeros(8, dtype=torch.int32, device="cuda")
    with pytest.raises(binding.MGError):
        mg.token_logprobs(x[:8], ids, flat[:8])
    a = torch.zeros(16, device="cuda")
    with pytest.raises(binding.MGError):
        mg.token_logprobs(x[:8], ids, a[:8], entropy=a[4:12])
    st = torch.zeros(8, 2, device="cuda")
    for dx in (x[1:9], x[:8, :32], flat[4:4 + 8 * 60].view(8, 60)):
        with pytest.raises(binding.MGError):
            mg.token_logprobs_backward(x[:8, :dx.shape[1]] if dx.shape[1] != 32 else x[:8, 16:48], ids, st, a[:8], dx)


def test_rows_past_2_31_elements():
    rows, v, ld = 70001, 32000, 32064
    x = torch.zeros(rows, ld, device="cuda", dtype=torch.bfloat16)[:, :v]
    at = [0, 1, 66000, 66975, 67000, rows - 1]
    x[at] = _logits(len(at), v, "bf16", 30)
    ids = torch.full((rows,), 7, dtype=torch.int32, device="cuda")
    o = _forward(x, ids, 3)
    _check(x[at], ids[at], {n: o[n][at] for n in o}, 3)
    assert (o["logp"] < 0).all()
    dx = torch.full((rows, ld), 2.0, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(rows, device="cuda")
    mg.token_logprobs_backward(x, ids, o["stats"], g, dx[:, :v])
    want, tol = _formula(x[at], ids[at], o["stats"][at], g[at], None, None, 1.0)
    assert ((dx[at, :v].double() - want).abs() <= tol * 1.01 + HALF["bf16"] * want.abs()).all()
    assert (dx[:, v:] == 2).all() and (dx[:, 7] > 0).all()


@pytest.mark.parametrize("rows,vocab", [(2, 131072), (300, 5000)])
def test_stream_and_graph(rows, vocab):
    x = _logits(rows, vocab, "bf16", 40)
    ids = _ids(rows, vocab, 41)
    dx = torch.zeros_like(x)
    g = torch.ones(rows, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o = _forward(x, ids, 9, stream=s)
        mg.token_logprobs_backward(x, ids, o["stats"], g, dx, stream=s)
    for seed in (42, 43):
        x.copy_(_logits(rows, vocab, "bf16", seed))
        graph.replay()
        torch.cuda.synchronize()
        _check(x, ids, o, 9)
        want, tol = _formula(x, ids, o["stats"], g, None, None, 1.0)
        assert ((dx.double() - want).abs() <= tol * 1.01 + HALF["bf16"] * want.abs() + 2.0 ** -140).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab", [(5, 31), (5, 32000), (700, 1003), (5, 200001)])
def test_rows_of_nan_alone(rows, vocab, t):
    """A row of NaN, or of NaN beside -inf, has NaN in its results and in all of its gradient; one of -inf alone has none."""
    x = _logits(rows, vocab, t, 60)
    x[0] = NAN
    x[1] = -INF
    x[1, vocab // 2] = NAN
    x[2] = -INF
    x[3, ::2] = NAN
    x[3, 1::2] = -INF
    ids = _ids(rows, vocab, 61)
    o = _forward(x, ids, 4)
    bad, rest = [0, 1, 3], [r for r in range(rows) if r not in (0, 1, 3)]
    for n in ("logp", "entropy", "top_logp"):
        assert torch.isnan(o[n][bad]).all() and not torch.isnan(o[n][rest]).any()
    one = torch.ones(rows, device="cuda")
    for g, h in ((one, None), (None, one), (one, one)):
        out = torch.full_like(x, 3.0)
        mg.token_logprobs_backward(x, ids, o["stats"], g, out, entropy=None if h is None else o["entropy"], dentropy=h)
        assert torch.isnan(out[bad]).all()
        assert (out[2] == 0).all() and torch.isfinite(out[rest]).all()
    mg.token_logprobs_backward(x, ids, o["stats"], one, x)          # in place
    assert torch.isnan(x[bad]).all() and torch.isfinite(x[rest]).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_logits_and_their_gradient_as_columns_of_one_buffer(t):
    rows, v = 9, 1003
    x = _logits(rows, v, t, 70)
    ids = _ids(rows, v, 71, pad=True)
    o = _forward(x, ids)
    g = torch.ones(rows, device="cuda")
    for first, second, stride in ((0, v, 2 * v), (v, 0, 2 * v), (5, v + 9, 2 * v + 40), (v + 9, 5, 2 * v + 40)):
        buf = torch.full((rows, stride), 5.0, dtype=DT[t], device="cuda")
        a, b = buf[:, first:first + v], buf[:, second:second + v]
        a.copy_(x)
        _gradient(a, ids, o, t, 1.0, out=b)
        assert torch.equal(a, x)
        rest = torch.ones(stride, dtype=torch.bool, device="cuda")
        rest[first:first + v] = rest[second:second + v] = False
        assert (buf[:, rest] == 5).all()
    # columns that meet: by one, across the end of a row, and in rows of another width
    buf = torch.zeros(rows + 2, 2 * v, dtype=DT[t], device="cuda")
    flat = buf.view(-1)
    for b in (buf[:rows, v - 1:2 * v - 1], flat[v + 1:v + 1 + rows * 2 * v].view(rows, 2 * v)[:, :v],
              flat[v:v + rows * (2 * v - 1)].view(rows, 2 * v - 1)[:, :v]):
        with pytest.raises(binding.MGError):
            mg.token_logprobs_backward(buf[:rows, :v], ids, o["stats"], g, b)
