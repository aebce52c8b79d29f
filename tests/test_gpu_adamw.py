"""AdamW over lists of tensors, with 32- and 8-bit moments.

Tolerances, u = 2^-24.  A moment is two products and a sum, of factors that are
themselves rounded (beta, 1 - beta, and with clipping the gradient's factor and
product): m within 6 u (beta1 |m| + (1 - beta1) |g'|), v within 8 u of itself.  The
update m / (root / root_bc + eps) lr / bc: magnitudes of m's terms, its root and
quotient to 2^-21 at worst, each factor and operation one u: 30 u of lr / bc (beta1
|m| + (1 - beta1) |g'|) / denominator; the parameter 4 u of itself (the decay's factor,
its product, the sum); then half a step of the stored type.

8-bit moments: every operation of the codes is one fp32 rounding, so a host that
does the same has the same codes, scales and bits (checked as such)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
B = binding.ADAMW_BLOCK


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _make(sizes, seed, pt="f32", gt="f32", shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda n, s: torch.randn(n + shift, generator=g, device="cuda") * s  # noqa: E731
    types = lambda t, i: DT[t.split("+")[i % len(t.split("+"))]]  # noqa: E731
    d = {"p": [rnd(n, 0.05).to(types(pt, i))[shift:] for i, n in enumerate(sizes)],
         "g": [rnd(n, 10.0 ** -(i % 4)).to(types(gt, i))[shift:] for i, n in enumerate(sizes)],
         "m": [rnd(n, 0.1 * 10.0 ** -(i % 4))[shift:] for i, n in enumerate(sizes)],
         "v": [(rnd(n, 0.3 * 10.0 ** -(i % 4)).square())[shift:] for i, n in enumerate(sizes)]}
    return d


SIZES = {"one": [1], "empty_among": [0, 5, 0, 300], "edges": [8192, 8191, 8193, 16384 + 7, 256, 255, 257],
         "mlp": [784 * 1024, 1024, 1024 * 1024, 1024, 10240, 10], "many": [(i * 37) % 501 + 1 for i in range(600)],
         "large": [9_000_001]}
HYPER = dict(betas=(0.9, 0.999), eps=1e-8)


def _step32(d, lr, t, wd, betas, eps, norm=None, max_norm=math.inf):
    """The definition in 64 bits: (p, m, v) and their bounds before the stored rounding, tensor by tensor."""
    b1, b2 = betas
    out = []
    c = 1.0 if norm is None or not norm > max_norm else max_norm / norm
    for i, p in enumerate(d["p"]):
        w = wd[i] if isinstance(wd, list) else wd
        pp, g, m, v = p.double(), d["g"][i].double() * c, d["m"][i].double(), d["v"][i].double()
        ma = b1 * m.abs() + (1 - b1) * g.abs()
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        den = (v / (1 - b2 ** t)).sqrt() + eps
        s = lr / (1 - b1 ** t)
        new = pp * (1 - lr * w) - s * m / den
        tiny = 2.0 ** -148                    # products below the normal range
        out.append(((new, 4 * U * (pp.abs() + new.abs()) + 30 * U * s * ma / den), (m, 6 * U * ma + tiny),
                    (v, 8 * U * v + tiny)))
    return out


def _check32(d, want):
    for p, m, v, w in zip(d["p"], d["m"], d["v"], want):
        for got, (x, tol) in zip((p, m, v), w):
            assert ((got.double() - x).abs() <= tol + HALF[got.dtype] * (x.abs() + tol)).all()


@pytest.mark.parametrize("case", sorted(SIZES))
@pytest.mark.parametrize("pt,gt,shift", [("f32", "f32", 0), ("f32", "bf16", 0), ("bf16", "bf16", 0), ("f32+bf16", "bf16+f32", 1)])
def test_32_bit(case, pt, gt, shift):
    d = _make(SIZES[case], 1, pt, gt, shift)
    wd = [0.1 * (i % 3) for i in range(len(d["p"]))]
    copies = [torch.full((p.numel() + shift,), 7.0, dtype=torch.bfloat16, device="cuda")[shift:] if i % 2 == 0 else None
              for i, p in enumerate(d["p"])]
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], copies=copies, weight_decay=wd, **HYPER)
    for t in (1, 2, 1000):
        want = _step32(d, 1e-2, t, wd, **HYPER)
        opt.step(1e-2, t)
        _check32(d, want)
    for p, c, w in zip(d["p"], copies, want):
        if c is not None:
            x, tol = w[0]
            assert ((c.double() - x).abs() <= tol + 2.0 ** -8 * (x.abs() + tol)).all()
    opt.close()


@pytest.mark.parametrize("betas", [(0.0, 0.0), (0.0, 0.999), (0.9, 0.0), (0.5, 0.95)])
def test_betas(betas):
    d = _make([1000, 77], 2)
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], betas=betas, eps=1e-3, weight_decay=0.0)
    for t in (1, 7):
        want = _step32(d, 0.1, t, 0.0, betas, 1e-3)
        opt.step(0.1, t)
        _check32(d, want)
    opt.close()


# ---- 8 bits, on the host -----------------------------------------------------------
F = np.float32


def _mix(z):
    with np.errstate(over="ignore"):
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        return z ^ (z >> np.uint64(31))


def _random16(seed, step, place, n):
    with np.errstate(over="ignore"):
        key = _mix(np.uint64(seed) * np.uint64(1000003) + np.uint64(step))
        i = np.arange(place, place + n, dtype=np.uint64)
        word = _mix(key + (i // np.uint64(4) + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15))
        return ((word >> (np.uint64(16) * (i % np.uint64(4)))) & np.uint64(0xFFFF)).astype(np.uint32)


_E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) / 8 * 2.0 ** -6 if not c >> 3 & 15 else
                                               (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7)) for c in range(256)], F)
_E4M3[[127, 255]] = np.nan


def _decode(codes, scales):
    return _E4M3[codes] * np.repeat(scales, B)[: codes.size]


def _encode(x, rnd, least):
    n = x.size
    pad = np.zeros(-(-n // B) * B, F)
    pad[:n] = np.abs(x)
    top = pad.reshape(-1, B).max(1).view(np.uint32)
    scale = np.maximum((((top + np.uint32(0x20A3C4)) & np.uint32(0x7F800000)).view(F) * F(2.0 ** -8)), F(2.0 ** -126))
    y = np.abs(x) / np.repeat(scale, B)[:n]
    # the code below, and one more where the distance to it in 2^16ths and the random number pass a whole
    ulp = np.exp2(np.maximum(np.floor(np.log2(np.maximum(y.astype(np.float64), 2.0 ** -200))), -6) - 3)
    q = y.astype(np.float64) / ulp
    frac = np.floor((q - np.floor(q)) * 2 ** 20)
    val = (np.floor(q) + (frac + rnd.astype(np.float64) * 16 >= 2 ** 20)) * ulp
    codes = np.searchsorted(_E4M3[:127], val.astype(F)).astype(np.uint8)
    assert np.array_equal(_E4M3[codes].astype(np.float64), val)
    codes = np.where((x != 0) & (codes < least), least, codes).astype(np.uint8)
    return codes | (np.signbit(x).astype(np.uint8) << 7), scale


def _host(d):
    """The list's tensors as host arrays (codes as bytes)."""
    def one(t):
        if t.dtype in (torch.float8_e4m3fn, torch.uint8):
            return t.view(torch.uint8).cpu().numpy().copy()
        return t.float().cpu().numpy().copy()
    return {k: [one(t) for t in v] for k, v in d.items()}


def _step8(h, i, place, seed, lr, t, wd, betas, eps, c=1.0):
    """New (m codes, v codes, m scales, v scales), and the parameters in 64 bits with their bound, of tensor i."""
    b1, b2 = F(betas[0]), F(betas[1])
    o1, o2 = F(1.0 - betas[0]), F(1.0 - betas[1])
    m, v = _decode(h["m"][i], h["ms"][i]), _decode(h["v"][i], h["vs"][i])
    g = h["g"][i] * F(c)
    ma = np.abs(m).astype(np.float64) * float(b1) + np.abs(g).astype(np.float64) * float(o1)
    m, v = m * b1 + g * o1, v * v * b2 + g * g * o2
    root = np.sqrt(v)
    rnd = _random16(seed, t, place, m.size)
    mc, ms = _encode(m, rnd, 0)
    vc, vs = _encode(root, rnd, 1)
    p = h["p"][i].astype(np.float64)
    den = root / math.sqrt(1 - betas[1] ** t) + eps
    s = lr / (1 - betas[0] ** t)
    new = p * (1 - lr * wd) - s * m / den
    return (mc, vc, ms, vs), new, 4 * U * (np.abs(p) + np.abs(new)) + 30 * U * s * ma / den


def _make8(sizes, seed, pt="f32", gt="f32", shift=0):
    d = _make(sizes, seed, pt, gt, shift)
    d["m"], d["v"], d["ms"], d["vs"] = mg.adamw_state(d["p"], 8)
    if shift:
        d["m"], d["v"] = ([torch.zeros(t.numel() + 3, dtype=torch.uint8, device="cuda")[3:] for t in d[k]] for k in ("m", "v"))
    return d


@pytest.mark.parametrize("case", ["one", "empty_among", "edges", "many"])
@pytest.mark.parametrize("pt,gt,shift", [("f32", "f32", 0), ("bf16", "bf16", 0), ("f32", "bf16", 0), ("bf16+f32", "f32+bf16", 1)])
def test_8_bit(case, pt, gt, shift):
    """Five steps, changing gradients, every code and scale as the host has it."""
    d = _make8(SIZES[case], 3, pt, gt, shift)
    copies = [torch.zeros(p.numel(), dtype=torch.bfloat16, device="cuda") for p in d["p"]]
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], d["ms"], d["vs"], copies, weight_decay=0.1, seed=5, **HYPER)
    for t in range(1, 6):
        h = _host(d)
        opt.step(1e-2, t)
        place = 0
        for i, p in enumerate(d["p"]):
            n = p.numel()
            if n == 0:
                continue
            (mc, vc, ms, vs), new, tol = _step8(h, i, place, 5, 1e-2, t, 0.1, **HYPER)
            place += -(-n // B) * B
            got = _host({k: [d[k][i]] for k in ("m", "v", "ms", "vs", "p")})
            assert np.array_equal(got["ms"][0], ms) and np.array_equal(got["vs"][0], vs)
            assert np.array_equal(got["m"][0], mc) and np.array_equal(got["v"][0], vc)
            half = HALF[p.dtype]
            assert (np.abs(got["p"][0] - new) <= tol + half * (np.abs(new) + tol)).all()
            assert (np.abs(copies[i].double().cpu().numpy() - new) <= tol + 2.0 ** -8 * (np.abs(new) + tol)).all()
        for k, x in zip(d["g"], _make(SIZES[case], 30 + t, pt, gt, shift)["g"]):
            k.copy_(x)
    opt.close()


def test_8_bit_extremes():
    """Magnitudes from the smallest to the largest, whole blocks of zeros, one value among zeros."""
    n = 12 * B
    g = torch.zeros(n, device="cuda").view(-1, B)
    r = torch.randn(12, B, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    for k, s in enumerate((1e-44, 1e-40, 1e-30, 1e-10, 1.0, 1e10, 1e18)):
        g[k] = r[k] * s
    g[8, 17] = 3.0
    g[9] = 448.0
    g[10] = torch.exp2(-torch.arange(B, device="cuda").float() / 6)
    g[11] = 1e-20
    g[11, 0] = 1e15
    d = {"p": [torch.zeros(n, device="cuda")], "g": [g.view(-1)]}
    d["m"], d["v"], d["ms"], d["vs"] = mg.adamw_state(d["p"], 8)
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], d["ms"], d["vs"], weight_decay=0.0, seed=2 ** 63 + 9, **HYPER)
    for t in range(1, 4):
        h = _host(d)
        opt.step(1e-3, t)
        (mc, vc, ms, vs), new, tol = _step8(h, 0, 0, 2 ** 63 + 9, 1e-3, t, 0.0, **HYPER)
        got = _host(d)
        for a, b in zip((mc, vc, ms, vs), (got["m"][0], got["v"][0], got["ms"][0], got["vs"][0])):
            assert np.array_equal(a, b)
        assert (np.abs(got["p"][0] - new) <= tol + HALF[torch.float32] * (np.abs(new) + tol) + 1e-40).all()
        # an update is bounded where the second moment is known; none is divided by eps alone
        assert np.abs(got["p"][0]).max() <= t * 1e-3 * 12
    opt.close()


def test_8_bit_moments_are_unbiased():
    """Over many elements the mean of the codes is the moment: the rounding's variance is at most a quarter of a step
    squared, so the mean of n equal elements lies within 6 steps / (2 sqrt(n)) of it (six deviations)."""
    n = 1 << 20
    for value in (0.3, 1.01, 17.3):
        d = {"p": [torch.zeros(n, device="cuda")], "g": [torch.full((n,), value, device="cuda")]}
        d["g"][0].view(-1, B)[:, 0] = 20.0
        d["m"], d["v"], d["ms"], d["vs"] = mg.adamw_state(d["p"], 8)
        opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], d["ms"], d["vs"], weight_decay=0.0, seed=3, **HYPER)
        opt.step(1e-3, 1)
        for k, scale, want in (("m", "ms", 0.1 * value), ("v", "vs", math.sqrt(0.001) * value)):
            x = d[k][0].float().view(-1, B)[:, 1:].double() * d[scale][0].double()[:, None]
            step = want / 8
            assert abs(float(x.mean()) - want) <= 6 * step / (2 * math.sqrt(x.numel())) + want * 2.0 ** -16
            assert len(torch.unique(x)) == 2
        opt.close()


def test_8_bit_moments_follow_the_gradients():
    """Gradients that grow and then shrink by ten: the mean over all elements of the second moment's root goes with
    the 32-bit one (rounded to nearest it would stay at its first value, a factor of ten off).

    Bound on the mean of the ratio.  A step moves a code by one place at most, a factor of 9/8 or less, with the
    probability of the distance, so on the way over ln 10 the logarithm's variance is at most ln 10 / 8 = 0.29.  The
    root of beta r^2 + (1 - beta) g^2 is convex in r with a second derivative of at most 1 / r, which biases the
    mean by at most half that variance, 0.145; and the mean of 10240 elements lies within six deviations, 6 sqrt(0.29 /
    10240) = 0.032, of its expectation: 0.18."""
    n = 40 * B
    gen = torch.Generator(device="cuda").manual_seed(4)
    base = torch.exp(torch.randn(n, generator=gen, device="cuda"))
    d = {"p": [torch.zeros(n, device="cuda")], "g": [base.clone()]}
    d["m"], d["v"], d["ms"], d["vs"] = mg.adamw_state(d["p"], 8)
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], d["ms"], d["vs"], betas=(0.9, 0.99), weight_decay=0.0)
    v = torch.zeros(n, dtype=torch.float64, device="cuda")
    t = 0
    for factor in (0.1, 1.0, 0.1):
        d["g"][0].copy_(base * factor)
        for _ in range(300):
            t += 1
            opt.step(1e-4, t)
            v = 0.99 * v + 0.01 * d["g"][0].double() ** 2
        root = d["v"][0].double() * d["vs"][0].double().repeat_interleave(B)
        ratio = root / v.sqrt()
        assert abs(float(ratio.mean()) - 1) <= 0.18
    opt.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_and_skipping(bits):
    sizes = [5000, 33, 70001]
    d = _make8(sizes, 6) if bits == 8 else _make(sizes, 6)
    grads = mg.GradList(d["g"])
    stats = torch.zeros(2, device="cuda")
    more = (d["ms"], d["vs"]) if bits == 8 else ()
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"], *more, weight_decay=0.1, **HYPER)
    grads.clip(math.inf, stats)
    norm = float(stats[0])
    for t, limit in ((1, 0.5), (2, norm * 2), (3, 0.0)):
        h = _host(d)
        c = float(F(limit) / F(norm)) if norm > limit else 1.0
        if bits == 32:
            want = _step32(d, 1e-2, t, 0.1, norm=norm, max_norm=limit, **HYPER)
        opt.step(1e-2, t, norm=stats, max_norm=limit)
        if bits == 32:
            _check32(d, want)
            continue
        place = 0
        for i, n in enumerate(sizes):
            (mc, vc, ms, vs), new, tol = _step8(h, i, place, 0, 1e-2, t, 0.1, c=c, **HYPER)
            place += -(-n // B) * B
            got = _host({k: [d[k][i]] for k in ("m", "v", "p")})
            assert np.array_equal(got["m"][0], mc) and np.array_equal(got["v"][0], vc)
            assert (np.abs(got["p"][0] - new) <= tol + U * (np.abs(new) + tol)).all()
    before = {k: [x.clone() for x in v] for k, v in d.items()}
    for bad in (math.nan, math.inf):
        d["g"][1][3] = bad
        grads.clip(math.inf, stats)
        opt.step(1e-2, 4, norm=stats, max_norm=1.0)
        for k in set(d) - {"g"}:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(d[k], before[k]))
    # without a norm what is not finite reaches its own element (8 bits: its block's states)
    opt.step(1e-2, 4)
    assert not torch.isfinite(d["p"][1][3]) and torch.isfinite(d["p"][0]).all() and torch.isfinite(d["p"][2]).all()
    assert not math.isfinite(float(d["m"][1].float()[3])) and int((~torch.isfinite(d["p"][1])).sum()) == 1
    opt.step(1e-2, 5)
    assert not math.isfinite(float(d["m"][1].float()[3]))
    opt.close()
    grads.close()


@pytest.mark.parametrize("bits", [32, 8])
def test_device_scalars_in_a_graph(bits):
    """lr and t read on the device: a replayed step goes on as launched ones do.  The corrections 1 - beta^t are fp32
    there: expm1 of a rounded exponent, 4 u more."""
    sizes = [9000, 70, 8192]
    a, b = ((_make8(sizes, 8) if bits == 8 else _make(sizes, 8)) for _ in range(2))
    new = lambda d: mg.AdamW(d["p"], d["g"], d["m"], d["v"], d.get("ms"), d.get("vs"), weight_decay=0.1, seed=1, **HYPER)  # noqa: E731
    one, two = new(a), new(b)
    lr, t = torch.zeros(1, device="cuda"), torch.zeros((), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        one.step(lr, t, stream=s)
    for k, rate in ((1, 1e-2), (2, 5e-3), (1000, 1e-3), (50000, 2e-2)):
        lr.fill_(rate)
        t.fill_(k)
        keep = [p.clone() for p in b["p"]]
        graph.replay()
        two.step(rate, k)
        torch.cuda.synchronize()
        for x, y in zip(a["m"] + a["v"], b["m"] + b["v"]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        for x, y, z in zip(a["p"], b["p"], keep):
            assert ((x.double() - y.double()).abs() <= 2 * U * y.double().abs() + 64 * U * (y - z).double().abs() + 64 * U * rate).all()
            y.copy_(x)
    # one of the two on the device
    one.step(lr, 50001)
    two.step(2e-2, torch.tensor([50001], dtype=torch.int32, device="cuda"))
    for x, y in zip(a["p"], b["p"]):
        assert ((x.double() - y.double()).abs() <= 2 * U * y.double().abs() + 64 * U * 2e-2 * 12).all()
    one.close()
    two.close()


def test_overlap_is_refused():
    z = lambda: torch.zeros(600, device="cuda")  # noqa: E731
    p, g, m, v = z(), z(), z(), z()
    for args in (([p, p], [g, z()], [m, z()], [v, z()]), ([p], [p], [m], [v]), ([p], [g], [m], [m]),
                 ([p[:300], p[200:]], [g[:300], g[200:]], [m[:300], z()[:400]], [v[:300], z()[:400]])):
        with pytest.raises(binding.MGError) as e:
            mg.AdamW(*args)
        assert e.value.status == binding.MG_ERR_INVALID_ARG
    # one gradient for two tensors, and neighbours in one buffer: allowed
    mg.AdamW([p[:300], p[300:]], [g[:300], g[:300]], [m[:300], m[300:]], [v[:300], v[300:]]).close()


def test_refused_steps():
    d = _make([10], 1)
    opt = mg.AdamW(d["p"], d["g"], d["m"], d["v"])
    for args, kw in (((-1.0, 1), {}), ((math.nan, 1), {}), ((0.1, 0), {}), ((0.1, 1), dict(norm=torch.zeros(1, device="cuda"), max_norm=-1.0)),
                     ((torch.zeros(2, device="cuda"), 1), {}), ((0.1, torch.ones(1, device="cuda")), {}),
                     ((0.1, 1), dict(norm=torch.zeros(1))), ((0.1, 2 ** 63), {}), ((0.1, 1), dict(norm=d["v"][0][3:5])),
                     ((d["p"][0][9:], 1), {})):
        with pytest.raises(binding.MGError):
            opt.step(*args, **kw)
    opt.close()


def test_tensor_past_2_31_elements():
    n = 2 ** 31 + 1000
    p = torch.zeros(n, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros_like(p)
    at = [0, 2 ** 31 - 1, 2 ** 31, n - 1]
    g[at] = 2.0
    m, v, ms, vs = mg.adamw_state([p], 8)
    opt = mg.AdamW([p], [g], m, v, ms, vs, weight_decay=0.0)
    opt.step(0.5, 1)
    # the first step is lr sign(g); bf16
    assert ((p[at].float() + 0.5).abs() <= 0.5 * 2.0 ** -8).all()
    assert int((p != 0).sum()) == len(at)
    assert int((m[0].view(torch.uint8) != 0).sum()) == len(at)
    opt.close()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, 1e30])
@pytest.mark.parametrize("pt,gt,shift", [("f32", "f32", 0), ("bf16", "bf16", 0), ("f32", "bf16", 1)])
def test_8_bit_neighbours_of_a_moment_that_is_not_finite(pt, gt, shift, bad):
    """A gradient that is not finite, or whose square is not, reaches its own element alone: all others have the codes,
    scales and parameters that they have when its element is 0, step after step.  (A first moment that is large and finite
    decides its block's scale, and with it its neighbours' first moments.)"""
    own = ("v", "vs") if abs(bad) < math.inf else ("m", "v", "ms", "vs", "p")
    sizes = [5 * B + 100, 7]
    at = [(0, 3), (0, 2 * B + 255), (0, 5 * B + 99), (1, 6)]     # in whole blocks, and at the tensors' ends
    d, w = _make8(sizes, 21, pt, gt, shift), _make8(sizes, 21, pt, gt, shift)
    opts = [mg.AdamW(q["p"], q["g"], q["m"], q["v"], q["ms"], q["vs"], weight_decay=0.1, seed=4, **HYPER) for q in (d, w)]
    others = [torch.ones(n, dtype=torch.bool, device="cuda") for n in sizes]
    for i, j in at:
        others[i][j] = False
    for t in range(1, 5):
        for i, g in enumerate(_make(sizes, 40 + t, pt, gt, shift)["g"]):
            for q in (d, w):
                q["g"][i].copy_(g)
        for i, j in at:
            d["g"][i][j] = bad if t == 1 else 0.5
            w["g"][i][j] = 0.0
        for o in opts:
            o.step(1e-2, t)
        for i in range(len(sizes)):
            for k in own:
                a, b = (q[k][i] if k in ("ms", "vs", "p") else q[k][i].view(torch.uint8) for q in (d, w))
                keep = others[i] if k in ("m", "v", "p") else slice(None)
                assert torch.equal(a[keep], b[keep])
        for i, j in at:
            assert int(d["v"][i].view(torch.uint8)[j]) & 0x7F == 0x7F
            if not abs(bad) < math.inf:
                assert int(d["m"][i].view(torch.uint8)[j]) & 0x7F == 0x7F
    for o in opts:
        o.close()
