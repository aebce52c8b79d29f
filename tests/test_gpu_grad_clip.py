"""Global gradient norm and clipping over lists of tensors, against the
definitions in 64 bits.

Tolerances.  32 squares are added in fp32 (eight running sums of four, three
more additions: at most seven roundings a term, relative 7 * 2^-24 of a sum of
nonnegative terms), the rest in fp64; the root halves that, and rounding the
result adds 2^-24: 4.5 * 2^-24 for the norm.  The factor adds one rounding, the
product another: 6.5 * 2^-24 in fp32, and bf16's 2^-8 for a bf16 output."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402
from static_graph_nn_gb300 import binding  # noqa: E402

U32, U16 = 2.0 ** -24, 2.0 ** -8
NORM_TOL, F32_TOL, BF16_TOL = 4.5 * U32, 6.5 * U32, U16 + 7 * U32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _make(sizes, types, seed, mag=1.0, shift=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = torch.bfloat16 if types[i % len(types)] == "bf16" else torch.float32
        x = torch.randn(n + shift, generator=g, device="cuda") * mag * 10.0 ** (-(i % 3))
        out.append(x.to(t)[shift:])
    return out


def _want(grads, max_norm):
    norm = math.sqrt(math.fsum(float(x.double().square().sum()) for x in grads))
    c = max_norm / norm if math.isfinite(norm) and norm > max_norm else 1.0
    return norm, c


def _check(grads, outs, stats, max_norm):
    norm, c = _want(grads, max_norm)
    assert abs(float(stats[0]) - norm) <= NORM_TOL * norm
    assert abs(float(stats[1]) - c) <= (NORM_TOL + U32) * c
    for g, o in zip(grads, outs):
        tol = BF16_TOL if o.dtype == torch.bfloat16 else F32_TOL
        w = g.double() * c
        assert ((o.double() - w).abs() <= tol * w.abs() + 1e-45).all()


CASES = {
    "one_value": ([1], ["f32"], 0),
    "empty_among": ([0, 5, 0, 17], ["f32"], 0),
    "chunk_edges": ([16384, 16383, 16385, 32768 + 16], ["f32", "bf16"], 0),
    "mlp": ([784 * 1024, 1024, 1024 * 1024, 1024, 10240, 10], ["f32"], 0),
    "many": ([(i * 37) % 501 + 1 for i in range(700)], ["bf16", "f32"], 0),
    "unaligned": ([1000, 33, 70001], ["f32", "bf16"], 1),
    "large": ([30_000_001], ["bf16"], 0),
}


@pytest.mark.parametrize("case", sorted(CASES))
@pytest.mark.parametrize("max_norm", [0.25, 1e9])
def test_clip(case, max_norm):
    sizes, types, shift = CASES[case]
    grads = _make(sizes, types, 1, shift=shift)
    stats = torch.empty(2, device="cuda")
    outs = [torch.full_like(x, 9.0) for x in grads]
    lst = mg.GradList(grads, outs)
    keep = [x.clone() for x in grads]
    lst.clip(max_norm, stats)
    _check(keep, outs, stats, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    first = [stats.clone()] + [o.clone() for o in outs]
    lst.clip(max_norm, stats)                       # the same bits again
    assert all(torch.equal(a, b) for a, b in zip(first, [stats] + outs))
    lst.close()
    # in place
    lst = mg.GradList(grads)
    lst.clip(max_norm, stats)
    _check(keep, grads, stats, max_norm)
    lst.close()


@pytest.mark.parametrize("mag", [1e-30, 1e-42, 1e-22, 1e18, 1e30, 3e38])
def test_range(mag):
    """Squares that leave fp32's range do not."""
    x = torch.full((5000,), mag, device="cuda")
    x[::3] = 0.0
    x[1::3] *= 0.5
    stats = torch.empty(2, device="cuda")
    out = [torch.empty_like(x)]
    lst = mg.GradList([x], out)
    lst.clip(mag, stats)
    norm, c = _want([x], float(torch.tensor(mag, dtype=torch.float32)))
    if norm > 3.4028235e38:          # the norm itself is beyond fp32
        assert math.isinf(float(stats[0]))
        assert abs(float(stats[1]) - c) <= (NORM_TOL + U32) * c
    else:
        assert abs(float(stats[0]) - norm) <= NORM_TOL * norm + 1e-45
        # below the normal range a value's spacing is 2^-149
        want = x.double() * c
        assert ((out[0].double() - want).abs() <= F32_TOL * want.abs() + 2.0 ** -149).all()
    lst.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_not_finite(bad):
    """The norm says so, and the gradients are left as they are."""
    grads = _make([300, 20000, 7], ["f32", "bf16"], 3)
    grads[1][12345] = bad
    keep = [x.clone() for x in grads]
    outs = [torch.empty_like(x) for x in grads]
    stats = torch.empty(2, device="cuda")
    for lst, got in ((mg.GradList(grads), grads), (mg.GradList(grads, outs), outs)):
        lst.clip(0.1, stats)
        assert not math.isfinite(float(stats[0]))
        assert math.isnan(float(stats[0])) == math.isnan(bad)
        assert float(stats[1]) == 1.0
        for a, b in zip(keep, got):
            assert torch.equal(a.view(torch.int16 if a.element_size() == 2 else torch.int32),
                               b.view(torch.int16 if a.element_size() == 2 else torch.int32))
        lst.close()


def test_zero_and_infinite_limits():
    grads = _make([1000, 17], ["f32"], 4)
    keep = [x.clone() for x in grads]
    stats = torch.empty(2, device="cuda")
    lst = mg.GradList(grads)
    lst.clip(math.inf, stats)
    assert float(stats[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(keep, grads))
    lst.clip(0.0, stats)
    assert float(stats[1]) == 0.0 and all((x == 0).all() for x in grads)
    lst.clip(0.0, stats)                            # all zero: norm 0
    assert float(stats[0]) == 0.0 and float(stats[1]) == 1.0
    for v in (-1.0, float("nan")):
        with pytest.raises(binding.MGError):
            lst.clip(v, stats)
    lst.close()


def test_all_empty():
    stats = torch.full((2,), 5.0, device="cuda")
    lst = mg.GradList([torch.empty(0, device="cuda")])
    lst.clip(1.0, stats)
    assert stats.tolist() == [0.0, 1.0]
    lst.close()


def test_overlap_is_refused():
    x = torch.zeros(100, device="cuda")
    y = torch.zeros(100, device="cuda")
    for args in (([x, x],), ([x, x[10:20]],), ([x, y], [y, x]), ([x[:50], y], [x[25:75], y]),
                 ([x, y[:100]], [y, torch.zeros(100, device="cuda")])):
        with pytest.raises(binding.MGError) as e:
            mg.GradList(*args)
        assert e.value.status == binding.MG_ERR_INVALID_ARG
    # read only twice, written apart: allowed
    o = [torch.empty(100, device="cuda") for _ in range(2)]
    mg.GradList([x, x], o).close()
    # neighbours in one buffer: allowed
    mg.GradList([x[:50], x[50:]]).close()


def test_streams_and_graph_replay():
    grads = _make([5000, 70000, 3], ["f32", "bf16"], 5)
    outs = [torch.empty_like(x) for x in grads]
    stats = torch.empty(2, device="cuda")
    lst = mg.GradList(grads, outs)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lst.clip(0.5, stats, stream=s)
    for seed in (6, 7):
        for a, b in zip(grads, _make([5000, 70000, 3], ["f32", "bf16"], seed, mag=seed - 5)):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        _check(grads, outs, stats, 0.5)
    lst.close()


def test_list_is_ready_for_any_stream():
    """Clipping on a stream that does not wait for the default one, directly
    after the list was made (its table and counters are complete by then)."""
    s = torch.cuda.Stream()
    for i in range(20):
        grads = _make([70001] * 16, ["f32"], i)
        norm, c = _want(grads, 1.0)
        stats = torch.zeros(2, device="cuda")
        torch.cuda.synchronize()
        gl = mg.GradList(grads)
        gl.clip(1.0, stats, stream=s)
        s.synchronize()
        gl.close()
        assert abs(float(stats[0]) - norm) <= NORM_TOL * norm
        assert abs(float(stats[1]) - c) <= (NORM_TOL + U32) * c
