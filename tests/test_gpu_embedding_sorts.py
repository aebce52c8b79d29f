"""The embedding gradient on both sides of every size at which its sort changes:
positions up to 65536 are sorted by one cluster of four or eight CTAs with one,
two, four or eight positions a thread, more by several launches.

Tolerances as in test_gpu_embedding: (c + 1) half steps of the sum of the
magnitudes for a sum of c terms and the factor."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_embedding import _bwd, _bwd_check, _ids, _randn   # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


# with vocabulary * width above 2048 n (four CTAs) and below (eight); widths that
# are multiples of 8, even and odd; vocabularies of one, two and three digits
@pytest.mark.parametrize("n,v,d", [
    (4096, 9000, 1024), (4097, 9000, 1030), (8192, 9000, 2048), (8192, 17000, 999),
    (8193, 17001, 1000), (12289, 32000, 1024), (16384, 33000, 1025), (16384, 300000, 120),
    (4097, 5, 64), (8192, 700, 33), (8193, 500, 64), (16384, 500, 65), (16384, 40000, 40),
    (16385, 300, 24), (32768, 90000, 40), (32768, 31, 17), (32769, 700, 40), (65535, 70000, 16),
    (65536, 3, 24), (65536, 511, 33), (65537, 3, 24), (65537, 70000, 9)])
@pytest.mark.parametrize("t,kind", [("f32", "i64"), ("bf16", "i32")])
def test_every_sort(n, v, d, t, kind):
    dout = _randn((n, d), t, 3)
    for hot, bad in ((0.3, 0.1), (0.0, 0.0)):
        ids = _ids(n, v, kind, 4, bad=bad, hot=hot)
        got = _bwd(dout, ids, v, -0.37)
        _bwd_check(dout, ids, v, -0.37, got)
        assert torch.equal(got, _bwd(dout, ids, v, -0.37))


@pytest.mark.parametrize("n", [8192, 16384, 32768, 65536])
@pytest.mark.parametrize("order", ["one", "ascending", "descending"])
def test_extreme_orders(n, order):
    """All positions under one id, and ids in order and against it."""
    v, d = n, 8
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    ids = {"one": torch.full_like(i, v - 1), "ascending": i, "descending": n - 1 - i}[order]
    dout = _randn((n, d), "f32", 5)
    got = _bwd(dout, ids, v, 1.0)
    _bwd_check(dout, ids, v, 1.0, got)
