"""The language-model operators on several streams at once, launched and replayed
from graphs, each call with a workspace (a list) of its own: the same bits as one
after the other."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _randn(shape, t, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=t)


def _grouped(rows, e, k, n, t, seed):
    """The three products; returns (call, outputs)."""
    x, dy, w = _randn((rows, k), t, seed), _randn((rows, n), t, seed + 1), _randn((e, k, n), t, seed + 2)
    cut = torch.randint(0, rows + 1, (e - 1,), generator=torch.Generator().manual_seed(seed)).sort().values.tolist()
    off = torch.tensor([0] + cut + [rows], dtype=torch.int32, device="cuda")
    ws = torch.zeros(mg.grouped_linear_workspace_bytes(rows, e, k, n), dtype=torch.uint8, device="cuda")
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros(e, k, n, device="cuda")

    def call(s):
        mg.grouped_linear_forward(x, off, w, y, ws, stream=s)
        mg.grouped_linear_backward_input(dy, off, w, dx, ws, stream=s)
        mg.grouped_linear_backward_weight(x, dy, off, dw, ws, stream=s)
    call.keep = (x, dy, w, off, ws)
    return call, [y, dx, dw]


def _embedding(n, v, d, t, seed):
    ids = torch.randint(-1, v, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32).cuda()
    ids[: n // 3] = 1
    dout, dt, out = _randn((n, d), t, seed), torch.zeros(v, d, device="cuda"), torch.zeros(n, d, dtype=t, device="cuda")
    ws = torch.zeros(mg.embedding_workspace_bytes(n, v, d), dtype=torch.uint8, device="cuda")

    def call(s):
        mg.embedding_backward(dout, ids, dt, ws, stream=s)
        mg.embedding_forward(dt, ids, out, stream=s)
    call.keep = (ids, dout, ws)
    return call, [dt, out]


def _clip(sizes, t, seed):
    grads = [_randn((s,), t, seed + i) for i, s in enumerate(sizes)]
    outs = [torch.zeros_like(g) for g in grads]
    stats = torch.zeros(2, device="cuda")
    lst = mg.GradList(grads, outs)

    def call(s):
        lst.clip(0.5, stats, stream=s)
    call.keep = (grads, lst)
    return call, outs + [stats]


def _work():
    bf, f32 = torch.bfloat16, torch.float32
    return [_clip([8192 * 450], f32, 1), _clip([1000, 3_000_000, 7], bf, 2), _clip([8192] * 400, f32, 3),
            _clip([9_000_001], f32, 4), _grouped(4000, 5, 512, 1024, bf, 5), _grouped(20, 6, 2048, 1000, bf, 6),
            _grouped(900, 3, 601, 1003, bf, 7), _grouped(700, 3, 300, 517, f32, 8), _embedding(9000, 4000, 512, bf, 9),
            _embedding(70001, 500, 40, f32, 10)]


@pytest.mark.parametrize("replayed", [False, True])
def test_many_streams_at_once(replayed):
    work = _work()
    for call, _ in work:
        call(None)
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in work]
    streams = [torch.cuda.Stream() for _ in work]
    graphs = []
    if replayed:
        for (call, _), s in zip(work, streams):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call(s)
            graphs.append(g)
    for _, outs in work:
        for o in outs:
            o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(25):
        for i, ((call, _), s) in enumerate(zip(work, streams)):
            if replayed:
                with torch.cuda.stream(s):
                    graphs[i].replay()
            else:
                call(s)
    torch.cuda.synchronize()
    for (call, outs), w in zip(work, want):
        for a, b in zip(outs, w):
            assert torch.equal(a, b)
