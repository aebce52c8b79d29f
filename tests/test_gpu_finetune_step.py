"""The operators around a language model's step together, as a fine-tuning step uses
them: token ids, a block between the residual stream's norms, a head, the given
tokens' log probabilities with an entropy bonus, the gradients back to every
parameter, their norm, and AdamW.  And all of them on many streams at once.

Bound of the gradients.  Five stages (embedding, block, norms, head, loss) forward
and as many back, each sum of at most 200 terms: 10 (200 + 30) 2^-24 = 1.4e-4 of
the terms' magnitudes; cancellation among terms of random signs leaves sums of n
terms at least about sqrt(n) smaller than their magnitudes, 14 for 200: 2e-3 of a
gradient's largest value."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import static_graph_nn_gb300 as mg   # noqa: E402

V, D, R, EPS, SCALE, BONUS, TEMP = 190, 96, 61, 1e-6, 0.7, 0.03, 0.9
BOUND = 2e-3


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Model:
    """table -> (w, post norm, gate, scaled residual, pre norm) -> head; fp32."""

    def __init__(self, seed, bits):
        g = _gen(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.p = {"table": rnd(V, D), "w": rnd(1, D, D) / math.sqrt(D), "post": 1 + 0.2 * rnd(D), "gate": 0.5 + 0.2 * rnd(D),
                  "pre": 1 + 0.2 * rnd(D), "head": rnd(1, D, V) / math.sqrt(D)}
        self.g = {k: torch.full_like(v, 7.0) for k, v in self.p.items()}
        new = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.x, self.y, self.xo, self.h = (new(R, D) for _ in range(4))
        self.dh, self.dy, self.dx, self.dxb = (new(R, D) for _ in range(4))
        self.logits, self.dlogits = new(R, V), new(R, V)
        self.rstd, self.stats, self.logp, self.entropy = new(R, 2), new(R, 2), new(R), new(R)
        self.off = torch.tensor([0, R], dtype=torch.int32, device="cuda")
        z = lambda n: torch.zeros(n, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws = [z(mg.grouped_linear_workspace_bytes(R, 1, D, D)), z(mg.grouped_linear_workspace_bytes(R, 1, D, V)),
                   z(mg.embedding_workspace_bytes(R, V, D)), z(mg.norm_residual_workspace_bytes(R, D, 1))]
        self.norm = new(2)
        grads = list(self.g.values())
        self.grads = mg.GradList(grads)
        params = list(self.p.values())
        self.state = mg.adamw_state(params, bits)
        decay = [0.1 if k in ("w", "head") else 0.0 for k in self.p]
        self.opt = mg.AdamW(params, grads, *self.state, weight_decay=decay)

    def gradients(self, ids, targets, weights, bonus, s=None):
        p, g = self.p, self.g
        mg.embedding_forward(p["table"], ids, self.x, stream=s)
        mg.grouped_linear_forward(self.x, self.off, p["w"], self.y, self.ws[0], stream=s)
        mg.norm_residual_forward(self.y, self.x, self.xo, self.h, gamma_post=p["post"], gate=p["gate"], gamma_pre=p["pre"],
                                 scale=SCALE, eps=EPS, rstd=self.rstd, stream=s)
        mg.grouped_linear_forward(self.h, self.off, p["head"], self.logits, self.ws[1], stream=s)
        mg.token_logprobs(self.logits, targets, self.logp, self.stats, self.entropy, temperature=TEMP, stream=s)
        mg.token_logprobs_backward(self.logits, targets, self.stats, weights, self.dlogits, entropy=self.entropy,
                                   dentropy=bonus, temperature=TEMP, stream=s)
        mg.grouped_linear_backward_weight(self.h, self.dlogits, self.off, g["head"], self.ws[1], stream=s)
        mg.grouped_linear_backward_input(self.dlogits, self.off, p["head"], self.dh, self.ws[1], stream=s)
        mg.norm_residual_backward(None, self.dh, self.y, self.x, self.rstd, self.dy, self.dx, self.ws[3],
                                  gamma_post=p["post"], gate=p["gate"], gamma_pre=p["pre"], dgamma_post=g["post"],
                                  dgate=g["gate"], dgamma_pre=g["pre"], scale=SCALE, stream=s)
        mg.grouped_linear_backward_weight(self.x, self.dy, self.off, g["w"], self.ws[0], stream=s)
        mg.grouped_linear_backward_input(self.dy, self.off, p["w"], self.dxb, self.ws[0], stream=s)

    def step(self, batch, lr, t, s=None):
        self.gradients(*batch, s=s)
        if s is None:
            self.dx += self.dxb
        else:
            with torch.cuda.stream(s):
                self.dx += self.dxb
        mg.embedding_backward(self.dx, batch[0], self.g["table"], self.ws[2], stream=s)
        self.grads.clip(math.inf, self.norm, stream=s)
        self.opt.step(lr, t, norm=self.norm, max_norm=0.5, stream=s)

    def reference(self, batch):
        """Gradients by autograd in 64 bits."""
        ids, targets, weights, bonus = batch
        p = {k: v.double().requires_grad_() for k, v in self.p.items()}
        norm = lambda v: v * (v.square().mean(1, keepdim=True) + EPS).rsqrt()  # noqa: E731
        x = p["table"][ids.long()]
        xo = SCALE * x + p["gate"] * (norm(x @ p["w"][0]) * p["post"])
        lp = torch.log_softmax((norm(xo) * p["pre"]) @ p["head"][0] / TEMP, 1)
        live = (targets >= 0).double()
        given = lp.gather(1, targets.clamp(0)[:, None].long())[:, 0]
        ((weights.double() * given + bonus.double() * -(lp.exp() * lp).sum(1)) * live).sum().backward()
        return {k: v.grad for k, v in p.items()}, given * live


def _batch(seed):
    g = _gen(seed)
    ids = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    targets = torch.randint(0, V, (R,), generator=g, device="cuda", dtype=torch.int32)
    targets[::7] = -1
    return ids, targets, -torch.rand(R, generator=g, device="cuda") / R, torch.full((R,), -BONUS / R, device="cuda")


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step(bits):
    m = Model(1, bits)
    for t in range(1, 4):
        batch = _batch(t)
        want, given = m.reference(batch)
        before = {k: v.clone() for k, v in m.p.items()}
        m.step(batch, 1e-2, t)
        for k in want:
            assert (m.g[k].double() - want[k]).abs().max() <= BOUND * want[k].abs().max(), k
        assert ((m.logp.double() - given).abs() <= 1e-4).all()
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in m.g.values()))
        assert abs(float(m.norm[0]) - norm) <= 1e-6 * norm
        if t == 1:       # the first update is lr sign(g) beside the decay
            for k, v in m.p.items():
                big = want[k].abs() > 1e-3 * want[k].abs().max()
                keep = 1 - 1e-2 * (0.1 if k in ("w", "head") else 0.0)
                d = (v.double() - before[k].double() * keep)[big]
                assert ((d + 1e-2 * want[k][big].sign()).abs() <= 1e-4).all(), k


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_goes_on_as_launched_ones_do(bits):
    a, b = Model(2, bits), Model(2, bits)
    batch = _batch(9)
    lr, t = torch.zeros(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.gradients(*batch, s=s)                       # (a first run outside of the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.step(batch, lr, t, s=s)
    for k in range(1, 6):
        for x, y in zip(batch, _batch(20 + k)):
            x.copy_(y)
        lr.fill_(1e-2 / k)
        t.fill_(k)
        graph.replay()
        b.step(batch, lr, t)
        torch.cuda.synchronize()
        for x, y in zip(list(a.p.values()) + list(a.g.values()) + a.state[0] + a.state[1],
                        list(b.p.values()) + list(b.g.values()) + b.state[0] + b.state[1]):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ---- many streams -----------------------------------------------------------------
def _logp_work(rows, vocab, t, k, seed):
    x = (2 * torch.randn(rows, vocab, generator=_gen(seed), device="cuda")).to(t)
    ids = torch.randint(-1, vocab, (rows,), generator=_gen(seed), device="cuda", dtype=torch.int32)
    new = lambda *s, d=torch.float32: torch.zeros(*s, device="cuda", dtype=d)  # noqa: E731
    o = [new(rows), new(rows, 2), new(rows), new(rows, k, d=torch.int32), new(rows, k), torch.zeros_like(x)]
    g = torch.randn(rows, generator=_gen(seed + 1), device="cuda")

    def call(s):
        mg.token_logprobs(x, ids, o[0], o[1], o[2], o[3], o[4], stream=s)
        mg.token_logprobs_backward(x, ids, o[1], g, o[5], entropy=o[2], dentropy=g, stream=s)
    call.keep = (x, ids, g)
    return call, o


def _norm_work(rows, dim, t, gates, seed):
    rnd = lambda n, *s: torch.randn(*s, generator=_gen(seed + n), device="cuda")  # noqa: E731
    y, x, dxo, dh = (rnd(i, rows, dim).to(t) for i in range(4))
    g1, g2, gate = 1 + 0.1 * rnd(5, dim), 1 + 0.1 * rnd(6, dim), rnd(7, gates, dim)
    o = [torch.zeros_like(x) for _ in range(4)] + [torch.zeros(rows, 2, device="cuda"), torch.zeros(dim, device="cuda"),
                                                    torch.zeros(dim, device="cuda"), torch.zeros_like(gate)]
    ws = torch.zeros(mg.norm_residual_workspace_bytes(rows, dim, gates), dtype=torch.uint8, device="cuda")

    def call(s):
        mg.norm_residual_forward(y, x, o[0], o[1], gamma_post=g1, gate=gate, gamma_pre=g2, rstd=o[4], stream=s)
        mg.norm_residual_backward(dxo, dh, y, x, o[4], o[2], o[3], ws, gamma_post=g1, gate=gate, gamma_pre=g2,
                                  dgamma_post=o[5], dgate=o[7], dgamma_pre=o[6], stream=s)
    call.keep = (y, x, dxo, dh, g1, g2, gate, ws)
    return call, o


def _adamw_work(n, bits, seed):
    """Always the first step, from parameters that are put back before it."""
    keep = torch.randn(n, generator=_gen(seed), device="cuda")
    p, g = keep.clone(), torch.randn(n, generator=_gen(seed + 1), device="cuda")
    m, v, ms, vs = mg.adamw_state([p], bits)
    opt = mg.AdamW([p], [g], m, v, ms, vs)
    outs = [p, m[0], v[0]] + ([ms[0], vs[0]] if bits == 8 else [])

    def call(s):
        with torch.cuda.stream(s or torch.cuda.current_stream()):
            p.copy_(keep)
            for t in outs[1:]:
                t.view(torch.uint8).zero_()
        opt.step(1e-2, 1, stream=s)
    call.keep = (keep, g, opt)
    return call, outs


@pytest.mark.parametrize("replayed", [False, True])
def test_many_streams_at_once(replayed):
    bf, f32 = torch.bfloat16, torch.float32
    work = [_logp_work(3, 131072, bf, 20, 1), _logp_work(900, 5003, f32, 7, 2), _logp_work(700, 1000, bf, 32, 3),
            _norm_work(2000, 2048, bf, 1, 4), _norm_work(300, 777, f32, 3, 5), _norm_work(40, 16384, bf, 2, 6),
            _norm_work(500, 200, bf, 5, 7), _norm_work(64, 8192, f32, 1, 8), _adamw_work(3_000_001, 32, 9),
            _adamw_work(500_000, 8, 10)]
    for call, _ in work:
        call(None)
    torch.cuda.synchronize()
    want = [[o.clone() for o in outs] for _, outs in work]
    streams = [torch.cuda.Stream() for _ in work]
    graphs = []
    if replayed:
        for (call, _), s in zip(work, streams):
            s.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call(s)
            graphs.append(g)
    for _, outs in work:
        for o in outs:
            o.view(torch.uint8).fill_(1)
    torch.cuda.synchronize()
    for _ in range(15):
        for i, ((call, _), s) in enumerate(zip(work, streams)):
            if replayed:
                with torch.cuda.stream(s):
                    graphs[i].replay()
            else:
                call(s)
    torch.cuda.synchronize()
    for (call, outs), w in zip(work, want):
        for a, b in zip(outs, w):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
