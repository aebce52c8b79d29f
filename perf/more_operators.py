"""Workloads of the operators around a language model's training step: log probabilities of given tokens with
entropy and top alternatives, the residual stream's norms with gate and scale, and AdamW over many tensors.

Each case is one call as a training or serving program makes it, in a plain form of elementary torch
operations (own = False) or through this package's entry points (own = True), on the same seeded inputs."""
import math

import torch

own = False

BLOCK = 256                       # elements under one scale of an 8-bit state
# the largest magnitude under a scale: just inside e4m3's 448, where sums of short numbers do not fall, so that
# no rounding decides a block's scale
LARGEST = 256.0 * (1.0 + 0x5F5C3B / 2.0 ** 23)


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 32 sequences that answers with 20 alternatives; constrained: a share of the
        # vocabulary is masked with -inf
        {"name": "logp_decode", "op": "logp_fwd", "rows": 32, "vocab": 32000, "stride": 32000, "dtype": "bf16",
         "ids": "i64", "pad": 0.0, "mask": 0.3, "temp": 0.7, "top": 20, "entropy": True},
        # scoring the 16384 tokens of a training step, a tenth of them padding
        {"name": "logp_score_train", "op": "logp_fwd", "rows": 16384, "vocab": 32000, "stride": 32000, "dtype": "bf16",
         "ids": "i32", "pad": 0.1, "mask": 0.0, "temp": 1.0, "top": 0, "entropy": True},
        # an evaluation in fp32 over an odd vocabulary kept in padded rows, with the 5 best alternatives
        {"name": "logp_eval_odd_f32", "op": "logp_fwd", "rows": 1037, "vocab": 50021, "stride": 50048, "dtype": "f32",
         "ids": "i32", "pad": 0.05, "mask": 0.0, "temp": 1.0, "top": 5, "entropy": False},
        # gradient of a policy's loss with an entropy bonus
        {"name": "logp_bwd_train", "op": "logp_bwd", "rows": 16384, "vocab": 32000, "stride": 32000, "dtype": "bf16",
         "ids": "i32", "pad": 0.1, "mask": 0.0, "temp": 1.0, "top": 0, "entropy": True},
        # one decoding step of 32 sequences between two blocks: latency only
        {"name": "norm_decode", "op": "norm_fwd", "rows": 32, "dim": 2048, "dtype": "bf16", "post": True, "pre": True,
         "gates": 1, "scale": 1.0},
        # between two blocks of the 16384-token residual network
        {"name": "norm_fwd_train", "op": "norm_fwd", "rows": 16384, "dim": 2048, "dtype": "bf16", "post": True,
         "pre": True, "gates": 1, "scale": 0.7071},
        # its gradients
        {"name": "norm_bwd_train", "op": "norm_bwd", "rows": 16384, "dim": 2048, "dtype": "bf16", "post": True,
         "pre": True, "gates": 1, "scale": 0.7071},
        # odd width in fp32, a gate for each of 7 sequences
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "rows": 7 * 431, "dim": 777, "dtype": "f32", "post": True,
         "pre": True, "gates": 7, "scale": 1.0},
        # the six tensors of the 784-1024-1024-10 MLP: latency counts
        {"name": "adamw_mlp", "op": "adamw", "layout": "mlp", "total": 1863690, "tensors": 6, "dtype": "f32",
         "grad": "f32", "bits": 32, "copy": False, "clip": True},
        # the 334M-parameter residual network: master weights and a bf16 copy, gradients from the backward in fp32
        {"name": "adamw_resnet", "op": "adamw", "layout": "resmlp", "total": 333987840, "tensors": 25, "dtype": "f32",
         "grad": "f32", "bits": 32, "copy": True, "clip": True},
        # the same with 8-bit states
        {"name": "adamw8_resnet", "op": "adamw", "layout": "resmlp", "total": 333987840, "tensors": 25, "dtype": "f32",
         "grad": "f32", "bits": 8, "copy": True, "clip": True},
        # many ragged tensors kept in bf16 alone
        {"name": "adamw8_ragged_bf16", "op": "adamw", "layout": "ragged", "total": 24000000, "tensors": 400,
         "dtype": "bf16", "grad": "bf16", "bits": 8, "copy": False, "clip": False},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp_fwd", "logp_fwd", "logp_bwd", "norm_fwd", "norm_bwd", "norm_bwd", "adamw", "adamw"])
    if op.startswith("logp"):
        c = {"op": op, "rows": _logint(rng, 1, 16384), "vocab": _logint(rng, 500, 200000),
             "dtype": rng.choice(["bf16", "f32"]), "ids": rng.choice(["i32", "i64"]), "pad": rng.choice([0.0, 0.1]),
             "mask": rng.choice([0.0, 0.0, 0.5]), "temp": rng.choice([1.0, 0.7, 1.3]),
             "top": rng.choice([0, 1, 5, 20, 32]), "entropy": rng.random() < 0.7}
        if rng.random() < 0.5:
            c["vocab"] = c["vocab"] // 8 * 8
        c["stride"] = c["vocab"] if rng.random() < 0.7 else (c["vocab"] + 127) // 64 * 64
        es = 2 if c["dtype"] == "bf16" else 4
        while c["rows"] * c["vocab"] * es > 16384 * 32000 * 2:
            c["rows"] = max(1, c["rows"] // 2)
        if op == "logp_bwd" or c["rows"] * c["vocab"] > 1 << 27:
            c["top"] = 0
        return c
    if op.startswith("norm"):
        c = {"op": op, "rows": _logint(rng, 1, 32768), "dim": _logint(rng, 64, 16384),
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "post": rng.random() < 0.8, "pre": rng.random() < 0.8,
             "gates": rng.choice([0, 1, 1, 4]), "scale": rng.choice([1.0, 0.7071, 0.5])}
        if rng.random() < 0.7:
            c["dim"] = c["dim"] // 8 * 8
        es = 2 if c["dtype"] == "bf16" else 4
        while c["rows"] * c["dim"] * es > 16384 * 2048 * 2:
            c["rows"] = max(1, c["rows"] // 2)
        if c["gates"] > 1:
            c["gates"] = min(c["gates"], c["rows"])
            c["rows"] = c["rows"] // c["gates"] * c["gates"]
        return c
    t = _logint(rng, 1, 400)
    dt = rng.choice(["f32", "f32", "bf16"])
    return {"op": "adamw", "layout": "ragged", "tensors": t, "total": _logint(rng, max(1000, 20 * t), 100000000),
            "dtype": dt, "grad": rng.choice(["f32", "bf16"]), "bits": rng.choice([8, 32]),
            "copy": dt == "f32" and rng.random() < 0.5, "clip": rng.random() < 0.5}


# --------------------------------------------------------------------------------------------- inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_HYPER = {"lr": 3e-4, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1, "seed": 11, "max_norm": 1.0}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logp_inputs(case, g):
    """Logits as a model gives them: a broad bell, a few raised tokens in each row, the given token often among
    them; with `mask` a share of the vocabulary at -inf."""
    r, v, ld = case["rows"], case["vocab"], case["stride"]
    buf = torch.randn(r, ld, generator=g, device="cuda", dtype=_DT[case["dtype"]]).mul_(2.0)
    logits = buf[:, :v]
    ids = torch.randint(0, v, (r,), generator=g, device="cuda")
    raised = torch.randint(0, v, (r, 8), generator=g, device="cuda")
    raised[:, 0] = ids
    logits.scatter_(1, raised, (8.0 + 2.0 * _randn(g, r, 8)).to(logits.dtype))
    if case["mask"]:
        off = torch.rand(v, generator=g, device="cuda") < case["mask"]
        logits.masked_fill_(off, -math.inf)
    if case["pad"]:
        gone = torch.rand(r, generator=g, device="cuda") < case["pad"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return {"logits": logits, "ids": ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)}


def _norm_inputs(case, g):
    r, d, dt = case["rows"], case["dim"], _DT[case["dtype"]]
    st = {"y": _randn(g, r, d).to(dt), "x": (2.0 * _randn(g, r, d)).to(dt)}
    st["gamma_post"] = 1.0 + 0.2 * _randn(g, d) if case["post"] else None
    st["gamma_pre"] = 1.0 + 0.2 * _randn(g, d) if case["pre"] else None
    st["gate"] = 0.5 + 0.2 * _randn(g, case["gates"], d) if case["gates"] else None
    if case["op"] == "norm_bwd":
        st["dxo"] = (1e-3 * _randn(g, r, d)).to(dt)
        st["dh"] = (1e-3 * _randn(g, r, d)).to(dt) if case["pre"] else None
    return st


def _tensor_sizes(case):
    if case["layout"] == "mlp":
        return [784 * 1024, 1024, 1024 * 1024, 1024, 1024 * 10, 10]
    if case["layout"] == "resmlp":
        return 8 * [2048, 2048 * 8192, 8192 * 2048] + [2048 * 32000]
    # ragged: geometric weights, at least one element each, summing to the total
    t, total = case["tensors"], case["total"]
    w = [math.exp(6.0 * ((i * 7919) % t) / t) for i in range(t)]
    s = sum(w)
    sizes = [max(1, int(total * x / s)) for x in w]
    sizes[0] += max(0, total - sum(sizes))
    return sizes


def _starts(sizes):
    """All tensors in one buffer, each at a multiple of BLOCK elements: the starts and the whole length."""
    starts, top = [], 0
    for s in sizes:
        starts.append(top)
        top += (s + BLOCK - 1) // BLOCK * BLOCK
    return starts, top


def _adamw_inputs(case, g):
    """Parameters, gradients and states some steps into a training run, zero between the tensors."""
    sizes = _tensor_sizes(case)
    starts, top = _starts(sizes)
    inside = torch.zeros(top + 1, device="cuda", dtype=torch.int8)
    edges = torch.tensor([a for s, n in zip(starts, sizes) for a in (s, s + n)], device="cuda")
    inside.index_add_(0, edges, torch.tensor([1, -1] * len(sizes), device="cuda", dtype=torch.int8))
    inside = torch.cumsum(inside[:-1], 0, dtype=torch.int8).bool()

    def noise(scale):
        return torch.randn(top, generator=g, device="cuda").mul_(scale).mul_(inside)

    # gradients of very different size from block to block, as layers have them
    size = torch.exp(2.0 * _randn(g, top // BLOCK, 1)).mul_(1e-4)
    st = {"params": noise(0.02).to(_DT[case["dtype"]]),
          "grads": (noise(1.0).view(-1, BLOCK) * size).view(-1).to(_DT[case["grad"]]),
          "sizes": sizes, "starts": starts, "step": 41}
    m = (noise(0.3).view(-1, BLOCK) * size).view(-1)
    root = (noise(0.3).abs_().add_(0.5 * inside).view(-1, BLOCK) * size).view(-1)   # of the second moment
    if case["bits"] == 32:
        st["m"], st["v"] = m, root.square_()
    else:
        for name, x in (("m", m), ("v", root)):
            top_bits = x.abs().view(-1, BLOCK).amax(1).view(torch.int32)
            scale = ((top_bits + 0x20A3C4) & 0x7F800000).view(torch.float32) * 2.0 ** -8
            scale = scale.clamp_(min=2.0 ** -126)
            st[name] = (x.view(-1, BLOCK) / scale[:, None]).view(-1).to(torch.float8_e4m3fn)
            st[name + "_scales"] = scale
    if case["copy"]:
        st["copy"] = st["params"].to(torch.bfloat16)
    st["norm"] = st["grads"].double().square().sum().sqrt().float().view(1) if case["clip"] else None
    return st


def _inputs(case, seed):
    g = _gen(seed)
    if case["op"].startswith("logp"):
        return _logp_inputs(case, g)
    if case["op"].startswith("norm"):
        return _norm_inputs(case, g)
    return _adamw_inputs(case, g)


def _row_statistics(x, temp):
    """(maximum, log of the sum of exponentials) of each row, and the entropy, as a forward pass saved them."""
    x = x.float()
    m = x.amax(1, keepdim=True)
    t = (x - m) / temp
    e = torch.exp(t)
    s = e.sum(1)
    ent = torch.log(s) - (e * torch.where(e > 0, t, torch.zeros_like(t))).sum(1) / s
    return torch.stack([m[:, 0], torch.log(s)], 1), ent


def prepare(case, seed):
    """The inputs, the outputs' buffers, what a forward pass saved for its backward, and what a program keeps
    between calls: a workspace, the optimizer with its list of tensors."""
    st = _inputs(case, seed)
    st["case"] = case
    op = case["op"]
    new = lambda *shape, dtype=torch.float32: torch.empty(*shape, device="cuda", dtype=dtype)  # noqa: E731
    if op == "logp_fwd":
        r, k = case["rows"], case["top"]
        st |= {"logp": new(r), "stats": new(r, 2), "entropy": new(r) if case["entropy"] else None,
               "top_ids": new(r, k, dtype=torch.int32) if k else None, "top_logp": new(r, k) if k else None}
    elif op == "logp_bwd":
        g = _gen(seed + 77)
        r, v = case["rows"], case["vocab"]
        parts = [_row_statistics(st["logits"][a:a + 2048], case["temp"]) for a in range(0, r, 2048)]
        st["stats"] = torch.cat([p[0] for p in parts])
        st["entropy"] = torch.cat([p[1] for p in parts])
        st["dlogp"] = _randn(g, r) / r
        st["dentropy"] = 0.01 * _randn(g, r) / r if case["entropy"] else None
        st["dlogits"] = torch.zeros(r, case["stride"], device="cuda", dtype=_DT[case["dtype"]])[:, :v]
    elif op.startswith("norm"):
        r, d, dt = case["rows"], case["dim"], _DT[case["dtype"]]
        if op == "norm_fwd":
            st |= {"x_out": new(r, d, dtype=dt), "h": new(r, d, dtype=dt) if case["pre"] else None,
                   "rstd": new(r, 2)}
        else:
            st["rstd"] = _norm_plain(case, st)["rstd"]
            st |= {"dy": new(r, d, dtype=dt), "dx": new(r, d, dtype=dt),
                   "dgamma_post": new(d) if case["post"] else None, "dgamma_pre": new(d) if case["pre"] else None,
                   "dgate": new(case["gates"], d) if case["gates"] else None}
    if own:
        import static_graph_nn_gb300 as mg
        if op == "norm_bwd":
            nb = mg.norm_residual_workspace_bytes(case["rows"], case["dim"], case["gates"])
            st["ws"] = torch.zeros(nb, dtype=torch.uint8, device="cuda")
        elif op == "adamw":
            cut = lambda t: None if t is None else [t[a:a + n] for a, n in zip(st["starts"], st["sizes"])]  # noqa: E731
            per = lambda t: None if t is None else [t[a // BLOCK:(a + n + BLOCK - 1) // BLOCK]  # noqa: E731
                                                    for a, n in zip(st["starts"], st["sizes"])]
            st["opt"] = mg.AdamW(cut(st["params"]), cut(st["grads"]), cut(st["m"]), cut(st["v"]),
                                 m_scales=per(st.get("m_scales")), v_scales=per(st.get("v_scales")),
                                 copies=cut(st.get("copy")), betas=_HYPER["betas"], eps=_HYPER["eps"],
                                 weight_decay=_HYPER["weight_decay"], seed=_HYPER["seed"])
    return st


# ------------------------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    return _run_own(case, st) if own else _run_plain(case, st)


def _given(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _run_own(case, st):
    import static_graph_nn_gb300 as mg
    op = case["op"]
    s = torch.cuda.current_stream()
    if op == "logp_fwd":
        mg.token_logprobs(st["logits"], st["ids"], st["logp"], stats=st["stats"], entropy=st["entropy"],
                          top_ids=st["top_ids"], top_logp=st["top_logp"], temperature=case["temp"], stream=s)
        return _given(logp=st["logp"], entropy=st["entropy"], top_ids=st["top_ids"], top_logp=st["top_logp"],
                      stats=st["stats"])
    if op == "logp_bwd":
        mg.token_logprobs_backward(st["logits"], st["ids"], st["stats"], st["dlogp"], st["dlogits"],
                                   entropy=st["entropy"] if case["entropy"] else None, dentropy=st["dentropy"],
                                   temperature=case["temp"], stream=s)
        return {"dlogits": st["dlogits"]}
    if op == "norm_fwd":
        mg.norm_residual_forward(st["y"], st["x"], st["x_out"], st["h"], gamma_post=st["gamma_post"],
                                 gate=st["gate"], gamma_pre=st["gamma_pre"], rstd=st["rstd"], scale=case["scale"],
                                 eps=1e-6, stream=s)
        return _given(x_out=st["x_out"], h=st["h"], rstd=st["rstd"])
    if op == "norm_bwd":
        mg.norm_residual_backward(st["dxo"], st["dh"], st["y"], st["x"], st["rstd"], st["dy"], st["dx"], st["ws"],
                                  gamma_post=st["gamma_post"], gate=st["gate"], gamma_pre=st["gamma_pre"],
                                  dgamma_post=st["dgamma_post"], dgate=st["dgate"], dgamma_pre=st["dgamma_pre"],
                                  scale=case["scale"], stream=s)
        return _given(dy=st["dy"], dx=st["dx"], dgamma_post=st["dgamma_post"], dgate=st["dgate"],
                      dgamma_pre=st["dgamma_pre"])
    st["opt"].step(_HYPER["lr"], st["step"], norm=st["norm"], max_norm=_HYPER["max_norm"], stream=s)
    st["step"] += 1
    return _state(st)


def _state(st):
    return _given(params=st["params"], m=st["m"], v=st["v"], m_scales=st.get("m_scales"),
                  v_scales=st.get("v_scales"), copy=st.get("copy"))


def _run_plain(case, st):
    if case["op"] == "logp_fwd":
        return _logp_plain(case, st)
    if case["op"] == "logp_bwd":
        return _logp_backward_plain(case, st)
    if case["op"] == "norm_fwd":
        out = _norm_plain(case, st)
        return _given(x_out=out["x_out"].to(st["x"].dtype), rstd=out["rstd"],
                      h=out["h"].to(st["x"].dtype) if case["pre"] else None)
    if case["op"] == "norm_bwd":
        return _norm_backward_plain(case, st)
    return _adamw_plain(case, st)


def _logp_plain(case, st):
    x, v = st["logits"].float(), case["vocab"]
    ids = st["ids"].long()
    ok = (ids >= 0) & (ids < v)
    m = x.amax(1, keepdim=True)
    t = (x - m) / case["temp"]
    e = torch.exp(t)
    s = e.sum(1)
    logs = torch.log(s)
    zero = torch.zeros_like(s)
    out = {"logp": torch.where(ok, t.gather(1, torch.where(ok, ids, 0)[:, None])[:, 0] - logs, zero),
           "stats": torch.stack([m[:, 0], logs], 1) * ok[:, None]}
    if case["entropy"]:
        plogp = (e * torch.where(e > 0, t, torch.zeros_like(t))).sum(1) / s
        out["entropy"] = torch.where(ok, logs - plogp, zero)
    if case["top"]:
        # the order of the values, then of the positions from the front: one integer for both
        bits = x.view(torch.int32).long()
        key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) * (1 << 20)
        key += (1 << 20) - 1 - torch.arange(v, device=x.device)
        best = torch.topk(key, case["top"], dim=1)[0]
        top = ((1 << 20) - 1) - (best & ((1 << 20) - 1))
        out["top_logp"] = torch.where(ok[:, None], t.gather(1, top) - logs[:, None], zero[:, None])
        out["top_ids"] = torch.where(ok[:, None], top, -torch.ones_like(top)).int()
    return out


def _logp_backward_plain(case, st):
    x, temp = st["logits"].float(), case["temp"]
    ids = st["ids"].long()
    ok = (ids >= 0) & (ids < case["vocab"])
    logp = (x - st["stats"][:, :1]) / temp - st["stats"][:, 1:]
    p = torch.exp(logp)
    g = st["dlogp"][:, None]
    d = -(p * g)
    if case["entropy"]:
        d -= st["dentropy"][:, None] * p * (torch.where(p > 0, logp, torch.zeros_like(p)) + st["entropy"][:, None])
    d.scatter_add_(1, torch.where(ok, ids, 0)[:, None], g)
    st["dlogits"].copy_(torch.where(ok[:, None], d / temp, torch.zeros_like(d)))
    return {"dlogits": st["dlogits"]}


def _gate_rows(case, st):
    """The gate of every row, or None."""
    return None if st["gate"] is None else st["gate"].repeat_interleave(case["rows"] // case["gates"], 0)


def _norm_plain(case, st):
    y, x = st["y"].float(), st["x"].float()
    r1 = torch.rsqrt(y.square().mean(1) + 1e-6) if case["post"] else torch.ones_like(y[:, 0])
    u = y * r1[:, None] * st["gamma_post"] if case["post"] else y
    if case["gates"]:
        u = u * _gate_rows(case, st)
    x_out = case["scale"] * x + u
    r2 = torch.rsqrt(x_out.square().mean(1) + 1e-6) if case["pre"] else torch.ones_like(r1)
    h = x_out * r2[:, None] * st["gamma_pre"] if case["pre"] else None
    return {"x_out": x_out, "h": h, "rstd": torch.stack([r1, r2], 1)}


def _norm_backward_plain(case, st):
    y, x, dt = st["y"].float(), st["x"].float(), st["x"].dtype
    r1, r2 = st["rstd"][:, :1], st["rstd"][:, 1:]
    u = y * r1 * st["gamma_post"] if case["post"] else y
    gate = _gate_rows(case, st)
    t = st["dxo"].float()
    out = {}
    if case["pre"]:
        xo = case["scale"] * x + (u if gate is None else gate * u)
        dh = st["dh"].float()
        a = dh * st["gamma_pre"]
        t = t + r2 * (a - xo * r2.square() * (a * xo).mean(1, keepdim=True))
        out["dgamma_pre"] = (dh * xo * r2).sum(0)
    if gate is not None:
        out["dgate"] = (t * u).view(case["gates"], -1, case["dim"]).sum(1)
    du = t if gate is None else gate * t
    if case["post"]:
        out["dgamma_post"] = (du * y * r1).sum(0)
        b = du * st["gamma_post"]
        out["dy"] = (r1 * (b - y * r1.square() * (b * y).mean(1, keepdim=True))).to(dt)
    else:
        out["dy"] = du.to(dt)
    out["dx"] = (case["scale"] * t).to(dt)
    return out


def _signed(z):
    return z - (1 << 64) if z >= 1 << 63 else z


_GAMMA, _M1, _M2 = (_signed(z) for z in (0x9E3779B97F4A7C15, 0xBF58476D1CE4E5B9, 0x94D049BB133111EB))


def _mix(z):
    """SplitMix64's finalizer on int64 tensors (logical shifts)."""
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _M1
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _M2
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _random16(n, step):
    """16 random bits for each element of the whole list: a 64-bit word for four of them."""
    key = _mix(torch.tensor([_HYPER["seed"] * 1000003 + step], device="cuda"))
    word = _mix(key + (torch.arange(n // 4, device="cuda") + 1) * _GAMMA)
    return ((word[:, None] >> torch.tensor([0, 16, 32, 48], device="cuda")) & 0xFFFF).view(-1).int()


def _encode(x, rnd, least):
    """Blocks of x in e4m3 under power-of-two scales, rounded up or down by the random bits; a value that is not
    zero is at least the code `least`."""
    blocks = x.view(-1, BLOCK)
    top_bits = blocks.abs().amax(1).view(torch.int32)
    scale = (((top_bits + 0x20A3C4) & 0x7F800000).view(torch.float32) * 2.0 ** -8).clamp_(min=2.0 ** -126)
    bits = ((blocks / scale[:, None]).view(-1) * 2.0 ** -120).view(torch.int32)
    code = ((bits & 0x7FFFFFFF) + rnd * 16) >> 20
    if least:
        code = torch.maximum(code, (x != 0).int() * least)
    return (code | torch.where(bits < 0, 128, 0)).to(torch.uint8).view(torch.float8_e4m3fn), scale


def _adamw_plain(case, st):
    p, g = st["params"].float(), st["grads"].float()
    b1, b2 = _HYPER["betas"]
    t, lr, n = st["step"], _HYPER["lr"], st["params"].numel()
    if case["clip"]:
        norm = st["norm"]
        g = g * torch.where(norm > _HYPER["max_norm"], _HYPER["max_norm"] / norm, torch.ones_like(norm))
    if case["bits"] == 8:
        m = (st["m"].float().view(-1, BLOCK) * st["m_scales"][:, None]).view(-1)
        v = (st["v"].float().view(-1, BLOCK) * st["v_scales"][:, None]).view(-1).square()
    else:
        m, v = st["m"], st["v"]
    m = m * b1 + g * (1.0 - b1)
    v = v * b2 + g * g * (1.0 - b2)
    root = torch.sqrt(v)
    p = p * (1.0 - lr * _HYPER["weight_decay"]) - m * (lr / (1.0 - b1 ** t)) / (
        root * (1.0 / math.sqrt(1.0 - b2 ** t)) + _HYPER["eps"])
    st["params"].copy_(p)
    if case["bits"] == 8:
        rnd = _random16(n, t)
        for name, x, least in (("m", m, 0), ("v", root, 1)):
            code, scale = _encode(x, rnd, least)
            st[name].copy_(code)
            st[name + "_scales"].copy_(scale)
    else:
        st["m"].copy_(m)
        st["v"].copy_(v)
    if case["copy"]:
        st["copy"].copy_(p)
    st["step"] += 1
    return _state(st)


# ------------------------------------------------------------------------------------------ arithmetic
def work(case):
    op = case["op"]
    es = 2 if case.get("dtype") == "bf16" else 4
    if op.startswith("logp"):
        live = case["rows"] * (1.0 - case["pad"])
        n = live * case["vocab"]
        idb = 4 if case["ids"] == "i32" else 8
        if op == "logp_fwd":
            return {"bytes": int(es * n + case["rows"] * (idb + 12 + 4 * case["entropy"] + 8 * case["top"])),
                    "flops": 5 * n}
        return {"bytes": int(es * (n + case["rows"] * case["vocab"]) + case["rows"] * (idb + 12 + 8 * case["entropy"])),
                "flops": 8 * n}
    if op.startswith("norm"):
        n = case["rows"] * case["dim"]
        vec = 4 * case["dim"] * (case["post"] + case["pre"] + case["gates"])
        if op == "norm_fwd":
            return {"bytes": es * n * (3 + case["pre"]) + vec + 8 * case["rows"], "flops": 10 * n}
        return {"bytes": es * n * (5 + case["pre"]) + 2 * vec + 8 * case["rows"], "flops": 25 * n}
    n = sum(_tensor_sizes(case))
    states = 16 if case["bits"] == 32 else 4 + 16.0 / BLOCK
    per = 2 * es + (2 if case["grad"] == "bf16" else 4) + states + 2 * case["copy"]
    return {"bytes": int(per * n), "flops": 16 * n}


def exact(case, seed):
    """The definitions in 64 bits, rows in blocks."""
    op = case["op"]
    if op.startswith("logp"):
        return _exact_logp(case, seed)
    if op.startswith("norm"):
        return _exact_norm(case, seed)
    return _exact_adamw(case, seed)


def _exact_logp(case, seed):
    st = prepare(case, seed) if case["op"] == "logp_bwd" else _inputs(case, seed)
    f8, v = torch.float64, case["vocab"]
    parts = []
    for a in range(0, case["rows"], 1024):
        z = st["logits"][a:a + 1024].to(f8) / case["temp"]
        ids = st["ids"][a:a + 1024].long()
        live = ((ids >= 0) & (ids < v)).to(f8)
        at = ids.clamp(0, v - 1)[:, None]
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        p = lp.exp()
        h = -torch.special.xlogy(p, p).sum(1)
        if case["op"] == "logp_bwd":
            # the statistics are inputs: the saved ones, in fp32
            sav = st["stats"][a:a + 1024].to(f8)
            lp = z - sav[:, :1] / case["temp"] - sav[:, 1:]
            p = lp.exp()
            one = torch.zeros_like(z).scatter_(1, at, 1.0)
            d = st["dlogp"][a:a + 1024, None].to(f8) * (one - p)
            if case["entropy"]:
                d -= st["dentropy"][a:a + 1024, None].to(f8) * (
                    torch.special.xlogy(p, p) + p * st["entropy"][a:a + 1024, None].to(f8))
            parts.append({"dlogits": d * live[:, None] / case["temp"]})
            continue
        m = st["logits"][a:a + 1024].amax(1).to(f8)
        none = live == 0
        o = {"logp": lp.gather(1, at)[:, 0].masked_fill(none, 0.0),
             "stats": torch.stack([m, lse - m / case["temp"]], 1) * live[:, None]}
        if case["entropy"]:
            o["entropy"] = h * live
        if case["top"]:
            idx = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :case["top"]]
            o["top_ids"] = idx.masked_fill(none[:, None], -1).int()
            o["top_logp"] = lp.gather(1, idx).masked_fill(none[:, None], 0.0)
        parts.append(o)
    return {k: torch.cat([o[k] for o in parts]) for k in parts[0]}


def _exact_norm(case, seed):
    st = prepare(case, seed)
    f8 = torch.float64
    r, d, n = case["rows"], case["dim"], max(1, case["gates"])
    up = lambda t: None if t is None else t.to(f8)  # noqa: E731
    y, x, s = up(st["y"]).view(n, -1, d), up(st["x"]).view(n, -1, d), case["scale"]
    g1 = up(st["gamma_post"]) if case["post"] else 1.0
    g2 = up(st["gamma_pre"]) if case["pre"] else 1.0
    a = up(st["gate"])[:, None, :] if case["gates"] else 1.0
    if case["op"] == "norm_fwd":
        one = torch.ones(n, r // n, 1, dtype=f8, device="cuda")
        r1 = 1.0 / torch.sqrt(torch.einsum("nrd,nrd->nr", y, y)[..., None] / d + 1e-6) if case["post"] else one
        xo = s * x + a * (g1 * (y * r1))
        r2 = 1.0 / torch.sqrt(torch.einsum("nrd,nrd->nr", xo, xo)[..., None] / d + 1e-6) if case["pre"] else one
        out = {"x_out": xo.view(r, d), "rstd": torch.cat([r1.view(r, 1), r2.view(r, 1)], 1)}
        return out | ({"h": (g2 * (xo * r2)).view(r, d)} if case["pre"] else {})
    r1, r2 = up(st["rstd"])[:, 0].view(n, -1, 1), up(st["rstd"])[:, 1].view(n, -1, 1)
    u = g1 * (y * r1) if case["post"] else y
    t = up(st["dxo"]).view(n, -1, d)
    out = {}
    if case["pre"]:
        xh = (s * x + a * u) * r2
        dh = up(st["dh"]).view(n, -1, d)
        out["dgamma_pre"] = torch.einsum("nrd,nrd->d", dh, xh)
        q = dh * g2
        t = t + r2 * (q - xh * torch.einsum("nrd,nrd->nr", q, xh)[..., None] / d)
    if case["gates"]:
        out["dgate"] = torch.einsum("nrd,nrd->nd", t, u)
    w = a * t
    dy = w
    if case["post"]:
        yh = y * r1
        out["dgamma_post"] = torch.einsum("nrd,nrd->d", w, yh)
        q = w * g1
        dy = r1 * (q - yh * torch.einsum("nrd,nrd->nr", q, yh)[..., None] / d)
    return out | {"dy": dy.reshape(r, d), "dx": (s * t).reshape(r, d)}


def _exact_adamw(case, seed):
    st = _inputs(case, seed)
    f8 = torch.float64
    b1, b2 = _HYPER["betas"]
    t, lr = st["step"], _HYPER["lr"]
    g = st["grads"].to(f8)
    if case["clip"]:
        g *= min(1.0, _HYPER["max_norm"] / float(st["norm"]))
    m, v = st["m"].to(f8), st["v"].to(f8)
    if case["bits"] == 8:
        m *= st["m_scales"].to(f8).repeat_interleave(BLOCK)
        v = (v * st["v_scales"].to(f8).repeat_interleave(BLOCK)) ** 2
    m = torch.lerp(g, m, b1)
    v = torch.lerp(g * g, v, b2)
    p = st["params"].to(f8)
    p = p - lr * (_HYPER["weight_decay"] * p + (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + _HYPER["eps"]))
    out = {"params": p}
    if case["bits"] == 32:
        out |= {"m": m, "v": v}
    else:
        rnd = _random16(p.numel(), t).to(f8) / 65536.0
        for name, x in (("m", m), ("v", v.sqrt())):
            mag = x.abs()
            top = mag.view(-1, BLOCK).amax(1)
            # the least power of two that keeps the block within the largest magnitude
            e = torch.ceil(torch.log2((top / LARGEST).clamp(min=2.0 ** -200)))
            scale = torch.exp2(e.clamp(min=-126.0))
            mag /= scale.repeat_interleave(BLOCK)
            ulp = torch.exp2(torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))) - 3.0)
            code = torch.floor(mag / ulp + rnd) * ulp
            if name == "v":
                code = torch.where((mag > 0) & (code < 2.0 ** -9), torch.full_like(code, 2.0 ** -9), code)
            out |= {name: torch.copysign(code, x), name + "_scales": scale}
    if case["copy"]:
        out["copy"] = p
    return out
