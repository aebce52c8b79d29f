"""Workloads of the language-model operators: embedding lookup and its gradient, matrix products grouped by
expert, and the global gradient norm with clipping.

Each case is one call as a training or serving program makes it, in a plain form of elementary torch
operations (own = False) or through this package's entry points (own = True), on the same seeded inputs."""
import math

import torch

own = False


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 32 sequences: a lookup of single tokens, latency only
        {"name": "embed_fwd_decode", "op": "embed_fwd", "n": 32, "vocab": 32000, "dim": 2048,
         "dtype": "bf16", "ids": "i32", "pad": 0.0, "scale": 1.0},
        # the input of the 16384-token residual network's step
        {"name": "embed_fwd_train", "op": "embed_fwd", "n": 16384, "vocab": 32000, "dim": 2048,
         "dtype": "bf16", "ids": "i32", "pad": 0.0, "scale": 45.25483399593904},
        # its gradient: word frequencies as text has them, so a few ids are very frequent
        {"name": "embed_bwd_train", "op": "embed_bwd", "n": 16384, "vocab": 32000, "dim": 2048,
         "dtype": "bf16", "ids": "i32", "pad": 0.0, "scale": 45.25483399593904},
        # a small odd vocabulary in fp32 with a padded batch
        {"name": "embed_bwd_odd_f32", "op": "embed_bwd", "n": 5003, "vocab": 10007, "dim": 777,
         "dtype": "f32", "ids": "i64", "pad": 0.1, "scale": 0.5},
        # the six gradients of the 784-1024-1024-10 MLP: latency counts
        {"name": "clip_mlp", "op": "clip", "layout": "mlp", "total": 1863690, "tensors": 6,
         "dtype": "f32", "max_norm": 1.0},
        # the gradients of the 334M-parameter residual network
        {"name": "clip_resnet", "op": "clip", "layout": "resmlp", "total": 333987840, "tensors": 25,
         "dtype": "f32", "max_norm": 1.0},
        # many ragged tensors, bf16
        {"name": "clip_ragged_bf16", "op": "clip", "layout": "ragged", "total": 24000000, "tensors": 400,
         "dtype": "bf16", "max_norm": 0.5},
        # one decoding step of 12 sequences routed to two experts each: bound by the experts' weights
        {"name": "experts_fwd_decode", "op": "experts_fwd", "rows": 24, "groups": 8, "d_in": 2048,
         "d_out": 8192, "dtype": "bf16", "skew": 0.5},
        # the widening layer of a training step, forward, input gradient and weight gradient
        {"name": "experts_fwd_train", "op": "experts_fwd", "rows": 16384, "groups": 8, "d_in": 2048,
         "d_out": 8192, "dtype": "bf16", "skew": 0.5},
        {"name": "experts_dx_train", "op": "experts_dx", "rows": 16384, "groups": 8, "d_in": 2048,
         "d_out": 8192, "dtype": "bf16", "skew": 0.5},
        {"name": "experts_dw_train", "op": "experts_dw", "rows": 16384, "groups": 8, "d_in": 2048,
         "d_out": 8192, "dtype": "bf16", "skew": 0.5},
        # the strict-f32 path with odd widths and many small groups
        {"name": "experts_fwd_strict", "op": "experts_fwd", "rows": 4096, "groups": 16, "d_in": 1001,
         "d_out": 517, "dtype": "f32", "skew": 1.0},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_fwd", "embed_bwd", "clip", "experts_fwd", "experts_dx", "experts_dw"])
    if op.startswith("embed"):
        c = {"op": op, "n": _logint(rng, 1, 32768), "vocab": _logint(rng, 1000, 64000),
             "dim": _logint(rng, 64, 4096), "dtype": rng.choice(["bf16", "f32"]),
             "ids": rng.choice(["i32", "i64"]), "pad": rng.choice([0.0, 0.1]),
             "scale": rng.choice([1.0, 0.5, 45.25483399593904])}
        if rng.random() < 0.6:
            c["dim"] = max(8, c["dim"] // 8 * 8)
        return c
    if op == "clip":
        t = _logint(rng, 1, 400)
        return {"op": "clip", "layout": "ragged", "tensors": t,
                "total": _logint(rng, max(1000, 20 * t), 100000000),
                "dtype": rng.choice(["bf16", "f32"]), "max_norm": rng.choice([0.5, 1.0, 1e6])}
    dt = "f32" if rng.random() < 0.2 else "bf16"
    c = {"op": op, "rows": _logint(rng, 1, 16384), "groups": _logint(rng, 1, 64),
         "d_in": _logint(rng, 64, 8192), "d_out": _logint(rng, 64, 8192), "dtype": dt,
         "skew": rng.choice([0.0, 0.5, 1.0])}
    if rng.random() < 0.8:
        c["d_in"], c["d_out"] = c["d_in"] // 8 * 8, c["d_out"] // 8 * 8
    mac = 16384 * 2048 * 8192 if dt == "bf16" else 4096 * 1001 * 517
    wmax = 8 * 2048 * 8192 if dt == "bf16" else 16 * 1001 * 517
    while c["rows"] * c["d_in"] * c["d_out"] > mac:
        c["rows"] = max(1, c["rows"] // 2)
        if c["rows"] == 1:
            break
    while c["groups"] * c["d_in"] * c["d_out"] > wmax and c["groups"] > 1:
        c["groups"] //= 2
    while c["d_in"] * c["d_out"] > wmax:
        c["d_in"] = max(64, c["d_in"] // 2)
        c["d_out"] = max(64, c["d_out"] // 2)
    return c


# --------------------------------------------------------------------------------------------- inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ids(case, g):
    """Token ids with the frequencies of text (one over the rank), spread over the vocabulary, and a share
    of padding (-1)."""
    v, n = case["vocab"], case["n"]
    p = 1.0 / (torch.arange(v, device="cuda", dtype=torch.float64) + 3.0)
    cdf = torch.cumsum(p / p.sum(), 0)
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    rank = torch.searchsorted(cdf, u).clamp_(max=v - 1)
    ids = torch.randperm(v, generator=g, device="cuda")[rank]
    if case["pad"]:
        pad = torch.rand(n, generator=g, device="cuda") < case["pad"]
        ids = torch.where(pad, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32 if case["ids"] == "i32" else torch.int64)


def _sizes(case, seed):
    """Rows of each expert: a router's choice with unequal popularity."""
    g = torch.Generator()
    g.manual_seed(seed)
    e = case["groups"]
    p = torch.softmax(case["skew"] * torch.randn(e, generator=g), 0)
    ids = torch.multinomial(p, case["rows"], replacement=True, generator=g)
    return torch.bincount(ids, minlength=e).tolist()


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


def _flat(sizes, dt):
    """One buffer of all tensors, each starting on a multiple of 64 elements, zero between them, and the views
    of the tensors, as an optimizer holds them."""
    starts, top = [], 0
    for s in sizes:
        starts.append(top)
        top += (s + 63) // 64 * 64
    flat = torch.zeros(top, device="cuda", dtype=dt)
    return flat, [flat[a:a + s] for a, s in zip(starts, sizes)]


def _inputs(case, seed):
    g = _gen(seed)
    op = case["op"]
    dt = _DT[case["dtype"]]
    if op == "embed_fwd":
        table = torch.randn(case["vocab"], case["dim"], generator=g, device="cuda", dtype=dt).mul_(0.02)
        return {"table": table, "ids": _ids(case, g)}
    if op == "embed_bwd":
        dout = torch.randn(case["n"], case["dim"], generator=g, device="cuda", dtype=dt).mul_(1e-3)
        return {"dout": dout, "ids": _ids(case, g)}
    if op == "clip":
        sizes = _tensor_sizes(case)
        flat, grads = _flat(sizes, dt)
        for i, x in enumerate(grads):
            x.copy_(torch.randn(x.numel(), generator=g, device="cuda", dtype=dt)).mul_(10.0 ** (-(i % 4)))
        return {"grads": grads}
    rows, e, k, n = case["rows"], case["groups"], case["d_in"], case["d_out"]
    sizes = _sizes(case, seed)
    off = [0]
    for s in sizes:
        off.append(off[-1] + s)
    d = {"sizes": sizes, "offsets": torch.tensor(off, dtype=torch.int32, device="cuda")}
    if op in ("experts_fwd", "experts_dw"):
        d["x"] = torch.randn(rows, k, generator=g, device="cuda", dtype=dt)
    if op in ("experts_dx", "experts_dw"):
        d["dy"] = torch.randn(rows, n, generator=g, device="cuda", dtype=dt).mul_(1e-3)
    if op in ("experts_fwd", "experts_dx"):
        d["w"] = torch.randn(e, k, n, generator=g, device="cuda", dtype=dt).mul_(1.0 / math.sqrt(k))
    return d


def prepare(case, seed):
    """The inputs, the outputs' buffers and what a program keeps between calls: a workspace, the list of
    gradient tensors."""
    st = _inputs(case, seed)
    st["case"] = case
    op = case["op"]
    dt = _DT[case["dtype"]]
    if op == "embed_fwd":
        st["out"] = torch.empty(case["n"], case["dim"], device="cuda", dtype=dt)
    elif op == "embed_bwd":
        st["dtable"] = torch.empty(case["vocab"], case["dim"], device="cuda")
    elif op == "clip":
        st["flat"], st["out"] = _flat([x.numel() for x in st["grads"]], dt)
        st["stats"] = torch.empty(2, device="cuda")
    elif op == "experts_fwd":
        st["y"] = torch.empty(case["rows"], case["d_out"], device="cuda", dtype=dt)
    elif op == "experts_dx":
        st["dx"] = torch.empty(case["rows"], case["d_in"], device="cuda", dtype=dt)
    else:
        st["dw"] = torch.empty(case["groups"], case["d_in"], case["d_out"], device="cuda")
    if own:
        import static_graph_nn_gb300 as mg
        if op == "embed_bwd":
            nb = mg.embedding_workspace_bytes(case["n"], case["vocab"], case["dim"])
            st["ws"] = torch.empty(nb, dtype=torch.uint8, device="cuda")
        elif op == "clip":
            st["list"] = mg.GradList(st["grads"], st["out"])
        elif op.startswith("experts"):
            nb = mg.grouped_linear_workspace_bytes(case["rows"], case["groups"], case["d_in"], case["d_out"])
            st["ws"] = torch.zeros(nb, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    return _run_own(case, st) if own else _run_plain(case, st)


def _run_own(case, st):
    import static_graph_nn_gb300 as mg
    op = case["op"]
    s = torch.cuda.current_stream()
    if op == "embed_fwd":
        mg.embedding_forward(st["table"], st["ids"], st["out"], scale=case["scale"], stream=s)
        return st["out"]
    if op == "embed_bwd":
        mg.embedding_backward(st["dout"], st["ids"], st["dtable"], st["ws"], scale=case["scale"], stream=s)
        return st["dtable"]
    if op == "clip":
        st["list"].clip(case["max_norm"], st["stats"], stream=s)
        return {"norm": st["stats"][0], "grads": st["flat"]}
    if op == "experts_fwd":
        mg.grouped_linear_forward(st["x"], st["offsets"], st["w"], st["y"], st["ws"], stream=s)
        return st["y"]
    if op == "experts_dx":
        mg.grouped_linear_backward_input(st["dy"], st["offsets"], st["w"], st["dx"], st["ws"], stream=s)
        return st["dx"]
    mg.grouped_linear_backward_weight(st["x"], st["dy"], st["offsets"], st["dw"], st["ws"], stream=s)
    return st["dw"]


def _run_plain(case, st):
    op = case["op"]
    if op == "embed_fwd":
        ids = st["ids"].long()
        ok = (ids >= 0) & (ids < case["vocab"])
        rows = st["table"][torch.where(ok, ids, torch.zeros_like(ids))].float() * case["scale"]
        return (rows * ok[:, None]).to(st["out"].dtype)
    if op == "embed_bwd":
        ids = st["ids"].long()
        ok = (ids >= 0) & (ids < case["vocab"])
        d = st["dtable"]
        d.zero_()
        d.index_add_(0, torch.where(ok, ids, torch.zeros_like(ids)), st["dout"].float() * ok[:, None])
        return d.mul_(case["scale"])
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for x in st["grads"]:
            total += x.float().square().sum(dtype=torch.float64)
        norm = total.sqrt()
        mx = case["max_norm"]
        c = torch.where(torch.isfinite(norm) & (norm > mx), mx / norm, torch.ones_like(norm)).float()
        for x, o in zip(st["grads"], st["out"]):
            o.copy_(x.float() * c)
        return {"norm": norm.float(), "grads": st["flat"]}
    r = 0
    for e, s in enumerate(st["sizes"]):
        if op == "experts_fwd":
            st["y"][r:r + s] = (st["x"][r:r + s].float() @ st["w"][e].float()).to(st["y"].dtype)
        elif op == "experts_dx":
            st["dx"][r:r + s] = (st["dy"][r:r + s].float() @ st["w"][e].float().t()).to(st["dx"].dtype)
        else:
            st["dw"][e] = st["x"][r:r + s].float().t() @ st["dy"][r:r + s].float()
        r += s
    return st["y"] if op == "experts_fwd" else st["dx"] if op == "experts_dx" else st["dw"]


# ------------------------------------------------------------------------------------------ arithmetic
def work(case):
    op = case["op"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op == "clip":
        n = sum(_tensor_sizes(case))
        return {"bytes": 2 * es * n, "flops": 3 * n}
    if op.startswith("embed"):
        idb = 4 if case["ids"] == "i32" else 8
        nd = case["n"] * case["dim"]
        if op == "embed_fwd":
            # each distinct row of the table once: the expected number of distinct ids is below both n and V
            rows = min(case["n"], case["vocab"])
            return {"bytes": case["n"] * idb + es * (rows * case["dim"] + nd), "flops": nd}
        return {"bytes": case["n"] * idb + es * nd + 4 * case["vocab"] * case["dim"], "flops": nd}
    t, e, k, n = case["rows"], case["groups"], case["d_in"], case["d_out"]
    used = e * (1.0 - (1.0 - 1.0 / e) ** t)          # experts that get a row, with equal popularity
    w = (4 * e if op == "experts_dw" else es * used) * k * n
    return {"bytes": int(es * t * (k + n) + w + 4 * (e + 1)), "flops": 2 * t * k * n}


def exact(case, seed):
    """The definitions in 64 bits, row block by row block."""
    st = _inputs(case, seed)
    op = case["op"]
    f8 = torch.float64
    if op == "embed_fwd":
        out = torch.zeros(case["n"], case["dim"], dtype=f8, device="cuda")
        sel = ((st["ids"] >= 0) & (st["ids"] < case["vocab"])).nonzero()[:, 0]
        out[sel] = st["table"].index_select(0, st["ids"][sel].long()).to(f8) * case["scale"]
        return out
    if op == "embed_bwd":
        out = torch.zeros(case["vocab"], case["dim"], dtype=f8, device="cuda")
        sel = ((st["ids"] >= 0) & (st["ids"] < case["vocab"])).nonzero()[:, 0]
        out.index_put_((st["ids"][sel].long(),), st["dout"][sel].to(f8) * case["scale"], accumulate=True)
        return out
    if op == "clip":
        sq = [float((x.to(f8) ** 2).sum()) for x in st["grads"]]
        norm = math.sqrt(math.fsum(sq))
        c = min(1.0, case["max_norm"] / norm) if math.isfinite(norm) and norm > 0 else 1.0
        parts = []
        for x in st["grads"]:
            parts += [x.to(f8) * c, torch.zeros(-x.numel() % 64, dtype=f8, device="cuda")]
        return {"norm": torch.tensor(norm, dtype=f8, device="cuda"), "grads": torch.cat(parts)}
    bounds = torch.tensor([0] + st["sizes"]).cumsum(0).tolist()
    if op == "experts_dw":
        return torch.stack([torch.einsum("tk,tn->kn", st["x"][a:b].to(f8), st["dy"][a:b].to(f8))
                            for a, b in zip(bounds, bounds[1:])])
    src, sub = (st["x"], "tk,kn->tn") if op == "experts_fwd" else (st["dy"], "tn,kn->tk")
    return torch.cat([torch.einsum(sub, src[a:b].to(f8), st["w"][e].to(f8))
                      for e, (a, b) in enumerate(zip(bounds, bounds[1:]))])
