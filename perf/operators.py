"""The training-step operators around the expert layer, as measured cases.

Five operators, each as the plain torch form and as the library's call:

``route``            logits -> expert ids and gates (scores, balance bias, groups, top-k, renormalised)
``route_backward``   dgates -> dlogits
``balance``          expert loads and the update of the balance bias
``router_backward``  dgates -> gradients of the router's input and weight
``clip``             global norm of many gradients, and the gradients scaled to a largest norm

Inputs follow the package's synthetic workloads: unit-variance logits plus a
per-expert offset (a trained router is skewed), a balance bias in steps of its
update rate, unit-variance activations, router weights of variance 1/d.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # decoding one token: pure latency
        dict(name="route one token", op="route", T=1, N=256, k=8, dt="f32", score="sigmoid",
             bias=True, renorm=True, scale=2.5, groups=8, keep=4, gscore="top2"),
        # a ragged batch of bf16 logits over a number of experts that is no power of two
        dict(name="route ragged", op="route", T=4099, N=60, k=6, dt="bf16", score="softmax",
             bias=True, renorm=False, scale=1.0, groups=1, keep=1, gscore="max"),
        # the largest workload's tokens and experts, with every part of the choice at work
        dict(name="route large", op="route", T=32768, N=256, k=8, dt="f32", score="sigmoid",
             bias=True, renorm=True, scale=2.5, groups=8, keep=4, gscore="top2"),
        # the headline batch: gradient of gates renormalised over two of 64 experts
        dict(name="route_backward batch", op="route_backward", T=4096, N=64, k=2, dt="f32",
             score="softmax", renorm=True, scale=1.0),
        # the largest workload, gates of the full softmax: every logit has a gradient
        dict(name="route_backward large", op="route_backward", T=32768, N=256, k=4, dt="f32",
             score="softmax", renorm=False, scale=1.0),
        # loads of a small batch over 8 experts
        dict(name="balance small", op="balance", T=256, N=8, k=2),
        # loads of the largest workload
        dict(name="balance large", op="balance", T=32768, N=256, k=8),
        # router gradient of the headline layer
        dict(name="router_backward batch", op="router_backward", T=4096, d=512, N=64, k=2,
             dt="bf16", score="softmax", renorm=True, scale=1.0, add=True),
        # full softmax gates, so the gradient of the logits is dense (d = 2048, 64 experts)
        dict(name="router_backward dense", op="router_backward", T=16384, d=2048, N=64, k=2,
             dt="bf16", score="softmax", renorm=False, scale=1.0, add=True),
        # the largest workload
        dict(name="router_backward large", op="router_backward", T=32768, d=4096, N=256, k=4,
             dt="bf16", score="sigmoid", renorm=True, scale=1.0, add=True),
        # one headline layer's gradients: theta, phi, W, router
        dict(name="clip layer", op="clip", layers=1, d=512, N=64, router="f32", extra=0),
        # eight layers of d = 4096 with 256 experts, each with a bf16 tensor of odd size
        dict(name="clip model", op="clip", layers=8, d=4096, N=256, router="bf16", extra=50257),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "balance", "router_backward", "clip"])
    if op == "clip":
        d = 1 << rng.randint(6, 12)
        return dict(op=op, layers=rng.randint(1, 8), d=d, N=_log(rng, 4, 256),
                    router=rng.choice(["f32", "bf16"]), extra=rng.choice([0, _log(rng, 1, 60000)]))
    if op == "balance":
        N = _log(rng, 8, 512)
        return dict(op=op, T=_log(rng, 1, 32768), N=N, k=rng.randint(1, 8))
    score = rng.choice(["softmax", "sigmoid"])
    renorm = rng.random() < 0.6
    scale = rng.choice([1.0, 2.5])
    if op == "router_backward":
        N = _log(rng, 8, 256)
        d = 1 << rng.randint(6, 12)
        dense = score == "softmax" and not renorm
        T = _log(rng, 16, 16384 if dense else 32768)
        return dict(op=op, T=T, d=d, N=min(N, 64) if dense else N, k=rng.randint(1 + renorm, 4),
                    dt=rng.choice(["bf16", "bf16", "f32"]) if T * d <= 1 << 25 else "bf16",
                    score=score, renorm=renorm, scale=scale, add=rng.random() < 0.5)
    T = _log(rng, 1, 32768)
    dt = rng.choice(["f32", "bf16"])
    if op == "route_backward":
        N = _log(rng, 8, 256)
        # (one renormalised gate is constant: its gradient is zero)
        return dict(op=op, T=T, N=N, k=rng.randint(1 + renorm, 8), dt=dt, score=score,
                    renorm=renorm, scale=scale)
    groups = rng.choice([1, 1, 4, 8])
    if groups > 1:
        N = groups * rng.randint(8, 256 // groups)
        keep = rng.randint(1, groups // 2 + 1)
    else:
        N, keep = _log(rng, 8, 256), 1
    return dict(op=op, T=T, N=N, k=rng.randint(1, 8), dt=dt, score=score,
                bias=rng.random() < 0.6, renorm=renorm, scale=scale, groups=groups, keep=keep,
                gscore=rng.choice(["max", "top2"]))


# ---- inputs ----------------------------------------------------------------

def _logits(g, T, N):
    skew = torch.randn(N, generator=g, device="cuda") * 0.5
    return torch.randn(T, N, generator=g, device="cuda") + skew


def _ids(g, T, N, k):
    """k distinct experts a token, the hotter ones (low ids) more often."""
    u = torch.rand(T, N, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    keys = -torch.log(-torch.log(u)) - 0.7 * torch.log1p(torch.arange(N, device="cuda").float())
    return torch.topk(keys, k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "clip":
        d, N, L = case["d"], case["N"], case["d"].bit_length() - 1
        grads = []
        for _ in range(case["layers"]):
            for shape in ((N, L, d // 2), (N, L, d // 2), (d, d)):
                grads.append(torch.randn(shape, generator=g, device="cuda") * 0.01)
            grads.append((torch.randn(N, d, generator=g, device="cuda") * 0.1).to(_DT[case["router"]]))
            if case["extra"]:
                grads.append((torch.randn(case["extra"], generator=g, device="cuda") * 0.1).to(torch.bfloat16))
        s.update(grads=grads, out=[torch.empty_like(t) for t in grads], max_norm=1.0)
        return s
    T, N, k = case["T"], case["N"], case["k"]
    if op == "balance":
        s.update(ids=_ids(g, T, N, k), load=torch.zeros(N, dtype=torch.int32, device="cuda"),
                 bias=torch.randint(-100, 101, (N,), generator=g, device="cuda") * 1e-3, rate=1e-3)
        return s
    if op == "route":
        s.update(logits=_logits(g, T, N).to(_DT[case["dt"]]),
                 b=torch.randint(-100, 101, (N,), generator=g, device="cuda") * 1e-3
                 if case["bias"] else None,
                 ids=torch.empty(T, k, dtype=torch.int32, device="cuda"),
                 gates=torch.empty(T, k, device="cuda"))
        return s
    s.update(ids=_ids(g, T, N, k), dgates=torch.randn(T, k, generator=g, device="cuda"))
    if op == "route_backward":
        s.update(logits=_logits(g, T, N).to(_DT[case["dt"]]),
                 dlogits=torch.empty(T, N, device="cuda"))
        return s
    d, dt = case["d"], _DT[case["dt"]]
    x = torch.randn(T, d, generator=g, device="cuda").to(dt)
    w = (torch.randn(N, d, generator=g, device="cuda") / math.sqrt(d)).to(dt)
    s.update(x=x, w=w, logits=_logits(g, T, N),
             dx_add=torch.randn(T, d, generator=g, device="cuda").to(dt) if case["add"] else None,
             dx=torch.empty_like(x), dw=torch.empty(N, d, device="cuda"))
    return s


# ---- the plain forms -------------------------------------------------------

def _scores(l, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    # scores and their order in 64 bits: neighbouring choices differ by less than fp32 holds
    l = s["logits"].double()
    T, N = l.shape
    sc = _scores(l, s["score"])
    c = sc if s["b"] is None else sc + s["b"].double()
    if s["groups"] > 1:
        cg = c.view(T, s["groups"], N // s["groups"])
        if s["gscore"] == "max":
            gs = cg.amax(2)
        else:
            gs = torch.sort(cg, dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :s["keep"]]
        kept = torch.zeros(T, s["groups"], dtype=torch.bool, device=l.device).scatter_(1, best, True)
        c = torch.where(kept[:, :, None], cg, -math.inf).reshape(T, N)
    ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    g = sc.gather(1, ids)
    if s["renorm"]:
        g = g / g.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "gates": (g * s["scale"]).float()}


def _plain_dlogits(s):
    l, ids, dg = s["logits"].float(), s["ids"].long(), s["dgates"]
    sc = _scores(l, s["score"])
    chosen = sc.gather(1, ids)
    ds = s["scale"] * dg
    if s["renorm"]:
        total = chosen.sum(1, keepdim=True)
        p = chosen / total
        ds = (ds - (ds * p).sum(1, keepdim=True)) / total
    dsc = torch.zeros_like(sc).scatter_(1, ids, ds)
    if s["score"] == "sigmoid":
        return dsc * sc * (1 - sc)
    return sc * (dsc - (dsc * sc).sum(1, keepdim=True))


def _plain_balance(s):
    ids = s["ids"].reshape(-1).long()
    load = torch.zeros_like(s["load"]).index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    s["load"].copy_(load)
    total = load.long().sum()
    s["bias"] += s["rate"] * torch.sign(total - load.long() * s["N"]).float()
    return {"load": s["load"], "bias": s["bias"]}


def _plain_router_backward(s):
    dl = _plain_dlogits(s)
    dx = torch.matmul(dl, s["w"].float())
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": torch.matmul(dl.t(), s["x"].float())}


def _plain_clip(s):
    # a sum over up to a thousand million squares, in 64 bits
    total = torch.stack([(t.float() * t.float()).sum(dtype=torch.float64) for t in s["grads"]]).sum()
    norm = torch.sqrt(total).float()
    coef = torch.clamp(s["max_norm"] / norm, max=1.0)
    out = [(t.float() * coef).to(t.dtype) for t in s["grads"]]
    return {"norm": norm, "grads": out}


def run(state):
    op = state["op"]
    if not own:
        return {"route": _plain_route, "route_backward": _plain_dlogits, "balance": _plain_balance,
                "router_backward": _plain_router_backward, "clip": _plain_clip}[op](state)
    from butterfly_rotated_ternary_amd import bmoe
    s = state
    if op == "route":
        spec = bmoe.RouteSpec(s["score"], renorm=s["renorm"], scale=s["scale"],
                              n_groups=s["groups"], topk_groups=s["keep"],
                              group_score=s["gscore"])
        ids, gates = bmoe.route_logits(s["logits"], s["k"], spec, bias=s["b"], ids=s["ids"],
                                       gates=s["gates"])
        return {"ids": ids, "gates": gates}
    if op == "balance":
        bmoe.route_balance(s["ids"], s["load"], bias=s["bias"], rate=s["rate"])
        return {"load": s["load"], "bias": s["bias"]}
    if op == "clip":
        norm = bmoe.clip_grads(s["grads"], s["max_norm"], out=s["out"])
        return {"norm": norm, "grads": s["out"]}
    spec = bmoe.RouteSpec(s["score"], renorm=s["renorm"], scale=s["scale"])
    if op == "route_backward":
        return bmoe.route_logits_backward(s["logits"], s["ids"], s["dgates"], spec,
                                          dlogits=s["dlogits"])
    return bmoe.router_backward(s["x"], s["w"], s["logits"], s["ids"], s["dgates"], spec,
                                dx_add=s["dx_add"], dx=s["dx"], dw=s["dw"])


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    op = case["op"]
    if op == "clip":
        d, N, L = case["d"], case["N"], case["d"].bit_length() - 1
        n32 = case["layers"] * (N * L * d + d * d)
        n16 = case["layers"] * case["extra"]
        if case["router"] == "f32":
            n32 += case["layers"] * N * d
        else:
            n16 += case["layers"] * N * d
        return {"bytes": 2 * (4 * n32 + 2 * n16), "flops": 3 * (n32 + n16)}
    T, N, k = case["T"], case["N"], case["k"]
    if op == "balance":
        return {"bytes": 4 * T * k + 12 * N, "flops": T * k}
    e = 2 if case["dt"] == "bf16" else 4
    if op == "route":
        return {"bytes": T * N * e + 4 * N * case["bias"] + 8 * T * k, "flops": 4 * T * N}
    dense = case["score"] == "softmax" and not case["renorm"]
    seen = T * (N if dense else k)   # logits the gradient depends on
    if op == "route_backward":
        return {"bytes": seen * e + 8 * T * k + 4 * T * N, "flops": 4 * seen}
    d = case["d"]
    return {"bytes": T * d * e * (3 if case["add"] else 2) + N * d * (e + 4) + 4 * seen + 8 * T * k,
            "flops": 4 * seen * d}


# ---- the operators' definitions in 64 bits -----------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        sq = sum(float(torch.linalg.vector_norm(t.double())) ** 2 for t in s["grads"])
        norm = math.sqrt(sq)
        f = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
        return {"norm": torch.tensor(norm, dtype=torch.float64, device="cuda"),
                "grads": [t.double() * f for t in s["grads"]]}
    if op == "balance":
        load = torch.bincount(s["ids"].flatten().long(), minlength=case["N"])
        mean = case["T"] * case["k"] / case["N"]
        step = (load < mean).double() - (load > mean).double()
        return {"load": None, "bias": s["bias"].double() + s["rate"] * step}
    l = s["logits"].double()
    if case["score"] == "sigmoid":
        prob = torch.sigmoid(l)
    else:
        prob = torch.exp(l - torch.logsumexp(l, 1, keepdim=True))
    rows = torch.arange(case["T"], device=l.device)
    if op == "route":
        left = prob.clone() if s["b"] is None else prob + s["b"].double()
        G, size = case["groups"], case["N"] // case["groups"]
        if G > 1:
            by = torch.topk(left.view(-1, G, size), 2 if case["gscore"] == "top2" else 1, dim=2)
            value = by.values.sum(2)
            rank = (value[:, None, :] > value[:, :, None]).sum(2)
            left[(rank >= case["keep"]).repeat_interleave(size, 1)] = -math.inf
        picked = []
        for _ in range(case["k"]):
            best = left.argmax(1)
            picked.append(prob[rows, best])
            left[rows, best] = -math.inf
        gates = torch.stack(picked, 1)
        if case["renorm"]:
            gates = gates / gates.sum(1, keepdim=True)
        return {"ids": None, "gates": gates * case["scale"]}
    # the gradient by torch's own differentiation of the definition, in 64 bits
    l = l.requires_grad_()
    prob = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    gates = prob.gather(1, s["ids"].long())
    if case["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    (dl,) = torch.autograd.grad((gates * case["scale"] * s["dgates"].double()).sum(), l)
    if op == "route_backward":
        return dl
    dx = dl @ s["w"].double()
    if s["dx_add"] is not None:
        dx += s["dx_add"].double()
    return {"dx": dx, "dw": dl.t() @ s["x"].double()}
