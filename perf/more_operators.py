"""Operators around an expert block, as measured cases: dense experts, the norms
around the block, the orthogonalised update of its weights.

Each as the plain torch form and as the library's calls:

``product``           ids -> rows grouped by expert -> the experts' products, ragged groups
``product_backward``  gradients of the rows and of the experts' weights
``norm``              gate-weighted sum of a token's expert rows, post-norm, scaled residual, pre-norm
``norm_backward``     gradients of all of its inputs
``orthogonalize``     Newton-Schulz orthogonalisation of a gradient, or of one tensor's whole update step

Inputs follow the package's synthetic workloads: unit-variance activations,
weights of variance 1/K, ids uniform or skewed towards low experts.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_NS = (3.4445, -4.7750, 2.0315)   # quintic whose fifth iterate takes (0, 1] near 1
_EPS = 1e-6                       # of the norms
_NS_EPS = 1e-7


# ---- cases -----------------------------------------------------------------

def listed():
    return [
        # decoding one token: eight experts' weights are read for one row each
        dict(name="product one token", op="product", T=1, k=8, N=256, K=2048, O=1408, dt="bf16",
             skew=0.7),
        # a ragged batch of odd widths in fp32
        dict(name="product ragged", op="product", T=1003, k=3, N=60, K=100, O=203, dt="f32",
             skew=1.1),
        # the largest workload's tokens and experts, each a narrow projection of d = 4096
        dict(name="product large", op="product", T=32768, k=4, N=256, K=4096, O=1024, dt="bf16",
             skew=0.0),
        # the headline batch
        dict(name="product_backward batch", op="product_backward", T=4096, k=2, N=64, K=512,
             O=1024, dt="bf16", skew=0.0),
        # d = 2048, 64 experts, a skewed router
        dict(name="product_backward large", op="product_backward", T=16384, k=2, N=64, K=2048,
             O=2048, dt="bf16", skew=0.4),
        # one token through the tail of a block
        dict(name="norm one token", op="norm", T=1, d=4096, k=8, dt="bf16", routed=True,
             gates=True, post=True, pre=True),
        # the largest workload
        dict(name="norm large", op="norm", T=32768, d=4096, k=4, dt="bf16", routed=True,
             gates=True, post=True, pre=True),
        # the headline batch behind the butterfly layer (its gates are already in u), fp32
        dict(name="norm_backward batch", op="norm_backward", T=4096, d=512, k=1, dt="f32",
             routed=False, gates=False, post=True, pre=True),
        # d = 2048, two picks a token
        dict(name="norm_backward large", op="norm_backward", T=16384, d=2048, k=2, dt="bf16",
             routed=True, gates=True, post=True, pre=True),
        # the headline router's gradient
        dict(name="orthogonalize router", op="orthogonalize", B=1, rows=64, cols=512, dt="f32",
             step=False),
        # the headline experts' weights, tall matrices
        dict(name="orthogonalize experts", op="orthogonalize", B=64, rows=1024, cols=512,
             dt="bf16", step=False),
        # the substrate's latent weights at d = 4096: momentum, orthogonalisation, update
        dict(name="orthogonalize substrate step", op="orthogonalize", B=1, rows=4096, cols=4096,
             dt="f32", step=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row length: mostly whole 16-byte pieces, now and then any number."""
    if rng.random() < 0.2:
        return _log(rng, lo, min(hi, 500))
    return 8 * _log(rng, max(1, lo // 8), hi // 8)


def draw(rng):
    op = rng.choice(["product", "product_backward", "norm", "norm_backward", "orthogonalize"])
    if op == "orthogonalize":
        dt = rng.choice(["f32", "bf16"])
        rows, cols = _width(rng, 8, 4096), _width(rng, 8, 4096)
        m, n = min(rows, cols), max(rows, cols)
        most = min((1 << 36) // (m * m * n), (1 << 25) // (m * n), 64)
        return dict(op=op, B=_log(rng, 1, max(1, most)), rows=rows, cols=cols, dt=dt,
                    step=rng.random() < 0.4)
    if op in ("norm", "norm_backward"):
        d, k = _width(rng, 16, 8192), rng.choice([1, 1, 2, 4, 8])
        most = min(32768, (1 << 29) // (d * k), (1 << 27) // d)
        if op == "norm_backward":
            most = min(most, (1 << 26) // (d * k) + 1)
        post = rng.random() < 0.7
        return dict(op=op, T=_log(rng, 1, most), d=d, k=k, dt=rng.choice(["bf16", "bf16", "f32"]),
                    routed=k > 1 and rng.random() < 0.7, gates=k > 1 and rng.random() < 0.7,
                    post=post, pre=not post or rng.random() < 0.8)
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    N = _log(rng, 4, 256)
    K, O = _width(rng, 32, 4096), _width(rng, 32, 4096)
    while N * K * O > (1 << 29 if op == "product_backward" else 1 << 30):
        N = max(1, N // 2)
    k = rng.randint(1, min(8, N))
    work = (1 << 35) if dt == "f32" else (1 << 37) if op == "product_backward" else (1 << 39)
    most = min(32768, work // (K * O * k), (1 << 28) // (k * max(K, O)))
    return dict(op=op, T=_log(rng, 1, max(1, most)), k=k, N=N, K=K, O=O, dt=dt,
                skew=rng.choice([0.0, 0.4, 1.1]))


# ---- inputs ----------------------------------------------------------------

def _ids(g, T, N, k, skew):
    """k distinct experts a token, low ids more often with `skew`."""
    u = torch.rand(T, N, generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    keys = -torch.log(-torch.log(u)) - skew * torch.log1p(torch.arange(N, device="cuda").float())
    return torch.topk(keys, k, dim=1).indices.to(torch.int32)


def _tables(ids, N):
    """offsets, perm and inv of the rows grouped by expert, in order within one."""
    e, order = torch.sort(ids.reshape(-1).long(), stable=True)
    offsets = torch.zeros(N + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.cumsum(torch.bincount(e, minlength=N), 0)
    inv = torch.empty_like(order)
    inv[order] = torch.arange(order.numel(), device=ids.device)
    return offsets.to(torch.int32), order.to(torch.int32), inv.to(torch.int32)


def _randn(g, shape, dt, scale=1.0):
    """Normal values, drawn a slice at a time so that no fp32 copy of all is held."""
    out = torch.empty(shape, dtype=dt, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(scale).to(dt)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, dt = case["op"], _DT[case["dt"]]
    s = dict(case)
    if op == "orthogonalize":
        B, m, n = case["B"], case["rows"], case["cols"]
        grad = _randn(g, (B, m, n), torch.float32 if case["step"] else dt, 0.01)
        s.update(u=grad, out=torch.empty_like(grad))
        if case["step"]:
            s.update(w=_randn(g, (B, m, n), dt, 1 / math.sqrt(n)),
                     momentum=_randn(g, (B, m, n), torch.float32, 0.03),
                     lr=0.02, beta=0.95, decay=0.1, scale=math.sqrt(max(1.0, m / n)))
        return s
    if op in ("norm", "norm_backward"):
        T, d, k = case["T"], case["d"], case["k"]
        M = T * k
        s.update(u=_randn(g, (M, d), dt), res_scale=0.8, out_scale=1.25, inv=None, g=None,
                 w_post=1 + _randn(g, (d,), torch.float32, 0.1) if case["post"] else None,
                 w_pre=1 + _randn(g, (d,), torch.float32, 0.1) if case["pre"] else None)
        if case["routed"]:
            s["inv"] = _tables(_ids(g, T, 64, k, 0.0), 64)[2]
        if case["gates"]:
            s["g"] = torch.softmax(torch.randn(T, k, generator=g, device="cuda"), 1)
        if op == "norm":
            s.update(r=_randn(g, (T, d), dt, 2.0), r_out=torch.empty(T, d, dtype=dt, device="cuda"),
                     n=torch.empty(T, d, dtype=dt, device="cuda") if case["pre"] else None)
        else:
            s.update(r_out=_randn(g, (T, d), dt, 2.0), dr_out=_randn(g, (T, d), dt),
                     dn=_randn(g, (T, d), dt) if case["pre"] else None)
        return s
    T, k, N, K, O = (case[c] for c in ("T", "k", "N", "K", "O"))
    ids = _ids(g, T, N, k, case["skew"])
    s.update(a=_randn(g, (T, K), dt), w=_randn(g, (N, O, K), dt, 1 / math.sqrt(K)), ids=ids)
    if op == "product_backward":
        s["offsets"], s["perm"], _ = _tables(ids, N)
        s.update(dc=_randn(g, (T * k, O), dt), da=torch.empty(T * k, K, dtype=dt, device="cuda"),
                 dw=torch.empty(N, O, K, device="cuda"))
    return s


# ---- the plain forms -------------------------------------------------------

def _plain_product(s):
    offsets, perm, inv = _tables(s["ids"], s["N"])
    rows = perm.long() // s["k"]
    off = offsets.tolist()
    c = torch.empty(rows.numel(), s["O"], dtype=s["a"].dtype, device="cuda")
    for e in range(s["N"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            c[lo:hi] = torch.matmul(s["a"][rows[lo:hi]].float(), s["w"][e].float().t()).to(c.dtype)
    return {"offsets": offsets, "perm": perm, "inv": inv, "c": c}


def _plain_product_backward(s):
    rows = s["perm"].long() // s["k"]
    off = s["offsets"].tolist()
    da, dw = s["da"], s["dw"]
    for e in range(s["N"]):
        lo, hi = off[e], off[e + 1]
        dc = s["dc"][lo:hi].float()
        da[lo:hi] = torch.matmul(dc, s["w"][e].float()).to(da.dtype)
        dw[e] = torch.matmul(dc.t(), s["a"][rows[lo:hi]].float())
    return {"da": da, "dw": dw}


def _gathered(s):
    """u by token, [T][k][d] fp32."""
    u = s["u"] if s["inv"] is None else s["u"][s["inv"].long()]
    return u.float().view(s["T"], s["k"], s["d"])


def _rstd(v):
    return 1 / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + _EPS)


def _plain_norm(s):
    u = _gathered(s)
    z = u.sum(1) if s["g"] is None else (s["g"][:, :, None] * u).sum(1)
    if s["w_post"] is not None:
        z = z * _rstd(z) * s["w_post"]
    r = s["res_scale"] * s["r"].float() + s["out_scale"] * z
    out = {"r": r.to(s["r"].dtype)}
    if s["w_pre"] is not None:
        out["n"] = (r * _rstd(r) * s["w_pre"]).to(s["r"].dtype)
    return out


def _norm_grad(v, w, dout):
    """Gradients of v * rstd(v) * w with respect to v and w."""
    q = _rstd(v)
    h = v * q
    t = w * dout
    return q * (t - h * (t * h).sum(1, keepdim=True) / v.shape[1]), (dout * h).sum(0)


def _plain_norm_backward(s):
    dt = s["u"].dtype
    dr = s["dr_out"].float()
    out = {}
    if s["w_pre"] is not None:
        dv, out["dw_pre"] = _norm_grad(s["r_out"].float(), s["w_pre"], s["dn"].float())
        dr = dr + dv
    out["dr"] = (s["res_scale"] * dr).to(dt)
    u = _gathered(s)
    y = u.sum(1) if s["g"] is None else (s["g"][:, :, None] * u).sum(1)
    dy = s["out_scale"] * dr
    if s["w_post"] is not None:
        dy, out["dw_post"] = _norm_grad(y, s["w_post"], dy)
    if s["g"] is None:
        du = dy[:, None, :].expand(u.shape)
    else:
        du = s["g"][:, :, None] * dy[:, None, :]
        out["dgates"] = (u * dy[:, None, :]).sum(2)
    du = du.reshape(-1, s["d"])
    if s["inv"] is not None:
        du = torch.empty_like(du).index_copy_(0, s["inv"].long(), du)
    out["du"] = du.to(dt)
    return out


def _plain_newton_schulz(u):
    """u fp32 [B][rows][cols] -> the fifth iterate."""
    norm = torch.sqrt((u.double() * u.double()).sum((1, 2), keepdim=True)).float()
    x = u / (norm + _NS_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, c = _NS
    for _ in range(5):
        p = torch.matmul(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return x.transpose(1, 2).contiguous() if tall else x


def _plain_orthogonalize(s):
    if not s["step"]:
        return {"o": _plain_newton_schulz(s["u"].float()).to(s["u"].dtype)}
    m = s["momentum"].mul_(s["beta"]).add_(s["u"])
    o = _plain_newton_schulz(s["u"] + s["beta"] * m)
    w = (1 - s["lr"] * s["decay"]) * s["w"].float() - s["lr"] * s["scale"] * o
    s["w"].copy_(w.to(s["w"].dtype))
    return {"w": s["w"], "momentum": m}


def run(state):
    op, s = state["op"], state
    if not own:
        return {"product": _plain_product, "product_backward": _plain_product_backward,
                "norm": _plain_norm, "norm_backward": _plain_norm_backward,
                "orthogonalize": _plain_orthogonalize}[op](s)
    from butterfly_rotated_ternary_amd import bmoe
    if op == "product":
        offsets, perm, inv = bmoe.group_rows(s["ids"], s["N"])
        c = bmoe.grouped_product(s["a"], s["w"], offsets, perm=perm, k=s["k"])
        return {"offsets": offsets, "perm": perm, "inv": inv, "c": c}
    if op == "product_backward":
        return bmoe.grouped_product_backward(s["a"], s["w"], s["offsets"], s["dc"],
                                             perm=s["perm"], k=s["k"], da=s["da"], dw=s["dw"])
    if op == "orthogonalize":
        spec = bmoe.OrthoSpec(5, _NS, eps=_NS_EPS)
        if not s["step"]:
            return {"o": bmoe.orthogonalize(s["u"], spec, out=s["out"])}
        bmoe.orthogonal_step(s["w"], s["u"], s["momentum"], s["lr"], spec, beta=s["beta"],
                             nesterov=True, weight_decay=s["decay"], scale=s["scale"])
        return {"w": s["w"], "momentum": s["momentum"]}
    spec = bmoe.NormSpec(eps=_EPS, res_scale=s["res_scale"], out_scale=s["out_scale"])
    if op == "norm":
        r, n = bmoe.residual_norm(s["u"], s["r"], spec, k=s["k"], inv=s["inv"], gates=s["g"],
                                  w_post=s["w_post"], w_pre=s["w_pre"], r_out=s["r_out"], n=s["n"])
        return {"r": r} if n is None else {"r": r, "n": n}
    out = bmoe.residual_norm_backward(s["u"], s["r_out"], spec, k=s["k"], inv=s["inv"],
                                      gates=s["g"], w_post=s["w_post"], w_pre=s["w_pre"],
                                      dr_out=s["dr_out"], dn=s["dn"])
    return {key: v for key, v in out.items() if v is not None}


# ---- what a pass cannot do without -----------------------------------------

def work(case):
    op = case["op"]
    e = 2 if case["dt"] == "bf16" else 4
    if op == "orthogonalize":
        B, m, n = case["B"], min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        # the two square products are symmetric: half of each is enough
        flops = 5 * B * (m * (m + 1) * n + m * m * (m + 1) + 2 * m * m * n)
        return {"bytes": B * m * n * (12 + 2 * e if case["step"] else 2 * e), "flops": flops}
    if op in ("norm", "norm_backward"):
        T, d, k = case["T"], case["d"], case["k"]
        small = 4 * T * k * (case["routed"] + case["gates"]) + 4 * d * (case["post"] + case["pre"])
        if op == "norm":
            return {"bytes": T * d * e * (k + 2 + case["pre"]) + small, "flops": T * d * (2 * k + 10)}
        return {"bytes": T * d * e * (2 * k + 3 + case["pre"]) + 2 * small,
                "flops": T * d * (4 * k + 20)}
    T, k, N, K, O = (case[c] for c in ("T", "k", "N", "K", "O"))
    M = T * k
    used = N * (1 - (1 - k / N) ** T)     # experts with rows, ids drawn uniformly
    if op == "product":
        return {"bytes": int(e * (T * K + M * O + used * K * O)) + 12 * M + 4 * N,
                "flops": 2 * M * K * O}
    return {"bytes": int(e * (T * K + M * O + M * K + used * K * O)) + 4 * N * K * O + 4 * M,
            "flops": 4 * M * K * O}


# ---- the operators' definitions in 64 bits -----------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "orthogonalize":
        if case["step"]:
            m = s["beta"] * s["momentum"].double() + s["u"].double()
            u = s["u"].double() + s["beta"] * m
        else:
            u = s["u"].double()
        x = u / (u.flatten(1).norm(dim=1)[:, None, None] + _NS_EPS)
        a, b, c = _NS
        wide = x.shape[2] >= x.shape[1]
        eye = torch.eye(min(x.shape[1:]), dtype=torch.float64, device="cuda")
        for _ in range(5):
            xt = x.mT.contiguous()
            p = x @ xt if wide else xt @ x
            q = (c * p + b * eye) @ p + a * eye
            x = q @ x if wide else x @ q
        if not case["step"]:
            return {"o": x}
        keep = 1 - s["lr"] * s["decay"]
        return {"w": keep * s["w"].double() - s["lr"] * s["scale"] * x, "momentum": m}
    if op in ("norm", "norm_backward"):
        T, d, k = case["T"], case["d"], case["k"]
        back = op == "norm_backward"
        u = s["u"].double().requires_grad_(back)
        g = None if s["g"] is None else s["g"].double().requires_grad_(back)
        ws = {key: None if s[key] is None else s[key].double().requires_grad_(back)
              for key in ("w_post", "w_pre")}
        rows = u if s["inv"] is None else u.index_select(0, s["inv"].long())
        rows = rows.view(T, k, d)
        y = rows.sum(1) if g is None else torch.einsum("tk,tkd->td", g, rows)

        def rms(v, w):
            return w * v / torch.sqrt(v.square().mean(1, keepdim=True) + _EPS)
        z = y if ws["w_post"] is None else rms(y, ws["w_post"])
        if not back:
            r = s["res_scale"] * s["r"].double() + s["out_scale"] * z
            return {"r": r} if ws["w_pre"] is None else {"r": r, "n": rms(r, ws["w_pre"])}
        # differentiated by torch in two parts, joined at the residual stream
        dr = s["dr_out"].double()
        out = {}
        if ws["w_pre"] is not None:
            r = s["r_out"].double().requires_grad_()
            dv, out["dw_pre"] = torch.autograd.grad(rms(r, ws["w_pre"]), (r, ws["w_pre"]),
                                                    s["dn"].double())
            dr = dr + dv
        out["dr"] = s["res_scale"] * dr
        names = ["du"] + ["dgates"] * (g is not None) + ["dw_post"] * (ws["w_post"] is not None)
        leaves = [u] + [t for t in (g, ws["w_post"]) if t is not None]
        out.update(zip(names, torch.autograd.grad(z, leaves, s["out_scale"] * dr)))
        return {key: out[key] for key in ("dw_pre", "dr", "dw_post", "dgates", "du") if key in out}
    T, k, N = case["T"], case["k"], case["N"]
    ids = s["ids"].reshape(-1).long()
    token = torch.arange(T, device="cuda").repeat_interleave(k)
    if op == "product":
        c = [s["a"].double()[token[ids == e]] @ s["w"][e].double().t() for e in range(N)]
        return {"offsets": None, "perm": None, "inv": None, "c": torch.cat(c)}
    a = s["a"].double()
    da, dw, done = [], [], 0
    for e in range(N):
        at = token[ids == e]
        dc = s["dc"][done:done + at.numel()].double()
        done += at.numel()
        da.append(dc @ s["w"][e].double())
        dw.append(dc.t() @ a[at])
    return {"da": torch.cat(da), "dw": torch.stack(dw)}
