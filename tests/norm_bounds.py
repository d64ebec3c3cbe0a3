"""residual_norm() and its gradient in 64 bits, with how far each entry of a float32
implementation may be off: every operation's rounding carried on to first order.

u = 2^-24 is a rounding's relative error. A sum over the d values of a row is at most
16 terms one by one in a thread, six steps across a wave and 16 waves: 38 roundings,
40 allowed (SUM) of the sum of the terms' magnitudes. A sum over tokens is a chain in
each of at least 384 workgroups (or one of a token), up to 16 rows of a workgroup, then
64 bits. So the bounds grow with a row's values, not with their count, and a wrong
formula, a missing term or a lost part of a sum lies far outside of them."""
import numpy as np
import torch

U = 2.0 ** -24
SUM = 40
BF, F32 = torch.bfloat16, torch.float32
SCALES = dict(eps=1e-6, res_scale=0.75, out_scale=1.25)


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def half(dt):
    return 2.0 ** -8 if dt == BF else 2.0 ** -24


def draw(T, d, k, dt, seed, routed=True, gates=True, post=True, pre=True, pad=0.0):
    g = torch.Generator().manual_seed(seed)
    s = dict(T=T, d=d, k=k, dt=dt, inv=None, gates=None, w_post=None, w_pre=None, dn=None,
             u=torch.randn(T * k, d, generator=g).to(dt),
             r=(2 * torch.randn(T, d, generator=g)).to(dt),
             dr_out=torch.randn(T, d, generator=g).to(dt))
    if routed:
        s["inv"] = torch.randperm(T * k, generator=g).int()
        if pad:
            s["inv"][torch.rand(T * k, generator=g) < pad] = -1
    if gates:
        s["gates"] = torch.softmax(torch.randn(T, k, generator=g), 1)
    if post:
        s["w_post"] = 1 + 0.1 * torch.randn(d, generator=g)
    if pre:
        s["w_pre"] = 1 + 0.1 * torch.randn(d, generator=g)
        s["dn"] = torch.randn(T, d, generator=g).to(dt)
    return s


def mean(x):
    return np.mean(x, axis=1, keepdims=True)


def _picks(s):
    """u's rows by token [T][k][d], the gates, and which picks there are."""
    T, k = s["T"], s["k"]
    at = np.arange(T * k) if s["inv"] is None else f64(s["inv"]).astype(np.int64)
    ok = (at >= 0) & (at < len(s["u"]))
    rows = np.where(ok[:, None], f64(s["u"])[np.where(ok, at, 0)], 0.0).reshape(T, k, -1)
    g = np.ones((T, k)) if s["gates"] is None else f64(s["gates"])
    return rows, np.where(ok.reshape(T, k), g, 0.0), ok.reshape(T, k), at.reshape(T, k)


def _rstd(v, ev):
    """1 / sqrt(mean v^2 + eps) and its relative error; v off by at most ev."""
    ms = mean(v * v) + SCALES["eps"]
    off = mean(SUM * U * v * v + 2 * np.abs(v) * ev) / ms
    return 1 / np.sqrt(ms), 0.5 * off + 6 * U


def _norm(v, ev, w):
    q, rho = _rstd(v, ev)
    out = v * q * w
    return out, np.abs(q * w) * ev + np.abs(out) * (rho + 2 * U)


def _summed(s):
    rows, g, _, _ = _picks(s)
    y = np.einsum("tk,tkd->td", g, rows)
    return y, s["k"] * U * np.einsum("tk,tkd->td", np.abs(g), np.abs(rows))


def forward(s):
    """{name: (value, tolerance)} of r and n."""
    z, ez = _summed(s)
    if s["w_post"] is not None:
        z, ez = _norm(z, ez, f64(s["w_post"]))
    a = SCALES["res_scale"] * f64(s["r"])
    r = a + SCALES["out_scale"] * z
    er = SCALES["out_scale"] * ez + U * (np.abs(a) + np.abs(r))
    h = half(s["dt"])
    out = {"r": (r, er + h * (np.abs(r) + er))}
    if s["w_pre"] is not None:
        n, en = _norm(r, er, f64(s["w_pre"]))
        out["n"] = (n, en + h * (np.abs(n) + en))
    return out


def _norm_back(v, ev, w, d, ed, wrong):
    """Gradient of v / rms(v) * w to v from d, and to w, with their errors."""
    q, rho = _rstd(v, ev)
    t, et = w * d, np.abs(w) * ed + U * np.abs(w * d)
    cols = slice(0, v.shape[1] * 7 // 8) if wrong == "part of a row's sum" else slice(None)
    m = np.sum((t * v)[:, cols], axis=1, keepdims=True) / v.shape[1]
    em = (SUM + 3) * U * mean(np.abs(t * v)) + mean(np.abs(v) * et + np.abs(t) * ev)
    em = em * q ** 2 + np.abs(m) * q ** 2 * (2 * rho + 4 * U)
    m = m * q ** 2 * (0.0 if wrong == "no projection" else 1.0)
    inner = t - v * m
    ein = et + np.abs(v) * em + np.abs(m) * ev + 2 * U * (np.abs(t) + np.abs(v * m))
    dv = q * inner
    edv = q * ein + np.abs(dv) * (rho + U)
    term = d * v * q
    eterm = np.abs(v * q) * ed + np.abs(d * q) * ev + np.abs(term) * (rho + 2 * U)
    chain = -(-len(v) // 384) + 19
    dw = term.sum(0)
    return dv, edv, dw, eterm.sum(0) + chain * U * np.abs(term).sum(0) + U * np.abs(dw)


def backward(s, wrong=None):
    """{name: (value, tolerance)} of the gradients at r' = r; du only for named rows (a
    mask beside it). wrong: one of WRONG, a mistake made on purpose."""
    h, k = half(s["dt"]), s["k"]
    dr, edr = f64(s["dr_out"]), np.zeros((s["T"], s["d"]))
    out = {}

    def stored(v, e):
        return v, e + h * (np.abs(v) + e) + U * np.abs(v)
    if s["w_pre"] is not None:
        x = f64(s["r"])
        pre = None if wrong == "no projection behind the block" else wrong
        pre = "no projection" if wrong == "no projection before the next" else pre
        dv, edv, dw, edw = _norm_back(x, np.zeros_like(x), f64(s["w_pre"]), f64(s["dn"]),
                                      np.zeros_like(x), pre)
        out["dw_pre"] = dw * (0.99 if wrong == "dw_pre scaled" else 1.0), edw
        dr = dr + dv
        edr = edv + U * np.abs(dr)
    out["dr"] = stored(SCALES["res_scale"] * dr, SCALES["res_scale"] * edr)
    dz, edz = SCALES["out_scale"] * dr, SCALES["out_scale"] * edr
    edz = edz + U * np.abs(dz)
    rows, g, ok, at = _picks(s)
    y, ey = _summed(s)
    if wrong == "a pick missing":
        y = y - g[:, k - 1:] * rows[:, k - 1]
    if s["w_post"] is not None:
        post = "no projection" if wrong == "no projection behind the block" else wrong
        dz, edz, dw, edw = _norm_back(y, ey, f64(s["w_post"]), dz, edz, post)
        out["dw_post"] = dw * (1.01 if wrong == "dw_post scaled" else 1.0), edw
    du, edu, named = np.zeros((T_rows(s), s["d"])), np.zeros((T_rows(s), s["d"])), np.zeros(T_rows(s), bool)
    for j in range(k):
        here = ok[:, j]
        to = at[here, j]
        du[to] = (g[:, j:j + 1] * dz)[here]
        edu[to] = (np.abs(g[:, j:j + 1]) * edz)[here]
        named[to] = True
    out["du"] = stored(du, edu)
    if s["gates"] is not None:
        dg = np.einsum("td,tkd->tk", dz, rows)
        edg = np.einsum("td,tkd->tk", edz + SUM * U * np.abs(dz), np.abs(rows))
        if wrong == "no dgates":
            dg = 0 * dg
        if wrong == "dgates of the other sign":
            dg = -dg
        if wrong == "dgates of the first two picks only":
            dg[:, 2:] = 0.0
        out["dgates"] = dg, edg + U * np.abs(dg)
    return out, named


def T_rows(s):
    return len(s["u"])


WRONG = ["no dgates", "dgates of the other sign", "dgates of the first two picks only",
         "no projection behind the block", "no projection before the next", "part of a row's sum",
         "a pick missing", "dw_post scaled", "dw_pre scaled"]


def rounded(v, name, dt):
    """A value as the library stores it."""
    t = torch.from_numpy(np.asarray(v))
    return (t if name in ("dgates", "dw_pre", "dw_post") else t.to(dt)).double().numpy()


def outside(got, want):
    """How often the tolerance the worst entry is off, by output; only those past it."""
    bad = {}
    for name, (ref, tol) in want.items():
        over = np.abs(got[name] - ref) / np.maximum(tol, 1e-300)
        if not (over <= 1).all():
            bad[name] = float(np.nanmax(over))
    return bad
