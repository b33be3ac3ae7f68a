"""Plain float64 CPU definitions of the block operators, with bounds of what the kernels'
arithmetic may differ by.

Bounds are first-order rounding analysis, in the order the kernels compute.  e = 2^-24 is half
a step of float32, U[dtype] half a step of the feature type.  A float32 sum of m products is
off by at most (m + 1) e times the sum of the absolute products (any order); the hardware exp,
reciprocal and square root are good to about 1 ulp, taken as K = 16 e with the operations
around them.  The slopes: |act'| <= 1.1, |act''| <= 0.5 for SiLU and the sigmoid.  A bf16
operand formed inside a kernel (hidden units, attention weights, their gradients) adds
U[bf16] of its own magnitude; every output adds U[its type] of itself."""
import math

import torch

E = 2.0 ** -24
K = 16 * E
UBF = torch.finfo(torch.bfloat16).eps / 2


def U(dtype):
    return torch.finfo(dtype).eps / 2


def ubf(dtype):
    """rounding of an operand formed inside a kernel"""
    return UBF if dtype == torch.bfloat16 else 0.0


def act(z, name):
    return {"none": lambda: z, "silu": lambda: z * torch.sigmoid(z), "sigmoid": lambda: torch.sigmoid(z)}[name]()


def dact(z, name):
    s = torch.sigmoid(z)
    return {"none": lambda: torch.ones_like(z), "silu": lambda: s * (1 + z * (1 - s)), "sigmoid": lambda: s * (1 - s)}[name]()


def d64(*ts):
    return [None if t is None else t.detach().cpu().double() for t in ts]


def linear(x, w, b, a, res, dy):
    """{name: (value, bound)} of linear and its gradients"""
    dt, k, o, n = x.dtype, x.shape[1], w.shape[0], x.shape[0]
    x, w, b, res, dy = d64(x, w, b, res, dy)
    z = x @ w.T + (b if b is not None else 0)
    az = x.abs() @ w.abs().T + (b.abs() if b is not None else 0)
    ez = (k + 2) * E * az
    y0 = act(z, a)
    ey = (1.1 * ez + K * (1 + z.abs()) * y0.abs()) if a != "none" else ez
    y = y0 + (res if res is not None else 0)
    out = {"y": (y, ey + U(dt) * y.abs() + E * (y.abs() + y0.abs()))}
    if dy is None:
        return out
    dz = dy * dact(z, a)
    edz = dy.abs() * (0.5 * ez + K * (1 + z.abs())) if a != "none" else torch.zeros_like(dz)
    edzr = edz + (ubf(dt) * dz.abs() if a != "none" else 0)
    dx, dw = dz @ w, dz.T @ x
    out["dx"] = (dx, edzr @ w.abs() + (o + 1) * E * (dz.abs() @ w.abs()) + U(dt) * dx.abs())
    out["dw"] = (dw, edzr.T @ x.abs() + (n + 520) * E * (dz.abs().T @ x.abs()) + U(dt) * dw.abs())
    db = dz.sum(0)
    out["db"] = (db, edz.sum(0) + (n + 520) * E * dz.abs().sum(0) + E * db.abs())
    return out


def ffn(x, wg, wu, wd, a, res, dy):
    dt, c, f, n = x.dtype, x.shape[1], wg.shape[0], x.shape[0]
    x, wg, wu, wd, res, dy = d64(x, wg, wu, wd, res, dy)
    zg, zu = x @ wg.T, x @ wu.T
    eg, eu = (c + 1) * E * (x.abs() @ wg.abs().T), (c + 1) * E * (x.abs() @ wu.abs().T)
    av = act(zg, a)
    ea = 1.1 * eg + K * (1 + zg.abs()) * av.abs()
    h = av * zu
    eh = zu.abs() * ea + av.abs() * eu + (E + ubf(dt)) * h.abs()
    y = h @ wd.T + (res if res is not None else 0)
    out = {"y": (y, eh @ wd.abs().T + (f + 2) * E * (h.abs() @ wd.abs().T + (res.abs() if res is not None else 0))
                 + U(dt) * y.abs())}
    if dy is None:
        return out
    dh = dy @ wd
    edh = (c + 1) * E * (dy.abs() @ wd.abs())
    da = dact(zg, a)
    dzu, dzg = dh * av, dh * zu * da
    ezu = edh * av.abs() + dh.abs() * ea + (2 * E + ubf(dt)) * dzu.abs()
    ezg = (edh * zu.abs() + dh.abs() * eu) * da.abs() + (dh * zu).abs() * (0.5 * eg + K * (1 + zg.abs()))
    ezg = ezg + (2 * E + ubf(dt)) * dzg.abs()
    dx = dzg @ wg + dzu @ wu
    out["dx"] = (dx, ezg @ wg.abs() + ezu @ wu.abs() + (2 * f + 1) * E * (dzg.abs() @ wg.abs() + dzu.abs() @ wu.abs())
                 + U(dt) * dx.abs())
    for name, l, el, r in (("dwg", dzg, ezg, x), ("dwu", dzu, ezu, x), ("dwd", dy, None, h)):
        v = l.T @ r
        e = (eh if el is None else el)
        b = (l.abs().T @ e) if el is None else (e.T @ r.abs())
        out[name] = (v, b + (n + 520) * E * (l.abs().T @ r.abs()) + U(dt) * v.abs())
    return out


def norm(x, b, scale, gate, w_post, w_pre, eps, dy, du):
    """(y, u) and the gradients; bounds carry the magnitudes A of each value's summands"""
    dt, c, n = x.dtype, x.shape[1], x.shape[0]
    x, b, scale, gate, w_post, w_pre, dy, du = d64(x, b, scale, gate, w_post, w_pre, dy, du)
    one = torch.ones(c, dtype=torch.float64)
    sc, wp = (scale if scale is not None else one), (w_post if w_post is not None else one)
    e = (c + 32) * E
    ib = (b.square().mean(1, keepdim=True) + eps).rsqrt() if w_post is not None else torch.ones(n, 1, dtype=torch.float64)
    bn = b * ib
    g = torch.sigmoid(gate) if gate is not None else torch.ones_like(b)
    t0 = sc * g * wp * bn
    y = x + t0
    ay = x.abs() + t0.abs()
    out = {"y": (y, U(dt) * y.abs() + 2 * e * ay)}
    if w_pre is not None:
        iy = (y.square().mean(1, keepdim=True) + eps).rsqrt()
        yn = y * iy
        # an error d of y moves y / rms by iy (d + yn mean(|yn d|)) <= iy (d + |yn| rms(d))
        ayn = iy * (ay + yn.abs() * ay.square().mean(1, keepdim=True).sqrt()) + yn.abs()
        u = w_pre * yn
        out["u"] = (u, U(dt) * u.abs() + 4 * e * w_pre.abs() * ayn)
    if dy is None and du is None:
        return out
    dyt = dy if dy is not None else torch.zeros_like(x)
    ad = dyt.abs()
    if du is not None:
        t = du * w_pre
        m = (t * yn).mean(1, keepdim=True)
        am = (t.abs() * ayn).mean(1, keepdim=True)
        dyt = dyt + iy * (t - yn * m)
        # rms(y) itself is off by the relative error of y: iy carries mean(ayn |yn|) more
        ad = ad + iy * (t.abs() + 2 * ayn * am) * (1 + (ayn * yn.abs()).mean(1, keepdim=True))
        v = (du * yn).sum(0)
        out["dw_pre"] = (v, (8 * e + (n + 1100) * E) * (du.abs() * ayn).sum(0) + E * v.abs())
    out["dx"] = (dyt, U(dt) * dyt.abs() + 8 * e * ad)
    if scale is not None:
        v = (dyt * g * wp * bn).sum(0)
        out["dscale"] = (v, (10 * e + (n + 1100) * E) * (ad * g * (wp * bn).abs()).sum(0) + E * v.abs())
    if gate is not None:
        v = dyt * sc * wp * bn * g * (1 - g)
        # 1 - g loses its leading digits where the gate is open: K absolute
        out["dgate"] = (v, U(dt) * v.abs() + (ad * (sc * wp * bn).abs() * g) * (12 * e + K))
    t = dyt * sc * g
    at = ad * sc.abs() * g
    if w_post is not None:
        v = (t * bn).sum(0)
        out["dw_post"] = (v, (10 * e + (n + 1100) * E) * (at * bn.abs()).sum(0) + E * v.abs())
        t, at = t * wp, at * wp.abs()
        m, am = (t * bn).mean(1, keepdim=True), (at * bn.abs()).mean(1, keepdim=True)
        t, at = ib * (t - bn * m), ib * (at + 2 * bn.abs() * am)
    out["db"] = (t, U(dt) * t.abs() + 14 * e * at)
    return out


def attention(q, k, v, sptr, heads, pos=None, slope=None, L=0.0, mask=None, cap=0.0, dout=None, save=False):
    """Rows past the last structure are NaN in value and bound."""
    dt = q.dtype
    n, c = q.shape
    d = c // heads
    q, k, v, pos, slope, dout = d64(q, k, v, pos, slope, dout)
    on_all = torch.ones(n, dtype=torch.bool) if mask is None else mask.cpu() != 0
    names = ["out"] + (["dq", "dk", "dv"] if dout is not None else [])
    out = {m: [torch.full((n, c), math.nan, dtype=torch.float64) for _ in range(2)] for m in names}
    if dout is not None and pos is not None:
        out["dpos"] = [torch.full((n, 3), math.nan, dtype=torch.float64) for _ in range(2)]
        out["dslope"] = [torch.zeros(heads, dtype=torch.float64) for _ in range(2)]
    sp = sptr.cpu().tolist()
    split = save and dt == torch.bfloat16      # weights enter with twice the bits
    for s, e in zip(sp[:-1], sp[1:]):
        if e == s:
            continue
        m = e - s
        on = on_all[s:e]
        hd = lambda t: t[s:e].view(m, heads, d).transpose(0, 1)  # noqa: E731
        kk, vv = k[s:e].clone(), v[s:e].clone()
        kk[~on], vv[~on] = 0, 0                 # masked keys: whatever they hold
        Q = hd(q)
        Kh, V = kk.view(m, heads, d).transpose(0, 1), vv.view(m, heads, d).transpose(0, 1)
        sc = d ** -0.5
        t = Q @ Kh.transpose(1, 2) * sc
        et = (d + 4) * E * (Q.abs() @ Kh.abs().transpose(1, 2)) * sc
        th = torch.zeros_like(t)
        if cap:
            th = torch.tanh(t / cap)
            t = cap * th
            et = et * (1 - th * th) + cap * th.abs() * (K + (1.2e-5 if dt == torch.bfloat16 and not save else 0)) + E * t.abs()
        if pos is not None:
            p = pos[s:e].clone()
            delta = p[None] - p[:, None]        # x_j - x_i
            if L:
                delta = delta - L * torch.round(delta / L)
            r = delta.square().sum(2).sqrt()
            r = torch.where(on[None, :], r, torch.zeros_like(r))
            t = t - slope[:, None, None] * r
            # the difference of two coordinates: one rounding, or 2^-32 of the box
            er = 6 * E * r + (3 * L * 2.0 ** -32 if L else 0)
            et = et + slope.abs()[:, None, None] * er
        et = et + 3 * E * t.abs()
        t = t.masked_fill(~on[None, None], -math.inf)
        et = et.masked_fill(~on[None, None], 0.0)
        mx = t.amax(2, keepdim=True)
        mx = torch.where(mx == -math.inf, torch.zeros_like(mx), mx)
        et = et + 3 * E * ((t - mx).masked_fill(~on[None, None], 0).abs() + mx.abs())
        a = torch.exp(t - mx)
        z = a.sum(2, keepdim=True)
        a = torch.where(z > 0, a / z.clamp(min=1e-300), torch.zeros_like(a))
        # relative error of a weight: its own exponent, and the sum's
        ra = et + (a * et).sum(2, keepdim=True) + (m + 16) * E + K
        o = a @ V
        eo = (a * (ra + (m + 2) * E + (2.0 ** -18 if split else ubf(dt)))) @ V.abs()
        cat = lambda x: x.transpose(0, 1).reshape(m, c)  # noqa: E731
        out["out"][0][s:e], out["out"][1][s:e] = cat(o), cat(eo + U(dt) * o.abs())
        if dout is None:
            continue
        dO = hd(dout)
        dv = a.transpose(1, 2) @ dO
        edv = (a * (ra + ubf(dt) + (m + 2) * E)).transpose(1, 2) @ dO.abs()
        dp = dO @ V.transpose(1, 2)
        edp = (d + 1) * E * (dO.abs() @ V.abs().transpose(1, 2))
        D = (dO * o).sum(2, keepdim=True)
        eD = (dO.abs() * (eo + (d + 2) * E * o.abs())).sum(2, keepdim=True)
        dl = a * (dp - D)
        edl = a * ((ra + 2 * E) * (dp - D).abs() + edp + eD + E * (dp.abs() + D.abs()))
        f = 1 - th * th
        ds = dl * f
        eds = edl * f + dl.abs() * (2 * th.abs() * (et / cap if cap else 0) + (K if cap else 0)) + ubf(dt) * ds.abs()
        dq, dk = ds @ Kh * sc, ds.transpose(1, 2) @ Q * sc
        eq = (eds + (m + 3) * E * ds.abs()) @ Kh.abs() * sc
        ek = (eds + (m + 3) * E * ds.abs()).transpose(1, 2) @ Q.abs() * sc
        dk[:, ~on], dv[:, ~on] = 0, 0
        for name, val, er_ in (("dq", dq, eq), ("dk", dk, ek), ("dv", dv, edv)):
            out[name][0][s:e], out[name][1][s:e] = cat(val), cat(er_ + U(dt) * val.abs())
        if pos is not None:
            w = (slope[:, None, None] * dl).sum(0)
            ew = (slope.abs()[:, None, None] * (edl + (heads + 8) * E * dl.abs())).sum(0)
            u = torch.where(r[..., None] > 0, delta / r.clamp(min=1e-300)[..., None], torch.zeros_like(delta))
            u = torch.where(on[None, :, None], u, torch.zeros_like(u))
            eu = torch.where(r > 0, 3 * L * 2.0 ** -32 / r.clamp(min=1e-300) + 12 * E, torch.zeros_like(r))
            dpos = (w[..., None] * u).sum(1) - (w[..., None] * u).sum(0)
            ep = (ew[..., None] * u.abs() + (w.abs() * (eu + 2 * (m + 8) * E))[..., None])
            out["dpos"][0][s:e], out["dpos"][1][s:e] = dpos, ep.sum(1) + ep.sum(0) + E * dpos.abs()
            out["dslope"][0] -= (dl * r).sum((1, 2))
            nn = max(n, 1) + 64
            out["dslope"][1] += ((edl + nn * E * dl.abs()) * r + dl.abs() * er).sum((1, 2))
    return {key: (val[0], val[1]) for key, val in out.items()}


def check(name, got, ref, bound):
    """got within bound of ref, everywhere; returns the largest error as a share of its bound"""
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert bool(torch.isfinite(got).all()), f"{name}: non-finite"
    err = (got - ref).abs()
    tiny = 1e-37
    share = float((err / (bound + tiny)).max()) if err.numel() else 0.0
    scale = float(ref.abs().max()) if ref.numel() else 0.0
    print(f"  {name}: max err {float(err.max()) if err.numel() else 0:.2e} of {scale:.2e}, {share:.3f} of its bound",
          flush=True)
    assert share <= 1.0, f"{name}: error {share:.3f} times its bound"
    return share
