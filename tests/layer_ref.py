"""Plain 64-bit forms of the layer operators (convolution, selective scan, norms) on the
CPU, written from their definitions, and the error bounds of the kernels.

Every form can be evaluated on magnitudes (`mag`): each term of each sum replaced by its
absolute value.  A kernel's fp32 sums of those terms are off by at most a small multiple
of 2^-24 of that magnitude, whatever cancels, which is what the tests' bounds count; see
`close`."""
import numpy as np
import torch

F64 = torch.float64


def bounds_of(x, cu):
    B, T = x.shape[:2]
    if cu is None:
        return [(i * T, (i + 1) * T) for i in range(B)]
    c = [int(v) for v in cu]
    return list(zip(c[:-1], c[1:]))


def d(t):
    return None if t is None else t.detach().to("cpu", F64)


def close(got, ref, mag, steps, name):
    """|got - ref| <= half a step of got's type at ref + steps 2^-24 mag, elementwise."""
    g = d(got)
    assert g.shape == ref.shape, f"{name}: shape {tuple(g.shape)} != {tuple(ref.shape)}"
    half = torch.finfo(got.dtype).eps / 2
    bound = half * ref.abs() + steps * 2.0 ** -24 * (mag + ref.abs()) + 1e-37
    bad = ~((g - ref).abs() <= bound)
    if bad.any():
        worst = ((g - ref).abs() / bound).nan_to_num(nan=float("inf"))
        i = int(worst.reshape(-1).argmax())
        at = tuple(int(v) for v in np.unravel_index(i, tuple(ref.shape)))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                             f"{worst.reshape(-1)[i]:.3g} at {at}: {g[at]:.9g} for {ref[at]:.9g}")


def sig(p):
    return 1 / (1 + torch.exp(-p))


def silu(p):
    return p * sig(p)


def dsilu(p):
    s = sig(p)
    return s * (1 + p * (1 - s))


# -------------------------------------------------------------- convolution --
def conv(x, w, b, init, cu, act, dout=None, dfin=None, mag=False):
    """(out, final) or, with dout, the dict of gradients."""
    B, T, C = x.shape
    W = w.shape[1]
    bounds = bounds_of(x, cu)
    N = len(bounds)
    x, w, b, init, dout, dfin = map(d, (x, w, b, init, dout, dfin))
    X = x.reshape(B * T, C)
    b = torch.zeros(C, dtype=F64) if b is None else b
    I = torch.zeros(N, W - 1, C, dtype=F64) if init is None else init
    A = (lambda v: v.abs()) if mag else (lambda v: v)
    out = torch.zeros(B * T, C, dtype=F64)
    fin = I.clone()
    if dout is not None:
        dout = dout.reshape(B * T, C)
    dx, dw, db, di = torch.zeros_like(X), torch.zeros_like(w), torch.zeros(C, dtype=F64), torch.zeros_like(I)
    for n, (p, q) in enumerate(bounds):
        full = torch.cat([I[n], X[p:q]])
        L = q - p
        pre = b + sum(full[j:j + L] * w[:, j] for j in range(W))
        pa = b.abs() + sum((full[j:j + L] * w[:, j]).abs() for j in range(W))
        if dout is None:
            out[p:q] = silu(pre) if act == "silu" else pre
            if mag:  # an error e of pre is one of silu'(pre) e, |silu'| < 1.1; and the factor's own
                out[p:q] = pa * 1.1 + pre.abs() * (2 + pre.abs())
            fin[n] = full[L:]
            continue
        dp = dout[p:q] * (dsilu(pre) if act == "silu" else 1)
        if mag:  # |silu''| <= 0.5: an error of pre moves dp by half of it; and the factor's own
            dp = dout[p:q].abs() * ((4 + pre.abs() + 0.5 * pa) if act == "silu" else 1)
        dfull = torch.zeros_like(full)
        for j in range(W):
            dfull[j:j + L] += dp * A(w[:, j])
            dw[:, j] += (dp * A(full[j:j + L])).sum(0)
        if dfin is not None:
            dfull[L:] += A(dfin[n])
        db += dp.sum(0)
        di[n] = dfull[:W - 1]
        dx[p:q] = dfull[W - 1:]
    if dout is None:
        return out.view(B, T, C), fin
    return {"dx": dx.view(B, T, C), "dweight": dw, "dbias": db, "dinitial_state": di}


# --------------------------------------------------------------------- scan --
def scan(x, dt, A_log, Bm, Cm, D, z, dt_bias, init, cu, dout=None, dfin=None, mag=False):
    """(out, final) or, with dout, the dict of gradients; token by token."""
    B, T, dim = x.shape
    G, n = Bm.shape[2:]
    bounds = bounds_of(x, cu)
    N = len(bounds)
    x, dt, A_log, Bm, Cm, D, z, dt_bias, init, dout, dfin = map(
        d, (x, dt, A_log, Bm, Cm, D, z, dt_bias, init, dout, dfin))
    M = B * T
    X, V = x.reshape(M, dim), dt.reshape(M, dim)
    V = V if dt_bias is None else V + dt_bias
    delta = torch.where(V > 30, V, torch.log1p(torch.exp(V.clamp(max=30))))
    A = -torch.exp(A_log)
    per = dim // G
    Bx = Bm.reshape(M, G, n).repeat_interleave(per, 1)
    Cx = Cm.reshape(M, G, n).repeat_interleave(per, 1)
    Z = None if z is None else z.reshape(M, dim)
    zs = 1.0 if Z is None else silu(Z)
    H0 = torch.zeros(N, dim, n, dtype=F64) if init is None else init
    Ds = torch.zeros(dim, dtype=F64) if D is None else D
    dsil = None if Z is None else dsilu(Z)
    if mag:
        X, Bx, Cx, H0, Ds = X.abs(), Bx.abs(), Cx.abs(), H0.abs(), Ds.abs()
        zs = 1.0 if Z is None else Z.abs() * (2 + Z.abs())
        dsil = None if Z is None else 4 + Z.abs()
    y, h = torch.zeros(M, dim, dtype=F64), torch.zeros(M, dim, n, dtype=F64)
    a = torch.exp(delta[..., None] * A)
    fin = H0.clone()
    for i, (p, q) in enumerate(bounds):
        s = H0[i]
        for t in range(p, q):
            s = a[t] * s + (delta[t] * X[t])[:, None] * Bx[t]
            h[t] = s
            y[t] = (s * Cx[t]).sum(-1) + Ds * X[t]
        fin[i] = s
    if dout is None:
        return (y * zs).view(B, T, dim), fin
    dout = dout.reshape(M, dim)
    if mag:
        dout = dout.abs()
    dy = dout * zs
    sg = torch.ones_like(V) if mag else sig(V)
    Aw = A.abs() if mag else A
    r = {"dx": torch.zeros(M, dim, dtype=F64), "ddt": torch.zeros(M, dim, dtype=F64),
         "dA_log": torch.zeros_like(A), "dB": torch.zeros(M, G, n, dtype=F64),
         "dC": torch.zeros(M, G, n, dtype=F64), "dinitial_state": torch.zeros_like(H0)}
    if Z is not None:
        r["dz"] = (dout * y * dsil).view(B, T, dim)
    live = torch.zeros(M, dtype=torch.bool)
    for i, (p, q) in enumerate(bounds):
        live[p:q] = True
        g = torch.zeros(dim, n, dtype=F64) if dfin is None else (dfin[i].abs() if mag else dfin[i])
        for t in range(q - 1, p - 1, -1):
            g = g + dy[t][:, None] * Cx[t]
            r["dC"][t] = (dy[t][:, None] * h[t]).view(G, per, n).sum(1)
            r["dB"][t] = ((delta[t] * X[t])[:, None] * g).view(G, per, n).sum(1)
            qq = (g * Bx[t]).sum(-1)
            g = g * a[t]
            w = g * (h[t - 1] if t > p else H0[i])
            r["dx"][t] = qq * delta[t] + dy[t] * Ds
            r["ddt"][t] = (qq * X[t] + (w * Aw).sum(-1)) * sg[t]
            r["dA_log"] += w * delta[t][:, None] * Aw
        r["dinitial_state"][i] = g
    r["dD"] = (dy * X)[live].sum(0)
    r["ddt_bias"] = r["ddt"].sum(0)
    r["dx"], r["ddt"] = r["dx"].view(B, T, dim), r["ddt"].view(B, T, dim)
    r["dB"], r["dC"] = r["dB"].view(B, T, G, n), r["dC"].view(B, T, G, n)
    return r


# -------------------------------------------------------------------- norms --
def prenorm(x, res, w, s, eps):
    x, res, w = d(x), d(res), d(w)
    s = d(s) if isinstance(s, torch.Tensor) else s
    h = s * x + (0 if res is None else res)
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w, h


def prenorm_bwd(dout, dh, h, w, x, s, eps):
    """(gradients, magnitudes)"""
    dout, dh, h, w, x = map(d, (dout, dh, h, w, x))
    s = d(s) if isinstance(s, torch.Tensor) else s
    r = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    u, du = h * r, dout * w
    dh0 = 0 if dh is None else dh
    g = dh0 + r * (du - u * (du * u).mean(-1, keepdim=True))
    m = abs(dh0) + r * (du.abs() + u.abs() * (du * u).abs().mean(-1, keepdim=True))
    flat = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    out = {"dresidual": g, "dx": g * s, "dweight": flat(dout * u)}
    mag = {"dresidual": m, "dx": m * abs(s), "dweight": flat((dout * u).abs())}
    if isinstance(s, torch.Tensor):
        out["dres_scale"], mag["dres_scale"] = flat(g * x), flat(m * x.abs())
    return out, mag


def act_of(act):
    return (silu, dsilu) if act == "silu" else (sig, lambda p: sig(p) * (1 - sig(p)))


def postnorm(x, w, gate, res, s, act, eps):
    x, w, gate, res = map(d, (x, w, gate, res))
    s = d(s) if isinstance(s, torch.Tensor) else s
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    if gate is not None:
        y = y * act_of(act)[0](gate)
    y = s * y
    return y if res is None else res + y


def postnorm_bwd(dout, x, w, gate, s, act, eps):
    dout, x, w, gate = map(d, (dout, x, w, gate))
    s = d(s) if isinstance(s, torch.Tensor) else s
    f, df = act_of(act)
    a = 1.0 if gate is None else f(gate)
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    u, dn = x * r, dout * s * a
    du = dn * w
    # the gate's own relative error grows with its argument
    k = 1.0 if gate is None else 2 + gate.abs()
    flat = lambda v: v.reshape(-1, v.shape[-1]).sum(0)  # noqa: E731
    out = {"dx": r * (du - u * (du * u).mean(-1, keepdim=True)), "dweight": flat(dn * u)}
    mag = {"dx": r * (k * du.abs() + u.abs() * (k * du * u).abs().mean(-1, keepdim=True)),
           "dweight": flat(k * (dn * u).abs())}
    if gate is not None:
        out["dgate"] = dout * s * u * w * df(gate)
        mag["dgate"] = (dout * s * u * w).abs() * (4 + gate.abs())
    if isinstance(s, torch.Tensor):
        out["dres_scale"], mag["dres_scale"] = flat(dout * u * w * a), flat(k * (dout * u * w * a).abs())
    return out, mag
