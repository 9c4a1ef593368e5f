"""Plain 64-bit form of the gated linear recurrence on the CPU, written from its definition
token by token, and the magnitudes that the kernels' error bounds count (see
tests/layer_ref.py): each term of each sum by its absolute value, times 1 + |gate| for
what a rounded gate argument does to a sigmoid."""
import torch

from tests.layer_ref import F64, bounds_of, d, dsilu, sig, silu


def linrec(x, r, i, A_log, z, r_bias, i_bias, init, cu, dout=None, dfin=None, mag=False):
    """(out, final) or, with dout, the dict of gradients."""
    B, T, D = x.shape
    M = B * T
    bounds = bounds_of(x, cu)
    N = len(bounds)
    x, r, i, A_log, z, r_bias, i_bias, init, dout, dfin = map(
        d, (x, r, i, A_log, z, r_bias, i_bias, init, dout, dfin))
    flat = lambda v: None if v is None else v.reshape(M, D)  # noqa: E731
    x, r, i, z, dout = map(flat, (x, r, i, z, dout))
    r = r if r_bias is None else r + r_bias
    i = i if i_bias is None else i + i_bias
    R, I = sig(r), sig(i)
    L = torch.exp(A_log) * R
    a, m = torch.exp(-L), torch.sqrt(-torch.expm1(-2 * L))
    h0 = torch.zeros(N, D, dtype=F64) if init is None else init
    wide = torch.ones_like(x)
    if mag:
        x, h0, wide = x.abs(), h0.abs(), 2 + r.abs() + i.abs()
        dout = None if dout is None else dout.abs()
        dfin = None if dfin is None else dfin.abs()
    b = m * I * x * wide
    before, h, fin = torch.zeros_like(x), torch.zeros_like(x), h0.clone()
    for n, (p, q) in enumerate(bounds):
        s = h0[n]
        for t in range(p, q):
            before[t] = s
            s = a[t] * s + b[t]
            h[t] = s
        fin[n] = s
    gate, slope = 1.0, None
    if z is not None:
        gate, slope = silu(z), dsilu(z)
        if mag:
            gate, slope = z.abs() * (2 + z.abs()) * sig(z), 4 + z.abs()
    if dout is None:
        return (h * gate).view(B, T, D), fin
    live = torch.zeros(M, 1, dtype=F64)
    dy = dout * gate
    g = torch.zeros_like(x)
    dinit = torch.zeros_like(h0) if dfin is None else dfin.clone()
    for n, (p, q) in enumerate(bounds):
        live[p:q] = 1
        c = torch.zeros(D, dtype=F64) if dfin is None else dfin[n]
        for t in range(q - 1, p - 1, -1):
            g[t] = dy[t] + c
            c = a[t] * g[t]
        if q > p:
            dinit[n] = c
    lm = torch.where(L > 0, L / m, 0)
    e = g * (a * a * lm * I * x - a * before * L) * live
    if mag:
        e = g * (a * a * lm * I * x + a * before * L) * wide * live
    gm = g * m * live * wide
    # 1 - sigmoid(v) = sigmoid(-v), which does not cancel
    out = {"dx": gm * I, "dr": e * sig(-r), "di": gm * x * I * sig(-i)}
    if z is not None:
        out["dz"] = dout * h * slope * live
    sums = {"dA_log": e.sum(0), "dr_bias": out["dr"].sum(0), "di_bias": out["di"].sum(0),
            "dinitial_state": dinit}
    return {**{k: v.view(B, T, D) for k, v in out.items()}, **sums}
