"""Plain 64-bit form of the gated feed-forward product, and the error bounds of the kernels.

A projection's sum of D products is accumulated in fp32 in an order of the hardware's: off by
at most (D + 8) 2^-24 of the sum of the products' magnitudes (they are exact in fp32), and the
tensor cores may drop what lies below the largest term's last bit, which the same bound
holds for, twice.  f and its slope are within 8 steps of fp32 plus what their arguments
are off by (|f'| <= 1.13, |f''| <= 0.8 for silu, gelu and sigmoid), and for arguments of
a size |g| 1.5 |g| steps more.  The backward's dg and du are rounded to bf16 (half a step,
eps / 2 = 2^-8 of the value) before they are summed with what they carry themselves.  Those
roundings are independent, so over a sum their norm stays at half a step over sqrt 3 of the
sum's: outputs rounded once are 1.7e-3 off in norm, with a rounding before the sum 2.4e-3;
`within` asks for 4e-3."""
import math

import torch

from tests.layer_ref import F64, d, sig

U = 2.0 ** -24          # half a step of fp32
HALF = 2.0 ** -8        # half a step of bf16, relative to the value
KEPT = 2.0 ** -10       # half a step of kept pre-activations, which have 9 bits of fraction


def kept_values(pre):
    """The values of a buffer of kept pre-activations: a sign, 6 bits of exponent (bias 31) and
    9 of fraction; below the smallest exponent the fraction has no leading one, above the
    largest there is no number."""
    b = pre.detach().cpu().contiguous().view(torch.int16).to(torch.int64) & 0xFFFF
    e, f = b >> 9 & 63, (b & 511).to(F64)
    v = torch.where(e > 0, torch.ldexp(1 + f / 512, e - 31), f / 512 * 2.0 ** -30)
    v = torch.where(e == 63, torch.nan, v)
    return torch.where(b >> 15 > 0, -v, v)


def act(g, fn):
    """f(g) and f'(g)"""
    if fn == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    s = sig(g)
    return (s, s * sig(-g)) if fn == "sigmoid" else (g * s, s + g * s * sig(-g))


def glu(x, wg, wu, fn, dout=None, pre=None):
    """{name: (value, bound)} of out, pre, and with dout of the gradients; `pre` (kept, rounded)
    takes the place of both projections in the backward."""
    shape = x.shape
    x, wg, wu = d(x).reshape(-1, shape[-1]), d(wg), d(wu)
    M, D = x.shape
    Fh = wg.shape[0]
    g, u = x @ wg.T, x @ wu.T
    eg, eu = ((x.abs() @ w.abs().T) * 2 * (D + 8) * U for w in (wg, wu))
    back = lambda v, n: v.reshape(*shape[:-1], n)  # noqa: E731
    if pre is not None:
        pre = kept_values(pre).reshape(M, 2 * Fh)
        g, u = pre[:, :Fh], pre[:, Fh:]
        eg, eu = torch.zeros_like(eg), torch.zeros_like(eu)
    f, df = act(g, fn)
    ef = 1.13 * eg + (8 + 2 * g.abs()) * U * (f.abs() + g.abs() * sig(g))
    out = f * u
    eout = ef * u.abs() + (f.abs() + ef) * eu + 2 * U * out.abs()
    kept = torch.cat([g, u], 1)
    r = {"out": (back(out, Fh), back(eout + HALF * (out.abs() + eout), Fh)),
         "pre": (back(kept, 2 * Fh), back(torch.cat([eg, eu], 1) * (1 + KEPT) + KEPT * kept.abs() + 2.0 ** -40, 2 * Fh))}
    if dout is None:
        return r
    dy = d(dout).reshape(M, Fh)
    dg, du = dy * u * df, dy * f
    edf = 0.8 * eg + (8 + 2 * g.abs()) * U * (1 + g.abs())
    edg = dy.abs() * (edf * u.abs() + (df.abs() + edf) * eu) + 4 * U * dg.abs()
    edu = dy.abs() * ef + 2 * U * du.abs()
    # rounded to bf16, then summed: of F (twice) or of M products
    edg, edu = edg * (1 + HALF) + HALF * dg.abs(), edu * (1 + HALF) + HALF * du.abs()
    ag, au = dg.abs() + edg, du.abs() + edu
    dx = dg @ wg + du @ wu
    edx = edg @ wg.abs() + edu @ wu.abs() + 2 * (2 * Fh + 8) * U * (ag @ wg.abs() + au @ wu.abs())
    grads = {"dx": (back(dx, D), back(edx + HALF * (dx.abs() + edx), D))}
    for k, v, e, a in (("dw_gate", dg, edg, ag), ("dw_up", du, edu, au)):
        dw = v.T @ x
        edw = e.T @ x.abs() + 2 * (M + 8) * U * (a.T @ x.abs())
        grads[k] = (dw, edw + HALF * (dw.abs() + edw))
    return {**r, **grads}


def within(got, ref, name):
    value, bound = ref
    got = kept_values(got) if name == "pre" else d(got)
    assert got.shape == value.shape, name
    bad = ~((got - value).abs() <= bound + 1e-37)
    if bad.any():
        i = int(((got - value).abs() / (bound + 1e-37)).nan_to_num(nan=float("inf")).argmax())
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} beyond the bound, worst "
                             f"{got.reshape(-1)[i]:.9g} for {value.reshape(-1)[i]:.9g} within "
                             f"{bound.reshape(-1)[i]:.3g}")
    # bounds of single values say little of an error that all share
    assert (got - value).norm() <= 4e-3 * value.norm() + 1e-30, f"{name}: norm of the error"
