"""The 64-bit forms that the layer operators are tested against: their gradients equal
central differences, and packed sequences equal sequences on their own."""
import pytest
import torch

from tests import layer_ref as R

F64 = torch.float64


def rnd(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=F64)


def check_differences(f, leaves, grads, weights):
    """<weights, f(leaves)> against its gradients along a random direction of each leaf."""
    gen = torch.Generator().manual_seed(3)
    for name, t in leaves.items():
        v = rnd(gen, *t.shape)
        eps = 1e-6
        vals = []
        for sgn in (1, -1):
            outs = f(**{**leaves, name: t + sgn * eps * v})
            vals.append(sum((o * w).sum() for o, w in zip(outs, weights)))
        num = (vals[0] - vals[1]) / (2 * eps)
        ana = (grads[name] * v).sum()
        assert abs(num - ana) <= 1e-6 * (1 + abs(ana)), f"{name}: {num} {ana}"


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 9]])
@pytest.mark.parametrize("act", ["silu", None])
def test_conv_gradients(cu, act):
    g = torch.Generator().manual_seed(1)
    B, T, C, W = (2, 5, 3, 4) if cu is None else (1, 9, 3, 4)
    N = B if cu is None else 4
    leaves = {"x": rnd(g, B, T, C), "w": rnd(g, C, W), "b": rnd(g, C), "init": rnd(g, N, W - 1, C)}
    dout, dfin = rnd(g, B, T, C), rnd(g, N, W - 1, C)
    r = R.conv(**leaves, cu=cu, act=act, dout=dout, dfin=dfin)
    grads = {"x": r["dx"], "w": r["dweight"], "b": r["dbias"], "init": r["dinitial_state"]}
    check_differences(lambda **k: R.conv(**k, cu=cu, act=act), leaves, grads, (dout, dfin))


@pytest.mark.parametrize("cu,G", [(None, 1), ([0, 3, 3, 4, 7], 2)])
def test_scan_gradients(cu, G):
    g = torch.Generator().manual_seed(2)
    B, T, dim, n = (2, 5, 4, 3) if cu is None else (1, 7, 4, 3)
    N = B if cu is None else 4
    leaves = {"x": rnd(g, B, T, dim), "dt": rnd(g, B, T, dim), "A_log": rnd(g, dim, n),
              "Bm": rnd(g, B, T, G, n), "Cm": rnd(g, B, T, G, n), "D": rnd(g, dim),
              "z": rnd(g, B, T, dim), "dt_bias": rnd(g, dim), "init": rnd(g, N, dim, n)}
    dout, dfin = rnd(g, B, T, dim), rnd(g, N, dim, n)
    r = R.scan(**leaves, cu=cu, dout=dout, dfin=dfin)
    grads = {"x": r["dx"], "dt": r["ddt"], "A_log": r["dA_log"], "Bm": r["dB"], "Cm": r["dC"],
             "D": r["dD"], "z": r["dz"], "dt_bias": r["ddt_bias"], "init": r["dinitial_state"]}
    check_differences(lambda **k: R.scan(**k, cu=cu), leaves, grads, (dout, dfin))


def test_scan_packed_equals_single():
    g = torch.Generator().manual_seed(4)
    T, dim, n, cu = 9, 3, 2, [0, 4, 4, 9]
    a = [rnd(g, 1, T, dim), rnd(g, 1, T, dim), rnd(g, dim, n), rnd(g, 1, T, 1, n), rnd(g, 1, T, 1, n)]
    init = rnd(g, 3, dim, n)
    out, fin = R.scan(*a, None, None, None, init, cu)
    for i, (p, q) in enumerate(zip(cu[:-1], cu[1:])):
        cut = [a[0][:, p:q], a[1][:, p:q], a[2], a[3][:, p:q], a[4][:, p:q]]
        o, f = R.scan(*cut, None, None, None, init[i:i + 1], None)
        assert torch.equal(o, out[:, p:q]) and torch.equal(f[0], fin[i])


@pytest.mark.parametrize("per_channel", [False, True])
def test_norm_gradients(per_channel):
    g = torch.Generator().manual_seed(5)
    rows, dim, eps = 3, 7, 1e-3
    x, res, w, gate = rnd(g, rows, dim), rnd(g, rows, dim), rnd(g, dim), rnd(g, rows, dim)
    s = rnd(g, dim) if per_channel else 0.7
    dout, dh = rnd(g, rows, dim), rnd(g, rows, dim)
    _, h = R.prenorm(x, res, w, s, eps)
    r, _ = R.prenorm_bwd(dout, dh, h, w, x, s, eps)
    leaves, grads = {"x": x, "res": res, "w": w}, {"x": r["dx"], "res": r["dresidual"], "w": r["dweight"]}
    if per_channel:
        leaves["s"], grads["s"] = s, r["dres_scale"]
    check_differences(lambda **k: R.prenorm(**{"s": s, **k}, eps=eps), leaves, grads, (dout, dh))
    for act in ("silu", "sigmoid"):
        r, _ = R.postnorm_bwd(dout, x, w, gate, s, act, eps)
        leaves = {"x": x, "w": w, "gate": gate}
        grads = {"x": r["dx"], "w": r["dweight"], "gate": r["dgate"]}
        if per_channel:
            leaves["s"], grads["s"] = s, r["dres_scale"]
        check_differences(lambda **k: (R.postnorm(**{"s": s, **k}, res=res, act=act, eps=eps),),
                          leaves, grads, (dout,))
