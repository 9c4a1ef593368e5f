"""Calls of the gated feed-forward product: arguments at the ends of their range, workspaces that held
another call's values, kept pre-activations as integers, no writes beyond the results."""
import ctypes

import pytest
import torch

from tests.glu_ref import glu, kept_values, within
from tests.test_gpu_glu import make
from tests.test_gpu_linrec_batches import guarded

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
NAMES = ("dx", "dw_gate", "dw_up")


@pytest.mark.parametrize("rows", [5, 300])
@pytest.mark.parametrize("fn", ["silu", "gelu", "sigmoid"])
def test_arguments_beyond_the_range_of_their_powers(kda_lib, rows, fn):
    """Pre-activations of 2^66 and 2^120 of both signs, whose cubes (and squares) fp32 does not hold:
    f is g or 0 (sigmoid: 1 or 0) and its slope 1 or 0 (0).  Powers of two, so that everything is exact."""
    import kimi_delta_attention_08_gb300 as kda
    w = torch.zeros(8, 8)
    w[:, 0] = torch.tensor([2.0 ** 66, -2.0 ** 66, 2.0 ** 44, -2.0 ** 44, 2.0 ** 120, -2.0 ** 120, 2.0 ** 20, -2.0 ** 20])
    x = torch.zeros(1, rows, 8)
    x[..., 0], x[..., 1] = 1, 0.5
    up = torch.zeros(8, 8)
    up[:, 1] = 4                             # u = 2
    dout = torch.full((1, rows, 8), 2.0 ** -60)
    dev = lambda v: v.to(BF).cuda()          # noqa: E731
    out = torch.empty(1, rows, 8, dtype=BF, device="cuda")
    kda.kda_glu_fwd(dev(x), dev(w), dev(up), out, activation=fn)
    g = w[:, 0].double()
    f, df = (torch.where(g > 0, g, 0), (g > 0).double()) if fn != "sigmoid" else ((g > 0).double(), 0 * g)
    assert torch.equal(out.cpu().double(), (2 * f).expand(1, rows, 8))
    got = kda.kda_glu_bwd(dev(x), dev(w), dev(up), dev(dout), activation=fn)
    dg, du = 2.0 ** -60 * 2 * df, 2.0 ** -60 * f
    dx = torch.zeros(8, dtype=torch.float64)
    dx[0], dx[1] = (dg * g).sum(), (du * 4).sum()
    want = {"dx": dx.expand(1, rows, 8), "dw_gate": rows * torch.outer(dg, x[0, 0].double()),
            "dw_up": rows * torch.outer(du, x[0, 0].double())}
    for k in NAMES:  # dx's sums have other terms that a rounding to bf16 drops: half a step of it
        assert ((got[k].cpu().double() - want[k]).abs() <= 2.0 ** -8 * want[k].abs()).all(), k


@pytest.mark.parametrize("size", [(97, 136, 6160), (300, 264, 2056), (513, 64, 2056), (1100, 264, 1032)])
@pytest.mark.parametrize("kept", [False, True])
def test_calls_in_turn_in_one_workspace(kda_lib, size, kept):
    """Sizes at which the weights' gradients start before dx ends: of calls in turn, each reads its own
    gradients of g and u, not those that the call before left in the workspace."""
    import kimi_delta_attention_08_gb300 as kda
    ws = kda.make_glu_bwd_workspace(size[0], size[2])
    sets, want = [make(*size, seed=k) for k in (1, 2)], []
    pres = [None, None]
    if kept:
        pres = [torch.empty(1, size[0], 2 * size[2], dtype=BF, device="cuda") for _ in sets]
        for (x, wg, wu, dout), pre in zip(sets, pres):
            kda.kda_glu_fwd(x, wg, wu, torch.empty_like(dout), pre=pre)
    for (x, wg, wu, dout), pre in zip(sets, pres):
        g = kda.kda_glu_bwd(x, wg, wu, dout, pre=pre)  # in memory of its own
        ref = glu(x, wg, wu, "silu", dout, pre)
        for k in NAMES:
            within(g[k], ref[k], k)
        want.append(g)
    torch.cuda.synchronize()
    got = [kda.kda_glu_bwd(*sets[n % 2], ws, pre=pres[n % 2]) for n in range(40)]
    for n, g in enumerate(got):
        for k in NAMES:
            assert torch.equal(g[k], want[n % 2][k]), (n, k)
    assert kda.kda_get_device_status(ws) == 0


@pytest.mark.parametrize("size", [(5, 72, 136), (300, 264, 2056)])
def test_kept_values_as_integers(kda_lib, size):
    """The buffer of kept pre-activations as int16, which no operation takes for numbers: the same bits."""
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(*size)
    out, shape = torch.empty_like(dout), (1, size[0], 2 * size[2])
    pre, same = torch.empty(shape, dtype=torch.int16, device="cuda"), torch.empty(shape, dtype=BF, device="cuda")
    kda.kda_glu_fwd(x, wg, wu, out, pre=pre)
    kda.kda_glu_fwd(x, wg, wu, out, pre=same)
    assert torch.equal(pre, same.view(torch.int16))
    within(pre, glu(x, wg, wu, "silu")["pre"], "pre")
    a, b = (kda.kda_glu_bwd(x, wg, wu, dout, pre=p) for p in (pre, same))
    for k in NAMES:
        assert torch.equal(a[k], b[k]), k
    assert kept_values(pre).isfinite().all()


@pytest.mark.parametrize("size", [(5, 72, 136), (130, 136, 264), (200, 1000, 9800), (300, 264, 2056)])
def test_nothing_beyond_the_results_is_written(kda_lib, size):
    """Few rows, tiles of both widths, split tiles; forward, and backward through the C entry point."""
    import kimi_delta_attention_08_gb300 as kda
    from kimi_delta_attention_08_gb300 import layer
    M, D, Fh = size
    x, wg, wu, dout = make(*size)
    (out, ok0), (pre, ok1) = guarded((1, M, Fh), BF), guarded((1, M, 2 * Fh), BF)
    kda.kda_glu_fwd(x, wg, wu, out)
    within(out, glu(x, wg, wu, "silu")["out"], "out")
    kda.kda_glu_fwd(x, wg, wu, out, pre=pre)
    assert ok0() and ok1()
    q, _ = layer._glu_problem(x, wg, wu, "silu", False)
    ws = kda.make_glu_bwd_workspace(M, Fh)
    for kept in (None, pre):
        grads = [guarded((1, M, D), BF), guarded((Fh, D), BF), guarded((Fh, D), BF)]
        layer._call("kda_glu_bwd", x.device, None, ctypes.byref(q), dout.data_ptr(),
                    None if kept is None else kept.data_ptr(), *[v.data_ptr() for v, _ in grads],
                    ws.data_ptr(), ws.numel())
        want = kda.kda_glu_bwd(x, wg, wu, dout, pre=kept)
        for nm, (v, ok) in zip(NAMES, grads):
            assert ok() and torch.equal(v, want[nm]), nm
