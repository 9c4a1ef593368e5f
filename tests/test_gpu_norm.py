"""The norms before and after a block against their 64-bit forms: one row to many, widths
on and off the vector size up to the limit, both types, the gate's slices, scales, in
place, rows of zeros and of large values.

Bounds: a row's sum of squares is added in a tree with at most 16 values in a row per
thread, so its relative error is under 30 steps of 2^-24 and rstd's under 17 with the
root's own; each output adds a few products, the gate the exponential (2^-22) and a
reciprocal: 64 steps of the magnitudes.  A weight's gradient is a sum over rows: one step
more per row."""
import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
EPS = 1e-6
SIZES = [(1, 4096), (33, 1), (5, 7), (300, 64), (1001, 128), (77, 192), (9, 257), (40, 512),
         (21, 1001), (13, 1024), (3, 2050), (6, 4096), (5, 5000), (3, 8191), (2, 8192)]


def rnd(g, *s, t=F, scale=1.0):
    return (torch.randn(*s, generator=g) * scale).to(t).cuda()


def scale_of(g, D, per_channel):
    return rnd(g, D) if per_channel else 0.5


def nan_like(t):
    return torch.full_like(t, float("nan"))


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("ty,sty,per_channel", [(BF, BF, False), (BF, F, True), (F, F, False)])
def test_prenorm(kda_lib, rows, D, ty, sty, per_channel):
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(rows * D)
    x, res, w, s = rnd(g, rows, D, t=ty), rnd(g, rows, D, t=sty, scale=2), rnd(g, D), scale_of(g, D, per_channel)
    out, ro = nan_like(x), nan_like(res)
    kda.kda_prenorm_fwd(x, res, w, out, ro, res_scale=s, eps=EPS)
    ref, h = R.prenorm(x, res, w, s, EPS)
    _, hm = R.prenorm(x.abs(), res.abs(), w, s.abs() if per_channel else s, EPS)
    R.close(ro, h, hm, 4, "residual_out")
    # out = h rstd w, where h carries the rounding of its own sum
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    R.close(out, ref, hm * rstd * R.d(w).abs(), 64, "out")
    inplace = res.clone()
    kda.kda_prenorm_fwd(x, inplace, w, out2 := nan_like(x), inplace, res_scale=s, eps=EPS)
    assert torch.equal(inplace, ro) and torch.equal(out2, out)

    dout, dh, h = rnd(g, rows, D, t=ty), rnd(g, rows, D, t=sty), ro
    r = kda.kda_prenorm_bwd(dout, dh, h, w, x, res_scale=s, eps=EPS)
    ref, mag = R.prenorm_bwd(dout, dh, h, w, x, s, EPS)
    assert set(r) - {"workspace"} == set(ref)
    for nm in ref:
        R.close(r[nm], ref[nm], mag[nm], 64 + (rows if nm in ("dweight", "dres_scale") else 0), nm)


@pytest.mark.parametrize("D", [128, 1000, 257])
def test_prenorm_parts_left_out(kda_lib, D):
    """No residual, no residual output, no gradient from elsewhere; scale 1 gives one buffer
    for both row gradients."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(D)
    x, w, dout = rnd(g, 50, D, t=BF), rnd(g, D), rnd(g, 50, D, t=BF)
    out = nan_like(x)
    kda.kda_prenorm_fwd(x, None, w, out, eps=EPS)
    ref, h = R.prenorm(x, None, w, 1.0, EPS)
    R.close(out, ref, ref.abs(), 64, "out")
    r = kda.kda_prenorm_bwd(dout, None, x, w, eps=EPS)
    assert r["dx"] is r["dresidual"]
    ref, mag = R.prenorm_bwd(dout, None, x, w, None, 1.0, EPS)
    for nm in ("dx", "dweight"):
        R.close(r[nm], ref[nm], mag[nm], 120, nm)


@pytest.mark.parametrize("rows,D", SIZES)
@pytest.mark.parametrize("ty,act,res,per_channel", [(BF, "sigmoid", False, False), (BF, "silu", True, True),
                                                     (F, "silu", False, False), (F, None, True, True)])
def test_postnorm(kda_lib, rows, D, ty, act, res, per_channel):
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(rows * D + 1)
    x, w, s = rnd(g, rows, D, t=ty), rnd(g, D), scale_of(g, D, per_channel)
    gate = None if act is None else rnd(g, rows, D, t=ty, scale=3)
    r0 = rnd(g, rows, D, t=ty) if res else None
    fn = act or "sigmoid"
    out = nan_like(x)
    kda.kda_postnorm_fwd(x, w, gate, out, r0, res_scale=s, activation=fn, eps=EPS)
    ref = R.postnorm(x, w, gate, r0, s, fn, EPS)
    part = R.postnorm(x, w, gate, None, s, fn, EPS).abs()
    mag = part * (1 if gate is None else 2 + R.d(gate).abs()) + (0 if r0 is None else R.d(r0).abs())
    R.close(out, ref, mag, 64, "out")
    same = x.clone()
    kda.kda_postnorm_fwd(same, w, gate, same, r0, res_scale=s, activation=fn, eps=EPS)
    assert torch.equal(same, out)

    dout = rnd(g, rows, D, t=ty)
    r = kda.kda_postnorm_bwd(dout, x, w, gate, res_scale=s, activation=fn, eps=EPS)
    ref, mag = R.postnorm_bwd(dout, x, w, gate, s, fn, EPS)
    assert set(r) - {"workspace"} == set(ref)
    for nm in ref:
        R.close(r[nm], ref[nm], mag[nm], 64 + (rows if nm in ("dweight", "dres_scale") else 0), nm)


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("D", [520, 1000, 2008])
def test_backward_after_other_rows(kda_lib, D, ty):
    """Widths that leave threads of a block without values, after a call whose rows were NaN
    everywhere: nothing of them is left in what the next call reads."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(D)
    bad = torch.full((2000, 2048), float("nan"), dtype=ty, device="cuda")
    x, dout, gate, w = rnd(g, 400, D, t=ty), rnd(g, 400, D, t=ty), rnd(g, 400, D, t=ty), rnd(g, D)
    s = rnd(g, D)
    kda.kda_prenorm_bwd(bad, bad, bad, torch.ones(2048, device="cuda"), bad,
                        res_scale=torch.ones(2048, device="cuda"), eps=EPS)
    r = kda.kda_prenorm_bwd(dout, gate, x, w, x, res_scale=s, eps=EPS)
    ref, mag = R.prenorm_bwd(dout, gate, x, w, x, s, EPS)
    for nm in ref:
        R.close(r[nm], ref[nm], mag[nm], 64 + (400 if nm in ("dweight", "dres_scale") else 0), nm)
    kda.kda_postnorm_bwd(bad, bad, torch.ones(2048, device="cuda"), bad, eps=EPS)
    r = kda.kda_postnorm_bwd(dout, x, w, gate, res_scale=s, activation="silu", eps=EPS)
    ref, mag = R.postnorm_bwd(dout, x, w, gate, s, "silu", EPS)
    for nm in ref:
        R.close(r[nm], ref[nm], mag[nm], 64 + (400 if nm in ("dweight", "dres_scale") else 0), nm)


@pytest.mark.parametrize("extra", [128, 5])
def test_gate_in_a_projection(kda_lib, extra):
    """The gate as a slice of wider rows [B, T, H, D]: the bits of a contiguous one."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(9)
    B, T, H, D = 2, 19, 3, 128
    x, w, dout = rnd(g, B, T, H, D, t=BF), rnd(g, D), rnd(g, B, T, H, D, t=BF)
    gate = rnd(g, B, T, H * D + extra, t=BF)[..., extra:].unflatten(2, (H, D))
    a, b = nan_like(x), nan_like(x)
    kda.kda_postnorm_fwd(x, w, gate, a)
    kda.kda_postnorm_fwd(x, w, gate.contiguous(), b)
    assert torch.equal(a, b)
    ga, gb = kda.kda_postnorm_bwd(dout, x, w, gate), kda.kda_postnorm_bwd(dout, x, w, gate.contiguous())
    for nm in ("dx", "dgate", "dweight"):
        R.close(ga[nm], R.d(gb[nm]), R.d(gb[nm]).abs(), 2 ** 12, nm)


def test_zero_and_large_rows(kda_lib):
    """A row of zeros stays zero (eps > 0); rows whose squares are far from 1 keep the
    relative accuracy; an infinity spoils its own row alone."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(11)
    x, w = rnd(g, 6, 1024), rnd(g, 1024)
    x[0] = 0
    x[1] *= 1e15
    x[2] *= 1e-12
    out = nan_like(x)
    kda.kda_postnorm_fwd(x, w, None, out, eps=1e-30)
    ref = R.postnorm(x, w, None, None, 1.0, "silu", 1e-30)
    assert not out[0].any()
    R.close(out, ref, ref.abs(), 64, "out")
    x[3, 5] = float("inf")
    kda.kda_postnorm_fwd(x, w, None, out2 := nan_like(x), eps=1e-30)
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(out2[keep], out[keep]) and not out2[3].isfinite().all()


def test_no_rows(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(64, device="cuda")
    kda.kda_prenorm_fwd(x, x, w, torch.empty_like(x), torch.empty_like(x))
    kda.kda_postnorm_fwd(x, w, x, torch.empty_like(x))
    r = kda.kda_postnorm_bwd(x, x, w, x, res_scale=w)
    assert not r["dweight"].any() and not r["dres_scale"].any()
    r = kda.kda_prenorm_bwd(x, x, x, w, x, res_scale=w)
    assert not r["dweight"].any() and not r["dres_scale"].any()
