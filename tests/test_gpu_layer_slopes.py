"""The slopes of sigmoid and SiLU where they come close to 0 or 1: the gradients of gates and of
the convolution's activation keep their relative accuracy at every argument.

Bounds, in steps of 2^-24 of the result: the exponential is within 2^-22 (4 steps) and its
argument's rounding adds up to 1.5 steps per unit of it; 1 + u, the reciprocal (2^-23), its
square and the products are 8; the norm's root and row sums 47 (tests/test_gpu_norm.py), the
convolution's own sum 16."""
import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def within(got, ref, mag, steps, name):
    """As R.close, with a bound of its own for each element: `steps` is a tensor."""
    g = R.d(got)
    bound = torch.finfo(got.dtype).eps / 2 * ref.abs() + steps * 2.0 ** -24 * mag + 1e-37
    bad = ~((g - ref).abs() <= bound)
    i = int(((g - ref).abs() / bound).nan_to_num(nan=float("inf")).reshape(-1).argmax())
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()}, worst {g.reshape(-1)[i]:.9g} "
                           f"for {ref.reshape(-1)[i]:.9g}")


GATES = [0.0, 0.5, 2.0, 8.0, 10.0, 12.0, 14.0, 17.0, 20.0, 40.0, 60.0]


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("D", [128, 1024, 257])
def test_gate_gradient_near_saturation(kda_lib, ty, act, D):
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(D)
    v = torch.tensor(GATES + [-x for x in GATES])
    gate = v[torch.randint(len(v), (40, D), generator=g)].to(ty).cuda()
    x, dout = torch.randn(40, D, generator=g).to(ty).cuda(), torch.randn(40, D, generator=g).to(ty).cuda()
    w = torch.randn(D, generator=g).cuda()
    r = kda.kda_postnorm_bwd(dout, x, w, gate, activation=act, eps=1e-6)
    p = R.d(gate)
    s, ds = R.sig(p), R.sig(p) * R.sig(-p)
    du = R.d(dout) * R.d(x) / torch.sqrt((R.d(x) ** 2).mean(-1, keepdim=True) + 1e-6) * R.d(w)
    ref, part = (du * ds, du.abs() * ds) if act == "sigmoid" else (du * (s + p * ds), du.abs() * (s + p.abs() * ds))
    within(r["dgate"], ref, part, 64 + 1.5 * p.abs(), "dgate")


LARGE = [3.0, 12.0, 17.0, 30.0, 1e3, 12345.678, 1e6, 1e8]


def silu_bounds(p):
    """silu'(p), and the error of s + p s (1 - s) from an s that is off by 8 + 1.5 |p| steps of
    itself (none where it has rounded to 1) and 1 - s by two steps of 1, p itself exact."""
    s, c = R.sig(p), R.sig(-p)
    live = p < 18
    rel = torch.where(live, 8 + 1.5 * p.abs(), torch.zeros_like(p))
    steps = s * (rel + 4) + (p * s).abs() * (c * (rel + 4) + torch.where(live, s * rel + 2, 0 * p))
    # beyond, 1 - s is zero: what is left out is p c
    return s + p * s * c, steps + torch.where(live, 0 * p, (p * c).abs() * 2.0 ** 24)


@pytest.mark.parametrize("C", [64, 37])
def test_convolution_slope_at_large_arguments(kda_lib, C):
    """Width 2 with weights (0, 1): the pre-activation is x itself and dx = dout silu'(x)."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(C)
    v = torch.tensor(LARGE + [-x for x in LARGE])
    x = v[torch.randint(len(v), (1, 200, C), generator=g)].cuda()
    w = torch.tensor([0.0, 1.0]).repeat(C, 1).cuda()
    dout = torch.randn(1, 200, C, generator=g).cuda()
    r = kda.kda_conv_bwd(x, w, None, dout)
    slope, steps = silu_bounds(R.d(x))
    ref = R.d(dout) * slope
    within(r["dx"], ref, R.d(dout).abs(), steps + 2, "dx")
    # dweight[1] = sum dout silu' x: as large as x, each term to its own error
    t = ref * R.d(x)
    err = (R.d(dout) * R.d(x)).abs() * (steps + 2)
    within(r["dweight"][:, 1], t.sum((0, 1)), t.abs().sum((0, 1)).clamp(min=1e-30),
           80 + err.sum((0, 1)) / t.abs().sum((0, 1)).clamp(min=1e-30), "dweight")


@pytest.mark.parametrize("dim", [64, 33])
def test_scan_gate_slope_at_large_arguments(kda_lib, dim):
    """Steps of zero and D = 1: y = x, so dz = dout x silu'(z)."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(dim)
    v = torch.tensor(LARGE + [-x for x in LARGE])
    z = v[torch.randint(len(v), (2, 50, dim), generator=g)].cuda()
    x, dout = (torch.randn(2, 50, dim, generator=g).cuda() for _ in range(2))
    B = torch.randn(2, 50, 1, 16, generator=g).cuda()
    r = kda.kda_scan_bwd(x, torch.full_like(x, -200.0), torch.zeros(dim, 16, device="cuda"), B, B, dout,
                         torch.ones(dim, device="cuda"), z)
    slope, steps = silu_bounds(R.d(z))
    du = R.d(dout) * R.d(x)
    within(r["dz"], du * slope, du.abs(), steps + 4, "dz")


FAR = [-85.0, -80.0, -60.0, -40.0, -20.0, -8.0, -1.0, 0.5, 3.0, 20.0, 85.0]


def far(g, *shape):
    """Arguments around FAR, not whole numbers: their products with log2 e are rounded."""
    v = torch.tensor(FAR)
    return (v[torch.randint(len(v), shape, generator=g)] * (1 + 0.02 * torch.rand(shape, generator=g))).clamp(-86, 86).cuda()


def test_fp32_activations_far_from_zero(kda_lib):
    """sigmoid and SiLU of fp32 rows to 16 steps of 2^-24 at any argument: the exponential (4),
    what is put back of its argument's rounding, 1 + e, the reciprocal (2) and the products
    (and 48 for the norm itself)."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(5)
    x = far(g, 1, 60, 64)
    w = torch.tensor([0.0, 1.0]).repeat(64, 1).cuda()
    out = torch.empty_like(x)
    kda.kda_conv_fwd(x, w, None, out)
    ref = R.silu(R.d(x))
    within(out, ref, ref.abs(), 16, "convolution")
    rows, step = x.view(60, 1, 64), torch.empty(60, 1, 64, device="cuda")
    kda.kda_conv_fwd(rows, w, None, step)
    assert torch.equal(step.view_as(out), out)
    u, gate = torch.randn(40, 128, generator=g).cuda(), far(g, 40, 128)
    wn, o = torch.ones(128, device="cuda"), torch.empty(40, 128, device="cuda")
    for act in ("sigmoid", "silu"):
        kda.kda_postnorm_fwd(u, wn, gate, o, activation=act)
        ref = R.postnorm(u, wn, gate, None, 1.0, act, 1e-6)
        within(o, ref, ref.abs(), 64, "gated norm " + act)
    # a scan with steps of zero and D = 1: out = x silu(z)
    for T in (40, 1):
        z, y = far(g, 2, T, 64), torch.randn(2, T, 64, generator=g).cuda()
        B, out = torch.randn(2, T, 1, 16, generator=g).cuda(), torch.empty(2, T, 64, device="cuda")
        kda.kda_scan_fwd(y, torch.full_like(y, -200.0), torch.zeros(64, 16, device="cuda"), B, B, out,
                         torch.ones(64, device="cuda"), z)
        ref = R.d(y) * R.silu(R.d(z))
        within(out, ref, ref.abs(), 16, "scan")


@pytest.mark.parametrize("ty", [BF, F])
def test_activations_at_infinity(kda_lib, ty):
    """sigmoid is 1 and 0 at the infinities, and what is no number stays none."""
    import kimi_delta_attention_08_gb300 as kda
    inf = float("inf")
    gate = torch.tensor([inf, -inf, float("nan"), 1e30, -1e30, 0.0, 90.0, -200.0]).to(ty).cuda().repeat(3, 16)
    x, w = torch.randn(3, 128).to(ty).cuda(), torch.ones(128, device="cuda")
    gated, plain = torch.empty_like(x), torch.empty_like(x)
    kda.kda_postnorm_fwd(x, w, gate, gated)
    kda.kda_postnorm_fwd(x, w, None, plain)
    for i, f in ((0, 1.0), (1, 0.0), (3, 1.0), (4, 0.0), (5, 0.5), (6, 1.0), (7, 0.0)):
        assert torch.equal(gated[:, i::8], plain[:, i::8] * f), i
    assert gated[:, 2::8].isnan().all()
    r = kda.kda_postnorm_bwd(x, x, w, gate)["dgate"]
    for i in (0, 1, 3, 4, 7):
        assert not r[:, i::8].any(), i
    assert r[:, 2::8].isnan().all() and r[:, 5::8].isfinite().all()
