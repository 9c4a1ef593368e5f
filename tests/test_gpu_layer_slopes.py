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
