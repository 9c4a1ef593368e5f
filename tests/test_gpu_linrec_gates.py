"""The backward of the gated linear recurrence where a gate is not a number, infinite or far out."""
import pytest
import torch

from tests import layer_ref as R
from tests.linrec_ref import linrec
from tests.test_gpu_linrec import make, ref_args

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("ty,dim", [(BF, 64), (BF, 33), (F, 40)])
@pytest.mark.parametrize("gate", ["r", "i"])
@pytest.mark.parametrize("row", [150, 299, 90, 0])
def test_a_gate_that_is_no_number(kda_lib, gate, row, ty, dim):
    """Within its sequence and channel what the 64-bit form makes of it, at a row within a sequence, at
    the last one, at a sequence's only one and at the first of all; elsewhere the same bits."""
    import kimi_delta_attention_08_gb300 as kda
    cu, T, ch = [0, 90, 91, 300, 430], 430, 7
    a, b, dout, dfin, cud = make((1, T, cu), dim, ty, 2)
    run = lambda: kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud)  # noqa: E731
    want = run()
    a[gate][0, row, ch] = float("nan")
    st = kda.make_linrec_states(T, dim)
    kda.kda_linrec_fwd(**a, out=torch.empty_like(dout), **b, cu_seqlens=cud, chunk_states=st)
    saved = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, cu_seqlens=cud, chunk_states=st)
    got, ref = run(), linrec(*ref_args(a, b, cu), dout=dout, dfin=dfin)
    n = next(n for n in range(4) if cu[n] <= row < cu[n + 1])
    here = torch.zeros(1, T, dim, dtype=torch.bool, device="cuda")
    here[0, cu[n]:cu[n + 1], ch] = True
    for k in ("dx", "dr", "di", "dz"):
        assert torch.equal(got[k].isnan().cpu(), ref[k].isnan()), k
        assert torch.equal(saved[k].isnan().cpu(), ref[k].isnan()), k
        assert torch.equal(got[k][~here], want[k][~here]), k
    for k in ("dx", "dr", "di"):
        assert got[k][0, row, ch].isnan(), k
    only = torch.arange(dim, device="cuda") != ch
    for k in ("dA_log", "dr_bias", "di_bias"):
        assert got[k][ch].isnan() and torch.equal(got[k][only], want[k][only]), k
    assert torch.equal(got["dinitial_state"].isnan().cpu(), ref["dinitial_state"].isnan())


FAR_R = [-200.0, -87.0, -85.0, -60.0, -9.0, 0.0, 9.0, 60.0, 85.0, 200.0]
FAR_I = [-200.0, -78.0, -60.0, -9.0, 0.0, 9.0, 60.0, 85.0, 200.0]


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("T", [3, 200])
def test_gates_far_out(kda_lib, ty, T):
    """A decay gate down to e^-87 and an input gate down to e^-78, which fp32 holds as they are computed
    (the input gate's sigmoid comes scaled by 2^-12), and beyond the range on both sides, where
    they are 0 and 1: gradients within the bound of tests/test_gpu_linrec.py.  Infinite gates give
    the same bits as those beyond the range."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(5)
    pick = lambda vals: torch.tensor(vals)[torch.randint(len(vals), (2, T, 64), generator=g)].to(ty).cuda()  # noqa: E731
    rnd = lambda t=ty: torch.randn(2, T, 64, generator=g).to(t).cuda()  # noqa: E731
    a = dict(x=rnd(), r=pick(FAR_R), i=pick(FAR_I), A_log=torch.linspace(-1, 2, 64).cuda())
    b = dict(z=rnd(), r_bias=None, i_bias=None, initial_state=torch.randn(2, 64, generator=g).cuda())
    dout = rnd()
    got = kda.kda_linrec_bwd(**a, dout=dout, **b)
    ref = linrec(*ref_args(a, b, None), dout=dout)
    mag = linrec(*ref_args(a, b, None), dout=dout, mag=True)
    for k in ref:
        if k in got:
            R.close(got[k], ref[k], mag[k], 16 * T + 256 + (2 * T if ref[k].dim() == 1 else 0), k)
    for nm in ("r", "i"):
        v = a[nm]
        a[nm] = torch.where(v.abs() == 200, v * float("inf"), v)
    inf = kda.kda_linrec_bwd(**a, dout=dout, **b)
    for k in got:
        if k != "workspace":
            assert torch.equal(inf[k], got[k]), k
