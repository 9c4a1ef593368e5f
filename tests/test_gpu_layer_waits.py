"""What a wait that ran out leaves where nobody reads a status word: no number, not a plausible
value.  (The test's hook makes the wait run out: a result that is never handed on, tiles that are
never loaded.)"""
import pytest
import torch

from tests import test_gpu_glu as G
from tests import test_gpu_linrec as L

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("ty,dim", [(BF, 64), (BF, 33), (F, 40)])
@pytest.mark.parametrize("T", [700, 4500])
def test_recurrence(kda_lib, T, ty, dim):
    """Every tile but the first one waits for it, directly or through those between."""
    import kimi_delta_attention_08_gb300 as kda
    a, b, dout, dfin, _ = L.make((1, T, None), dim, ty, 2)
    out, fin = torch.zeros_like(dout), torch.zeros_like(dfin)
    kda.kda_linrec_fwd(**a, out=out, **b, final_state=fin, debug_stall=True)
    assert out[:, :128].isfinite().all()
    assert out[:, 128:].isnan().all() and fin.isnan().all()
    g = kda.kda_linrec_bwd(**a, dout=dout, **b, dfinal_state=dfin, debug_stall=True)
    last = (T - 1) // 64 * 64
    assert g["dx"][:, last:].isfinite().all()
    for k in ("dx", "dr", "di"):
        assert g[k][:, :last].isnan().all(), k
    for k in ("dA_log", "dr_bias", "di_bias", "dinitial_state"):
        assert g[k].isnan().all(), k
    want, got = torch.empty_like(out), torch.empty_like(out)
    kda.kda_linrec_fwd(**a, out=want, **b)
    kda.kda_linrec_fwd(**a, out=got, **b)
    assert want.isfinite().all() and torch.equal(got, want)


@pytest.mark.parametrize("size", [(5, 1024, 256), (128, 256, 128), (300, 128, 256), (200, 1000, 9800), (1100, 264, 4104)])
@pytest.mark.parametrize("keep", [False, True])
def test_feed_forward(kda_lib, size, keep):
    """Few rows, tiles of both widths, more tiles than pairs."""
    import kimi_delta_attention_08_gb300 as kda
    from tests.glu_ref import glu, kept_values, within
    x, wg, wu, dout = G.make(*size)
    out = torch.zeros_like(dout)
    pre = torch.zeros(1, size[0], 2 * size[2], dtype=BF, device="cuda") if keep else None
    kda.kda_glu_fwd(x, wg, wu, out, pre=pre, debug_stall=True)
    assert out.isnan().all()
    if keep:
        assert kept_values(pre).isnan().all()
    kda.kda_glu_fwd(x, wg, wu, out, pre=pre)
    ref = glu(x, wg, wu, "silu")
    within(out, ref["out"], "out")
    if keep:
        within(pre, ref["pre"], "pre")
