"""What a wait that ran out leaves where nobody reads a status word: no number, not a plausible
value.  (The test's hook makes the wait run out: a result that is never handed on.)"""
import pytest
import torch

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
