"""What the norm of the linear recurrence's errors tells apart, on the 64-bit form."""
import pytest
import torch

from tests.linrec_norm import near
from tests.linrec_ref import linrec


def whole(T, D, carry):
    """The 64-bit form, 128 tokens at a time, the state between them held in `carry`."""
    g = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, r, i = rnd(1, T, D), rnd(1, T, D), rnd(1, T, D)
    A = torch.log(-8 * torch.log(0.9 + 0.099 * torch.rand(D, generator=g)))
    h0, out = torch.zeros(1, D, dtype=torch.float64), []
    for p in range(0, T, 128):
        q = slice(p, min(p + 128, T))
        y, h0 = linrec(x[:, q], r[:, q], i[:, q], A, None, None, None, h0.to(carry), None)
        out.append(y)
    return torch.cat(out, 1), h0


@pytest.mark.parametrize("T", [2112, 4500])
def test_a_state_carried_in_too_few_bits_is_told(T):
    ref, rfin = whole(T, 40, torch.float64)
    out, fin = whole(T, 40, torch.float32)
    near(out.float(), ref, "out")
    near(fin.float(), rfin, "state")
    out, fin = whole(T, 40, torch.bfloat16)
    with pytest.raises(AssertionError, match="norm"):
        near(out.float(), ref, "out")
    with pytest.raises(AssertionError, match="norm"):
        near(fin.float(), rfin, "state")


def test_a_small_error_that_all_values_share_is_told():
    ref, _ = whole(1000, 40, torch.float64)
    near(ref.to(torch.bfloat16), ref, "out")
    with pytest.raises(AssertionError, match="norm"):
        near((ref * (1 + 2e-5)).float(), ref, "out")
    with pytest.raises(AssertionError, match="norm"):
        near((ref.to(torch.bfloat16) * 1.01).to(torch.bfloat16), ref, "out")
