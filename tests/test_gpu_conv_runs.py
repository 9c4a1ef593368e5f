"""The convolution at every length of run that its rule on the number of values can choose
(forward 8, 16, 32 and 64 tokens, backward 8 to 256): sequences whose ends lie inside runs, off
multiples of 8, shorter than the window and longer than several runs, where the ring of rows
in shared memory turns many times, in both types and on both paths.

Bounds: as in tests/test_gpu_conv.py; a weight's gradient is added over a run's tokens, over 4
warps, over every 32nd row block and over 32 of those: run + 36 + blocks / 32 steps of 2^-24,
and 16 for each term."""
import pytest
import torch

from tests import layer_ref as R

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def lengths(total):
    """Uneven sequences that add up to at most `total`: around runs of 8 to 256 tokens."""
    cu, i = [0], 0
    want = [1, 263, 0, 2, 129, 517, 64, 31, 3, 95, 255, 16, 7, 190]
    while cu[-1] + want[i % len(want)] <= total:
        cu.append(cu[-1] + want[i % len(want)])
        i += 1
    return cu


def make(T, C, ty, cu, seed, W=4):
    g = torch.Generator().manual_seed(seed)
    N = 1 if cu is None else len(cu) - 1
    r = lambda *s, t=ty: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    return (r(1, T, C), r(C, W, t=F), r(C, t=F), r(N, W - 1, C), r(1, T, C), r(N, W - 1, C),
            None if cu is None else torch.tensor(cu, device="cuda"))


# tokens x channels on each side of the rule's borders: below 3, 8 and 20 million values
FORWARD = [(8, 700, 4096), (16, 1000, 4096), (32, 1500, 8192), (64, 1800, 12288), (64, 1300, 16001)]


@pytest.mark.parametrize("run,T,C", FORWARD)
@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("packed", [False, True])
def test_forward_runs(kda_lib, run, T, C, ty, packed):
    import kimi_delta_attention_08_gb300 as kda
    assert run == (8 if T * C < 3e6 else 16 if T * C < 8e6 else 32 if T * C < 20e6 else 64)
    cu = lengths(T - 5) if packed else None
    x, w, b, init, _, _, cud = make(T, C, ty, cu, T + C)
    out, fin = torch.full_like(x, float("nan")), torch.full_like(init, float("nan"))
    kda.kda_conv_fwd(x, w, b, out, init, fin, cud)
    ref, rfin = R.conv(x, w, b, init, cu, "silu")
    mag, _ = R.conv(x, w, b, init, cu, "silu", mag=True)
    end = T if cu is None else cu[-1]
    R.close(out[:, :end], ref[:, :end], mag[:, :end], 16, "out")
    assert out[:, end:].isnan().all()
    assert torch.equal(R.d(fin), rfin)


# below 1.5, 4, 7, 12 and 300 million values
BACKWARD = [(8, 300, 4096), (16, 700, 4096), (32, 1200, 4096), (64, 2000, 4096), (128, 1100, 12288),
            (128, 900, 16001)]


@pytest.mark.parametrize("run,T,C", BACKWARD)
@pytest.mark.parametrize("ty,dty", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("packed", [False, True])
def test_backward_runs(kda_lib, run, T, C, ty, dty, packed):
    import kimi_delta_attention_08_gb300 as kda
    v = T * C / 1e6
    assert run == (8 if v < 1.5 else 16 if v < 4 else 32 if v < 7 else 64 if v < 12 else 128)
    cu = lengths(T - 5) if packed else None
    x, w, b, init, dout, dfin, cud = make(T, C, ty, cu, T + C + 1)
    dout = dout.to(dty)
    g = kda.kda_conv_bwd(x, w, b, dout, init, dfin, cud)
    args = (x, w, b, init, cu, "silu", dout, dfin)
    ref, mag = R.conv(*args), R.conv(*args, mag=True)
    steps = 16 + run + 36 + T / (4 * run) / 32
    for nm in ref:
        R.close(g[nm], ref[nm], mag[nm], 16 if nm in ("dx", "dinitial_state") else steps, nm)


@pytest.mark.parametrize("packed", [False, True])
def test_backward_longest_run(kda_lib, packed):
    """256 tokens a run, from 300 million values on: all gradients at some of the channels, in
    64 bits on the GPU's own inputs."""
    import kimi_delta_attention_08_gb300 as kda
    T, C = 9203, 32768
    assert T * C >= 300e6
    cu = lengths(T - 5) if packed else None
    gen = torch.Generator("cuda").manual_seed(1)
    N = 1 if cu is None else len(cu) - 1
    r = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda").normal_(generator=gen)  # noqa: E731
    x, w, b, init, dout, dfin = r(1, T, C), r(C, 4, t=F), r(C, t=F), r(N, 3, C), r(1, T, C), r(N, 3, C)
    g = kda.kda_conv_bwd(x, w, b, dout, init, dfin, None if cu is None else torch.tensor(cu, device="cuda"))
    at = torch.tensor([0, 1, 2, 3, 127, 128, 5000, 16383, 16384, 32764, 32765, 32766, 32767], device="cuda")
    args = (x[..., at], w[at], b[at], init[..., at], cu, "silu", dout[..., at], dfin[..., at])
    ref, mag = R.conv(*args), R.conv(*args, mag=True)
    steps = 16 + 256 + 36 + T / 1024 / 32
    for nm, got in (("dx", g["dx"][..., at]), ("dinitial_state", g["dinitial_state"][..., at]),
                    ("dweight", g["dweight"][at]), ("dbias", g["dbias"][at])):
        R.close(got, ref[nm], mag[nm], 16 if nm in ("dx", "dinitial_state") else steps, nm)
