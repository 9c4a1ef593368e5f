"""The gated feed-forward product against its 64-bit form: every size at which the 256 x 256
tiles of 64 wide steps are cut off, activations, kept pre-activations, slices, no rows.
The bounds are derived in tests/glu_ref.py."""
import time

import pytest
import torch

from tests.glu_ref import glu, within

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# rows, dim, hidden: ragged and whole tiles, one step and many, more tiles than pairs of CTAs;
# up to 128 rows the forward splits the summed axis over clusters of 1 to 8, with a part left over
SIZES = [(1, 8, 8), (3, 64, 128), (17, 72, 136), (127, 200, 264), (128, 256, 128), (129, 128, 256),
         (256, 512, 512), (257, 520, 248), (300, 1000, 640), (513, 64, 2056), (1100, 264, 1032),
         (2, 1032, 200), (33, 2112, 72), (128, 4104, 1608), (64, 4096, 9800)]


def make(M, D, Fh, seed=0, B=1, wide=0):
    g = torch.Generator().manual_seed(seed + M + D + Fh)
    r = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(BF).cuda()  # noqa: E731
    x = r(B, M, D + wide)[..., :D]
    return x, r(Fh, D, k=D ** -0.5), r(Fh, D, k=D ** -0.5), r(B, M, Fh)


@pytest.mark.parametrize("fn", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("size", SIZES)
def test_forward(kda_lib, size, fn):
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(*size)
    out, pre = torch.full_like(dout, float("nan")), torch.full((1, size[0], 2 * size[2]), float("nan"), dtype=BF, device="cuda")
    ws = torch.full((256,), 0x5A, dtype=torch.uint8, device="cuda")
    kda.kda_glu_fwd(x, wg, wu, out, ws, activation=fn)
    assert kda.kda_get_device_status(ws) == 0
    ref = glu(x, wg, wu, fn)
    within(out, ref["out"], "out")
    again = torch.empty_like(out)
    kda.kda_glu_fwd(x, wg, wu, again, pre=pre, activation=fn)
    assert torch.equal(again, out)
    within(pre, ref["pre"], "pre")


@pytest.mark.parametrize("fn", ["silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_backward(kda_lib, size, fn, kept):
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(*size, seed=1)
    pre = None
    if kept:
        pre = torch.empty(1, size[0], 2 * size[2], dtype=BF, device="cuda")
        kda.kda_glu_fwd(x, wg, wu, torch.empty_like(dout), pre=pre, activation=fn)
    g = kda.kda_glu_bwd(x, wg, wu, dout, pre=pre, activation=fn)
    assert kda.kda_get_device_status(g["workspace"]) == 0
    ref = glu(x, wg, wu, fn, dout, pre)
    for k in ("dx", "dw_gate", "dw_up"):
        within(g[k], ref[k], k)


@pytest.mark.parametrize("size", [(97, 136, 6160), (300, 264, 2056), (3100, 264, 520), (3100, 1032, 2560)])
def test_tiles_that_several_pairs_compute(kda_lib, size):
    """Sizes at which dx's tiles (the first two), the weights' (the third) or the last turn of both are
    split along the summed axis: in a workspace of anything, and twice in the same one, the same
    gradients bit for bit."""
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(*size, seed=3)
    ref = glu(x, wg, wu, "silu", dout)
    ws = kda.make_glu_bwd_workspace(size[0], size[2])
    ws.fill_(0xFF)
    first = None
    for _ in range(4):
        g = kda.kda_glu_bwd(x, wg, wu, dout, ws)
        assert kda.kda_get_device_status(ws) == 0
        got = {k: v for k, v in g.items() if k != "workspace"}
        if first is None:
            first = got
            for k, v in got.items():
                within(v, ref[k], k)
        for k, v in got.items():
            assert torch.equal(v, first[k]), k


@pytest.mark.parametrize("fn", ["silu", "gelu"])
@pytest.mark.parametrize("size", [(200, 1000, 9800), (256, 136, 12288), (129, 72, 14592), (600, 264, 4008)])
def test_wide_tiles(kda_lib, size, fn):
    """Sizes whose tiles of 128 columns take a second turn: they are 160 (the first and the last) or
    192 wide, with fewer and more steps than stages; kept values, and a backward that computes
    them again."""
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(*size, seed=4)
    out, pre = torch.full_like(dout, float("nan")), torch.full((1, size[0], 2 * size[2]), float("nan"), dtype=BF, device="cuda")
    kda.kda_glu_fwd(x, wg, wu, out, pre=pre, activation=fn)
    ref = glu(x, wg, wu, fn, dout)
    within(out, ref["out"], "out")
    within(pre, glu(x, wg, wu, fn)["pre"], "pre")
    again = torch.full_like(dout, float("nan"))
    kda.kda_glu_fwd(x, wg, wu, again, activation=fn)
    assert torch.equal(again, out)
    g = kda.kda_glu_bwd(x, wg, wu, dout, activation=fn)
    assert kda.kda_get_device_status(g["workspace"]) == 0
    for k in ("dx", "dw_gate", "dw_up"):
        within(g[k], ref[k], k)


def test_many_tiles_in_batches_and_slices(kda_lib):
    """More tiles than pairs of CTAs in every pass, two sequences, rows of a wider projection,
    both weights as parts of one matrix."""
    import kimi_delta_attention_08_gb300 as kda
    x, _, _, dout = make(1500, 1224, 2200, B=2, wide=40)
    w = (torch.randn(4400, 1224, generator=torch.Generator().manual_seed(2)) / 35).to(BF).cuda()
    wg, wu = w[:2200], w[2200:]
    out = torch.empty_like(dout)
    kda.kda_glu_fwd(x, wg, wu, out)
    g = kda.kda_glu_bwd(x, wg, wu, dout)
    ref = glu(x, wg, wu, "silu", dout)
    within(out, ref["out"], "out")
    for k in ("dx", "dw_gate", "dw_up"):
        within(g[k], ref[k], k)


def test_nothing_beyond_the_outputs_is_written(kda_lib):
    """Outputs in the middle of a larger buffer: what lies before and behind them stays."""
    import kimi_delta_attention_08_gb300 as kda
    M, D, Fh = 130, 136, 264
    x, wg, wu, dout = make(M, D, Fh)
    for n, call in ((M * Fh, lambda o: kda.kda_glu_fwd(x, wg, wu, o.view(1, M, Fh))),):
        buf = torch.full((n + 8192,), 7.0, dtype=BF, device="cuda")
        call(buf[4096:4096 + n])
        assert (buf[:4096] == 7).all() and (buf[4096 + n:] == 7).all()
    pre = torch.full((M * 2 * Fh + 8192,), 7.0, dtype=BF, device="cuda")
    kda.kda_glu_fwd(x, wg, wu, torch.empty_like(dout), pre=pre[4096:-4096].view(1, M, 2 * Fh))
    assert (pre[:4096] == 7).all() and (pre[-4096:] == 7).all()


def test_no_rows(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(0, 64, 128)
    kda.kda_glu_fwd(x, wg, wu, dout)
    g = kda.kda_glu_bwd(x, wg, wu, dout)
    assert g["dx"].shape == x.shape and (g["dw_gate"] == 0).all() and (g["dw_up"] == 0).all()


def test_a_row_that_is_not_finite_stays_alone(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(300, 128, 256)
    want, got = torch.empty_like(dout), torch.empty_like(dout)
    kda.kda_glu_fwd(x, wg, wu, want)
    wdx = kda.kda_glu_bwd(x, wg, wu, dout)["dx"]
    x[0, 131, 5] = float("nan")
    kda.kda_glu_fwd(x, wg, wu, got)
    dx = kda.kda_glu_bwd(x, wg, wu, dout)["dx"]
    keep = torch.arange(300, device="cuda") != 131
    assert torch.equal(got[0, keep], want[0, keep]) and torch.equal(dx[0, keep], wdx[0, keep])
    assert got[0, 131].isnan().all() and dx[0, 131].isnan().all()


@pytest.mark.parametrize("fn", ["silu", "gelu", "sigmoid"])
def test_far_arguments(kda_lib, fn):
    """Pre-activations of up to 200: values and slopes near saturation and far from zero."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(4)
    x = torch.randn(1, 64, 64, generator=g).to(BF).cuda()
    wg = (torch.randn(256, 64, generator=g) * torch.logspace(-3, 0.7, 256)[:, None]).to(BF).cuda()
    wu = torch.randn(256, 64, generator=g).to(BF).cuda()
    dout = torch.randn(1, 64, 256, generator=g).to(BF).cuda()
    out = torch.empty_like(dout)
    kda.kda_glu_fwd(x, wg, wu, out, activation=fn)
    got = kda.kda_glu_bwd(x, wg, wu, dout, activation=fn)
    ref = glu(x, wg, wu, fn, dout)
    within(out, ref["out"], "out")
    for k in ("dx", "dw_gate", "dw_up"):
        within(got[k], ref[k], k)


def test_kept_values_of_every_size(kda_lib):
    """Pre-activations from 2^-36 to 2^34 of both signs, zero and NaN, as they are kept: within
    half a step, and not a number beyond 2^32."""
    import kimi_delta_attention_08_gb300 as kda
    from tests.glu_ref import kept_values
    e = torch.arange(-36, 35)
    w = torch.zeros(8 * len(e) + 16, 8)
    w[:8 * len(e), 0] = torch.ldexp(torch.tensor([1.0, -1, 1.25, -1.5, 1.75, 1.9921875, -1.0078125, 1.5]).repeat(len(e)),
                                    e.repeat_interleave(8))
    x = torch.zeros(1, 200, 8, dtype=BF)
    x[..., 0] = 1
    x[0, 1, 0], x[0, 2, 0] = 0, float("nan")
    w, x = w.to(BF).cuda(), x.cuda()
    for rows in (5, 200):       # both kernels
        out, pre = (torch.empty(1, rows, k * len(w), dtype=BF, device="cuda") for k in (1, 2))
        kda.kda_glu_fwd(x[:, :rows].contiguous(), w, w, out, pre=pre)
        got, want = kept_values(pre)[0, 0, :len(w)], w[:, 0].cpu().double()
        small = want.abs() < 2.0 ** 32
        assert got[~small].isnan().all()
        # half a step: of the value, or of the smallest exponent's fraction
        assert ((got - want).abs()[small] <= torch.clamp(want.abs()[small] * 2.0 ** -10, min=2.0 ** -40)).all()
        assert (kept_values(pre)[0, 1] == 0).all() and kept_values(pre)[0, 2].isnan().all()


@pytest.mark.parametrize("rows", [5, 300])
def test_a_wait_that_runs_out_is_reported(kda_lib, rows):
    """Nothing is loaded: the products and the epilogue give up, and the next call is right."""
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(rows, 1024 if rows == 5 else 128, 256)
    out, ws = torch.empty_like(dout), torch.empty(256, dtype=torch.uint8, device="cuda")
    t0 = time.time()
    kda.kda_glu_fwd(x, wg, wu, out, ws, debug_stall=True)
    assert kda.kda_get_device_status(ws) == 8
    g = kda.kda_glu_bwd(x, wg, wu, dout, debug_stall=True)
    assert kda.kda_get_device_status(g["workspace"]) == 8
    assert time.time() - t0 < 10
    kda.kda_glu_fwd(x, wg, wu, out, ws)
    assert kda.kda_get_device_status(ws) == 0
    within(out, glu(x, wg, wu, "silu")["out"], "out")


def test_runs_are_the_same_bits_and_captured(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    x, wg, wu, dout = make(700, 512, 1024)
    out, pre = torch.empty_like(dout), torch.empty(1, 700, 2048, dtype=BF, device="cuda")
    ws = kda.make_glu_bwd_workspace(700, 1024)

    def step():
        kda.kda_glu_fwd(x, wg, wu, out, pre=pre)
        return kda.kda_glu_bwd(x, wg, wu, dout, ws, pre=pre)
    first = {k: v.clone() for k, v in step().items() if k != "workspace"}
    first["out"] = out.clone()
    for _ in range(5):
        g = step()
        assert all(torch.equal(v, out if k == "out" else g[k]) for k, v in first.items())
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        g = step()
    x.copy_(torch.randn_like(x))
    gr.replay()
    torch.cuda.synchronize()
    got = {k: v.clone() for k, v in g.items() if k != "workspace"}
    got["out"] = out.clone()
    g = step()
    assert all(torch.equal(v, out if k == "out" else g[k]) for k, v in got.items())
