"""A layer of a hybrid model from the library's operators, as a program runs it: norm, short
convolution, gated linear recurrence and gated norm, then norm and the gated feed-forward
product, with the projections between them as plain matrix products.  Prompt, single tokens with
carried states, and a training step; every operator's result is checked against its 64-bit
form on the inputs that it got there, within that operator's own bounds."""
import pytest
import torch

from tests import layer_ref as R
from tests.glu_ref import glu, within
from tests.linrec_ref import linrec

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
D, H, W = 192, 512, 4           # model width, feed-forward width, convolution width


class Layer:
    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, t=BF, k=1.0: (torch.randn(*s, generator=g) * k).to(t).cuda()  # noqa: E731
        self.n1, self.n2, self.n3 = (1 + r(D, t=F, k=0.1) for _ in range(3))
        self.p_in, self.p_out = r(4 * D, D, k=D ** -0.5), r(D, D, k=D ** -0.5)
        self.cw, self.cb = r(D, W, t=F, k=0.5), r(D, t=F, k=0.1)
        self.A, self.rb, self.ib = r(D, t=F, k=0.5) - 1, r(D, t=F), r(D, t=F)
        self.wg, self.wu, self.wd = r(H, D, k=D ** -0.5), r(H, D, k=D ** -0.5), r(D, H, k=H ** -0.5)

    def states(self, n):
        return torch.zeros(n, W - 1, D, dtype=BF, device="cuda"), torch.zeros(n, D, device="cuda")

    def forward(self, kda, x, conv, rec, cu=None, keep=False):
        """The layer on x [B, T, D], its states updated in place; returns all it computed."""
        B, T, _ = x.shape
        t = {"x": x}
        new = lambda *s, ty=BF: torch.empty(B, T, *s, dtype=ty, device="cuda")  # noqa: E731
        t["y"] = new(D)
        kda.kda_prenorm_fwd(x, None, self.n1, t["y"])
        proj = t["y"] @ self.p_in.T
        t["u"], t["r"], t["i"], t["z"] = proj.split(D, 2)
        t["conv0"], t["rec0"] = conv.clone(), rec.clone()
        t["c"] = torch.zeros(B, T, D, dtype=BF, device="cuda")
        kda.kda_conv_fwd(t["u"], self.cw, self.cb, t["c"], conv, conv, cu)
        t["o"] = torch.zeros(B, T, D, dtype=BF, device="cuda")
        t["cs"] = kda.make_linrec_states(B * T, D) if keep else None
        kda.kda_linrec_fwd(t["c"], t["r"], t["i"], self.A, t["o"], None, self.rb, self.ib, rec, rec, cu,
                           chunk_states=t["cs"])
        t["conv1"], t["rec1"] = conv.clone(), rec.clone()
        t["n"] = new(D)
        kda.kda_postnorm_fwd(t["o"], self.n2, t["z"].contiguous(), t["n"])
        t["m"] = t["n"] @ self.p_out.T
        t["res"], t["h"] = new(D), new(D)
        kda.kda_prenorm_fwd(t["m"], x, self.n3, t["h"], t["res"])
        t["f"], t["pre"] = new(H), new(2 * H) if keep else None
        kda.kda_glu_fwd(t["h"], self.wg, self.wu, t["f"], pre=t["pre"])
        t["out"] = t["res"] + t["f"] @ self.wd.T
        return t

    def check(self, t, cu):
        ends = t["x"].shape[1] if cu is None else cu[-1]
        live = lambda v: v[:, :ends]  # noqa: E731
        ref, _ = R.prenorm(t["x"], None, self.n1, 1.0, 1e-6)
        R.close(live(t["y"]), live(ref), live(ref).abs() * 2, 64, "norm")
        args = (t["u"], self.cw, self.cb, t["conv0"], cu, "silu")
        (ref, fin), mag = R.conv(*args), R.conv(*args, mag=True)[0]
        R.close(live(t["c"]), live(ref), live(mag), 16, "convolution")
        assert torch.equal(R.d(t["conv1"]), fin)
        args = (t["c"], t["r"], t["i"], self.A, None, self.rb, self.ib, t["rec0"], cu)
        (ref, fin), (mag, mfin) = linrec(*args), linrec(*args, mag=True)
        R.close(live(t["o"]), live(ref), live(mag), 8 * ends + 64, "recurrence")
        R.close(t["rec1"], fin, mfin, 8 * ends + 64, "its state")
        ref = R.postnorm(t["o"], self.n2, t["z"], None, 1.0, "sigmoid", 1e-6)
        R.close(t["n"], ref, ref.abs() * (2 + R.d(t["z"]).abs()), 64, "gated norm")
        ref, res = R.prenorm(t["m"], t["x"], self.n3, 1.0, 1e-6)
        R.close(t["res"], res, R.d(t["m"]).abs() + R.d(t["x"]).abs(), 8, "residual")
        R.close(t["h"], ref, ref.abs() * 2 + (R.d(t["m"]).abs() + R.d(t["x"]).abs()), 64, "second norm")
        within(t["f"], glu(t["h"], self.wg, self.wu, "silu")["out"], "feed-forward")


def prompt(T, seed=0, B=1):
    return torch.randn(B, T, D, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


@pytest.mark.parametrize("B,T,cu", [(2, 150, None), (1, 300, [0, 1, 1, 130, 300]), (1, 100, [0, 64, 90])])
def test_prompt(kda_lib, B, T, cu):
    import kimi_delta_attention_08_gb300 as kda
    layer = Layer()
    conv, rec = layer.states(B if cu is None else len(cu) - 1)
    conv.normal_(), rec.normal_()
    cud = None if cu is None else torch.tensor(cu, device="cuda")
    t = layer.forward(kda, prompt(T, B=B), conv, rec, cud)
    layer.check(t, cu)


def test_tokens_after_a_prompt(kda_lib):
    """Five sequences: a prompt of 70 tokens, then tokens one at a time with the carried states;
    the states that they end with are those of the whole sequence at once, up to what the
    chain's bf16 roundings leave (the inputs of the recurrence differ by them)."""
    import kimi_delta_attention_08_gb300 as kda
    layer, x = Layer(1), prompt(76, 3, 5)
    conv, rec = layer.states(5)
    layer.check(layer.forward(kda, x[:, :70].contiguous(), conv, rec), None)
    for t in range(70, 76):
        layer.check(layer.forward(kda, x[:, t:t + 1].contiguous(), conv, rec), None)
    conv2, rec2 = layer.states(5)
    layer.forward(kda, x, conv2, rec2)
    # the projections may sum in another order for one token: a step of bf16 of their largest values
    assert (conv.float() - conv2.float()).abs().max() <= 2 * 2.0 ** -8 * conv2.float().abs().max()
    assert (rec - rec2).norm() <= 0.01 * rec2.norm()


def backward(layer, kda, t, cu, dout):
    """The gradients of a forward that kept its states, operator by operator."""
    g = {"df": dout @ layer.wd}
    b = kda.kda_glu_bwd(t["h"], layer.wg, layer.wu, g["df"], pre=t["pre"])
    g["glu"] = b
    n = kda.kda_prenorm_bwd(b["dx"], dout, t["res"], layer.n3, t["m"])
    g["dn"] = (n["dx"] @ layer.p_out).contiguous()
    p = kda.kda_postnorm_bwd(g["dn"], t["o"], layer.n2, t["z"].contiguous())
    g["post"] = p
    g["rec"] = kda.kda_linrec_bwd(t["c"], t["r"], t["i"], layer.A, p["dx"], None, layer.rb, layer.ib,
                                  t["rec0"], None, cu, chunk_states=t["cs"])
    g["conv"] = kda.kda_conv_bwd(t["u"], layer.cw, layer.cb, g["rec"]["dx"], t["conv0"], None, cu)
    dproj = torch.cat([g["conv"]["dx"], g["rec"]["dr"], g["rec"]["di"], p["dgate"]], 2)
    first = kda.kda_prenorm_bwd((dproj @ layer.p_in).contiguous(), None, t["x"], layer.n1, t["x"])
    g["dx"] = n["dresidual"] + first["dx"]
    return g


@pytest.mark.parametrize("cu", [None, [0, 70, 70, 200]])
def test_training_step(kda_lib, cu):
    import kimi_delta_attention_08_gb300 as kda
    layer, T = Layer(2), 200
    conv, rec = layer.states(1 if cu is None else 3)
    cud = None if cu is None else torch.tensor(cu, device="cuda")
    t = layer.forward(kda, prompt(T, 5), conv, rec, cud, keep=True)
    g = backward(layer, kda, t, cud, prompt(T, 6))
    ref = glu(t["h"], layer.wg, layer.wu, "silu", g["df"], t["pre"])
    for k in ("dx", "dw_gate", "dw_up"):
        within(g["glu"][k], ref[k], k)
    args = (t["c"], t["r"], t["i"], layer.A, None, layer.rb, layer.ib, t["rec0"], cu)
    ref = linrec(*args, dout=g["post"]["dx"])
    mag = linrec(*args, dout=g["post"]["dx"], mag=True)
    for k in ref:
        R.close(g["rec"][k], ref[k], mag[k], 16 * T + 256 + (T if ref[k].dim() == 1 else 0), k)
    args = (t["u"], layer.cw, layer.cb, t["conv0"], cu, "silu", g["rec"]["dx"])
    ref, mag = R.conv(*args), R.conv(*args, mag=True)
    for k in ref:
        R.close(g["conv"][k], ref[k], mag[k], 16 + T, k)
    assert g["dx"].isfinite().all()


def test_captured_training_step(kda_lib):
    """The whole step in one graph, replayed on new inputs: the bits of a direct step."""
    import kimi_delta_attention_08_gb300 as kda
    layer, x, dout = Layer(3), prompt(200, 1), prompt(200, 2)

    def step():
        conv, rec = layer.states(1)
        t = layer.forward(kda, x, conv, rec, keep=True)
        g = backward(layer, kda, t, None, dout)
        return [t["out"], g["dx"], g["glu"]["dw_gate"], g["rec"]["dA_log"], g["rec"]["dr_bias"], g["conv"]["dweight"]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        outs = step()
    x.copy_(prompt(200, 8))
    gr.replay()
    torch.cuda.synchronize()
    for got, want in zip(outs, step()):
        assert torch.equal(got, want)


def calls(kda):
    """(name, call(stream)) of the operators that allocate what they return."""
    g = torch.Generator().manual_seed(3)
    r = lambda *s, t=BF: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    x, a, b, d = (r(2, 700, 256) for _ in range(4))
    A, init = r(256, t=F), r(2, 256, t=F)
    wg, wu, dh = r(384, 256), r(384, 256), r(2, 700, 384)
    return {"linrec": lambda s: kda.kda_linrec_bwd(x, a, b, A, d, None, A, A, init, stream=s),
            "glu": lambda s: kda.kda_glu_bwd(x, wg, wu, dh, stream=s)}


@pytest.mark.parametrize("name", ["linrec", "glu"])
def test_results_do_not_take_memory_that_is_still_read(kda_lib, name):
    """Tensors that were freed while the current stream still has to read them: a call on another
    stream right after that must not write its results or its workspace there."""
    import kimi_delta_attention_08_gb300 as kda
    run = calls(kda)[name]
    want = {k: v.clone() for k, v in run(None).items()}
    sizes = [v.numel() * v.element_size() for v in want.values()]
    s = torch.cuda.Stream()
    old = [(torch.arange(n, device="cuda") % 251).to(torch.uint8) for n in sizes * 2]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                       # some 50 ms
    kept = [t.clone() for t in old]                      # queued behind it
    del old
    got = run(s)
    torch.cuda.synchronize()
    for t, n in zip(kept, sizes * 2):
        assert torch.equal(t, (torch.arange(n, device="cuda") % 251).to(torch.uint8))
    for k, v in want.items():
        if k != "workspace":
            assert torch.equal(got[k], v), k


@pytest.mark.parametrize("name", ["linrec", "glu"])
def test_two_streams_at_once(kda_lib, name):
    """Calls that run side by side, each in its stream's memory: the bits of single calls, though
    the recurrence's tiles wait for one another on a GPU that others use too."""
    import kimi_delta_attention_08_gb300 as kda
    run = calls(kda)[name]
    want = {k: v.clone() for k, v in run(None).items() if k != "workspace"}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [run(s) for _ in range(20) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert kda.kda_get_device_status(g["workspace"]) == 0
        assert all(torch.equal(g[k], v) for k, v in want.items())


def test_feed_forward_beyond_32_bits(kda_lib):
    """More than 2^31 values in the output: rows from its start, middle and end."""
    import kimi_delta_attention_08_gb300 as kda
    M, K, N = 70000, 64, 32768
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, M, K, generator=g).to(BF).cuda()
    wg, wu = (torch.randn(N, K, generator=g).to(BF).cuda() / 8 for _ in range(2))
    out = torch.empty(1, M, N, dtype=BF, device="cuda")
    kda.kda_glu_fwd(x, wg, wu, out)
    rows = [0, 1, 255, 256, 35001, 65535, 65536, 69998, 69999]
    within(out[:, rows], glu(x[:, rows], wg, wu, "silu")["out"], "out")


def test_recurrence_beyond_32_bits(kda_lib):
    """More than 2^31 values: its last rows depend on some hundred tokens, so a call on the last
    2,000 alone gives them too, up to what its other tiles round differently."""
    import kimi_delta_attention_08_gb300 as kda
    T, C, n = (1 << 19) + 130, 4104, 2000
    x = torch.empty(1, T, C, dtype=BF, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for p in range(0, T, 1 << 16):
        x[:, p:p + (1 << 16)] = torch.randn(1, min(1 << 16, T - p), C, generator=g, device="cuda").to(BF)
    A = torch.zeros(C, device="cuda")
    out = torch.empty_like(x)
    ws = kda.make_linrec_workspace(1, T, C)
    fin, fin2 = torch.empty(1, C, device="cuda"), torch.empty(1, C, device="cuda")
    kda.kda_linrec_fwd(x, x, x, A, out, final_state=fin, workspace=ws)
    assert kda.kda_get_device_status(ws) == 0
    tail, o2 = x[:, -n:].contiguous(), torch.empty(1, n, C, dtype=BF, device="cuda")
    kda.kda_linrec_fwd(tail, tail, tail, A, o2, final_state=fin2)
    # states of size one, a few hundred roundings of 2^-24 that decay; outputs a step of bf16 apart
    assert (fin - fin2).abs().max() < 1e-4
    a, b = out[:, -64:].float(), o2[:, -64:].float()
    assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-4).all()
