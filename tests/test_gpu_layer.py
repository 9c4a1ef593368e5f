"""The layer operators together and with kda_fwd / kda_bwd, as a layer runs them: prompts,
single tokens and training; captured graphs; streams; buffers beyond 2^31 elements.

Each operator of a chain is compared with its 64-bit form on the inputs that it really got
(the stages before it store bf16), at its own bound; the recurrence with its oracle."""
import numpy as np
import pytest
import torch

import oracle
from tests import layer_ref as R
from tests.kda_testutil import CHUNK_BWD_TOL, OUT_TOL, STATE_TOL

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32
EPS = 1e-6


def bits(t):
    return t.detach().cpu().contiguous().view(torch.int16).numpy().view(np.uint16)


class Layer:
    """A KDA layer's weights; H heads of 128, input width d."""

    def __init__(self, d=256, H=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, k=1.0, t=F: (torch.randn(*s, generator=g) * k).to(t).cuda()  # noqa: E731
        self.d, self.H, self.C = d, H, 3 * H * 128
        self.w_in, self.w_post = 1 + r(d, k=0.1), 1 + r(128, k=0.1)
        self.proj = r(d, self.C + 2 * H * 128 + H, k=d ** -0.5, t=BF)   # q, k, v | g | gate | beta
        self.conv_w, self.conv_b = r(self.C, 4, k=0.5), r(self.C, k=0.1)
        self.proj_out = r(H * 128, d, k=(H * 128) ** -0.5, t=BF)
        self.A_log, self.dt_bias = r(H), r(H, 128)
        self.rnd = r

    def forward(self, kda, x, res, cu, conv_state, state, in_place=False):
        B, T = x.shape[:2]
        H, HD, C = self.H, self.H * 128, self.C
        N = B if cu is None else cu.numel() - 1
        s = {"x": x, "res": res}
        s["h"], s["y"] = torch.empty_like(res), torch.empty_like(x)
        kda.kda_prenorm_fwd(x, res, self.w_in, s["y"], s["h"], res_scale=0.5, eps=EPS)
        p = s["p"] = s["y"] @ self.proj
        s["qkv"] = p[..., :C]                                        # slices of one projection
        s["g"] = p[..., C:C + HD].reshape(B, T, H, 128).contiguous()
        s["gate"] = p[..., C + HD:C + 2 * HD].unflatten(2, (H, 128))
        s["beta"] = p[..., C + 2 * HD:].contiguous()
        qkv = [torch.empty(B, T, H, 128, dtype=BF, device="cuda") for _ in range(3)]
        s["conv_in"], s["state_in"] = conv_state, state
        s["conv_out"] = conv_state if in_place else torch.empty_like(conv_state)
        s["state_out"] = state if in_place else torch.empty_like(state)
        kda.kda_conv_fwd(s["qkv"], self.conv_w, self.conv_b, qkv, conv_state, s["conv_out"], cu)
        s["q"], s["k"], s["v"] = qkv
        s["o"] = torch.empty_like(s["v"])
        s["ws"] = kda.make_workspace(B * T, H)
        kda.kda_fwd(*qkv, s["g"], s["beta"], 128 ** -0.5, s["o"], self.A_log, self.dt_bias, -5.0, state,
                    s["state_out"], cu, s["ws"])
        s["n"] = torch.empty_like(s["o"])
        kda.kda_postnorm_fwd(s["o"], self.w_post, s["gate"], s["n"], eps=EPS)
        s["out"] = s["n"].flatten(2) @ self.proj_out
        return s

    def states(self, N):
        return self.rnd(N, 3, self.C, t=BF), self.rnd(N, self.H, 128, 128, k=0.1)


def check_forward(L, s, cu, conv_in, state_in):
    ref, h = R.prenorm(s["x"], s["res"], L.w_in, 0.5, EPS)
    R.close(s["y"], ref, ref.abs() * 2, 64, "prenorm")
    cul = None if cu is None else cu.tolist()
    args = (s["qkv"], L.conv_w, L.conv_b, conv_in, cul, "silu")
    (out, fin), (mag, _) = R.conv(*args), R.conv(*args, mag=True)
    got = torch.cat([s[k].flatten(2) for k in "qkv"], 2)
    R.close(got, out, mag, 16, "conv")
    assert torch.equal(R.d(s["conv_out"]), fin)
    o, f, _ = oracle.fwd(bits(s["q"]), bits(s["k"]), bits(s["v"]), bits(s["g"]), bits(s["beta"]),
                         L.A_log.cpu().numpy(), L.dt_bias.cpu().numpy(), -5.0, 128 ** -0.5,
                         state_in.cpu().numpy(), None if cu is None else cu.cpu().numpy(), want_final=True)
    eo = np.abs(R.d(s["o"]).numpy().reshape(o.shape) - o).max() / np.abs(o).max()
    es = np.linalg.norm(R.d(s["state_out"]).numpy() - f) / np.linalg.norm(f)
    assert eo <= OUT_TOL and es <= STATE_TOL, (eo, es)
    ref = R.postnorm(s["o"], L.w_post, s["gate"], None, 1.0, "sigmoid", EPS)
    R.close(s["n"], ref, ref.abs() * (2 + R.d(s["gate"]).abs()), 64, "postnorm")


@pytest.mark.parametrize("cu", [None, [0, 1, 1, 40, 130]])
def test_kda_layer_prompt(kda_lib, cu):
    import kimi_delta_attention_08_gb300 as kda
    L = Layer()
    B, T = (2, 70) if cu is None else (1, 130)
    cud = None if cu is None else torch.tensor(cu, device="cuda")
    x, res = L.rnd(B, T, L.d, t=BF), L.rnd(B, T, L.d, t=BF)
    conv_state, state = L.states(B if cu is None else len(cu) - 1)
    s = L.forward(kda, x, res, cud, conv_state, state)
    assert kda.kda_get_device_status(s["ws"]) == 0
    check_forward(L, s, cud, conv_state, state)


def test_kda_layer_decode(kda_lib):
    """Single tokens with both states updated in place, each step against its reference."""
    import kimi_delta_attention_08_gb300 as kda
    L = Layer(seed=1)
    conv_state, state = L.states(5)
    for _ in range(3):
        before = conv_state.clone(), state.clone()
        x, res = L.rnd(5, 1, L.d, t=BF), L.rnd(5, 1, L.d, t=BF)
        s = L.forward(kda, x, res, None, conv_state, state, in_place=True)
        check_forward(L, s, None, *before)


def test_kda_layer_training(kda_lib):
    """The chain backwards: the gated norm, kda_bwd, the convolution fed with kda_bwd's fp32
    dq, dk and dv as they are, and the norm before the block."""
    import kimi_delta_attention_08_gb300 as kda
    L = Layer(seed=2)
    B, T, H = 2, 100, L.H
    x, res = L.rnd(B, T, L.d, t=BF), L.rnd(B, T, L.d, t=BF)
    conv_state, state = L.states(B)
    s = L.forward(kda, x, res, None, conv_state, state)
    dn, dh = L.rnd(B, T, H, 128, t=BF), L.rnd(B, T, L.d, t=BF)
    gp = kda.kda_postnorm_bwd(dn, s["o"], L.w_post, s["gate"], eps=EPS)
    ref, mag = R.postnorm_bwd(dn, s["o"], L.w_post, s["gate"], 1.0, "sigmoid", EPS)
    for nm in ref:
        R.close(gp[nm], ref[nm], mag[nm], 64 + (B * T * H if nm == "dweight" else 0), nm)
    gk = kda.kda_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], 128 ** -0.5, L.A_log, L.dt_bias, -5.0,
                     gp["dx"], state)
    assert kda.kda_get_device_status(gk["workspace"]) == 0
    want = oracle.bwd(bits(s["q"]), bits(s["k"]), bits(s["v"]), bits(s["g"]), bits(s["beta"]),
                      L.A_log.cpu().numpy(), L.dt_bias.cpu().numpy(), -5.0, 128 ** -0.5, bits(gp["dx"]),
                      state.cpu().numpy(), None, None)
    for nm in ("dq", "dk", "dv", "dg"):
        e = np.abs(R.d(gk[nm]).numpy().reshape(want[nm].shape) - want[nm]).max() / np.abs(want[nm]).max()
        assert e <= CHUNK_BWD_TOL, (nm, e)
    dqkv = [gk["dq"], gk["dk"], gk["dv"]]
    gc = kda.kda_conv_bwd(s["qkv"], L.conv_w, L.conv_b, dqkv, conv_state)
    args = (s["qkv"], L.conv_w, L.conv_b, conv_state, None, "silu", torch.cat([t.flatten(2) for t in dqkv], 2))
    ref, mag = R.conv(*args), R.conv(*args, mag=True)
    for nm in ref:
        R.close(gc[nm], ref[nm], mag[nm], 16 if nm in ("dx", "dinitial_state") else 96, nm)
    dy = (gc["dx"] @ L.proj[:, :L.C].T).contiguous()
    gn = kda.kda_prenorm_bwd(dy, dh, s["h"], L.w_in, res_scale=0.5, eps=EPS)
    ref, mag = R.prenorm_bwd(dy, dh, s["h"], L.w_in, None, 0.5, EPS)
    for nm in ref:
        R.close(gn[nm], ref[nm], mag[nm], 64 + (B * T if nm == "dweight" else 0), nm)


def scan_block(dim=96, n=16, B=2, T=300, seed=0, ty=BF):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, k=1.0, t=ty: (torch.randn(*s, generator=g) * k).to(t).cuda()  # noqa: E731
    return dict(x=r(B, T, dim), w=r(dim, 4, t=F), b=r(dim, t=F), dt=r(B, T, dim),
                A_log=torch.log(torch.arange(1, n + 1.0)).expand(dim, n).contiguous().cuda(),
                B=r(B, T, 1, n), C=r(B, T, 1, n), D=r(dim, t=F), z=r(B, T, dim), bias=r(dim, t=F) - 3,
                dout=r(B, T, dim), wn=1 + r(dim, k=0.1, t=F))


def run_block(kda, a, **kw):
    """convolution -> scan -> norm, and all of it backwards; every output."""
    u, y, n = (torch.empty_like(a["x"]) for _ in range(3))
    B, T, dim = a["x"].shape
    kda.kda_conv_fwd(a["x"], a["w"], a["b"], u, **kw)
    states = kda.make_scan_states(B * T, B, dim, a["A_log"].shape[1])
    kda.kda_scan_fwd(u, a["dt"], a["A_log"], a["B"], a["C"], y, a["D"], a["z"], a["bias"],
                     chunk_states=states, **kw)
    kda.kda_postnorm_fwd(y, a["wn"], a["z"], n, a["x"], activation="silu", **kw)
    g1 = kda.kda_postnorm_bwd(a["dout"], y, a["wn"], a["z"], activation="silu", **kw)
    g2 = kda.kda_scan_bwd(u, a["dt"], a["A_log"], a["B"], a["C"], g1["dx"], a["D"], a["z"], a["bias"],
                          chunk_states=states, **kw)
    g3 = kda.kda_conv_bwd(a["x"], a["w"], a["b"], g2["dx"], **kw)
    keep = [u, y, n]
    for g in (g1, g2, g3):
        keep += [g[k] for k in sorted(g) if k != "workspace"]
    return keep


def same(a, b):
    return all(torch.equal(x.view(torch.int16 if x.dtype == BF else torch.int32),
                           y.view(torch.int16 if y.dtype == BF else torch.int32)) for x, y in zip(a, b))


def test_scan_block_matches_its_references(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    a = scan_block(T=60)
    u, y, n = run_block(kda, a)[:3]
    ref, _ = R.conv(a["x"], a["w"], a["b"], None, None, "silu")
    mag, _ = R.conv(a["x"], a["w"], a["b"], None, None, "silu", mag=True)
    R.close(u, ref, mag, 16, "conv")
    args = (u, a["dt"], a["A_log"], a["B"], a["C"], a["D"], a["z"], a["bias"], None, None)
    (ref, _), (mag, _) = R.scan(*args), R.scan(*args, mag=True)
    R.close(y, ref, mag, 6 * 60 + 64, "scan")
    ref = R.postnorm(y, a["wn"], a["z"], a["x"], 1.0, "silu", EPS)
    part = R.postnorm(y, a["wn"], a["z"], None, 1.0, "silu", EPS).abs()
    R.close(n, ref, part * (2 + R.d(a["z"]).abs()) + R.d(a["x"]).abs(), 64, "norm")


def test_captured_and_replayed(kda_lib):
    """One graph of the whole block, forward and backward, replayed on new inputs while
    direct calls run in between: the bits of direct calls."""
    import kimi_delta_attention_08_gb300 as kda
    a = scan_block(seed=1)
    run_block(kda, a)                                       # first calls outside capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_block(kda, a)
    for seed in (2, 3):
        b = scan_block(seed=seed)
        for k in a:
            a[k].copy_(b[k])
        want = run_block(kda, b)
        graph.replay()
        run_block(kda, scan_block(seed=9))                  # a direct call after the replay
        torch.cuda.synchronize()
        assert same(got, want)


def test_two_graphs_with_one_workspace(kda_lib):
    """Two captured calls that share a caller's workspace, replayed one after the other."""
    import kimi_delta_attention_08_gb300 as kda
    a, b = scan_block(seed=4, T=600), scan_block(seed=5, T=600)
    ws = kda.make_scan_workspace(2, 600, 96, 16, backward=True)
    run = lambda s: kda.kda_scan_bwd(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["dout"], s["D"], s["z"],  # noqa: E731
                                     s["bias"], workspace=ws)
    names = ("dx", "ddt", "dA_log", "dB", "dC", "dD", "dz", "ddt_bias")
    want = [[t.clone() for t in map(run(s).get, names)] for s in (a, b)]
    torch.cuda.synchronize()
    graphs, got = [], []
    for s in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append([run(s)[k] for k in names])
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert same(got[0], want[0]) and same(got[1], want[1])


def test_other_streams(kda_lib):
    """Two blocks at once on two streams that are not the current one, workspaces from the
    allocator: the bits of calls one after the other."""
    import kimi_delta_attention_08_gb300 as kda
    blocks = [scan_block(seed=6), scan_block(seed=7)]
    want = [run_block(kda, a) for a in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [run_block(kda, a, stream=s) for a, s in zip(blocks, streams)]
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


def test_a_raw_stream_needs_a_workspace(kda_lib):
    import kimi_delta_attention_08_gb300 as kda
    a = scan_block()
    h = torch.cuda.current_stream().cuda_stream
    out = torch.empty_like(a["x"])
    kda.kda_conv_fwd(a["x"], a["w"], a["b"], out, stream=h)          # none needed
    with pytest.raises(ValueError):
        kda.kda_conv_bwd(a["x"], a["w"], a["b"], a["dout"], stream=h)
    ws = kda.make_conv_bwd_workspace(600, 96, 4)
    g = kda.kda_conv_bwd(a["x"], a["w"], a["b"], a["dout"], workspace=ws, stream=h)
    assert torch.equal(g["dx"], kda.kda_conv_bwd(a["x"], a["w"], a["b"], a["dout"])["dx"])


def test_beyond_two_to_the_31_elements(kda_lib):
    """The last sequence of a packed batch of 2.3 G elements equals the sequence alone."""
    import kimi_delta_attention_08_gb300 as kda
    C, T, last = 32768, 70000, 50
    x = torch.empty(1, T, C, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    cu = torch.tensor([0, T - last, T], device="cuda")
    w = torch.randn(C, 4, device="cuda")
    out = torch.empty_like(x)
    kda.kda_conv_fwd(x, w, None, out, None, None, cu)
    tail = x[:, T - last:].contiguous()
    alone = torch.empty_like(tail)
    kda.kda_conv_fwd(tail, w, None, alone)
    assert torch.equal(out[:, T - last:], alone)
    g = kda.kda_conv_bwd(x, w, None, x, None, None, cu)
    assert torch.equal(g["dx"][:, T - last:], kda.kda_conv_bwd(tail, w, None, tail)["dx"])
    del g
    wn = torch.ones(8192, device="cuda")
    rows = x.view(-1, 8192)
    kda.kda_postnorm_fwd(rows, wn, rows, out.view(-1, 8192))
    kda.kda_postnorm_fwd(tail.view(-1, 8192), wn, tail.view(-1, 8192), alone.view(-1, 8192))
    assert torch.equal(out[:, T - last:], alone)
    # the scan, whose plan goes by the whole batch: the same sequence within its own rounding
    A = torch.log(torch.arange(1, 9.0)).expand(C, 8).contiguous().cuda()
    bc = torch.randn(1, T, 1, 8, device="cuda").to(BF)
    kda.kda_scan_fwd(x, x, A, bc, bc, out, cu_seqlens=cu)
    bt = bc[:, T - last:].contiguous()
    kda.kda_scan_fwd(tail, tail, A, bt, bt, alone)
    d = (out[:, T - last:].float() - alone.float()).abs().max() / alone.float().abs().max()
    assert d <= 2 ** -8, float(d)
