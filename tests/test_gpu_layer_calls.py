"""How the layer operators are called: from several host threads at once, on streams that are
not the current one, in place; the results are the bits of single calls one after the other."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


def norm_case(D, seed, ty=BF):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, t=ty: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    return dict(dout=r(64, D), h=r(64, D), x=r(64, D), w=r(D, t=F), s=r(D, t=F))


def run_norm(kda, op, a):
    if op == "prenorm":
        r = kda.kda_prenorm_bwd(a["dout"], None, a["h"], a["w"], a["x"], res_scale=a["s"])
    else:
        r = kda.kda_postnorm_bwd(a["dout"], a["h"], a["w"], a["x"], res_scale=a["s"])
    return {k: v for k, v in r.items() if k != "workspace"}


@pytest.mark.parametrize("op", ["prenorm", "postnorm"])
def test_two_widths_from_two_threads(kda_lib, op, monkeypatch):
    """4,096 wide rows keep their next rows in more shared memory than a block has without a
    request, 2,048 wide ones in half of it: neither call may take the limit away from the
    other between its request and its launch.  The library is called with the binding's
    arguments, so that the threads spend their time there."""
    import kimi_delta_attention_08_gb300 as kda
    from kimi_delta_attention_08_gb300 import layer
    cases = [norm_case(4096, 1, F), norm_case(2048, 2, F)]
    want = [run_norm(kda, op, a) for a in cases]
    torch.cuda.synchronize()
    calls = []
    monkeypatch.setattr(layer, "_call", lambda name, dev, stream, *args: calls.append((name, args)))
    got = [run_norm(kda, op, a) for a in cases]
    space = [kda.make_norm_bwd_workspace(64, 4096) for _ in cases]
    monkeypatch.undo()
    streams = [torch.cuda.Stream() for _ in cases]
    bad, go = [], threading.Barrier(2)

    def work(i):
        name, args = calls[i]
        fn, args = getattr(kda_lib, name), (*args[:-2], space[i].data_ptr(), space[i].numel(),
                                            streams[i].cuda_stream)
        go.wait(30)
        for _ in range(20):
            bad.extend(s for s in [fn(*args) for _ in range(500)] if s)
            streams[i].synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, f"{len(bad)} of 20000 calls failed with status {set(bad)}"
    for g, w in zip(got, want):
        for k in w:
            assert torch.equal(g[k], w[k]), k


def backward(kda, op):
    """A call that allocates what it returns, as a function of (stream, workspace), and a
    workspace for it."""
    g = torch.Generator().manual_seed(3)
    T, C = 300, 256
    r = lambda *s, t=BF: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    x, dt, z, dout = (r(2, T, C) for _ in range(4))
    w, b, B, Cm = r(C, 4, t=F), r(C, t=F), r(2, T, 1, 16), r(2, T, 1, 16)
    A, wn, init, st = r(C, 16, t=F), r(C, t=F), r(2, 3, C), r(2, C, 16, t=F)
    kw = lambda s, ws: dict(stream=s, workspace=ws)  # noqa: E731
    if op == "conv":
        return (lambda s, ws: kda.kda_conv_bwd(x, w, b, dout, init, **kw(s, ws)),
                kda.make_conv_bwd_workspace(2 * T, C, 4))
    if op == "scan":
        return (lambda s, ws: kda.kda_scan_bwd(x, dt, A, B, Cm, dout, wn, z, b, st, **kw(s, ws)),
                kda.make_scan_workspace(2, T, C, 16, backward=True))
    ws = kda.make_norm_bwd_workspace(2 * T, C)
    if op == "prenorm":
        return lambda s, ws: kda.kda_prenorm_bwd(dout, None, x, wn, z, res_scale=b, **kw(s, ws)), ws
    return lambda s, ws: kda.kda_postnorm_bwd(dout, x, wn, z, res_scale=b, **kw(s, ws)), ws


@pytest.mark.parametrize("op", ["conv", "scan", "prenorm", "postnorm"])
@pytest.mark.parametrize("raw", [False, True])
def test_results_do_not_take_memory_that_is_still_read(kda_lib, op, raw):
    """Tensors that were freed while the current stream still has to read them: a call on
    another stream (an object, or a raw handle with a workspace) right after that must not
    write its results there."""
    import kimi_delta_attention_08_gb300 as kda
    run, ws = backward(kda, op)
    want = {k: v.clone() for k, v in run(None, None).items() if k != "workspace"}
    sizes = [v.numel() * v.element_size() for v in want.values()] + [ws.numel()]
    s = torch.cuda.Stream()
    old = [(torch.arange(n, device="cuda") % 251).to(torch.uint8) for n in sizes * 2]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                       # some 50 ms
    kept = [t.clone() for t in old]                      # queued behind it
    del old
    got = run(s.cuda_stream, ws) if raw else run(s, None)
    torch.cuda.synchronize()
    for t, n in zip(kept, sizes * 2):
        assert torch.equal(t, (torch.arange(n, device="cuda") % 251).to(torch.uint8))
    for k, v in want.items():
        assert torch.equal(got[k], v), k


@pytest.mark.parametrize("ty", [BF, F])
@pytest.mark.parametrize("N,T,C", [(301, 1, 512), (301, 1, 259), (97, 2, 1024), (50, 32, 264), (9, 33, 1024),
                                   (3, 700, 259)])
def test_convolution_state_in_place(kda_lib, ty, N, T, C):
    """Every kernel that writes a final state (single tokens, runs that are whole sequences,
    runs of longer ones), with the initial state in the same buffer, call after call."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(N * T + C)
    w, b = torch.randn(C, 4, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    one = torch.randn(N, 3, C, generator=g).to(ty).cuda()
    two = one.clone()
    for _ in range(4):
        x = torch.randn(N, T, C, generator=g).to(ty).cuda()
        a, o, end = torch.empty_like(x), torch.empty_like(x), torch.empty_like(one)
        kda.kda_conv_fwd(x, w, b, a, two, end)
        two = end
        kda.kda_conv_fwd(x, w, b, o, one, one)
        assert torch.equal(a, o) and torch.equal(one, two)
        assert torch.equal(one[:, max(0, 3 - T):], x[:, max(0, T - 3):])


def test_recurrence_gradients_do_not_take_memory_that_is_still_read(kda_lib):
    """The same for kda_bwd on another stream."""
    import kimi_delta_attention_08_gb300 as kda
    g = torch.Generator().manual_seed(4)
    r = lambda *s, t=BF: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    q, k, v, gt, dout, beta = (*(r(2, 100, 2, 128) for _ in range(5)), r(2, 100, 2))
    A, bias = r(2, t=F), r(2, 128, t=F)
    run = lambda s: kda.kda_bwd(q, k, v, gt, beta, 128 ** -0.5, A, bias, -5.0, dout, stream=s)  # noqa: E731
    want = {n: t.clone() for n, t in run(None).items() if n != "workspace"}
    sizes = [t.numel() * 4 for t in want.values()] + [kda.make_bwd_workspace(200, 2, 2).numel()]
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
    for n, t in want.items():
        assert torch.equal(got[n], t), n


def test_shards_on_another_stream(kda_lib):
    """A sharded forward on a stream that is not the current one, which is busy: the zeros of a
    piece, the copies between the phases and the final state are in that stream's order."""
    from kimi_delta_attention_08_gb300 import shard
    g = torch.Generator().manual_seed(6)
    r = lambda *s, t=BF: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    x = [r(1, 200, 2, 128) for _ in range(4)] + [r(1, 200, 2)]
    A, bias = r(2, t=F), r(2, 128, t=F)
    cut = [[t[:, a:b].contiguous() for t in x] for a, b in ((0, 80), (80, 200))]

    def run(stream):
        outs = [torch.full_like(c[2], float("nan")) for c in cut]
        fins = [torch.full((1, 2, 128, 128), float("nan"), device="cuda") for _ in cut]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)                   # some 50 ms of the current stream
        args = lambda i: (*cut[i], 128 ** -0.5, outs[i], A, bias, -5.0)  # noqa: E731
        pieces = [shard.shard_piece(i, *args(i), stream=stream) for i in range(2)]
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            pieces = torch.stack(pieces)
        for i in range(2):
            shard.shard_finish(i, pieces, *args(i), fins[i], stream=stream)
        torch.cuda.synchronize()
        return outs + fins

    for a, b in zip(run(None), run(torch.cuda.Stream())):
        assert torch.equal(a, b)


@pytest.mark.parametrize("op", ["prenorm", "postnorm"])
def test_two_widths_in_one_graph(kda_lib, op):
    """Rows of 4,096, 2,048 and 4,096 again in one captured graph, direct calls of another width
    between its replays."""
    import kimi_delta_attention_08_gb300 as kda
    cases = [norm_case(D, D, F) for D in (4096, 2048, 4096)]
    want = [run_norm(kda, op, a) for a in cases]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [run_norm(kda, op, a) for a in cases]
    other = norm_case(1024, 3, F)
    for _ in range(3):
        for r in got:
            for t in r.values():
                t.fill_(float("nan"))
        run_norm(kda, op, other)
        graph.replay()
        torch.cuda.synchronize()
        for r, w in zip(got, want):
            for k in w:
                assert torch.equal(r[k], w[k]), k


@pytest.mark.parametrize("op", ["conv", "scan", "prenorm", "postnorm"])
def test_captured_on_a_side_stream(kda_lib, op):
    """A call on a stream that a capture forks to, its memory from there: replays give the bits
    of a direct call, also while another graph of the same call is alive."""
    import kimi_delta_attention_08_gb300 as kda
    run, ws = backward(kda, op)
    want = {k: v.clone() for k, v in run(None, None).items() if k != "workspace"}
    torch.cuda.synchronize()
    s, graphs, got = torch.cuda.Stream(), [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.wait_stream(torch.cuda.current_stream())
            got.append(run(s, None))
            torch.cuda.current_stream().wait_stream(s)
    for _ in range(2):
        for r in got:
            for k in want:
                r[k].fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for r in got:
            for k, v in want.items():
                assert torch.equal(r[k], v), k
