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
