"""Calls of the 8-bit and backward entry points that a program may make beside the plain
one: handles of streams, host threads, shared and in-place tensors, tokens that are not finite."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = float(np.float32(1e-6))


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _site(T, S, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    R, n = (2 + S) * S, S * H
    return dict(x=r(T, S, H), f=r(T, H), w=r(R, n) / n ** 0.5, scale=0.5 + r(3).abs(),
                base=0.3 * r(R), g=r(T, S, H), dy=r(T, H), dpost=r(T, S), dcomb=r(T, S, S),
                dx_in=r(T, S, H))


def _pre_bwd(mhc, d, x=None, **kw):
    return mhc.site_pre_bwd(d["x"] if x is None else x, d["w"], d["scale"], d["base"], 20, EPS,
                            d["dy"], d["dpost"], d["dcomb"], **kw)


def _same(a, b):
    return all(torch.equal(p.contiguous().view(torch.uint8), q.contiguous().view(torch.uint8))
               for p, q in zip(a, b))


def test_the_default_stream_by_handle(mhc):
    print("[case] stream handles", flush=True)
    d = _site(20, 4, 260, 1)
    x = d["x"].view(80, 260)
    kept = mhc.f8_encode(x)
    post, comb = torch.sigmoid(d["dpost"]), torch.softmax(d["dcomb"], 2)
    calls = [lambda **k: mhc.f8_encode(x, **k), lambda **k: mhc.f8_repack(*kept, 260, **k),
             lambda **k: (mhc.f8_decode(*kept, 260, **k),),
             lambda **k: (mhc.f8_matmul(*kept, *kept, **k),),
             lambda **k: mhc.site_post_bwd(d["g"], d["x"], d["f"], post, comb, **k),
             lambda **k: _pre_bwd(mhc, d, **k)]
    for k, call in enumerate(calls):
        want = call()
        for how in (0, torch.cuda.default_stream(), torch.cuda.current_stream().cuda_stream):
            got = call(stream=how)
            torch.cuda.synchronize()
            assert _same(got, want), (k, how)


def test_calls_from_two_threads(mhc):
    """Each with its own stream and scratch: what they give alone."""
    print("[case] two threads", flush=True)
    sites = [_site(150 + 100 * k, 4, 516, k) for k in range(2)]
    want = [_pre_bwd(mhc, d) for d in sites]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(k):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[k] = _pre_bwd(mhc, sites[k])
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == [] and all(_same(g, w) for g, w in zip(got, want))


@pytest.mark.parametrize("T,S,H", [(40, 1, 260), (300, 4, 516), (1500, 4, 1028), (700, 8, 388)])
@pytest.mark.parametrize("f8", [True, False])
def test_dx_in_place(mhc, T, S, H, f8):
    """dx_in and dx one tensor, over several ranges of tokens and columns."""
    print(f"[case] in place T={T} S={S} H={H} f8={f8}", flush=True)
    d = _site(T, S, H, 3)
    x = mhc.f8_encode(d["x"]) if f8 else d["x"]
    want = _pre_bwd(mhc, d, x, dx_in=d["dx_in"])
    dx = d["dx_in"].clone()
    got = _pre_bwd(mhc, d, x, dx_in=dx, out=(dx, *(torch.empty_like(t) for t in want[1:])))
    assert got[0] is dx and _same(got, want)


@pytest.mark.parametrize("T,S,H", [(9, 3, 260), (40, 4, 516), (300, 4, 516), (200, 8, 388)])
@pytest.mark.parametrize("what", ["x", "dy", "dpost", "dcomb", "dx_in"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_fp32_token_keeps_to_itself(mhc, T, S, H, what, bad):
    print(f"[case] bad {what} T={T} S={S} H={H} {bad}", flush=True)
    d = _site(T, S, H, 4)
    want = _pre_bwd(mhc, d, dx_in=d["dx_in"])[0]
    t = T // 2
    d[what] = d[what].clone()
    d[what][t].view(-1)[-1] = bad
    got = _pre_bwd(mhc, d, dx_in=d["dx_in"])[0]
    rest = [k for k in range(T) if k != t]
    assert not torch.isfinite(got[t]).all() and torch.equal(got[rest], want[rest])


def test_tensors_that_are_inputs_twice(mhc):
    print("[case] shared inputs", flush=True)
    d = _site(50, 4, 516, 5)
    want = _pre_bwd(mhc, d, dpre=d["dpost"].clone(), dx_in=d["x"].clone())
    assert _same(_pre_bwd(mhc, d, dpre=d["dpost"], dx_in=d["x"]), want)
    kept = mhc.f8_encode(d["dy"][:48].contiguous())
    assert torch.equal(mhc.f8_matmul(*kept, *kept),
                       mhc.f8_matmul(*kept, *(t.clone() for t in kept)))
    comb, post = torch.softmax(d["dcomb"], 2), torch.sigmoid(d["dpost"])
    assert _same(mhc.site_post_bwd(d["x"], d["x"], d["f"], post, comb),
                 mhc.site_post_bwd(d["x"], d["x"].clone(), d["f"], post, comb))


@pytest.mark.parametrize("rows,cols", [(5, 260), (300, 516)])
def test_transposed_square_alone(mhc, rows, cols):
    print(f"[case] transposed square {rows}x{cols}", flush=True)
    x = _site(rows, 1, cols, 6)["dy"]
    assert _same(mhc.f8_encode(x, transposed="only", square=True),
                 mhc.f8_encode(x, transposed=True, square=True)[2:])


def test_graphs_replayed_in_turn(mhc):
    """Two captured calls with one scratch between them, replayed one after the other with
    eager work in between: a replay is over before the next one begins on the same stream."""
    print("[case] two graphs", flush=True)
    sites = [_site(100 + 60 * k, 4, 516, 7 + k) for k in range(2)]
    want = [_pre_bwd(mhc, d) for d in sites]
    work = torch.empty(max(mhc.site_pre_bwd_work_bytes(d["x"].shape[0], 4, 516) for d in sites),
                       device="cuda", dtype=torch.uint8)
    outs = [tuple(torch.empty_like(t) for t in w) for w in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = [torch.cuda.CUDAGraph() for _ in sites]
    for g, d, o in zip(graphs, sites, outs):
        with torch.cuda.stream(s):
            _pre_bwd(mhc, d, out=o, work=work)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            _pre_bwd(mhc, d, out=o, work=work)
    for rep in range(3):
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(_same(o, w) for o, w in zip(outs, want)), rep
        _pre_bwd(mhc, sites[0], work=work)
