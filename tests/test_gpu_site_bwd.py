"""The backward passes of a site's two halves on the GPU, against 64-bit forms and
against differences of the forward pass."""
import numpy as np
import pytest

import plain_forms as pf

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
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    R, n = (2 + S) * S, S * H
    return dict(x=r(T, S, H), f=r(T, H), w=r(R, n) / n ** 0.5, scale=0.5 + torch.rand(3, generator=g),
                base=0.3 * r(R), g=r(T, S, H), dy=r(T, H), dpre=r(T, S), dpost=r(T, S),
                dcomb=r(T, S, S), dx_in=r(T, S, H))


def _keep(mhc, t, f8):
    """What the call is given for t, and the float64 values that stands for."""
    if not f8:
        return t.cuda(), t.double()
    kept = mhc.f8_encode(t.cuda())
    return kept, mhc.f8_decode(*kept, t.shape[-1]).double().cpu()


# An fp32 sum of n products is off by at most n * 2^-24 of the sum of magnitudes (one
# rounding a term, the first product included).
def _check_sum(got, want, magnitude, terms, name):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    over = (got - want).abs() - (terms + 1) * 2.0 ** -24 * magnitude
    assert over.max() <= 0, f"{name}: {over.max()} past the bound"


SHAPES = [(1, 4, 4096), (4, 4, 128), (5, 1, 4), (7, 2, 1028), (37, 3, 132), (3, 8, 7168),
          (20, 5, 516), (9, 6, 260), (6, 7, 384), (130, 4, 512), (33, 8, 64)]


@pytest.mark.parametrize("T,S,H", SHAPES)
@pytest.mark.parametrize("xf8,ff8", [(False, False), (True, True), (True, False), (False, True)])
def test_post_bwd(mhc, T, S, H, xf8, ff8):
    print(f"[case] post_bwd T={T} S={S} H={H} {xf8} {ff8}", flush=True)
    d = _site(T, S, H, T + S + H)
    post, comb = 2 * torch.sigmoid(d["dpost"]), torch.softmax(d["dcomb"], 2)
    kx, x = _keep(mhc, d["x"], xf8)
    kf, f = _keep(mhc, d["f"], ff8)
    got = mhc.site_post_bwd(d["g"].cuda(), kx, kf, post.cuda(), comb.cuda())
    g, post, comb = d["g"].double(), post.double(), comb.double()
    forms = [lambda g, x, f, p, c: c @ g, lambda g, x, f, p, c: (p.unsqueeze(1) @ g).squeeze(1),
             lambda g, x, f, p, c: (g @ f.unsqueeze(2)).squeeze(2),
             lambda g, x, f, p, c: x @ g.transpose(1, 2)]
    args = (g, x, f, post, comb)
    for k, (form, terms) in enumerate(zip(forms, (S, S, H, H))):
        _check_sum(got[k], form(*args), form(*(a.abs() for a in args)), terms,
                   ("dx", "df", "dpost", "dcomb")[k])


# The chain has up to n + 6 * iters + 50 fp32 roundings on a path; worst-case signs
# would add up to (n + ...) * 2^-24, but the terms of the long sums round
# independently, so an error of order sqrt(n) * 2^-24 plus the short part's
# 170 * 2^-24 = 1e-5 is what arithmetic gives: for n up to 57344 below 2.5e-5 of the
# largest entry of a gradient, which every entry's own terms are bounded by.
BWD_REL = 2.5e-5


def _check_rel(got, want, name, scale=None):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    scale = max(want.abs().max().item(), 1e-6) if scale is None else scale
    rel = (got - want).abs().max().item() / scale
    assert rel <= BWD_REL, f"{name}: {rel:.3e} of the largest entry"


NAMES = ("dx", "dfn_w", "dscale", "dbase")


def _pre_bwd(mhc, kx, d, iters, **kw):
    a = {k: v.cuda() for k, v in d.items() if k in ("w", "scale", "base", "dy", "dpost", "dcomb")}
    return mhc.site_pre_bwd(kx, a["w"], a["scale"], a["base"], iters, EPS, a["dy"], a["dpost"],
                            a["dcomb"], **kw)


@pytest.mark.parametrize("T,S,H", SHAPES)
@pytest.mark.parametrize("f8", [False, True])
@pytest.mark.parametrize("iters", [1, 20])
def test_pre_bwd(mhc, T, S, H, f8, iters):
    print(f"[case] pre_bwd T={T} S={S} H={H} f8={f8} iters={iters}", flush=True)
    d = _site(T, S, H, 3 * T + S + H)
    kx, x = _keep(mhc, d["x"], f8)
    got = _pre_bwd(mhc, kx, d, iters, dpre=d["dpre"].cuda(), dx_in=d["dx_in"].cuda())
    want = pf.pre_grads(x, d["w"], d["scale"], d["base"], iters, EPS, d["dy"], d["dpre"],
                        d["dpost"], d["dcomb"], d["dx_in"])
    # dscale and dbase share their sums' terms: the size of dbase bounds both
    scale = max(want[3].abs().max().item(), want[2].abs().max().item(), 1e-6)
    for k, n in enumerate(NAMES):
        _check_rel(got[k], want[k], n, scale if k >= 2 else None)


def test_pre_bwd_many_tokens(mhc):
    """Several token ranges and hidden ranges, a ragged end."""
    T, S, H = 1027, 4, 260
    print(f"[case] pre_bwd T={T}", flush=True)
    d = _site(T, S, H, 9)
    for f8 in (False, True):
        kx, x = _keep(mhc, d["x"], f8)
        got = _pre_bwd(mhc, kx, d, 20)
        want = pf.pre_grads(x, d["w"], d["scale"], d["base"], 20, EPS, d["dy"], None, d["dpost"],
                            d["dcomb"], None)
        scale = max(want[3].abs().max().item(), want[2].abs().max().item())
        for k, n in enumerate(NAMES):
            _check_rel(got[k], want[k], n, scale if k >= 2 else None)
        again = _pre_bwd(mhc, kx, d, 20)
        for a, b in zip(got, again):
            assert torch.equal(a, b)


def test_pre_bwd_in_place_and_most_rounds(mhc):
    print("[case] pre_bwd in place, 120 rounds, zero input", flush=True)
    d = _site(6, 4, 132, 4)
    d["x"][2] = 0
    dx = d["dx_in"].cuda()
    e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    out = (dx, e(24, 528), e(3), e(24))
    got = _pre_bwd(mhc, d["x"].cuda(), d, 120, dx_in=dx, out=out)
    assert got[0] is dx
    want = pf.pre_grads(d["x"], d["w"], d["scale"], d["base"], 120, EPS, d["dy"], None,
                        d["dpost"], d["dcomb"], d["dx_in"])
    # an all-zero token has 1/sqrt(eps) = 1000 in front of its gradient: token by token
    for t in range(6):
        _check_rel(got[0][t], want[0][t], f"dx of token {t}")
    for k in (1, 2, 3):
        _check_rel(got[k], want[k], NAMES[k], max(want[3].abs().max().item(),
                                                  want[2].abs().max().item()) if k > 1 else None)


@pytest.mark.parametrize("S", [4, 8])
@pytest.mark.parametrize("T", [1, 30])
def test_pre_bwd_of_saturated_gates(mhc, S, T):
    """With W = 0 a gate's argument is its base, and the gradient of base is the gate's slope
    p (1 - p) (twice that for post): every slope to its own size.  exp, a sum, a reciprocal
    and three products: at most 16 roundings, 2^-20, but for fp32's least normal number."""
    print(f"[case] pre_bwd saturated gates T={T} S={S}", flush=True)
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    R, H = (2 + S) * S, 132
    for lo, hi in ((-40, 40), (0, 20), (-100, 100), (10, 17.5)):
        base = torch.zeros(R)
        base[:2 * S] = torch.linspace(lo, hi, 2 * S)
        one = z(T, S)
        one[T // 2] = 1.0
        got = mhc.site_pre_bwd(z(T, S, H), z(R, S * H), z(3) + 1, base.cuda(), 20, EPS, z(T, H),
                               one, z(T, S, S), dpre=one)[3].double().cpu()
        b = base.double()
        want = torch.sigmoid(b) * torch.sigmoid(-b)
        want[S:2 * S] *= 2
        want[2 * S:] = 0
        bound = 2.0 ** -20 * want + 2.0 ** -126
        assert ((got - want).abs() <= bound).all(), (got / want)[:2 * S]


def test_pre_bwd_of_no_tokens_is_zero(mhc):
    print("[case] pre_bwd T=0", flush=True)
    d = _site(1, 4, 128, 4)
    z = {k: (v[:0] if k in ("x", "dy", "dpost", "dcomb") else v) for k, v in d.items()}
    e = lambda *s: torch.full(s, 5.0, device="cuda")  # noqa: E731
    out = (e(0, 4, 128), e(24, 512), e(3), e(24))
    _pre_bwd(mhc, z["x"].cuda(), z, 20, out=out)
    assert all((o == 0).all() for o in out[1:])
    got = mhc.site_post_bwd(e(0, 4, 128), e(0, 4, 128), e(0, 128), e(0, 4), e(0, 4, 4))
    assert got[0].shape == (0, 4, 128)


def test_gradients_match_differences(mhc):
    """Central differences of the float64 forward pass along random directions.  With
    h = 1e-5 and values of order one a difference is off by about h^2 plus 1e-16 / h,
    1e-10, far inside the gradient's own fp32 error."""
    T, S, H, iters, h = 3, 4, 64, 20, 1e-5
    print("[case] differences", flush=True)
    d = _site(T, S, H, 21)
    seeds = [d[k].double() for k in ("dpre", "dpost", "dcomb", "dy")]
    args = [d[k].double() for k in ("x", "w", "scale", "base")]

    def loss(a):
        return sum((o * s).sum() for o, s in zip(pf.site_pre(*a, iters, EPS), seeds))

    grads = _pre_bwd(mhc, d["x"].cuda(), d, iters, dpre=d["dpre"].cuda())
    post, comb = 2 * torch.sigmoid(d["dpost"]), torch.softmax(d["dcomb"], 2)
    pargs = [t.double() for t in (d["x"], d["f"], post, comb)]

    def ploss(a):
        return (pf.site_post(*a) * d["g"].double()).sum()

    pgrads = mhc.site_post_bwd(d["g"].cuda(), d["x"].cuda(), d["f"].cuda(), post.cuda(),
                               comb.cuda())
    gen = torch.Generator().manual_seed(5)
    for fn, at, got in ((loss, args, grads), (ploss, pargs, pgrads)):
        for i, gr in enumerate(got):
            v = torch.randn(at[i].shape, generator=gen, dtype=torch.float64)
            up, dn = list(at), list(at)
            up[i], dn[i] = at[i] + h * v, at[i] - h * v
            diff = (fn(up) - fn(dn)) / (2 * h)
            dot = (gr.double().cpu() * v).sum()
            size = gr.double().cpu().norm() * v.norm()
            assert abs(dot - diff) <= BWD_REL * size, (i, dot.item(), diff.item())


def test_site_trained_together(mhc):
    """A site as training runs it: pre, branch in 8 bits, post, with x, z and f kept in
    8 bits; then the backward passes in order, captured and replayed from a graph."""
    T, S, H = 50, 4, 256
    print(f"[case] site step T={T}", flush=True)
    d = {k: v.cuda() for k, v in _site(T, S, H, 30).items()}
    wb = mhc.f8_encode(torch.randn(H, H, device="cuda") / 16, transposed=True, square=True)

    def step():
        pre, post, comb, y = mhc.site_pre(d["x"], d["w"], d["scale"], d["base"], 20, EPS)
        kx, kz = mhc.f8_encode(d["x"]), mhc.f8_encode(y)
        f = mhc.f8_matmul(*kz, wb[0], wb[1])
        xo = mhc.site_post(d["x"], f, post, comb)
        kf = mhc.f8_encode(f)
        dx, df, dpost, dcomb = mhc.site_post_bwd(d["g"], kx, kf, post, comb)
        dc, ds, dct, dst = mhc.f8_encode(df, transposed=True)
        dy = mhc.f8_matmul(dc, ds, wb[2], wb[3])
        dwb = mhc.f8_matmul(dct, dst, *mhc.f8_repack(*kz, H))
        return (xo, dwb, *mhc.site_pre_bwd(kx, d["w"], d["scale"], d["base"], 20, EPS, dy, dpost,
                                           dcomb, dx_in=dx), post, comb, f, dy, dx, dpost, dcomb)

    want = [t.clone() for t in step()]
    kx, kf = mhc.f8_encode(d["x"]), mhc.f8_encode(want[8])
    x = mhc.f8_decode(*kx, H).double().cpu()
    f = mhc.f8_decode(*kf, H).double().cpu()
    g, post, comb = (t.double().cpu() for t in (d["g"], want[6], want[7]))
    _check_sum(want[10], comb @ g, comb @ g.abs(), S, "dx of the post half")
    _check_sum(want[11], (g @ f.unsqueeze(2)).squeeze(2),
               (g.abs() @ f.abs().unsqueeze(2)).squeeze(2), H, "dpost")
    _check_sum(want[12], x @ g.transpose(1, 2), x.abs() @ g.abs().transpose(1, 2), H, "dcomb")
    grads = pf.pre_grads(x, d["w"].cpu(), d["scale"].cpu(), d["base"].cpu(), 20, EPS,
                         want[9].cpu(), None, want[11].cpu(), want[12].cpu(), want[10].cpu())
    scale = max(grads[2].abs().max().item(), grads[3].abs().max().item())
    for k, n in enumerate(NAMES):
        _check_rel(want[2 + k], grads[k], n, scale if k >= 2 else None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for rep in range(3):
        for t in got:
            t.fill_(float("nan"))
        step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (rep, k)


def test_two_calls_on_two_streams(mhc):
    """Each call has its own scratch: two streams at once give what they give alone."""
    print("[case] two streams", flush=True)
    ds = [_site(200, 4, 512, s) for s in (1, 2)]
    xs = [d["x"].cuda() for d in ds]
    want = [[t.clone() for t in _pre_bwd(mhc, x, d, 20)] for x, d in zip(xs, ds)]
    dev = [{k: v.cuda() for k, v in d.items()} for d in ds]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [mhc.site_pre_bwd(x, d["w"], d["scale"], d["base"], 20, EPS, d["dy"], d["dpost"],
                                d["dcomb"], stream=s) for x, d, s in zip(xs, dev, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
