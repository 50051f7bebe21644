"""fp32 accuracy of the pre half's gradient, entry by entry: inputs whose sums are the
rounding errors of single products (tests/plane_inputs.py), so that a wrong, missing or
misplaced plane of W, x or u stands whole in the result."""
import pytest

import plane_inputs as pi

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _call(mhc, d, f8, iters, eps, scale=1.0, **kw):
    """The gradient with what d does not name at zero."""
    T, S, H = d["x"].shape
    R = (2 + S) * S
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    p = {k: v.cuda() for k, v in d.items() if k not in ("want", "size", "leaks")}
    x = mhc.f8_encode(p["x"]) if f8 else p["x"]
    if f8:
        assert torch.equal(mhc.f8_decode(*x, H), p["x"])
    return mhc.site_pre_bwd(x, p.get("w", z(R, S * H)), z(3) + scale, z(R), iters, eps,
                            p.get("dy", z(T, H)), p.get("dpost", z(T, S)),
                            p.get("dcomb", z(T, S, S)),
                            dpre=p.get("dpre"), dx_in=p.get("dx_in"), **kw)


def _check(got, d, bound, name):
    over = ((got.double().cpu() - d["want"]).abs() / bound).max().item()
    assert over <= 1, f"{name}: {over:.2f} of the bound"


# Few tokens (W cut on the way), one group of them, many; one to eight streams
SHAPES = [(3, 1, 260), (16, 4, 1028), (1, 4, 4096), (9, 8, 260), (50, 7, 516), (40, 2, 36),
          (64, 4, 516), (100, 8, 260), (37, 3, 1028), (200, 1, 388), (150, 4, 260), (300, 8, 516),
          (200, 5, 64), (1100, 4, 132), (130, 6, 68)]


@pytest.mark.parametrize("T,S,H", SHAPES)
@pytest.mark.parametrize("f8", [False, True])
def test_dots(mhc, T, S, H, f8):
    """dx of the one column in which x is zero is the pre gate, 1 / (1 + exp(-scale r dot)).
    The gate is off by at most eight roundings (exp, sum, reciprocal, the products of its
    argument), its argument by 80 * 2^-24 where the gate lies between 0.11 and 0.89, the dot
    by that over scale r; r is at least one here."""
    print(f"[case] planes of the dots T={T} S={S} H={H} f8={f8}", flush=True)
    d = pi.dots(T, S, H, T + S, f8)
    scale = 2.0 ** (13 if f8 else 18)
    dx = _call(mhc, d, f8, 1, 1e-6, scale)[0]
    r = (d["x"].double().square().mean((1, 2)) + 1e-6).rsqrt().unsqueeze(1)
    p = dx[:, :, H - 1].double().cpu()
    assert (r >= 1).all() and ((p > 0.11) & (p < 0.89)).all()
    got = torch.log(p / (1 - p)) / (scale * r)
    left_out = 0 if f8 else pi.KEPT  # a code is one plane: three products are all of them
    _check(got, d, (left_out + pi.SUMS) * d["size"] + 80 * 2.0 ** -24 / (scale * r), "dots")


@pytest.mark.parametrize("T,S,H", [(3, 1, 260), (16, 4, 1028), (9, 8, 260), (50, 7, 516),
                                   (40, 2, 36), (64, 4, 516), (100, 8, 260), (200, 4, 388),
                                   (300, 8, 516), (200, 5, 64)])
@pytest.mark.parametrize("f8", [False, True])
def test_dots_of_every_row(mhc, T, S, H, f8):
    """With a gradient at one gate of one token, dscale of its group is that gradient times
    the dot over rms (one product rounded)."""
    print(f"[case] planes of every row T={T} S={S} H={H} f8={f8}", flush=True)
    d = pi.rows(T, S, H, T + S, f8)
    R = (2 + S) * S
    g = torch.Generator().manual_seed(5)
    left_out = 0 if f8 else pi.KEPT
    for r in range(R):
        t = int(torch.randint(0, T, (), generator=g))
        u = torch.zeros(T, R)
        u[t, r] = 1.0
        got = _call(mhc, {"x": d["x"], "w": d["w"], **pi.seeds(u, S)}, f8, 1, pi.EPS,
                    2.0 ** -30)[2] / pi.UNIT_RMS
        group = 0 if r < S else 1 if r < 2 * S else 2
        one = {"want": d["want"][t, r]}
        _check(got[group], one, (left_out + pi.SUMS) * d["size"][t, r]
               + 2.0 ** -23 * one["want"].abs() + pi.LEAK, f"row {r}")
        assert not got[[k for k in range(3) if k != group]].any()


@pytest.mark.parametrize("T,S,H", SHAPES)
@pytest.mark.parametrize("f8", [False, True])
def test_gradient_of_the_state(mhc, T, S, H, f8):
    print(f"[case] planes of dx T={T} S={S} H={H} f8={f8}", flush=True)
    d = pi.streams(T, S, H, T + S)
    dx = _call(mhc, d, f8, 1, pi.EPS)[0] / pi.UNIT_RMS
    _check(dx, d, (pi.KEPT + pi.SUMS + pi.ROUND * d["leaks"]) * d["size"] + pi.LEAK, "dx")


@pytest.mark.parametrize("T,S,H", [(16, 4, 260), (40, 1, 516), (64, 8, 132), (33, 8, 36),
                                   (100, 2, 1028), (300, 4, 516), (500, 8, 388), (1100, 4, 132),
                                   (2100, 3, 260), (90, 5, 260), (70, 6, 64), (77, 7, 132)])
@pytest.mark.parametrize("f8", [False, True])
def test_gradient_of_the_weight(mhc, T, S, H, f8):
    print(f"[case] planes of dW T={T} S={S} H={H} f8={f8}", flush=True)
    d = pi.weights(T, S, H, T + S, f8)
    dw = _call(mhc, d, f8, 1, pi.EPS)[1] / pi.UNIT_RMS
    left_out = 0 if f8 else pi.KEPT
    _check(dw, d, (left_out + pi.SUMS + pi.ROUND * d["leaks"]) * d["size"] + pi.LEAK, "dW")


@pytest.mark.parametrize("T,S,H", [(16, 4, 1028), (50, 7, 516), (37, 3, 132), (300, 4, 516),
                                   (200, 8, 388)])
@pytest.mark.parametrize("f8", [False, True])
def test_small_tokens_beside_large_ones(mhc, T, S, H, f8):
    """The gradient is linear in what comes in, token by token: a token's gradients times a
    power of two give that power times its dx, bit for bit, whatever its neighbours have."""
    print(f"[case] powers of two T={T} S={S} H={H} f8={f8}", flush=True)
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    R = (2 + S) * S
    fixed = dict(x=r(T, S, H), w=r(R, S * H) / (S * H) ** 0.5)
    grads = dict(dy=r(T, H), dpre=r(T, S), dpost=r(T, S), dcomb=r(T, S, S), dx_in=r(T, S, H))
    by = 2.0 ** (torch.arange(T) * 7 % 41 - 20).float()
    if f8:
        fixed["x"] = mhc.f8_decode(*mhc.f8_encode(fixed["x"].cuda()), H).cpu()
    want = _call(mhc, fixed | grads, f8, 20, 1e-6)[0].cpu()
    scaled = {k: v * by.reshape(-1, *[1] * (v.dim() - 1)) for k, v in grads.items()}
    got = _call(mhc, fixed | scaled, f8, 20, 1e-6)[0].cpu()
    assert torch.equal(got, want * by.reshape(-1, 1, 1))


def test_entries_above_the_largest_bf16(mhc):
    """An fp32 entry that rounds to an infinity in bf16 is still itself: a weight that meets
    no gradient, and one that does."""
    print("[case] planes of the largest entries", flush=True)
    T, S, H = 40, 2, 132
    big = torch.finfo(torch.float32).max
    R = (2 + S) * S
    d = dict(x=torch.zeros(T, S, H), w=torch.zeros(R, S * H), dpre=torch.zeros(T, S))
    d["w"][0, ::3], d["w"][1, 1::3] = big, -big
    d["dpre"][7, 0], d["dpre"][9, 1] = 2.0 ** -30, 2.0 ** -30
    for n in (40, 1):
        part = {k: v if k == "w" else v[:n] for k, v in d.items()}
        dx = _call(mhc, part, False, 3, 1.0)[0].double().cpu()
        want = torch.zeros(n, S, H, dtype=torch.float64)
        if n > 9:
            want[7] = (d["w"][0].double() * 2.0 ** -32).reshape(S, H)
            want[9] = (d["w"][1].double() * 2.0 ** -32).reshape(S, H)
        assert torch.equal(dx, want)
