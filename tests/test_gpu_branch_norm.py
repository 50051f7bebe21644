"""The norms around a branch and their gradients on the GPU, against 64-bit forms."""
import pytest

import branch_forms as bf
from branch_forms import ULP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
EPS = 1e-5
EPS64 = float(torch.tensor(EPS, dtype=torch.float32))  # what the call is given
BF16 = 2.0 ** -8  # half a step of bf16, relative

# Roundings of 1/sqrt(mean v^2 + eps), relative: a thread adds up to 32 squares and the
# block's tree another 6 + 16, all positive, so the sum is off by at most 54 half steps; the
# root halves that; the mean, the epsilon and the reciprocal root (one unit) add 4.
RINV = 31
# ... of a gate's factor: the exponential and the reciprocal are good to a unit (two half
# steps) each, the sum under it and three products a half step each.
GATE = 12


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _rand(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g)


def _within(got, want, bound, name):
    got = got.double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all(), name
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, f"{name}: {over} past the bound"


def _same(a, b):
    return all(p is q is None or torch.equal(p.contiguous().view(torch.uint8),
                                             q.contiguous().view(torch.uint8))
               for p, q in zip(a, b))


NORM_SHAPES = [(1, 4), (3, 128), (5, 256), (7, 260), (37, 1028), (1, 4096), (9, 4100), (2, 7168),
               (3, 8192), (1500, 132), (1100, 1024), (4, 8188), (1023, 1028), (1024, 1028),
               (1030, 4096)]


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("bf16", [False, True])
def test_branch_norm(mhc, T, H, bf16):
    print(f"[case] branch_norm T={T} H={H} bf16={bf16}", flush=True)
    r = _rand(T + H)
    y, nw = r(T, H) * torch.exp(r(T, 1)), 1 + 0.2 * r(H)
    if T > 2:
        y[1] = 0
    got = mhc.branch_norm(y.cuda(), nw.cuda(), EPS, dtype=torch.bfloat16 if bf16 else None)
    assert got.dtype == (torch.bfloat16 if bf16 else torch.float32)
    want = bf.branch(y.double(), nw.double(), EPS64)
    _within(got, want, want.abs() * ((RINV + 3) * ULP + (BF16 * 1.01 if bf16 else 0)), "z")


def _keep(mhc, t, kind):
    """What the call is given for t, and the float64 values that stands for."""
    if kind == "f8":
        kept = mhc.f8_encode(t.cuda())
        return kept, mhc.f8_decode(*kept, t.shape[-1]).double().cpu()
    t = t.bfloat16() if kind == "bf16" else t
    return t.cuda(), t.double()


@pytest.mark.parametrize("T,H", NORM_SHAPES)
@pytest.mark.parametrize("dz_kind,f8", [("f32", False), ("bf16", True), ("f32", True)])
def test_branch_norm_bwd(mhc, T, H, dz_kind, f8):
    print(f"[case] branch_norm_bwd T={T} H={H} {dz_kind} f8={f8}", flush=True)
    r = _rand(3 * T + H)
    gz, dz = _keep(mhc, r(T, H), dz_kind)
    gy, y = _keep(mhc, r(T, H), "f8" if f8 else "f32")
    nw = 1 + 0.2 * r(H)
    dy, dnw = mhc.branch_norm_bwd(gz, gy, nw.cuda(), EPS)
    w_dy, w_dnw, alone, row, size = bf.norm_bwd(dz, dz.abs(), y, nw.double(), EPS64)
    # r enters three times in the part that goes with the row, whose sum has H terms
    _within(dy, w_dy, ((RINV + 4) * alone + (H + 3 * RINV + 8) * row) * ULP, "dy")
    _within(dnw, w_dnw, (T + RINV + 4) * ULP * size, "dnw")
    again = mhc.branch_norm_bwd(gz, gy, nw.cuda(), EPS)
    assert _same((dy, dnw), again)


POST_SHAPES = [(1, 4, 4096), (4, 4, 128), (5, 1, 4), (7, 2, 1028), (37, 3, 132), (3, 8, 7168),
               (20, 5, 516), (9, 6, 260), (6, 7, 384), (200, 4, 2052), (130, 4, 512),
               (33, 8, 64), (2, 1, 8192), (150, 2, 8188), (1100, 2, 256), (300, 4, 5000)]
GATES = [("none", "f32", None), ("channel", "f32", None), ("token", "bf16", "sigmoid"),
         ("channel", "bf16", "silu"), ("token", "f32", "silu"), ("channel", "f32", "sigmoid"),
         ("token", "f32", None)]


def _site(T, S, H, seed, gate, gate_kind):
    r = _rand(seed)
    d = dict(x=r(T, S, H), f=r(T, H) * torch.exp(r(T, 1)), nw=1 + 0.2 * r(H),
             post=2 * torch.sigmoid(r(T, S)), comb=torch.softmax(r(T, S, S), 2), g=r(T, S, H),
             gate=None)
    if gate != "none":
        d["gate"] = 2 * r(*((H,) if gate == "channel" else (T, H)))
        if gate_kind == "bf16":
            d["gate"] = d["gate"].bfloat16()
    return d


def _cuda(t):
    return None if t is None else t.cuda()


def _double(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("T,S,H", POST_SHAPES)
@pytest.mark.parametrize("k", range(len(GATES)))
def test_site_post_norm(mhc, T, S, H, k):
    gate, gate_kind, how = GATES[k]
    f_kind = "bf16" if k % 2 else "f32"
    print(f"[case] site_post_norm T={T} S={S} H={H} {GATES[k]} f={f_kind}", flush=True)
    d = _site(T, S, H, T + S + H + k, gate, gate_kind)
    gf, f = _keep(mhc, d["f"], f_kind)
    got = mhc.site_post_norm(d["x"].cuda(), gf, d["nw"].cuda(), d["post"].cuda(),
                             d["comb"].cuda(), EPS, gate=_cuda(d["gate"]), gate_act=how,
                             alpha=-0.75)
    want, size = bf.site_post_norm(d["x"].double(), f, d["nw"].double(), d["post"].double(),
                                   d["comb"].double(), EPS64, _double(d["gate"]), how, -0.75)
    _within(got, want, (RINV + GATE + 5 + S + 1) * ULP * size, "x'")


@pytest.mark.parametrize("T,S,H", POST_SHAPES)
@pytest.mark.parametrize("k", range(len(GATES)))
def test_site_post_norm_bwd(mhc, T, S, H, k):
    gate, gate_kind, how = GATES[k]
    f_kind, xf8 = ("f32", "bf16", "f8")[k % 3], k % 2 == 0
    print(f"[case] site_post_norm_bwd T={T} S={S} H={H} {GATES[k]} f={f_kind} x8={xf8}",
          flush=True)
    alpha = -0.75
    d = _site(T, S, H, 5 * T + S + H + k, gate, gate_kind)
    gf, f = _keep(mhc, d["f"], f_kind)
    gx, x = _keep(mhc, d["x"], "f8" if xf8 else "f32")
    got = mhc.site_post_norm_bwd(d["g"].cuda(), gx, gf, d["nw"].cuda(), d["post"].cuda(),
                                 d["comb"].cuda(), EPS, gate=_cuda(d["gate"]), gate_act=how,
                                 alpha=alpha)
    g, nw, post, comb = (d[n].double() for n in ("g", "nw", "post", "comb"))
    gt = _double(d["gate"])
    a, slope, slope_size = bf.act(gt, how)
    _within(got[0], comb @ g, (S + 1) * ULP * (comb.abs() @ g.abs()), "dx")
    gT = g.transpose(1, 2).contiguous()
    _within(got[3], x @ gT, (H + 1) * ULP * (x.abs() @ gT.abs()), "dcomb")
    h = bf.branch(f, nw, EPS64, gt, how, alpha)
    each = RINV + GATE + S + 8  # roundings of a term beside those of its sum
    _within(got[2], (g @ h.unsqueeze(2)).squeeze(2),
            (H + each) * ULP * (g.abs() @ h.abs().unsqueeze(2)).squeeze(2), "dpost")
    e = (post.unsqueeze(1) @ g).squeeze(1)
    e_size = (post.abs().unsqueeze(1) @ g.abs()).squeeze(1)
    df, dnw, alone, row, size = bf.norm_bwd(alpha * e * a, abs(alpha) * e_size * a.abs(), f, nw,
                                            EPS64)
    _within(got[1], df, (each * alone + (H + each + 2 * RINV) * row) * ULP, "df")
    _within(got[4], dnw, (T + each) * ULP * size, "dnw")
    if gt is None:
        assert got[5] is None
    else:
        base = bf.branch(f, nw, EPS64)
        dg = alpha * e * slope * base
        dg_size = abs(alpha) * e_size * slope_size * base.abs()
        if gate == "channel":
            dg, dg_size = dg.sum(0), dg_size.sum(0)
        _within(got[5], dg, (T + each + GATE) * ULP * dg_size, "dgate")
    again = mhc.site_post_norm_bwd(d["g"].cuda(), gx, gf, d["nw"].cuda(), d["post"].cuda(),
                                   d["comb"].cuda(), EPS, gate=_cuda(d["gate"]), gate_act=how,
                                   alpha=alpha)
    assert _same(got, again)


@pytest.mark.parametrize("how", [None, "sigmoid", "silu"])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_gradient_against_differences(mhc, how, gate):
    """The gradient along a direction against central differences of the 64-bit forward:
    their error is h^2 times a third derivative (below 1e-6 of the size here), the gradient's
    own, over n terms of either sign, far below 1e-4 of the size of its terms."""
    T, S, H = 6, 4, 132
    print(f"[case] differences {how} {gate}", flush=True)
    d = _site(T, S, H, 11, gate, "f32")
    names = ("x", "f", "post", "comb", "nw", "gate")
    got = mhc.site_post_norm_bwd(d["g"].cuda(), d["x"].cuda(), d["f"].cuda(), d["nw"].cuda(),
                                 d["post"].cuda(), d["comb"].cuda(), EPS, gate=d["gate"].cuda(),
                                 gate_act=how, alpha=0.5)
    r = _rand(12)
    for name, grad in zip(names, got):
        v = r(*d[name].shape).double()

        def loss(h):
            q = {n: d[n].double() for n in names}
            q[name] = q[name] + h * v
            out, _ = bf.site_post_norm(q["x"], q["f"], q["nw"], q["post"], q["comb"], EPS64,
                                       q["gate"], how, 0.5)
            return (d["g"].double() * out).sum().item()

        h = 1e-4
        want = (loss(h) - loss(-h)) / (2 * h)
        have = (grad.double().cpu() * v).sum().item()
        size = (grad.double().cpu() * v).abs().sum().item()
        assert abs(have - want) <= 1e-4 * size, (name, have, want)


def test_plain_gate_and_scale_of_one_are_the_post_mix(mhc):
    """With the norm's result fed to site_post: the same mix of the same values."""
    print("[case] composed", flush=True)
    for T, S, H in ((1, 4, 4096), (300, 4, 516), (5, 8, 7168)):
        d = _site(T, S, H, 3, "none", "f32")
        x, f, nw, post, comb = (d[n].cuda() for n in ("x", "f", "nw", "post", "comb"))
        got = mhc.site_post_norm(x, f, nw, post, comb, EPS)
        want = mhc.site_post(x, mhc.branch_norm(f, nw, EPS), post, comb)
        size = (post.unsqueeze(2) * 8).abs().max().item() + x.abs().max().item()
        # both round h within RINV + 3 half steps
        assert (got - want).abs().max().item() <= 2 * (RINV + 4) * ULP * size


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["f", "gate", "x", "post"])
def test_a_bad_token_keeps_to_itself(mhc, what, bad):
    print(f"[case] bad {what} {bad}", flush=True)
    for T, S, H in ((9, 4, 260), (200, 4, 1028), (1500, 2, 132)):
        d = {k: v.cuda() for k, v in _site(T, S, H, 4, "token", "f32").items()}

        def both():
            out = mhc.site_post_norm(d["x"], d["f"], d["nw"], d["post"], d["comb"], EPS,
                                     gate=d["gate"], gate_act="silu")
            return (out,) + mhc.site_post_norm_bwd(
                d["g"], d["x"], d["f"], d["nw"], d["post"], d["comb"], EPS, gate=d["gate"],
                gate_act="silu")

        want = both()
        t = T // 2
        d[what] = d[what].clone()
        d[what][t].view(-1)[-1] = bad
        got = both()
        rest = [k for k in range(T) if k != t]
        assert not torch.isfinite(got[0][t]).all()
        for k in (0, 1, 2, 3, 4, 6):  # all but dnw, a sum over the tokens
            assert torch.equal(got[k][rest], want[k][rest]), k
        assert what == "x" or not torch.isfinite(got[5]).all()


def test_extreme_gates(mhc):
    """Saturated gates: exact ends of the sigmoid, its slope to its own size, no NaN."""
    print("[case] extreme gates", flush=True)
    T, S, H = 3, 2, 64
    d = _site(T, S, H, 8, "none", "f32")
    v = torch.tensor([-1e30, -200.0, -90.0, -30.0, -1.0, 0.0, 1.0, 30.0, 90.0, 200.0, 1e30])
    gate = v[torch.arange(H) % len(v)]
    for how in ("sigmoid", "silu"):
        got = mhc.site_post_norm_bwd(d["g"].cuda(), d["x"].cuda(), d["f"].cuda(), d["nw"].cuda(),
                                     d["post"].cuda(), d["comb"].cuda(), EPS, gate=gate.cuda(),
                                     gate_act=how)
        g64 = gate.double()
        a, slope, slope_size = bf.act(g64, how)
        e = (d["post"].double().unsqueeze(1) @ d["g"].double()).squeeze(1)
        e_size = (d["post"].double().unsqueeze(1) @ d["g"].double().abs()).squeeze(1)
        base = bf.branch(d["f"].double(), d["nw"].double(), EPS64)
        # exp(-90) and less are at or under fp32's normal numbers: they may count as zero
        bound = (T + RINV + 2 * GATE + S + 10) * ULP * (e_size * slope_size * base.abs()).sum(0)
        tiny = 2.0 ** -120 * (e_size * base.abs()).sum(0)
        if how == "silu":
            tiny = tiny * g64.abs().clamp(1, 200)
        _within(got[5], (e * slope * base).sum(0), bound + tiny, how)
        if how == "sigmoid":
            out = mhc.site_post_norm(d["x"].cuda(), d["f"].cuda(), d["nw"].cuda(),
                                     d["post"].cuda(), d["comb"].cuda(), EPS, gate=gate.cuda(),
                                     gate_act=how)
            zero = mhc.site_post(d["x"].cuda(), torch.zeros(T, H, device="cuda"),
                                 d["post"].cuda(), d["comb"].cuda())
            off = (gate <= -200).cuda()
            assert torch.equal(out[:, :, off], zero[:, :, off])


def test_no_tokens(mhc):
    print("[case] no tokens", flush=True)
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    nw, gate = e(128).fill_(1.0), e(128).fill_(1.0)
    assert mhc.branch_norm(e(0, 128), nw).shape == (0, 128)
    dy, dnw = mhc.branch_norm_bwd(e(0, 128), e(0, 128), nw)
    assert dy.shape == (0, 128) and torch.equal(dnw, torch.zeros_like(nw))
    assert mhc.site_post_norm(e(0, 4, 128), e(0, 128), nw, e(0, 4), e(0, 4, 4)).shape == (0, 4, 128)
    for g in (None, gate, e(0, 128)):
        got = mhc.site_post_norm_bwd(e(0, 4, 128), e(0, 4, 128), e(0, 128), nw, e(0, 4),
                                     e(0, 4, 4), gate=g)
        assert torch.equal(got[4], torch.zeros_like(nw))
        if g is gate:
            assert torch.equal(got[5], torch.zeros_like(nw))


def _calls(mhc, d):
    """Each entry point on a site's tensors, as a function of its keywords."""
    how = dict(gate=d["gate"], gate_act="sigmoid", alpha=0.5)
    a = (d["f"], d["nw"], d["post"], d["comb"], EPS)
    return [lambda **k: (mhc.branch_norm(d["f"], d["nw"], EPS, **k),),
            lambda **k: mhc.branch_norm_bwd(d["g"][:, 0].contiguous(), d["f"], d["nw"], EPS, **k),
            lambda **k: (mhc.site_post_norm(d["x"], *a, **how, **k),),
            lambda **k: mhc.site_post_norm_bwd(d["g"], d["x"], *a, **how, **k)]


@pytest.mark.parametrize("gate", ["channel", "token"])
def test_streams_outputs_and_scratch(mhc, gate):
    print(f"[case] streams {gate}", flush=True)
    d = {k: v.cuda() for k, v in _site(50, 4, 516, 6, gate, "f32").items()}
    work = torch.empty(mhc.norm_bwd_work_bytes(50, 516), device="cuda", dtype=torch.uint8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for k, call in enumerate(_calls(mhc, d)):
        want = call()
        for how in (0, torch.cuda.current_stream().cuda_stream, side, side.cuda_stream):
            got = call(stream=how)
            torch.cuda.synchronize()
            assert _same(got, want), (k, how)
        out = tuple(torch.full_like(t, float("nan")) for t in want)
        extra = dict(work=work) if k in (1, 3) else {}
        got = call(out=out if len(out) > 1 else out[0], **extra)
        assert all(p is q for p, q in zip(got, out)) and _same(got, want)
        with pytest.raises(ValueError):
            call(out=tuple(t[:-1] for t in out) if len(out) > 1 else out[0][:-1])
        if extra:
            with pytest.raises(mhc.MhcError, match="EINVAL"):
                call(work=work[:64])


def test_operands_that_are_refused(mhc):
    print("[case] refused", flush=True)
    d = {k: v.cuda() for k, v in _site(6, 4, 128, 6, "token", "f32").items()}
    a = (d["nw"], d["post"], d["comb"], EPS)
    wide = torch.empty(6, 256, device="cuda")[:, :128]
    with pytest.raises(ValueError, match="contiguous"):
        mhc.site_post_norm(d["x"], wide, *a)
    with pytest.raises(ValueError, match="contiguous"):
        mhc.branch_norm(wide, d["nw"])
    with pytest.raises(ValueError, match="shape"):
        mhc.site_post_norm(d["x"], d["f"], *a, gate=d["gate"][:3])
    with pytest.raises(ValueError, match="shape"):
        mhc.site_post_norm(d["x"], d["f"][:, :64].contiguous(), *a)
    with pytest.raises(mhc.MhcError, match="EOVERLAP"):
        mhc.site_post_norm(d["x"], d["f"], *a, out=d["x"])
    with pytest.raises(mhc.MhcError, match="EOVERLAP"):
        mhc.branch_norm(d["f"], d["nw"], out=d["f"])
    with pytest.raises(mhc.MhcError, match="EINVAL"):
        mhc.branch_norm(d["f"], d["nw"], 0.0)
    with pytest.raises(mhc.MhcError, match="EINVAL"):
        mhc.site_post_norm(d["x"], d["f"], *a, alpha=float("nan"))
    with pytest.raises(mhc.MhcError, match="EALIGN"):
        mhc.branch_norm(d["f"][:, :126].contiguous(), d["nw"][:126].contiguous())


@pytest.mark.parametrize("T,gate", [(1, "channel"), (70, "channel"), (1500, "token")])
def test_captured_and_replayed(mhc, T, gate):
    """Every call in one graph, replayed with eager work in between and new inputs."""
    print(f"[case] graph T={T} {gate}", flush=True)
    d = {k: v.cuda() for k, v in _site(T, 4, 260, 9, gate, "f32").items()}
    calls = _calls(mhc, d)
    outs = [tuple(torch.empty_like(t) for t in c()) for c in calls]
    work = torch.empty(mhc.norm_bwd_work_bytes(T, 260), device="cuda", dtype=torch.uint8)
    dz = torch.empty(T, 260, device="cuda")

    def all_calls():
        how = dict(gate=d["gate"], gate_act="sigmoid", alpha=0.5)
        a = (d["f"], d["nw"], d["post"], d["comb"], EPS)
        mhc.branch_norm(d["f"], d["nw"], EPS, out=outs[0][0])
        mhc.branch_norm_bwd(dz, d["f"], d["nw"], EPS, out=outs[1], work=work)
        mhc.site_post_norm(d["x"], *a, **how, out=outs[2][0])
        mhc.site_post_norm_bwd(d["g"], d["x"], *a, **how, out=outs[3], work=work)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        all_calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        all_calls()
    for rep in range(3):
        new = _site(T, 4, 260, 20 + rep, gate, "f32")
        for k in d:
            d[k].copy_(new[k])
        dz.copy_(d["g"][:, 0])
        for o in outs:
            for t in o:
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, c in enumerate(calls):
            assert _same(outs[k], c()), (rep, k)


def test_past_32_bits(mhc):
    """Byte offsets past 2^32 in x, f and the gate: the last tokens as a call of their own."""
    print("[case] large", flush=True)
    T, S, H, n = 140000, 1, 8192, 5
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    f, nw, post, comb = r(T, H), 1 + 0.2 * r(H), r(T, S), r(T, S, S)
    x, gate = f.view(T, 1, H), f
    last = slice(T - n, T)
    end = [t[last].clone() for t in (x, f, post, comb, gate)]

    def near(a, b):  # few tokens take another split of the same sums
        return (a - b).abs().max().item() <= 200 * ULP * b.abs().max().item()

    z = mhc.branch_norm(f, nw, EPS)
    assert near(z[last], mhc.branch_norm(end[1], nw, EPS))
    del z
    out = mhc.site_post_norm(x, f, nw, post, comb, EPS, gate=gate, gate_act="sigmoid")
    assert near(out[last], mhc.site_post_norm(end[0], end[1], nw, end[2], end[3], EPS,
                                              gate=end[4], gate_act="sigmoid"))
    del out
    got = mhc.site_post_norm_bwd(x, x, f, nw, post, comb, EPS, gate=gate, gate_act="sigmoid")
    want = mhc.site_post_norm_bwd(end[0], end[0], end[1], nw, end[2], end[3], EPS, gate=end[4],
                                  gate_act="sigmoid")
    for k in (0, 1, 2, 3, 5):
        assert torch.equal(got[k][last], want[k]), k
    del got
    dy, _ = mhc.branch_norm_bwd(f, f, nw, EPS)
    assert torch.equal(dy[last], mhc.branch_norm_bwd(end[1], end[1], nw, EPS)[0])
