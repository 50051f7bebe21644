"""Sizes at which the 8-bit product and the site's backward passes take their other
kernels, against 64-bit forms of the whole result."""
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


def _decode(codes, scales, cols, square=False):
    """float64 values, from torch's own conversion of a code."""
    s = torch.exp2(scales.double() - 127)
    if square:
        s = s.repeat_interleave(pf.BLOCK, 0)[:codes.shape[0]]
    return (codes.double() * s.repeat_interleave(pf.BLOCK, 1))[:, :cols].contiguous()


def _randn(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda")


# Few rows against short and long weights, one and two blocks of 16 rows past a full
# one, depths of 2 to 66 blocks; then squares of tiles of each size with ragged edges.
MKN = [(1, 8324, 260), (5, 132, 8196), (16, 4096, 8196), (16, 4100, 8196), (17, 4992, 4100),
       (32, 388, 8196), (31, 4224, 8196), (33, 260, 8188), (64, 4228, 4100), (64, 260, 8196),
       (50, 132, 516), (1795, 260, 1668), (1664, 1284, 1924), (3845, 260, 3332),
       (3584, 1412, 3588), (4093, 4, 4100), (24700, 132, 68), (100, 388, 24900),
       (70001, 260, 4), (12500, 260, 64), (66, 516, 65540), (16, 4096, 16388),
       (9, 8324, 16388), (16, 2048, 5124), (3, 260, 16388), (32, 516, 20004),
       (100, 1156, 1028), (200, 8452, 1988), (65, 1024, 16380), (3900, 516, 3988),
       (4100, 260, 4500), (250, 388, 49000)]


@pytest.mark.parametrize("M,K,N", MKN)
@pytest.mark.parametrize("square", [True, False])
def test_matmul(mhc, M, K, N, square):
    print(f"[case] matmul {M}x{N}x{K} square={square}", flush=True)
    # rows of sizes that differ by 2^16: a row of a neighbour shows
    x = _randn(M + K, M, K) * 2.0 ** (torch.arange(M, device="cuda") % 17 - 8).unsqueeze(1)
    ea = mhc.f8_encode(x)
    eb = mhc.f8_encode(_randn(N, N, K), square=square)
    a, b = _decode(*ea, K), _decode(*eb, K, square)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    # exact products; K additions, each off by at most a unit in the last place (2^-23, a
    # truncating adder included) of a partial sum of at most `size`
    bound = K * 2.0 ** -23 * size
    got = mhc.f8_matmul(*ea, *eb, dtype=torch.float32).double()
    over = ((got - want).abs() - bound).max().item()
    assert over <= 0, over
    got = mhc.f8_matmul(*ea, *eb, dtype=torch.bfloat16).double()
    # and one rounding to bf16 of a value of at most want + bound
    over = ((got - want).abs() - bound * (1 + 2.0 ** -8) - 2.0 ** -8 * want.abs()).max().item()
    assert over <= 0, over


def _site(T, S, H, seed):
    R, n = (2 + S) * S, S * H
    return dict(x=_randn(seed, T, S, H), f=_randn(seed + 1, T, H),
                w=_randn(seed + 2, R, n) / n ** 0.5, scale=0.5 + _randn(seed + 3, 3).abs(),
                base=0.3 * _randn(seed + 4, R), g=_randn(seed + 5, T, S, H),
                dy=_randn(seed + 6, T, H), dpost=_randn(seed + 7, T, S),
                dcomb=_randn(seed + 8, T, S, S), dx_in=_randn(seed + 9, T, S, H))


def _keep(mhc, t, f8):
    if not f8:
        return t, t
    kept = mhc.f8_encode(t)
    return kept, mhc.f8_decode(*kept, t.shape[-1])


@pytest.mark.parametrize("T,S,H", [(2345, 4, 7168), (2400, 8, 4100), (5000, 1, 7172)])
@pytest.mark.parametrize("f8", [True, False])
def test_post_bwd_past_the_cache(mhc, T, S, H, f8):
    print(f"[case] post_bwd T={T} S={S} H={H} f8={f8}", flush=True)
    assert T * (S + 1) * H * 4 > 256 << 20
    d = _site(T, S, H, T)
    post, comb = 2 * torch.sigmoid(d["dpost"]), torch.softmax(d["dcomb"], 2)
    kx, x = _keep(mhc, d["x"], f8)
    kf, f = _keep(mhc, d["f"], f8)
    got = mhc.site_post_bwd(d["g"], kx, kf, post, comb)
    for t0 in range(0, T, 500):  # 64-bit forms of 500 tokens at a time
        g, xs, fs, p, c = (t[t0:t0 + 500].double() for t in (d["g"], x, f, post, comb))
        forms = [lambda g, x, f, p, c: (c.unsqueeze(3) * g.unsqueeze(1)).sum(2),
                 lambda g, x, f, p, c: (p.unsqueeze(2) * g).sum(1),
                 lambda g, x, f, p, c: (g * f.unsqueeze(1)).sum(2),
                 lambda g, x, f, p, c: (x.unsqueeze(2) * g.unsqueeze(1)).sum(3)]
        args = (g, xs, fs, p, c)
        for k, (form, terms) in enumerate(zip(forms, (S, S, H, H))):
            want, size = form(*args), form(*(a.abs() for a in args))
            # one fp32 rounding a term and one for its product
            over = (got[k][t0:t0 + 500].double() - want).abs() - (terms + 1) * 2.0 ** -24 * size
            assert over.max() <= 0, (k, t0, over.max().item())


# of the largest entry of a gradient: the same count of roundings as at the small sizes
# (n up to 57344: sqrt(n) * 2^-24 of the long sums and 170 * 2^-24 of the short part)
BWD_REL = 2.5e-5


@pytest.mark.parametrize("T,S,H", [(513, 1, 132), (520, 2, 516), (777, 3, 260), (1100, 4, 1028),
                                   (530, 5, 388), (540, 6, 132), (550, 7, 260), (600, 8, 1028),
                                   (2049, 4, 260), (1601, 4, 4096), (1031, 8, 2052), (512, 4, 4),
                                   (4097, 4, 4096), (4100, 3, 4100), (2100, 2, 16388),
                                   (1200, 1, 32772), (3001, 4, 7168), (17, 1, 4), (64, 4, 1028),
                                   (65, 4, 1028), (50, 2, 4100), (100, 5, 388), (97, 6, 132),
                                   (112, 7, 260), (128, 8, 1028), (16, 8, 4100), (90, 8, 516)])
@pytest.mark.parametrize("f8", [True, False])
def test_pre_bwd(mhc, T, S, H, f8):
    print(f"[case] pre_bwd T={T} S={S} H={H} f8={f8}", flush=True)
    d = _site(T, S, H, 3 * T + S)
    kx, x = _keep(mhc, d["x"], f8)
    args = (kx, d["w"], d["scale"], d["base"], 20, EPS, d["dy"], d["dpost"], d["dcomb"])
    got = mhc.site_pre_bwd(*args, dx_in=d["dx_in"])
    want = pf.pre_grads(x, d["w"], d["scale"], d["base"], 20, EPS, d["dy"], None, d["dpost"],
                        d["dcomb"], d["dx_in"])
    # dscale and dbase share their sums' terms: the size of dbase bounds both
    short = max(want[2].abs().max().item(), want[3].abs().max().item())
    for k, n in enumerate(("dx", "dfn_w", "dscale", "dbase")):
        assert torch.isfinite(got[k]).all(), n
        size = short if k >= 2 else want[k].abs().max().item()
        rel = (got[k].double() - want[k]).abs().max().item() / size
        assert rel <= BWD_REL, f"{n}: {rel:.3e} of the largest entry"
    for a, b in zip(got, mhc.site_pre_bwd(*args, dx_in=d["dx_in"])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("S", [1, 2])
def test_pre_bwd_reads_each_slice_of_dy(mhc, S):
    """Several slices of the hidden axis to a block, each with a dy of its own.  With
    x = 1, W = 0 and base = 0 every pre gate is 1/2 and dz = dy.x / 4; all sums are of whole
    numbers with a common factor and below 2^24 of it, so they are exact: 64 * (1 + .. + 64)
    a token and stream."""
    T, H = 4096, 4096
    print(f"[case] pre_bwd slices of dy S={S}", flush=True)
    x = mhc.f8_encode(torch.ones(T, S, H, device="cuda"))
    dy = (torch.arange(H, device="cuda") // 64 + 1).float().expand(T, H).contiguous()
    R = (2 + S) * S
    z = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    dx, _, _, dbase = mhc.site_pre_bwd(x, z(R, S * H), z(3) + 1, z(R), 20, EPS, dy, z(T, S),
                                       z(T, S, S))
    assert (dbase[:S] == T * 64 * 2080 / 4).all(), dbase[:S]
    assert torch.equal(dx, (dy / 2).unsqueeze(1).expand(T, S, H))


def test_pre_bwd_keeps_a_bad_token_to_itself(mhc):
    """A token with a NaN code, in one stream: every other token's gradient is what it
    is without it."""
    T, S, H = 700, 4, 516
    print(f"[case] pre_bwd NaN T={T}", flush=True)
    d = _site(T, S, H, 2)
    codes, scales = mhc.f8_encode(d["x"])

    def call(codes):
        return mhc.site_pre_bwd((codes, scales), d["w"], d["scale"], d["base"], 20, EPS,
                                d["dy"], d["dpost"], d["dcomb"])[0]

    want = call(codes)
    bad = codes.clone()
    bad.view(torch.uint8)[333, 2, 515] = 0x7f
    got = call(bad)
    assert torch.isnan(got[333]).any()
    rest = [t for t in range(T) if t != 333]
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("f8", [True, False])
def test_pre_bwd_at_the_widest_site(mhc, f8):
    """S * H = 2^24, where 32 tokens' rows are 2^31 bytes: offsets past 31 bits."""
    T, S, H = 35, 2, 1 << 23
    print(f"[case] pre_bwd T={T} S={S} H={H} f8={f8}", flush=True)
    d = _site(T, S, H, 1)
    kx, x = _keep(mhc, d["x"], f8)
    args = (d["w"], d["scale"], d["base"], 20, EPS, d["dy"], d["dpost"], d["dcomb"])
    got = mhc.site_pre_bwd(kx, *args)
    want = pf.pre_grads(x, *args[:6], None, *args[6:], None)
    short = max(want[2].abs().max().item(), want[3].abs().max().item())
    for k, n in enumerate(("dx", "dfn_w", "dscale", "dbase")):
        size = short if k >= 2 else want[k].abs().max().item()
        # sums of 2^24 terms: sqrt(n) * 2^-24 = 2.4e-4 in place of the 1.4e-5 of n = 57344
        rel = (got[k].double() - want[k]).abs().max().item() / size
        assert rel <= BWD_REL + 2.4e-4, f"{n}: {rel:.3e} of the largest entry"


def test_outputs_belong_to_the_stream_given(mhc):
    """A call on another stream must not get memory that pending work of the current
    stream still writes: a long product, then a fill of a block that is freed at once."""
    print("[case] outputs on a side stream", flush=True)
    x = _randn(1, 2048, 4, 512)
    g, f = _randn(2, 2048, 4, 512), _randn(3, 2048, 512)
    post, comb = _randn(4, 2048, 4), _randn(5, 2048, 4, 4)
    codes, scales = mhc.f8_encode(x)
    wc, ws = mhc.f8_encode(_randn(6, 512, 512), square=True)
    z = mhc.f8_encode(f)
    w = _randn(7, 24, 2048)
    small = _randn(8, 24)
    calls = [lambda **k: mhc.f8_encode(x, **k),
             lambda **k: (mhc.f8_decode(codes, scales, 512, **k),),
             lambda **k: mhc.f8_repack(codes.view(8192, 512), scales.view(8192, 4), 512, **k),
             lambda **k: (mhc.f8_matmul(*z, wc, ws, **k),),
             lambda **k: mhc.site_post_bwd(g, x, f, post, comb, **k),
             lambda **k: mhc.site_pre_bwd(x, w, small[:3], small, 20, EPS, f, post, comb, **k)]
    want = [[t.clone() for t in call()] for call in calls]
    side = torch.cuda.Stream()
    a = _randn(9, 8192, 8192)
    for how in (side, side.cuda_stream):
        for k, call in enumerate(calls):
            torch.cuda.synchronize()
            a @ a  # some milliseconds
            for t in want[k]:
                torch.empty_like(t).view(torch.uint8).fill_(0x55)
            got = call(stream=how)
            torch.cuda.synchronize()
            for p, q in zip(got, want[k]):
                assert torch.equal(p.view(torch.uint8), q.view(torch.uint8)), k
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError):
            calls[0](stream=torch.cuda.Stream(device=1))


# ------------------------------------------------------------------ past 32 bits
def _same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_encode_past_32_bits(mhc):
    """2.2e9 entries, 4.4 GB: the last rows and columns are what they are alone."""
    rows, cols, tail = 128 * 4219, 4096, 1280
    print(f"[case] encode {rows}x{cols}", flush=True)
    x = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    x.copy_(_randn(1, 1, cols))
    x[-tail:] = _randn(2, tail, cols).bfloat16()
    got = mhc.f8_encode(x, transposed=True)
    want = mhc.f8_encode(x[-tail:], transposed=True)
    assert _same(got[0][-tail:], want[0]) and _same(got[1][-tail:], want[1])
    assert _same(got[2][:, -tail:], want[2]) and _same(got[3][:, -tail // 128:], want[3])
    alone = mhc.f8_encode(x)
    assert _same(alone[0], got[0]) and _same(alone[1], got[1])
    again = mhc.f8_repack(got[0], got[1], cols)
    part = mhc.f8_repack(got[0][-tail:], got[1][-tail:], cols)
    assert _same(again[0][:, -tail:], part[0]) and _same(again[1][:, -tail // 128:], part[1])
    back = mhc.f8_decode(got[0], got[1], cols)
    assert _same(back[-tail:], mhc.f8_decode(got[0][-tail:], got[1][-tail:], cols))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_matmul_past_32_bits(mhc, M):
    """4.5e9 codes, as the weight and as the activations of a product."""
    N, K, tail = 1100004, 4096, 100
    print(f"[case] matmul {M}x{N}x{K}", flush=True)
    b = torch.empty(N, K, device="cuda", dtype=torch.bfloat16)
    b.copy_(_randn(1, 1, K))
    b[-tail:] = _randn(2, tail, K).bfloat16()
    eb, ea = mhc.f8_encode(b), mhc.f8_encode(_randn(3, M, K))
    va, vb = _decode(*ea, K), _decode(eb[0][-tail:], eb[1][-tail:], K)
    bound = K * 2.0 ** -23 * (va.abs() @ vb.abs().t())  # as above
    got = mhc.f8_matmul(*ea, *eb)[:, -tail:].double()
    assert ((got - va @ vb.t()).abs() <= bound).all()
    got = mhc.f8_matmul(*eb, *mhc.f8_encode(b[-64:], square=True))
    va, vb = vb, _decode(*mhc.f8_encode(b[-64:], square=True), K, True)
    bound = K * 2.0 ** -23 * (va.abs() @ vb.abs().t())
    assert ((got[-tail:].double() - va @ vb.t()).abs() <= bound).all()


@pytest.mark.parametrize("N", [1 << 29, (1 << 31) - 4])
def test_matmul_of_no_depth_for_very_many_columns(mhc, N):
    """More columns than one launch's threads: K = 0 needs nothing but the output."""
    print(f"[case] matmul 1x{N}x0", flush=True)
    e = lambda r, k, t: torch.empty(r, k, device="cuda", dtype=t)  # noqa: E731
    out = torch.full((1, N), 3.0, device="cuda", dtype=torch.bfloat16)
    mhc.f8_matmul(e(1, 0, torch.float8_e4m3fn), e(1, 0, torch.uint8),
                  e(N, 0, torch.float8_e4m3fn), e(N, 0, torch.uint8), out=out)
    assert not out.view(torch.int16).any()


@pytest.mark.parametrize("M", [1, 6, 40])
@pytest.mark.parametrize("square", [True, False])
def test_matmul_in_several_launches(mhc, M, square):
    """The columns next to a launch's last one, and the last of all."""
    edge, N, K = 1 << 24, (1 << 24) + 132, 128
    print(f"[case] matmul {M}x{N}x{K} square={square}", flush=True)
    b = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
    b[:] = _randn(1, 1, K)
    b[edge - 256:] = _randn(2, 388, K).bfloat16() * 2.0 ** (torch.arange(388, device="cuda") %
                                                            9).unsqueeze(1)
    eb, ea = mhc.f8_encode(b, square=square), mhc.f8_encode(_randn(3, M, K))
    at = (edge - 256) // (128 if square else 1)
    va, vb = _decode(*ea, K), _decode(eb[0][edge - 256:], eb[1][at:], K, square)
    bound = K * 2.0 ** -23 * (va.abs() @ vb.abs().t())  # as above
    out = torch.full((M + 1, N), 7.0, device="cuda")
    got = mhc.f8_matmul(*ea, *eb, out=out[:M])[:, edge - 256:].double()
    assert ((got - va @ vb.t()).abs() <= bound).all()
    assert (out[M] == 7.0).all(), "the row behind the last one was written"
    same = mhc.f8_matmul(*ea, eb[0][:64].contiguous(), eb[1][:1 if square else 64].contiguous())
    assert torch.allclose(out[:M, :64], same, rtol=0, atol=2 * bound.max().item())


@pytest.mark.parametrize("f8", [True, False])
def test_site_bwd_past_32_bits(mhc, f8):
    """8.5 GB of state: the last tokens' gradients are what they are alone."""
    T, S, H, tail = 65500, 8, 4096, 100
    print(f"[case] site backward T={T} S={S} H={H} f8={f8}", flush=True)
    assert 2 ** 31 > T * S * H > 2 ** 31 * 0.99
    d = _site(T, S, H, 5)
    post, comb = 2 * torch.sigmoid(d["dpost"]), torch.softmax(d["dcomb"], 2)
    kx, _ = _keep(mhc, d["x"], f8)
    kf, _ = _keep(mhc, d["f"], f8)
    cut = lambda k: tuple(t[-tail:] for t in k) if f8 else k[-tail:]  # noqa: E731
    got = mhc.site_post_bwd(d["g"], kx, kf, post, comb)
    want = mhc.site_post_bwd(d["g"][-tail:], cut(kx), cut(kf), post[-tail:], comb[-tail:])
    for p, q in zip(got, want):
        assert _same(p[-tail:], q)
    dx = got[0]
    del got, want
    weights = (d["w"], d["scale"], d["base"], 20, EPS)
    want = mhc.site_pre_bwd(cut(kx), *weights, d["dy"][-tail:], d["dpost"][-tail:],
                            d["dcomb"][-tail:], dx_in=dx[-tail:])
    half = T // 2 + 7  # the sums over tokens, in two calls
    cuts = (slice(0, half), slice(half, T))
    parts = [mhc.site_pre_bwd(tuple(t[c] for t in kx) if f8 else kx[c], *weights, d["dy"][c],
                              d["dpost"][c], d["dcomb"][c])[1:] for c in cuts]
    got = mhc.site_pre_bwd(kx, *weights, d["dy"], d["dpost"], d["dcomb"], dx_in=dx, out=(
        dx, *(torch.empty_like(t) for t in parts[0])))
    # the dots' and the token sums' order differs with T: each side is within BWD_REL
    size = want[0].abs().max()
    assert (got[0][-tail:] - want[0]).abs().max() <= 2 * BWD_REL * size
    short = max((parts[0][k] + parts[1][k]).abs().max() for k in (1, 2))
    for k in range(3):
        both = parts[0][k].double() + parts[1][k].double()
        size = both.abs().max() if k == 0 else short
        assert (got[1 + k].double() - both).abs().max() <= 3 * BWD_REL * size, k
