"""4-bit groups on the GPU: encoding, values, and the product, against 64-bit forms."""
import numpy as np
import pytest

import branch_forms as bf
from branch_forms import ULP

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _hard_weight(N, K, seed):
    """Rows of several sizes, zero groups, ties, ends, infinities and NaN."""
    g = np.random.default_rng(seed)
    w = (g.standard_normal((N, K)) * 2.0 ** g.integers(-30, 30, (N, 1))).astype(np.float32)
    if N > 1:
        w[N // 2] = 0
    w[0] = np.round(w[0] / np.abs(w[0]).max() * 14) / 2  # halves: ties of a scale of one
    w[0, ::32] = 7
    if N > 4:
        w[1] = np.abs(w[1])
        w[2, 3], w[2, 17], w[2, 30] = np.nan, np.inf, -np.inf
        w[3] = 1e-40
        w[4] = 3.3e38 * np.sign(w[4])
    return w


@pytest.mark.parametrize("N,K", [(1, 32), (6, 96), (9, 160), (7, 1056), (64, 4096)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("bf16", [False, True])
def test_encode_and_decode(mhc, N, K, group, zeros, bf16):
    print(f"[case] encode N={N} K={K} G={group} zeros={zeros} bf16={bf16}", flush=True)
    w = torch.from_numpy(_hard_weight(N, K, N + K))
    if bf16:
        w = w.bfloat16()
    kept = mhc.q4_encode(w.cuda(), group=group, zeros=zeros)
    assert len(kept) == 3 if zeros else 2
    c, d, z = bf.encode(w.float().numpy(), group, zeros)
    np.testing.assert_array_equal(kept[1].float().cpu().numpy(), d)
    if zeros:
        np.testing.assert_array_equal(kept[2].cpu().numpy(), z)
    np.testing.assert_array_equal(bf.unpack(kept[0].cpu().numpy(), K), c)
    np.testing.assert_array_equal(kept[0].cpu().numpy(), bf.pack(c))  # padding is zero
    got = mhc.q4_decode(*kept, cols=K).double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = bf.decode(c, d, z if zeros else None, group).astype(np.float32)
    np.testing.assert_array_equal(got, want)


def test_encode_is_within_half_a_scale(mhc):
    """... and, at the ends of a range whose scale was rounded down, 2^-9 of the range."""
    print("[case] encode error", flush=True)
    g = torch.Generator().manual_seed(1)
    w = torch.randn(50, 512, generator=g)
    for group in (32, 64, 128):
        for zeros in (False, True):
            kept = mhc.q4_encode(w.cuda(), group=group, zeros=zeros)
            d = kept[1].float().cpu().repeat_interleave(group, 1)
            off = (mhc.q4_decode(*kept, cols=512).cpu() - w).abs()
            # the zero point is rounded as well: another half scale at the ends
            assert (off <= d * ((1.0 if zeros else 0.5) + 15 * 2.0 ** -9 + 1e-5)).all()


def _weight(N, K, group, zeros, f16, seed):
    """A weight's tensors on the GPU and its float64 values; scales over a wide range."""
    g = np.random.default_rng(seed)
    c = g.integers(0, 16, (N, K)).astype(np.uint8)
    kg = -(-K // group)
    d = torch.from_numpy((2.0 ** g.uniform(-8, -2, (N, kg))).astype(np.float32))
    d = d.half() if f16 else d.bfloat16()
    z = g.integers(0, 16, (N, kg)).astype(np.uint8) if zeros else None
    kept = (torch.from_numpy(bf.pack(c)).cuda(), d.cuda(),
            None if z is None else torch.from_numpy(z).cuda())
    w = bf.decode(c, d.float().numpy(), z, group)
    at = np.arange(K) // group
    # the sizes that are summed: code and zero point times the scale
    size = (c + (8.0 if z is None else z[:, at])) * d.double().numpy()[:, at]
    return kept, torch.from_numpy(w), torch.from_numpy(size)


def _act(M, K, kind, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn(M, K, generator=g) * (1 + 20 * (torch.rand(K, generator=g) > 0.97))
    if kind == "q8":
        d = a.view(M, -1, 32).abs().amax(2) / 127
        q = torch.round(a.view(M, -1, 32) / d.unsqueeze(2)).clamp(-127, 127).to(torch.int8)
        v = (q.double() * d.double().unsqueeze(2)).view(M, K)
        return (q.view(M, K).cuda(), d.cuda()), v
    a = a.bfloat16() if kind == "bf16" else a
    return a.cuda(), a.double()


SHAPES = [(1, 1, 32), (1, 16, 32), (2, 5, 96), (1, 100, 4096), (3, 33, 160), (8, 130, 1056),
          (1, 4099, 256), (5, 9000, 64), (16, 33, 128), (17, 64, 256), (40, 70, 384),
          (64, 129, 2080), (100, 257, 512), (333, 48, 1024), (130, 520, 224), (1, 64, 16384),
          (2, 8200, 512), (7, 16400, 128), (300, 700, 96), (65, 4100, 128),
          # one row: more rows of the weight than one turn of the waves, more depth than theirs
          (1, 30000, 64), (1, 70, 20000),
          # up to 16 rows: each width of a block, several stages and a short last one
          (4, 6000, 2080), (3, 16400, 2208), (9, 5000, 4128), (16, 8200, 1056), (16, 16390, 1120),
          # each tile: 32 x 128, 64 x 128, 32 x 128 past one round, 128 x 128, 96 x 128 (bf16)
          (40, 9000, 160), (120, 16000, 416), (130, 20000, 288), (128, 32700, 96),
          (90, 30000, 416)]


def _bound(kind, K, group, a, size, w):
    """Products are exact.  A matrix instruction adds 32 of them to its sum with at most 33
    roundings, a group has group/32 of them for each plane of a; the group's two sums are put
    together in 2 and added to the others in K/group more and one for each of 16 waves.  int8
    blocks of up to 16 rows are exact: one rounding a block, then as above; past that their
    values are rounded once and then go as fp32 does."""
    planes = 1 if kind == "bf16" else 3
    kg = -(-K // group)
    if kind == "q8" and a.shape[0] <= 16:
        return (group // 32 + 3 + kg + 18) * ULP * (a.abs() @ w.abs().t())
    n = 33 * group // 32 * planes + 5 + kg + 18
    return n * ULP * (a.abs() @ size.t())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("group,zeros,f16", [(128, False, False), (64, True, True),
                                             (32, True, False)])
def test_product(mhc, M, N, K, kind, group, zeros, f16):
    print(f"[case] product M={M} N={N} K={K} {kind} G={group} z={zeros} f16={f16}", flush=True)
    kept, w, size = _weight(N, K, group, zeros, f16, N + K)
    a, av = _act(M, K, kind, M + K)
    want = av @ w.t()
    bound = _bound(kind, K, group, av, size, w)
    got = mhc.q4_matmul(a, *kept).double().cpu()
    assert got.shape == (M, N) and torch.isfinite(got).all()
    assert ((got - want).abs() - bound).max() <= 0
    low = mhc.q4_matmul(a, *kept, dtype=torch.bfloat16)
    assert low.dtype == torch.bfloat16
    assert torch.equal(low.float().cpu(), got.float().bfloat16().float())


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
def test_whole_numbers_are_exact(mhc, M, N, K, kind):
    """Small integers and one power-of-two scale a row: every sum is an integer below 2^24
    times that scale (15 * 3 * 16384 < 2^20), so every rounding is exact."""
    print(f"[case] whole M={M} N={N} K={K} {kind}", flush=True)
    g = np.random.default_rng(K + N)
    c = g.integers(0, 16, (N, K)).astype(np.uint8)
    a = g.integers(-3, 4, (M, K)).astype(np.float32)
    for group in (32, 64, 128):
        kg = -(-K // group)
        d = np.repeat(2.0 ** g.integers(-3, 4, (N, 1)), kg, 1).astype(np.float32)
        z = g.integers(0, 16, (N, kg)).astype(np.uint8)
        t = torch.from_numpy(a).cuda()
        if kind == "bf16":
            t = t.bfloat16()
        elif kind == "q8":
            t = t.to(torch.int8), torch.ones(M, K // 32, device="cuda")
        for zeros in (z, None):
            got = mhc.q4_matmul(t, torch.from_numpy(bf.pack(c)).cuda(),
                                torch.from_numpy(d).half().cuda(),
                                None if zeros is None else torch.from_numpy(z).cuda())
            want = a.astype(np.float64) @ bf.decode(c, d, zeros, group).T
            np.testing.assert_array_equal(got.double().cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("M", [1, 4, 12, 40])
@pytest.mark.parametrize("ea,es", [(-110, 120), (-100, 127), (100, -126)])
def test_scales_at_the_ends_of_their_range(mhc, kind, M, ea, es):
    """Whole numbers times powers of two: exact in any order."""
    print(f"[case] q4_matmul M={M} {kind} a 2^{ea} scales 2^{es}", flush=True)
    g = np.random.default_rng(M)
    c = g.integers(0, 16, (70, 256)).astype(np.uint8)
    c[3], c[5, 64:128] = 8, 8  # a group, and a row, of zeros
    n = g.integers(-4, 5, (M, 256)).astype(np.float32)
    scales = torch.full((70, 4), 2.0 ** es, dtype=torch.bfloat16).cuda()
    v = torch.from_numpy(n)
    a = (v.to(torch.int8).cuda(), torch.full((M, 8), 2.0 ** ea).cuda()) if kind == "q8" else \
        (v * 2.0 ** ea).to(torch.bfloat16 if kind == "bf16" else torch.float32).cuda()
    got = mhc.q4_matmul(a, torch.from_numpy(bf.pack(c)).cuda(), scales).double().cpu()
    want = torch.from_numpy(n.astype(np.float64) @ (c.astype(np.float64) - 8).T)
    assert torch.equal(got, want * 2.0 ** (ea + es))


def test_one_column_at_a_time(mhc):
    """A unit activation picks a weight's column: every column's place and group."""
    print("[case] columns", flush=True)
    for N, K, group in ((20, 288, 64), (33, 160, 32), (17, 416, 128)):
        kept, w, _ = _weight(N, K, group, True, False, 5)
        eye = torch.eye(K)
        got = mhc.q4_matmul(eye.cuda(), *kept).double().cpu()
        assert torch.equal(got, w.t())
        one = torch.stack([mhc.q4_matmul(eye[k:k + 1].cuda(), *kept)[0] for k in range(0, K, 7)])
        assert torch.equal(one.double().cpu(), w.t()[::7])


@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("M", [1, 2, 5, 16, 40, 200])
def test_a_bad_row_keeps_to_itself(mhc, kind, M):
    """A row with an infinity or a NaN, also in the last, short block of the depth."""
    print(f"[case] bad row {kind} M={M}", flush=True)
    N, K = 70, 288
    kept, _, _ = _weight(N, K, 64, True, False, 3)
    a, _ = _act(M, K, kind, 4)
    want = mhc.q4_matmul(a, *kept)
    for bad in (float("nan"), float("inf"), float("-inf")):
        for k in (0, 100, K - 1):
            m = M // 2
            b = (a[0], a[1].clone()) if kind == "q8" else a.clone()
            if kind == "q8":
                b[1][m, k // 32] = bad
            else:
                b[m, k] = bad
            got = mhc.q4_matmul(b, *kept)
            rest = [i for i in range(M) if i != m]
            assert torch.equal(got[rest], want[rest])
            assert not torch.isfinite(got[m]).any() if kind != "q8" else \
                not torch.isfinite(got[m]).all()


def test_sizes_of_activations(mhc):
    """fp32 values over the whole range of exponents whose products stay in range."""
    print("[case] sizes", flush=True)
    N, K = 48, 256
    kept, w, size = _weight(N, K, 128, True, False, 6)
    g = torch.Generator().manual_seed(7)
    for M in (1, 6, 40):
        a = torch.randn(M, K, generator=g) * 2.0 ** torch.randint(-90, 90, (M, 1), generator=g)
        av = a.double()
        got = mhc.q4_matmul(a.cuda(), *kept).double().cpu()
        assert ((got - av @ w.t()).abs() - _bound("f32", K, 128, av, size, w)).max() <= 0


def test_calls(mhc):
    """Streams by handle, given outputs, refusals, no tokens."""
    print("[case] calls", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn(70, 160, generator=g, device="cuda")
    kept = mhc.q4_encode(w, group=64, zeros=True)
    a = torch.randn(5, 160, generator=g, device="cuda")
    calls = [lambda **k: mhc.q4_encode(w, group=64, zeros=True, **k),
             lambda **k: mhc.q4_decode(*kept, cols=160, **k),
             lambda **k: mhc.q4_matmul(a, *kept, **k)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for call in calls:
        want = call()
        tup = isinstance(want, tuple)
        for how in (0, side, side.cuda_stream, torch.cuda.default_stream()):
            got = call(stream=how)
            torch.cuda.synchronize()
            assert all(map(torch.equal, got if tup else [got], want if tup else [want]))
        out = tuple(torch.zeros_like(t) for t in want) if tup else torch.zeros_like(want)
        got = call(out=out)
        assert all(map(torch.equal, got if tup else [got], want if tup else [want]))
        assert got is out or tup
    low = torch.empty(5, 70, device="cuda", dtype=torch.bfloat16)
    assert mhc.q4_matmul(a, *kept, out=low) is low
    assert torch.equal(low, mhc.q4_matmul(a, *kept).bfloat16())
    assert mhc.q4_matmul(a[:0], *kept).shape == (0, 70)
    with pytest.raises(ValueError, match="contiguous"):
        mhc.q4_matmul(a.t().contiguous().t(), *kept)
    with pytest.raises(ValueError, match="groups"):
        mhc.q4_matmul(a[:, :128].contiguous(), *kept)
    with pytest.raises(ValueError, match="zeros"):
        mhc.q4_matmul(a, kept[0], kept[1], kept[2][:, :1].contiguous())
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        mhc.q4_matmul(a.half(), *kept)
    with pytest.raises(ValueError, match="d has shape"):
        mhc.q4_matmul((a.to(torch.int8), torch.ones(5, 4, device="cuda")), *kept)
    with pytest.raises(mhc.MhcError, match="EOVERLAP"):
        b = torch.zeros(160, 160, device="cuda")
        mhc.q4_matmul(b, *mhc.q4_encode(torch.ones(160, 160, device="cuda")), out=b)
    with pytest.raises(ValueError, match="multiple of 32"):
        mhc.q4_matmul(torch.zeros(2, 100, device="cuda"), *kept)
    with pytest.raises(mhc.MhcError, match="EALIGN"):
        mhc.q4_encode(torch.zeros(2, 100, device="cuda"))


@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("M", [1, 3, 16, 50, 300])
def test_repeatable_and_captured(mhc, kind, M):
    print(f"[case] graph {kind} M={M}", flush=True)
    kept, _, _ = _weight(1000, 544, 32, True, True, 3)
    a, _ = _act(M, 544, kind, 1)
    out = torch.empty(M, 1000, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mhc.q4_matmul(a, *kept, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        mhc.q4_matmul(a, *kept, out=out)
    for rep in range(3):
        new, _ = _act(M, 544, kind, 2 + rep)
        for t, n in zip(a if kind == "q8" else [a], new if kind == "q8" else [new]):
            t.copy_(n)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mhc.q4_matmul(a, *kept))


def test_past_32_bits(mhc):
    """Codes, scales and outputs at byte offsets past 2^32."""
    print("[case] large", flush=True)
    N, K, n = 140000, 65536, 37
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.rand(N, K // 128, device="cuda").bfloat16()
    end = (codes[-n:].clone(), scales[-n:].clone())
    for M in (1, 2, 6, 30):
        a = torch.randn(M, K, device="cuda").bfloat16()
        got, want = mhc.q4_matmul(a, codes, scales)[:, -n:], mhc.q4_matmul(a, *end)
        # another number of rows may take another split of the sum
        assert (got - want).abs().max() <= 1e-4 * want.abs().max()
    del codes, scales
    N, K = 520000, 64
    kept = mhc.q4_encode(torch.randn(N, K, device="cuda"), group=32)
    a = torch.randn(2100, K, device="cuda").bfloat16()
    got = mhc.q4_matmul(a, *kept)[-3:, -n:]
    want = mhc.q4_matmul(a[-3:].clone(), kept[0][-n:].clone(), kept[1][-n:].clone())
    assert (got - want).abs().max() <= 1e-4 * want.abs().max()


@pytest.mark.parametrize("T", [1, 4, 37])
def test_a_decode_site(mhc, T):
    """The calls in a row, as a decoding site makes them: pre half with the int8 epilogue,
    two products, the norm behind the branch and the post mix."""
    print(f"[case] site T={T}", flush=True)
    S, H, F = 4, 512, 1536
    g = torch.Generator(device="cuda").manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    R, n = (2 + S) * S, S * H
    x, fn_w, scale, base = r(T, S, H), r(R, n) / n ** 0.5, 0.5 + r(3).abs(), 0.3 * r(R)
    nw, nw2, gate = 1 + 0.2 * r(H), 1 + 0.2 * r(H), r(H)
    up, down = mhc.q4_encode(r(F, H) / H ** 0.5), mhc.q4_encode(r(H, F) / F ** 0.5, group=32,
                                                              zeros=True)
    pre, post, comb, y, z, q, d = mhc.site_pre_zq8(x, fn_w, scale, base, nw, 20, 1e-6)
    u = mhc.q4_matmul((q, d), *up)
    v = torch.nn.functional.silu(u).bfloat16()
    f = mhc.q4_matmul(v, *down, dtype=torch.bfloat16)
    out = mhc.site_post_norm(x, f, nw2, post, comb, 1e-5, gate=gate, gate_act="sigmoid",
                             alpha=0.5)
    c = lambda t: t.double().cpu()  # noqa: E731
    want_u = (c(q).view(T, -1, 32) * c(d).unsqueeze(2)).view(T, H) @ c(
        mhc.q4_decode(*up, cols=H)).t()
    assert (c(u) - want_u).abs().max() <= 1e-5 * want_u.abs().max()
    want_f = c(v) @ c(mhc.q4_decode(*down, cols=F)).t()
    assert (c(f) - want_f).abs().max() <= (2.0 ** -8 + 1e-5) * want_f.abs().max()
    want, size = bf.site_post_norm(c(x), c(f), c(nw2), c(post), c(comb), 1e-5, c(gate),
                                   "sigmoid", 0.5)
    assert ((c(out) - want).abs() - 60 * ULP * size).max() <= 0


def test_a_training_site(mhc):
    """... and as training does: norm, 8-bit products, norm behind, and the way back."""
    print("[case] training site", flush=True)
    T, S, H = 200, 4, 512
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    R, n = (2 + S) * S, S * H
    x, fn_w, scale, base = r(T, S, H), r(R, n) / n ** 0.5, 0.5 + r(3).abs(), 0.3 * r(R)
    nw, nw2, gate, G = 1 + 0.2 * r(H), 1 + 0.2 * r(H), r(T, H), r(T, S, H)
    wc, ws, wct, wst = mhc.f8_encode(r(H, H) / H ** 0.5, transposed=True, square=True)
    pre, post, comb, y = mhc.site_pre(x, fn_w, scale, base, 20, 1e-6)
    z = mhc.branch_norm(y, nw, 1e-5, dtype=torch.bfloat16)
    kz = mhc.f8_encode(z)
    f = mhc.f8_matmul(*kz, wc, ws, dtype=torch.bfloat16)
    how = dict(gate=gate, gate_act="silu", alpha=0.5)
    out = mhc.site_post_norm(x, f, nw2, post, comb, 1e-5, **how)
    dx, df, dpost, dcomb, dnw2, dgate = mhc.site_post_norm_bwd(G, x, f, nw2, post, comb, 1e-5,
                                                               **how)
    dz = mhc.f8_matmul(*mhc.f8_encode(df), wct, wst)
    dy, dnw = mhc.branch_norm_bwd(dz, y, nw, 1e-5)
    grads = mhc.site_pre_bwd(x, fn_w, scale, base, 20, 1e-6, dy, dpost, dcomb, dx_in=dx)
    # the same in float64 by automatic differentiation, z and f taking the values that the
    # 8-bit blocks and bf16 gave them (their rounding has slope one)
    import plain_forms as pf
    c = lambda t: t.double().cpu()  # noqa: E731
    as_kept = lambda v, kept: v + (c(kept) - v).detach()  # noqa: E731
    leaves = [c(t).requires_grad_() for t in (x, fn_w, scale, base, nw, nw2, gate)]
    X, W, sc, ba, n1, n2, ga = leaves
    _, p64, c64, y64 = pf.site_pre(X, W, sc, ba, 20, float(np.float32(1e-6)))
    z64 = as_kept(bf.branch(y64, n1, 1e-5), mhc.f8_decode(*kz, H))
    w64 = c(mhc.f8_decode(wct, wst.repeat_interleave(128, 0)[:H].contiguous(), H)).t()
    f64 = as_kept(z64 @ w64.t(), f)
    h64 = bf.branch(f64, n2, 1e-5, ga, "silu", 0.5)
    o64 = pf.site_post(X, h64, p64, c64)
    assert (c(out) - o64).abs().max() <= 1e-4 * o64.abs().max()
    o64.backward(c(G))
    # df was rounded to 8 bits on its way (2^-4 of an entry at most, and a random weight
    # stretches no direction more than twice its mean): what goes through dz is good to 2^-3
    for name, got, leaf, tol in zip(
            ("dx", "dfn_w", "dscale", "dbase", "dnw", "dnw2", "dgate"),
            (*grads, dnw, dnw2, dgate), leaves, (2 ** -3,) * 5 + (1e-4,) * 2):
        rel = (c(got) - leaf.grad).norm() / leaf.grad.norm()
        assert rel <= tol, (name, rel.item())
