"""8-bit blocks and their product on the GPU, against plain 64-bit forms."""
import numpy as np
import pytest

import plain_forms as pf

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _values(rows, cols, seed):
    """Values over many binades, rows of zeros and of subnormals, block maxima at and
    next to 448 * 2^e, ties between codes."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * 2.0 ** g.integers(-30, 30, (rows, 1))
    x *= 2.0 ** g.integers(-8, 1, (rows, cols))
    x = x.astype(np.float32)
    for r in range(0, rows, 7):
        x[r] = 0.0
    for r in range(1, rows, 11):
        x[r] = g.choice(np.array([448, 449, 447.99997, 464, 17, 19, 2.0 ** -7, 3 * 2.0 ** -10, 1e-30],
                                 np.float32), cols) * np.float32(2.0 ** (r % 5))
    for r in range(3, rows, 13):
        x[r] = x[r] * np.float32(1e-44)
    for r in range(5, rows, 17):
        x[r] = np.float32(3.4e38) * g.choice(np.array([1, -1, 0.5, 1e-6], np.float32), cols)
    return x


def _bytes(t):
    return t.view(torch.uint8).cpu().numpy()


def _check_codes(got, want, name):
    got, want = _bytes(got), np.asarray(want)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    nan = (want & 0x7f) == 0x7f
    assert np.array_equal((got & 0x7f) == 0x7f, nan), f"{name}: NaN codes"
    bad = np.argwhere((got != want) & ~nan)
    assert bad.size == 0, f"{name}: {len(bad)} codes differ, first at {bad[0]}"


SHAPES = [(1, 4), (1, 128), (3, 132), (2, 4096), (33, 260), (128, 128), (129, 516), (300, 1028),
          (1, 7168), (127, 4)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_encode_equals_the_definition(mhc, rows, cols, dtype):
    print(f"[case] encode {rows}x{cols} {dtype}", flush=True)
    x = torch.from_numpy(_values(rows, cols, rows + cols)).to(getattr(torch, dtype))
    x64 = x.double().numpy()
    with np.errstate(invalid="ignore"):
        x64 = np.where(np.isfinite(x64), x64, x64)
    want, wt = pf.encode(x64), pf.encode(x64.T)
    sq, sqt = pf.encode(x64, square=True), pf.encode(x64.T, square=True)
    xd = x.cuda()
    for tr in (False, True, "only"):
        got = mhc.f8_encode(xd, transposed=tr)
        parts = (want if tr != "only" else ()) + (wt if tr else ())
        assert len(got) == len(parts)
        for k, (a, b) in enumerate(zip(got, parts)):
            (_check_codes if k % 2 == 0 else
             lambda a, b, n: np.testing.assert_array_equal(_bytes(a), b, n))(a, b, f"{tr} {k}")
    got = mhc.f8_encode(xd, transposed=True, square=True)
    for k, (a, b) in enumerate(zip(got, sq + sqt)):
        (_check_codes if k % 2 == 0 else
         lambda a, b, n: np.testing.assert_array_equal(_bytes(a), b, n))(a, b, f"square {k}")
    only = mhc.f8_encode(xd, square=True)
    assert torch.equal(only[0].view(torch.uint8), got[0].view(torch.uint8))
    assert torch.equal(only[1], got[1])
    assert torch.equal(got[2][:, :rows].view(torch.uint8).t(), got[0][:, :cols].view(torch.uint8))


def test_every_code_round_trips_and_infinities_are_nan(mhc):
    print("[case] every code, infinities", flush=True)
    x = np.zeros((4, 128), np.float32)
    x[0, :127], x[1, :127] = pf.E4M3, -pf.E4M3
    x[2, :5] = [np.inf, -np.inf, np.nan, 1.0, -448.0]
    x[3] = np.inf
    codes, scales = mhc.f8_encode(torch.from_numpy(x).cuda())
    assert scales.flatten().tolist() == [127, 127, 127, 127]
    assert np.array_equal(_bytes(codes)[0, :127], np.arange(127))
    assert np.array_equal(_bytes(codes)[1, 1:127], np.arange(129, 255))
    back = mhc.f8_decode(codes, scales, 128).cpu().numpy()
    np.testing.assert_array_equal(back[:2], x[:2])
    assert np.isnan(back[2, :3]).all() and back[2, 3] == 1 and back[2, 4] == -448
    assert np.isnan(back[3]).all()


@pytest.mark.parametrize("rows,cols", [(5, 260), (130, 132), (300, 516)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_encode_of_infinities_and_nan(mhc, rows, cols, dtype):
    """In every form: single entries, a whole row and column, and a whole 128 x 128 square
    without a finite entry (scale 2^0, every code NaN)."""
    print(f"[case] encode non-finite {rows}x{cols} {dtype}", flush=True)
    g = np.random.default_rng(rows)
    bad = np.array([np.inf, -np.inf, np.nan])
    x = g.standard_normal((rows, cols)) * 2.0 ** g.integers(-20, 20, (rows, 1))
    x[g.random((rows, cols)) < 0.02] = np.inf
    x[g.random((rows, cols)) < 0.02] = np.nan
    x[3] = g.choice(bad, cols)
    x[:, 2] = g.choice(bad, rows)
    x[:, cols - 1] = -np.inf
    x[128:256, 128:256] = g.choice(bad, x[128:256, 128:256].shape)
    x[256:, :128] = g.choice(bad, x[256:, :128].shape)
    xd = torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype)).cuda()
    x = xd.double().cpu().numpy()
    assert np.isinf(x).any() and np.isnan(x).any()
    rows_form, cols_form = pf.encode(x), pf.encode(x.T)
    square = pf.encode(x, square=True) + pf.encode(x.T, square=True)
    got = [mhc.f8_encode(xd) + mhc.f8_encode(xd, transposed="only"),
           mhc.f8_encode(xd, transposed=True), mhc.f8_encode(xd, transposed=True, square=True)]
    for have, want in zip(got, (rows_form + cols_form, rows_form + cols_form, square)):
        for k in (0, 2):
            _check_codes(have[k], want[k], f"codes {k}")
            np.testing.assert_array_equal(_bytes(have[k + 1]), want[k + 1])
    values = pf.decode(*rows_form, cols)
    np.testing.assert_array_equal(mhc.f8_decode(*got[0][:2], cols).double().cpu().numpy(), values)
    again, want = mhc.f8_repack(*got[0][:2], cols), pf.encode(values.T)
    _check_codes(again[0], want[0], "repack")
    np.testing.assert_array_equal(_bytes(again[1]), want[1])


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_decode_and_repack(mhc, rows, cols):
    print(f"[case] decode, repack {rows}x{cols}", flush=True)
    x = _values(rows, cols, 7 * rows + cols)
    codes, scales = pf.encode(x)
    values = pf.decode(codes, scales, cols)
    c, s = torch.from_numpy(codes).cuda().view(F8), torch.from_numpy(scales).cuda()
    np.testing.assert_array_equal(mhc.f8_decode(c, s, cols).double().cpu().numpy(), values)
    got = mhc.f8_repack(c, s, cols)
    want = pf.encode(values.T)
    _check_codes(got[0], want[0], "repack")
    np.testing.assert_array_equal(_bytes(got[1]), want[1])


def test_encode_of_a_state_keeps_its_shape(mhc):
    print("[case] encode [T, S, H]", flush=True)
    x = torch.randn(5, 3, 260, device="cuda")
    codes, scales = mhc.f8_encode(x)
    assert codes.shape == (5, 3, 384) and scales.shape == (5, 3, 3)
    flat = mhc.f8_encode(x.view(15, 260))
    assert torch.equal(flat[0].view(torch.uint8), codes.view(15, 384).view(torch.uint8))
    assert torch.equal(flat[1], scales.view(15, 3))
    assert mhc.f8_decode(codes, scales, 260).shape == (5, 3, 260)
    empty = mhc.f8_encode(x[:0], transposed=True)
    assert empty[0].shape == (0, 3, 384) and empty[2].shape == (260, 0)


# ------------------------------------------------------------------ product
def _operands(M, N, K, square, seed):
    g = np.random.default_rng(seed)
    a = g.standard_normal((M, K)) * 2.0 ** g.integers(-12, 12, (M, 1))
    b = g.standard_normal((N, K)) * 2.0 ** g.integers(-6, 6, (1, K))
    if M > 2:
        a[1] = 0
    a, b = a.astype(np.float32), b.astype(np.float32)
    ea, eb = pf.encode(a), pf.encode(b, square=square)
    return ea, eb, pf.decode(*ea, K), pf.decode(*eb, K, square=square)


def _on_gpu(codes, scales):
    return torch.from_numpy(codes).cuda().view(F8), torch.from_numpy(scales).cuda()


# products of codes have 8 significant bits and are exact in fp32.  K of them are
# added in fp32, each addition off by at most one unit in the last place (2^-23
# relative, a truncating adder included) of a partial sum that is at most the sum
# of magnitudes; bf16 results are rounded once more, by at most 2^-8 (half of
# torch.finfo(bfloat16).eps) of their value.
def _check_product(out, a, b, name):
    want = a @ b.T
    bound = a.shape[1] * 2.0 ** -23 * (np.abs(a) @ np.abs(b).T)
    got = out.double().cpu().numpy()
    if out.dtype == torch.bfloat16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    finite = bool(np.isfinite(got).all())
    assert got.shape == want.shape and finite, name
    worst = float((np.abs(got - want) - bound).max(initial=-1))
    assert worst <= 0, f"{name}: {worst} past the bound"


MKN = [(1, 128, 4), (1, 4096, 512), (2, 256, 36), (16, 1024, 100), (17, 384, 260), (33, 512, 132),
       (64, 128, 64), (65, 896, 68), (100, 2048, 516), (129, 256, 1028), (255, 384, 260),
       (256, 512, 256), (257, 640, 772), (300, 1152, 300), (520, 256, 4), (1030, 384, 516)]


@pytest.mark.parametrize("M,K,N", MKN)
@pytest.mark.parametrize("square", [True, False])
def test_matmul_within_the_bound(mhc, M, K, N, square):
    print(f"[case] matmul {M}x{N}x{K} square={square}", flush=True)
    ea, eb, a, b = _operands(M, N, K, square, M + N + K)
    ga, gb = _on_gpu(*ea), _on_gpu(*eb)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.full((M + 1, N), 7.0, device="cuda", dtype=dtype)
        got = mhc.f8_matmul(*ga, *gb, out=out[:M])
        _check_product(got, a, b, str(dtype))
        assert (out[M] == 7.0).all(), "the row behind the last one was written"
        again = mhc.f8_matmul(*ga, *gb, dtype=dtype)
        assert torch.equal(got, again)


def test_matmul_of_nothing(mhc):
    print("[case] matmul K = 0, M = 0", flush=True)
    e = lambda *s: torch.empty(s, device="cuda", dtype=F8)  # noqa: E731
    u = lambda *s: torch.empty(s, device="cuda", dtype=torch.uint8)  # noqa: E731
    out = torch.full((5, 8), 3.0, device="cuda")
    mhc.f8_matmul(e(5, 0), u(5, 0), e(8, 0), u(8, 0), out=out)
    assert (out == 0).all()
    assert mhc.f8_matmul(e(0, 128), u(0, 1), e(8, 128), u(8, 1)).shape == (0, 8)


@pytest.mark.parametrize("M", [3, 300])
def test_matmul_keeps_nan_to_its_row(mhc, M):
    print(f"[case] matmul NaN M={M}", flush=True)
    ea, eb, a, b = _operands(M, 132, 256, True, 5)
    ea[0][2, 200] = 0x7f
    got = mhc.f8_matmul(*_on_gpu(*ea), *_on_gpu(*eb))
    assert torch.isnan(got[2]).all()
    keep = [i for i in range(M) if i != 2]
    _check_product(got[keep], a[keep], b, "the other rows")


@pytest.mark.parametrize("M", [1, 5, 24, 40, 300])
@pytest.mark.parametrize("K", [128, 384, 2176, 4224])
def test_matmul_of_an_infinite_value(mhc, M, K):
    """An entry above 248 * 2^120 decodes to an infinity (include/mhc.h): its row of the
    product is that infinity with the sign of the other operand, wherever it stands."""
    print(f"[case] matmul infinity M={M} K={K}", flush=True)
    N = 20
    for at in (3, K - 1):
        a, b = torch.zeros(M, K), torch.ones(N, K)
        a[0, at] = 3.4e38
        b[1::2] = -1.0
        for flip in (False, True):
            got = mhc.f8_matmul(*mhc.f8_encode(a.cuda()), *mhc.f8_encode(b.cuda())).cpu()
            want = torch.zeros(M, N)
            want[0, 0::2], want[0, 1::2] = float("inf"), float("-inf")
            assert torch.equal(got, want), (at, flip)
            a[0, 0] = 1.0  # and beside other entries
    ea, eb = mhc.f8_encode(b.cuda()), mhc.f8_encode(torch.cat([a, torch.zeros(4, K)]).cuda())
    got = mhc.f8_matmul(*ea, eb[0][:M - M % 4 + 4].contiguous(), eb[1][:M - M % 4 + 4].contiguous())
    assert torch.isinf(got[:, 0]).all() and not got[:, 1:].any()


@pytest.mark.parametrize("M", [4, 40, 300])
def test_matmul_at_the_ends_of_the_scales(mhc, M):
    """Scale bytes 1 and 247: products near the least and the largest fp32."""
    print(f"[case] matmul extreme scales M={M}", flush=True)
    ea, eb, a, b = _operands(M, 132, 256, True, 6)
    for byte_a, byte_b in ((1, 247), (247, 1), (1, 120), (240, 127)):
        sa, sb = np.full_like(ea[1], byte_a), np.full_like(eb[1], byte_b)
        got = mhc.f8_matmul(*_on_gpu(ea[0], sa), *_on_gpu(eb[0], sb))
        va, vb = pf.decode(ea[0], sa, 256), pf.decode(eb[0], sb, 256, square=True)
        # a code of 256 or more at 2^120 is past fp32 (an infinity): entries that such an
        # operand reaches have no finite value and are left out, and so are entries
        # whose sum of magnitudes is past fp32, where a partial sum may overflow
        with np.errstate(invalid="ignore"):
            want = va @ vb.T
            finite = np.abs(va) @ np.abs(vb).T <= 3.4e38
        va, vb = (np.where(np.isfinite(v), v, 0) for v in (va, vb))
        # operands under 2^-126 may count as zero (include/mhc.h), and so may sums
        small = (np.where(np.abs(va) < 2.0 ** -126, np.abs(va), 0) @ np.abs(vb).T
                 + np.abs(va) @ np.where(np.abs(vb) < 2.0 ** -126, np.abs(vb), 0).T)
        bound = 256 * (2.0 ** -23 * (np.abs(va) @ np.abs(vb).T) + 2.0 ** -126) + small
        far = np.abs(got.double().cpu().numpy()[finite] - want[finite]) - bound[finite]
        worst = far.max(initial=-1)
        assert finite.any() and worst <= 0, (byte_a, byte_b, worst)


# ------------------------------------------------------------------ together
def test_linear_forward_and_backward_together(mhc):
    """A projection as training runs it: encoded input kept, forward, input gradient with
    the transposed weight, weight gradient from the repacked checkpoint; on a side stream
    and replayed from a graph, with other work between the replays."""
    T, K, N = 77, 260, 388
    print(f"[case] linear T={T}", flush=True)
    g = torch.Generator().manual_seed(3)
    z, w = torch.randn(T, K, generator=g), torch.randn(N, K, generator=g)
    df = torch.randn(T, N, generator=g)
    zd, wd, dd = z.cuda(), w.cuda(), df.cuda()

    def step():
        wc, ws, wct, wst = mhc.f8_encode(wd, transposed=True, square=True)
        zc, zs = mhc.f8_encode(zd)
        f = mhc.f8_matmul(zc, zs, wc, ws)
        dc, ds, dct, dst = mhc.f8_encode(dd, transposed=True)
        dz = mhc.f8_matmul(dc, ds, wct, wst)
        zct, zst = mhc.f8_repack(zc, zs, K)
        dw = mhc.f8_matmul(dct, dst, zct, zst)
        return f, dz, dw

    want = [t.clone() for t in step()]
    ez, ew = pf.encode(z.numpy()), pf.encode(w.numpy(), square=True)
    ed, edt = pf.encode(df.numpy()), pf.encode(df.numpy().T)
    vz, vw = pf.decode(*ez, K), pf.decode(*ew, K, square=True)
    _check_product(want[0], vz, vw, "forward")
    _check_product(want[1], pf.decode(*ed, N), vw.T, "input gradient")
    _check_product(want[2], pf.decode(*edt, T), pf.decode(*pf.encode(vz.T), T), "weight gradient")
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
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
