"""The layout of 4-bit codes on the GPU: sixteen bytes hold 32 columns of a row, byte j column j
in its low half and column 16 + j in its high half.  Packed and unpacked here entry by entry, by
that sentence alone."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _pack(c):
    N, K = c.shape
    out = np.zeros((N, K // 2), np.uint8)
    for k in range(K):
        out[:, k // 32 * 16 + k % 16] += c[:, k] * (16 if k % 32 >= 16 else 1)
    return out


def _values(c, d, z, group):
    w = np.zeros(c.shape)
    for k in range(c.shape[1]):
        w[:, k] = d[:, k // group].astype(np.float64) * (c[:, k].astype(np.float64) - z[:, k // group])
    return w


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 17, 100])
@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
def test_product(mhc, M, kind, group):
    """Whole numbers and scales that are powers of two: every sum is exact."""
    for N, K in ((40, 32), (70, 96), (33, 160), (20, 224), (130, 512), (17, 4160)):
        print(f"[case] layout M={M} N={N} K={K} {kind} G={group}", flush=True)
        g = np.random.default_rng(M + N + K)
        c = g.integers(0, 16, (N, K)).astype(np.uint8)
        kg = -(-K // group)
        d = (2.0 ** g.integers(-2, 3, (N, kg))).astype(np.float32)
        z = g.integers(0, 16, (N, kg)).astype(np.uint8)
        a = g.integers(-3, 4, (M, K)).astype(np.float32)
        t = torch.from_numpy(a).cuda()
        if kind == "bf16":
            t = t.bfloat16()
        elif kind == "q8":
            t = t.to(torch.int8), torch.ones(M, K // 32, device="cuda")
        got = mhc.q4_matmul(t, torch.from_numpy(_pack(c)).cuda(),
                            torch.from_numpy(d).bfloat16().cuda(), torch.from_numpy(z).cuda())
        # 4160 entries of up to 3 * 15 * 4 each in steps of a quarter: below 2^22 steps
        np.testing.assert_array_equal(got.double().cpu().numpy(),
                                      a.astype(np.float64) @ _values(c, d, z, group).T)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_encode_and_decode(mhc, group, zeros):
    for N, K in ((1, 32), (5, 96), (3, 160), (9, 4128)):
        print(f"[case] layout encode N={N} K={K} G={group} zeros={zeros}", flush=True)
        # every entry is a code of its own group: a scale of one, and both ends of the range
        g = np.random.default_rng(K)
        c = g.integers(0 if zeros else 1, 16, (N, K)).astype(np.uint8)
        c[:, ::32], c[:, 1::32] = 15, 0 if zeros else 1
        w = c.astype(np.float32) - (6 if zeros else 8)
        kept = mhc.q4_encode(torch.from_numpy(w).cuda(), group=group, zeros=zeros)
        assert kept[0].shape == (N, K // 2)
        np.testing.assert_array_equal(kept[0].cpu().numpy(), _pack(c))
        assert (kept[1] == 1).all() and (not zeros or (kept[2] == 6).all())
        np.testing.assert_array_equal(mhc.q4_decode(*kept, cols=K).cpu().numpy(), w)


@pytest.mark.parametrize("M", [2, 4, 5, 16])
@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
def test_product_of_many_columns(mhc, M, kind):
    """On both sides of the numbers of columns where a block's shape changes."""
    for N in (4096, 4097, 8192, 8193, 16383, 16384, 28671, 28672):
        print(f"[case] columns M={M} N={N} {kind}", flush=True)
        g = np.random.default_rng(M + N)
        K, group = 96, 32
        c = g.integers(0, 16, (N, K)).astype(np.uint8)
        d = (2.0 ** g.integers(-2, 3, (N, K // group))).astype(np.float32)
        z = g.integers(0, 16, (N, K // group)).astype(np.uint8)
        a = g.integers(-3, 4, (M, K)).astype(np.float32)
        t = torch.from_numpy(a).cuda()
        if kind == "bf16":
            t = t.bfloat16()
        elif kind == "q8":
            t = t.to(torch.int8), torch.ones(M, K // 32, device="cuda")
        got = mhc.q4_matmul(t, torch.from_numpy(_pack(c)).cuda(),
                            torch.from_numpy(d).bfloat16().cuda(), torch.from_numpy(z).cuda())
        np.testing.assert_array_equal(got.double().cpu().numpy(),
                                      a.astype(np.float64) @ _values(c, d, z, group).T)
