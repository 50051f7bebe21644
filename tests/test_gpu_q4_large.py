"""The 4-bit groups on the GPU where an operand's bytes pass 2^32: activations, the scales of int8
ones, codes, scales and zero points.  All but the last rows are zero; these are whole numbers, so
that the results are exact."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
LAST = 5


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    yield m
    torch.cuda.empty_cache()


def _room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB")


def _whole(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device="cuda")


def _weight(g, N, K, group):
    """Codes, scales that are powers of two, zero points, and the float64 values."""
    c = _whole(g, 0, 16, N, K).to(torch.uint8)
    b = c.unflatten(1, (-1, 2, 16))
    kg = -(-K // group)
    d = torch.exp2(_whole(g, -2, 3, N, kg).float()).bfloat16()
    z = _whole(g, 0, 16, N, kg).to(torch.uint8)
    wide = [t.double().repeat_interleave(group, 1)[:, :K] for t in (d, z)]
    return ((b[:, :, 0] | (b[:, :, 1] << 4)).flatten(1).contiguous(), d, z,
            wide[0] * (c.double() - wide[1]))


def test_activations(mhc):
    print("[case] q4 large activations", flush=True)
    _room(16)
    g = torch.Generator(device="cuda").manual_seed(1)
    M, K = 70016, 32768  # 4.6 GB in bf16
    codes, d, z, w = _weight(g, 16, K, 128)
    a = torch.zeros(M, K, device="cuda", dtype=torch.bfloat16)
    a[-LAST:] = _whole(g, -3, 4, LAST, K).bfloat16()
    got = mhc.q4_matmul(a, codes, d, z)
    assert torch.equal(got[-LAST:].double(), a[-LAST:].double() @ w.t())
    assert not got[:-LAST].any()


def test_int8_scales(mhc):
    print("[case] q4 large int8", flush=True)
    _room(64)
    g = torch.Generator(device="cuda").manual_seed(2)
    M, K = 1 << 20, 32832  # 34 GB of codes, 4.3 GB of scales
    codes, d, z, w = _weight(g, 16, K, 64)
    q = torch.zeros(M, K, device="cuda", dtype=torch.int8)
    s = torch.zeros(M, K // 32, device="cuda")
    q[-LAST:] = _whole(g, -3, 4, LAST, K).to(torch.int8)
    s[-LAST:] = torch.exp2(_whole(g, 0, 2, LAST, K // 32).float())
    got = mhc.q4_matmul((q, s), codes, d, z)
    v = q[-LAST:].double() * s[-LAST:].double().repeat_interleave(32, 1)
    assert torch.equal(got[-LAST:].double(), v @ w.t())
    assert not got[:-LAST].any()


def test_weights(mhc):
    print("[case] q4 large weights", flush=True)
    _room(128)
    g = torch.Generator(device="cuda").manual_seed(3)
    N, K = (1 << 22) + 37, 32800  # 69 GB of codes, 8.6 of scales, 4.3 of zero points
    end = _weight(g, LAST, K, 32)
    kg = K // 32
    codes = torch.zeros(N, K // 2, device="cuda", dtype=torch.uint8)
    d = torch.zeros(N, kg, device="cuda", dtype=torch.bfloat16)
    z = torch.zeros(N, kg, device="cuda", dtype=torch.uint8)
    for t, e in zip((codes, d, z), end):
        t[-LAST:] = e
    for M in (1, 2, 6, 30):
        for kind in ("f32", "q8"):
            n = _whole(g, -3, 4, M, K)
            a = n.float() if kind == "f32" else (n.to(torch.int8),
                                                 torch.ones(M, kg, device="cuda"))
            got = mhc.q4_matmul(a, codes, d, z)
            assert torch.equal(got[:, -LAST:].double(), n.double() @ end[3].t()), (M, kind)
            assert not got[:, :-LAST].any(), (M, kind)


def test_encode_and_decode(mhc):
    print("[case] q4 large encode", flush=True)
    _room(80)
    g = torch.Generator(device="cuda").manual_seed(4)
    N, K = 262200, 32800  # 17 GB in bf16, 4.3 of codes, 34 of fp32 values
    w = torch.zeros(N, K, device="cuda", dtype=torch.bfloat16)
    w[-LAST:] = torch.randn(LAST, K, generator=g, device="cuda").bfloat16()
    kept = mhc.q4_encode(w, group=32, zeros=True)
    end = mhc.q4_encode(w[-LAST:].clone(), group=32, zeros=True)
    del w
    assert all(torch.equal(t[-LAST:], e) for t, e in zip(kept, end))
    got = mhc.q4_decode(*kept, cols=K)
    assert torch.equal(got[-LAST:], mhc.q4_decode(*end, cols=K))
    assert not got[:-LAST].any()
