"""The range of the 4-bit product's activations on the GPU: whole numbers times powers of two,
whose sums are exact in any order, at both ends of what include/mhc.h allows."""
import numpy as np
import pytest

import branch_forms as bf

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _case(M, kind, group, ea, es, seed, least):
    """a = n 2^ea, |n| from `least` to 1 (ones) or of both signs, scales 2^es."""
    g = np.random.default_rng(seed)
    N, K = 70, 384
    c = g.integers(0, 16, (N, K)).astype(np.uint8)
    c[:3] = 15
    z = g.integers(0, 16, (N, K // group)).astype(np.uint8)
    z[0], z[1] = 0, 15
    n = g.integers(least, 2, (M, K)).astype(np.float32)
    v = torch.from_numpy(n)
    a = (v.to(torch.int8).cuda(), torch.full((M, K // 32), 2.0 ** ea).cuda()) if kind == "q8" else \
        (v * 2.0 ** ea).to(torch.bfloat16 if kind == "bf16" else torch.float32).cuda()
    kept = (torch.from_numpy(bf.pack(c)).cuda(),
            torch.full((N, K // group), 2.0 ** es, dtype=torch.bfloat16).cuda(),
            torch.from_numpy(z).cuda())
    w = c.astype(np.float64) - np.repeat(z, group, 1)
    return a, kept, torch.from_numpy(n.astype(np.float64) @ w.T) * 2.0 ** (ea + es)


@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("M", [1, 2, 5, 16, 40, 200])
@pytest.mark.parametrize("group,ea", [(32, 119), (64, 118), (128, 117)])
@pytest.mark.parametrize("least", [1, -1])
def test_largest_activations(mhc, kind, M, group, ea, least):
    """A group's 15 * sum |a| is 15/16 of 2^128: no sum on the way overflows, and the scale
    brings the result back."""
    print(f"[case] q4 range M={M} {kind} G={group} a 2^{ea}", flush=True)
    a, kept, want = _case(M, kind, group, ea, -60, M, least)
    assert torch.equal(mhc.q4_matmul(a, *kept).double().cpu(), want)


@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("M", [1, 2, 5, 16, 40, 200])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("ea", [-118, -126])
def test_smallest_activations(mhc, kind, M, group, ea):
    """Normal numbers of any size count in full."""
    print(f"[case] q4 range M={M} {kind} G={group} a 2^{ea}", flush=True)
    a, kept, want = _case(M, kind, group, ea, 100, M, -1)
    assert torch.equal(mhc.q4_matmul(a, *kept).double().cpu(), want)


@pytest.mark.parametrize("kind,M", [("f32", 1), ("bf16", 1), ("bf16", 2), ("bf16", 5), ("bf16", 40)])
@pytest.mark.parametrize("e", [100, -100, -115, -125])
def test_values_keep_their_bits(mhc, kind, M, e):
    """One column a row, of any mantissa, and codes that are powers of two: products and sums
    are exact for normal numbers of every size."""
    print(f"[case] q4 bits {kind} M={M} 2^{e}", flush=True)
    g = np.random.default_rng(e + 200)
    N, K = 40, 256
    c = g.choice([0, 1, 2, 4, 8], (N, K)).astype(np.uint8)
    v = torch.from_numpy(((1 + g.random(M)) * 2.0 ** e).astype(np.float32))
    if kind == "bf16":
        v = v.bfloat16()
    col = torch.from_numpy(g.integers(0, K, M))
    a = torch.zeros(M, K, dtype=v.dtype)
    a[torch.arange(M), col] = v
    s = 2.0 ** (-e // 2)
    kept = (torch.from_numpy(bf.pack(c)).cuda(), torch.full((N, 2), s, dtype=torch.bfloat16).cuda(),
            torch.zeros(N, 2, dtype=torch.uint8).cuda())
    want = v.double()[:, None] * torch.from_numpy(c.astype(np.float64)).t()[col] * s
    assert torch.equal(mhc.q4_matmul(a.cuda(), *kept).double().cpu(), want)
