"""The 4-bit product on the GPU where it has to be exact to the last bit of an activation, and
where its errors have to be those of independent roundings: what a lost or misplaced part of an
fp32 value (the kernels multiply it as three bf16 ones) would break."""
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


# One row; two to four; five to sixteen, at each width of a block; then the tiles: 32 x 64, 32 x
# 128, 64 x 128, past one round 128 x 128, 32 x 128 and 96 x 128 (bf16).
SHAPES = [(1, 100, 160), (1, 4099, 4096), (2, 33, 96), (3, 6000, 288), (4, 9000, 160),
          (4, 16390, 128), (5, 4100, 2208), (8, 6000, 160), (12, 16400, 96), (16, 70, 1056),
          (16, 9000, 128), (17, 64, 256), (100, 257, 512), (40, 9000, 160), (120, 16000, 160),
          (128, 32700, 96), (130, 20000, 128), (90, 30000, 160), (333, 7168, 128)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_column_keeps_every_bit(mhc, M, N, K, kind, group):
    """A row with one activation, of a full mantissa, times codes that are powers of two with
    zero points of 0 and such scales: every product, and every sum of its parts, is a value of at
    most 24 bits.  (int8: the activation is the code times its scale, rounded to fp32 once.)"""
    g = torch.Generator(device="cuda").manual_seed(M + N + K + group)
    kg = -(-K // group)
    codes = torch.tensor([0, 1, 2, 4, 8], device="cuda", dtype=torch.uint8)[
        torch.randint(0, 5, (N, K), generator=g, device="cuda")]
    b = codes.unflatten(1, (-1, 2, 16))
    packed = (b[:, :, 0] | (b[:, :, 1] << 4)).flatten(1).contiguous()
    d = torch.exp2(torch.randint(-6, 7, (N, kg), generator=g, device="cuda").float())
    kept = packed, d.bfloat16(), torch.zeros(N, kg, device="cuda", dtype=torch.uint8)
    wide = d.repeat_interleave(group, 1)[:, :K]
    for turn in range(max(1, 24 // M)):  # few rows see many columns all the same
        print(f"[case] one column M={M} N={N} K={K} {kind} G={group} {turn}", flush=True)
        col = (torch.arange(M, device="cuda") * 37 + 11 * turn + 5) % K
        at = torch.arange(M, device="cuda"), col
        v = (1 + torch.rand(M, generator=g, device="cuda")) * torch.exp2(
            torch.randint(-20, 21, (M,), generator=g, device="cuda").float())
        if kind == "q8":
            n = torch.randint(-127, 128, (M,), generator=g, device="cuda").to(torch.int8)
            q = torch.zeros(M, K, device="cuda", dtype=torch.int8)
            s = 1 + torch.rand(M, K // 32, generator=g, device="cuda")
            q[at], s[at[0], col // 32] = n, v
            a, v = (q, s), n.float() * v
        else:
            v = v.bfloat16() if kind == "bf16" else v
            a = torch.zeros(M, K, device="cuda", dtype=v.dtype)
            a[at] = v
        want = v.float()[:, None] * (codes[:, col].float() * wide[:, col]).t()  # exact in fp32
        assert torch.equal(mhc.q4_matmul(a, *kept), want)


@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 17, 100])
@pytest.mark.parametrize("kind", ["f32", "bf16", "q8"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
def test_errors_are_independent_roundings(mhc, M, kind, group, zeros):
    """The root mean square of the error against 64 bits.  A rounding is off by at most half a
    step of the sum it rounds, 2^-24 of it, and by 1/sqrt(3) of that in the mean of squares.
    Sums of terms of either sign are as large as the root of their sum of squares.  A group has
    at most 33 roundings for 32 columns and each plane, and 5 more; the groups' sums K/group, 16
    for the waves and 6 across lanes: their squares add up.  int8: products and sums of 32
    columns are exact up to 16 rows, but the bound is left as it is for fp32."""
    N, K = 200, 512
    print(f"[case] rounding M={M} {kind} G={group} zeros={zeros}", flush=True)
    g = np.random.default_rng(M + group)
    kg = K // group
    c = g.integers(0, 16, (N, K)).astype(np.uint8)
    z = g.integers(0, 16, (N, kg)).astype(np.uint8) if zeros else None
    d = torch.from_numpy((2.0 ** g.uniform(-3, 0, (N, kg))).astype(np.float32)).bfloat16()
    t = torch.from_numpy(g.standard_normal((M, K)).astype(np.float32))
    if kind == "q8":
        s = t.view(M, -1, 32).abs().amax(2) / 127
        q = torch.round(t.view(M, -1, 32) / s.unsqueeze(2)).clamp(-127, 127).to(torch.int8)
        a, v = (q.view(M, K).cuda(), s.cuda()), (q.double() * s.double().unsqueeze(2)).view(M, K)
    else:
        t = t.bfloat16() if kind == "bf16" else t
        a, v = t.cuda(), t.double()
    w = torch.from_numpy(bf.decode(c, d.float().numpy(), z, group))
    zero = 8.0 if z is None else np.repeat(z, group, 1).astype(np.float64)
    size = torch.from_numpy((c + zero) * np.repeat(d.double().numpy(), group, 1))
    got = mhc.q4_matmul(a, torch.from_numpy(bf.pack(c)).cuda(), d.cuda(),
                        None if z is None else torch.from_numpy(z).cuda()).double().cpu()
    planes = 1 if kind == "bf16" else 3
    n = 33 * group // 32 * planes + 5 + kg + 22
    rms = ((v * v) @ (size * size).t()).mean().sqrt()
    off = (got - v @ w.t()).square().mean().sqrt()
    assert off <= ULP * (n / 3) ** 0.5 * rms, (off / (ULP * rms)).item()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_one_row_of_one_sign(mhc, kind):
    """Activations of one sign, as behind a relu: sum code * a and zero point * sum a are far
    larger than their difference.  One row sums a block of 32 columns, and its activations, in
    four chains of 8 and then the chains: the mean square of the error is at most that of
    independent roundings, each half a step of its partial sum at most and 1/sqrt(3) of that in
    the mean (the partial sums are taken in 64 bits here)."""
    print(f"[case] one sign {kind}", flush=True)
    g = np.random.default_rng(5)
    N, K, off, sums = 2000, 32, 0.0, 0.0
    for turn in range(40):
        c = g.integers(0, 16, (N, K)).astype(np.uint8)
        v = torch.from_numpy((0.5 + g.random(K)).astype(np.float32))
        v = v.bfloat16() if kind == "bf16" else v
        got = mhc.q4_matmul(v[None].cuda(), torch.from_numpy(bf.pack(c)).cuda(),
                            torch.ones(N, 1, dtype=torch.bfloat16).cuda()).double().cpu()[0]
        a = v.double().numpy()
        want = (c.astype(np.float64) - 8) @ a
        off += np.square(got.numpy() - want).mean()
        # columns 4 d .. + 3 and 16 + 4 d .. + 3 are chain d
        order = np.concatenate([np.r_[4 * d:4 * d + 4, 16 + 4 * d:20 + 4 * d] for d in range(4)])
        for terms, by in ((c[:, order] * a[order], 1.0), (a[None, order], 8.0)):
            p = np.cumsum(terms.reshape(-1, 4, 8), 2)
            t = p[:, :, 7]
            last = [t[:, 0] + t[:, 1], t[:, 2] + t[:, 3], t.sum(1)]
            sums += by ** 2 * (np.square(p).sum((1, 2)).mean() + sum(np.square(x).mean() for x in last))
        sums += np.square(want).mean()
    assert (off / 40) ** 0.5 <= ULP * (sums / 40 / 3) ** 0.5, ((off / sums * 3) ** 0.5 / ULP)
