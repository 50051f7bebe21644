"""The 8-bit product on whole numbers whose sums fp32 holds: no rounding is due anywhere, so
the results are equal to the definition's, bit for bit, whatever the order of the sums."""
import pytest

from test_gpu_f8 import MKN as SMALL
from test_gpu_train_large import MKN as LARGE

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
LOUD = 30  # columns of 256 .. 448 in both operands, among columns of 1 .. 4


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


def _operand(rows, K, loud, seed, device):
    """Whole numbers that are e4m3 codes times their block's scale, whichever block they
    are in: multiples of 32 up to 448, and 1 .. 4."""
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=device)  # noqa: E731
    x = r(1, 5, rows, K)
    x[:, loud] = 32 * r(8, 15, rows, len(loud))
    return (x * (1 - 2 * r(0, 2, rows, K))).float()


def _columns(K, seed):
    return torch.randperm(K, generator=torch.Generator().manual_seed(seed))[:LOUD]


@pytest.mark.parametrize("M,K,N", SMALL + LARGE)
@pytest.mark.parametrize("square", [True, False])
def test_matmul_of_whole_numbers(mhc, M, K, N, square):
    """Sums of magnitudes are at most 30 * 448^2 + K * 16 < 2^23 for K < 2^17."""
    print(f"[case] exact matmul {M}x{N}x{K} square={square}", flush=True)
    loud = _columns(K, M + N)
    a, b = _operand(M, K, loud, 1, "cuda"), _operand(N, K, loud, 2, "cuda")
    by = 2.0 ** (torch.arange(M, device="cuda") % 17 - 8).unsqueeze(1)  # moves exponents only
    ea, eb = mhc.f8_encode(a * by), mhc.f8_encode(b, square=square)
    assert torch.equal(mhc.f8_decode(*ea, K), a * by)
    want = a.double() @ b.double().t() * by
    assert torch.equal(mhc.f8_matmul(*ea, *eb).double(), want)
    # a whole number of 24 bits rounds once to bf16
    assert torch.equal(mhc.f8_matmul(*ea, *eb, dtype=torch.bfloat16), want.float().bfloat16())
