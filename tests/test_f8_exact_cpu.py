"""The whole numbers of tests/test_gpu_f8_exact.py tell sums of 24 bits from narrower ones."""
import torch

from test_gpu_f8_exact import _columns, _operand


def _sum_of_groups(a, b, bits, size=8):
    """Products in groups of `size`, aligned on a group's largest with `bits` bits kept."""
    p = (a.unsqueeze(1) * b.unsqueeze(0)).double().unflatten(2, (-1, size))
    top = torch.exp2(torch.floor(torch.log2(p.abs().amax(-1, keepdim=True))) - bits + 1)
    return (torch.trunc(p / top) * top).sum((-2, -1))


def test_narrow_sums_differ():
    K = 512
    loud = _columns(K, 7)
    a, b = _operand(40, K, loud, 1, "cpu"), _operand(36, K, loud, 2, "cpu")
    want = a.double() @ b.double().t()
    assert want.abs().max() < 2 ** 23
    assert torch.equal(_sum_of_groups(a, b, 24), want)
    for bits in (14, 16):
        assert (_sum_of_groups(a, b, bits) != want).double().mean() > 0.9
    for t in (a, b):
        assert torch.equal(t.to(torch.float8_e4m3fn).float(), t)
