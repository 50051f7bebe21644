"""The inputs of tests/plane_inputs.py tell a right product of planes from a wrong one: six
rounded products are within the bound, and each mistake is outside it."""
import pytest
import torch

import plane_inputs as pi


@pytest.fixture(scope="module")
def values():
    g = torch.Generator().manual_seed(1)
    return pi.rand24(g, 20000), pi.rand24(g, 20000)


def _over(values, **kw):
    a, b = values
    c, want = pi.pair(a, b)
    off = (pi.product(a, b, **kw) - c.double() - want).abs()
    return (off / (pi.KEPT * (a.double() * b.double()).abs())).max().item()


def test_six_products_of_rounded_planes_are_within_the_bound(values):
    assert 0.5 < _over(values) <= 1


@pytest.mark.parametrize("kw", [dict(cut=True)] + [dict(drop=((i, j),)) for i in range(3)
                                                    for j in range(3 - i)])
def test_mistakes_are_outside(values, kw):
    assert _over(values, **kw) > 4


def test_planes_that_are_cut_lose_one_sidedly(values):
    """The mean loss, not the largest, is what a long sum of them is off by."""
    a, b = values
    exact = a.double() * b.double()
    loss = [((exact - pi.product(a, b, cut=cut)) / exact).mean().item() * 2 ** 24
            for cut in (True, False)]
    assert loss[0] > 0.5 and abs(loss[1]) < 0.05


@pytest.mark.parametrize("T,S,H", [(40, 2, 36), (6, 4, 260)])
def test_sums_are_small(T, S, H):
    """What is left of each product is at most half a unit in its last place (f8: of 18 bits)."""
    for d in (pi.dots(T, S, H, 1, False), pi.streams(T, S, H, 2), pi.weights(T + 16, S, H, 3, False),
              pi.weights(T + 16, S, H, 4, True), pi.rows(T, S, H, 6, False)):
        assert (d["want"].abs() <= 2.0 ** -24 * d["size"] * (1 + 2.0 ** -20)).all()
        assert d["want"].abs().max() > 0
    for d in (pi.dots(T, S, H, 5, True), pi.rows(T, S, H, 7, True)):
        assert (d["want"].abs() <= 2.0 ** -18).all() and (d["want"] != 0).any()
