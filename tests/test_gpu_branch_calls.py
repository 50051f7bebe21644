"""Calls of the norms around a branch that their documentation allows, on the GPU."""
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


def _rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


@pytest.mark.parametrize("how", ["sigmoid", "silu"])
def test_an_activation_is_not_read_without_a_gate(mhc, how):
    print(f"[case] no gate, {how}", flush=True)
    T, S, H = 5, 3, 132
    r = _rand(1)
    x, f, nw, post, comb, g = r(T, S, H), r(T, H), r(H), r(T, S), r(T, S, S), r(T, S, H)
    want = mhc.site_post_norm(x, f, nw, post, comb)
    assert torch.equal(mhc.site_post_norm(x, f, nw, post, comb, gate_act=how), want)
    want = mhc.site_post_norm_bwd(g, x, f, nw, post, comb)
    got = mhc.site_post_norm_bwd(g, x, f, nw, post, comb, gate_act=how)
    assert want[5] is None and got[5] is None
    assert all(map(torch.equal, got[:5], want[:5]))


def test_rows_of_zeros_with_the_smallest_epsilon(mhc):
    """A row without a square is a row of zeros, whatever the epsilon, and its gradient is the
    incoming one times nw / sqrt(eps)."""
    print("[case] zero rows", flush=True)
    T, S, H = 6, 2, 260
    r = _rand(2)
    nw, post, comb, g = r(H), r(T, S), r(T, S, S), r(T, S, H)
    y = torch.zeros(T, H, device="cuda")
    x = r(T, S, H)
    for eps in (2.0 ** -126, 1e-30, 1e-5):
        assert not mhc.branch_norm(y, nw, eps).any()
        dz = r(T, H)
        dy, dnw = mhc.branch_norm_bwd(dz, y, nw, eps)
        want = dz.double() * nw.double() / eps ** 0.5
        assert ((dy.double() - want).abs() <= 1e-6 * want.abs()).all() and not dnw.any()
        assert torch.equal(mhc.site_post_norm(x, y, nw, post, comb, eps),
                           mhc.site_post(x, y, post, comb))
        got = mhc.site_post_norm_bwd(g, x, y, nw, post, comb, eps)
        assert all(torch.isfinite(t).all() for t in got[:5]) and not got[2].any() and not got[4].any()
