"""Every operand type of the norms around a branch with every other, on the GPU against 64-bit
forms: each is a kernel of its own, as is each range of hidden sizes and of streams."""
import pytest

import branch_forms as bf
from branch_forms import ULP
from test_gpu_branch_norm import (EPS, EPS64, GATE, NORM_SHAPES, RINV, _cuda, _double, _keep,
                                  _rand, _same, _site, _within)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def mhc():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mhc_hyper_connection_token_amd as m
    m.load_library()
    return m


@pytest.mark.parametrize("T,H", NORM_SHAPES)
def test_norm_gradient_of_bf16_and_an_fp32_row(mhc, T, H):
    print(f"[case] branch_norm_bwd T={T} H={H} bf16 fp32", flush=True)
    r = _rand(7 * T + H)
    gz, dz = _keep(mhc, r(T, H), "bf16")
    y, nw = r(T, H), 1 + 0.2 * r(H)
    dy, dnw = mhc.branch_norm_bwd(gz, y.cuda(), nw.cuda(), EPS)
    w_dy, w_dnw, alone, row, size = bf.norm_bwd(dz, dz.abs(), y.double(), nw.double(), EPS64)
    # r enters three times in the part that goes with the row, whose sum has H terms
    _within(dy, w_dy, ((RINV + 4) * alone + (H + 3 * RINV + 8) * row) * ULP, "dy")
    _within(dnw, w_dnw, (T + RINV + 4) * ULP * size, "dnw")


@pytest.mark.parametrize("T,H", [(2048, 1028), (2049, 1028), (2050, 4096), (2048, 4096)])
@pytest.mark.parametrize("bf16", [False, True])
def test_norm_on_both_sides_of_its_rule(mhc, T, H, bf16):
    """Up to 2048 tokens four waves hold a row, past it two."""
    print(f"[case] branch_norm T={T} H={H} bf16={bf16}", flush=True)
    r = _rand(T + H)
    y, nw = r(T, H) * torch.exp(r(T, 1)), 1 + 0.2 * r(H)
    y[T // 2] = 0
    got = mhc.branch_norm(y.cuda(), nw.cuda(), EPS, dtype=torch.bfloat16 if bf16 else None)
    want = bf.branch(y.double(), nw.double(), EPS64)
    _within(got, want, want.abs() * ((RINV + 3) * ULP + (2.0 ** -8 * 1.01 if bf16 else 0)), "z")


# A wave's rows, a block's up to 4096 and beyond; up to four streams and more; tokens that
# follow one another in a block (more than 1024 short ones or 256 long ones) and that do not.
SHAPES = [(9, 4, 260), (1100, 2, 132), (30, 6, 516), (7, 3, 1028), (270, 4, 1028), (6, 8, 2052),
          (5, 4, 5000), (262, 3, 4100), (4, 5, 4100), (260, 8, 4100)]
GATES = [None, "f32", "bf16"]


def _gate_of(n):
    """One row of it or one a token, and an activation, in turn."""
    return ("channel", "token")[n % 2], (None, "sigmoid", "silu")[n // 2 % 3]


@pytest.mark.parametrize("T,S,H", SHAPES + [(200, 1, 2052), (130, 7, 1028), (140, 4, 5000),
                                            (24, 4, 4096), (25, 4, 4096), (64, 8, 4100),
                                            (65, 8, 4100), (64, 3, 2048), (65, 3, 2048)])
@pytest.mark.parametrize("f_kind", ["f32", "bf16"])
@pytest.mark.parametrize("gate_kind", GATES)
def test_post_mix(mhc, T, S, H, f_kind, gate_kind):
    gate, how = _gate_of(T + S + H // 4) if gate_kind else ("none", None)
    print(f"[case] post T={T} S={S} H={H} f={f_kind} gate={gate_kind} {gate} {how}", flush=True)
    d = _site(T, S, H, T + S + H, gate, gate_kind)
    gf, f = _keep(mhc, d["f"], f_kind)
    got = mhc.site_post_norm(d["x"].cuda(), gf, d["nw"].cuda(), d["post"].cuda(),
                             d["comb"].cuda(), EPS, gate=_cuda(d["gate"]), gate_act=how, alpha=1.5)
    want, size = bf.site_post_norm(d["x"].double(), f, d["nw"].double(), d["post"].double(),
                                   d["comb"].double(), EPS64, _double(d["gate"]), how, 1.5)
    _within(got, want, (RINV + GATE + 5 + S + 1) * ULP * size, "x'")


@pytest.mark.parametrize("T,S,H", SHAPES)
@pytest.mark.parametrize("x_kind", ["f32", "f8"])
@pytest.mark.parametrize("f_kind", ["f32", "bf16", "f8"])
@pytest.mark.parametrize("gate_kind", GATES)
def test_post_mix_gradient(mhc, T, S, H, x_kind, f_kind, gate_kind):
    turn = T + S + H // 4 + (x_kind == "f8") + 2 * ("f32", "bf16", "f8").index(f_kind)
    gate, how = _gate_of(turn) if gate_kind else ("none", None)
    print(f"[case] post bwd T={T} S={S} H={H} x={x_kind} f={f_kind} gate={gate_kind} {gate} {how}",
          flush=True)
    alpha = 1.5
    d = _site(T, S, H, 3 * T + S + H, gate, gate_kind)
    gf, f = _keep(mhc, d["f"], f_kind)
    gx, x = _keep(mhc, d["x"], x_kind)
    args = (d["g"].cuda(), gx, gf, d["nw"].cuda(), d["post"].cuda(), d["comb"].cuda(), EPS)
    keys = dict(gate=_cuda(d["gate"]), gate_act=how, alpha=alpha)
    got = mhc.site_post_norm_bwd(*args, **keys)
    g, nw, post, comb = (d[n].double() for n in ("g", "nw", "post", "comb"))
    gt = _double(d["gate"])
    a, slope, slope_size = bf.act(gt, how)
    _within(got[0], comb @ g, (S + 1) * ULP * (comb.abs() @ g.abs()), "dx")
    gT = g.transpose(1, 2).contiguous()
    _within(got[3], x @ gT, (H + 1) * ULP * (x.abs() @ gT.abs()), "dcomb")
    h = bf.branch(f, nw, EPS64, gt, how, alpha)
    each = RINV + GATE + S + 8  # roundings of a term beside those of its sum
    _within(got[2], (g @ h.unsqueeze(2)).squeeze(2),
            (H + each) * ULP * (g.abs() @ h.abs().unsqueeze(2)).squeeze(2), "dpost")
    e = (post.unsqueeze(1) @ g).squeeze(1)
    e_size = (post.abs().unsqueeze(1) @ g.abs()).squeeze(1)
    df, dnw, alone, row, size = bf.norm_bwd(alpha * e * a, alpha * e_size * a.abs(), f, nw, EPS64)
    _within(got[1], df, (each * alone + (H + each + 2 * RINV) * row) * ULP, "df")
    _within(got[4], dnw, (T + each) * ULP * size, "dnw")
    if gt is None:
        assert got[5] is None
    else:
        base = bf.branch(f, nw, EPS64)
        dg = alpha * e * slope * base
        dg_size = alpha * e_size * slope_size * base.abs()
        if gate == "channel":
            dg, dg_size = dg.sum(0), dg_size.sum(0)
        _within(got[5], dg, (T + each + GATE) * ULP * dg_size, "dgate")
    assert _same(got, mhc.site_post_norm_bwd(*args, **keys))
