"""Host-side argument checks of the norms around a branch and the 4-bit groups (no GPU work)."""
import numpy as np
import pytest

import branch_forms as bf
import mhc_hyper_connection_token_amd as mhc

OK, EINVAL, EALIGN, EUNSUP, EHIP, EOVERLAP, ECAPTURE = range(7)
A = [(k + 1) << 36 for k in range(24)]  # aligned addresses far apart, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(mhc.LIB_PATH):
        pytest.skip("libmhc.so not built")
    return mhc.load_library()


def norm(**kw):
    a = dict(y=A[0], nw=A[1], T=9, H=260, eps=1e-5, z=A[2], z_type=0) | kw
    return mhc.branch_norm_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(z_type=1), OK), (dict(T=0, y=None, nw=None, z=None), OK),
    (dict(H=8192), OK), (dict(H=8196), EUNSUP), (dict(T=1 << 23), EUNSUP),
    (dict(T=1 << 19, H=4096), EUNSUP), (dict(T=-1), EINVAL), (dict(H=0), EINVAL),
    (dict(H=262), EALIGN), (dict(z_type=2), EINVAL), (dict(z_type=-1), EINVAL),
    (dict(eps=0.0), EINVAL), (dict(eps=-1e-5), EINVAL), (dict(eps=NAN), EINVAL),
    (dict(eps=INF), EINVAL), (dict(nw=None), EINVAL), (dict(y=A[0] + 8), EALIGN),
    (dict(z=A[0]), EOVERLAP), (dict(z=A[0] + 9 * 260 * 4 - 16), EOVERLAP),
    (dict(z=A[0] + 9 * 260 * 4), OK), (dict(z=A[1]), EOVERLAP)])
def test_branch_norm_check(kw, code):
    assert norm(**kw) == code


def norm_bwd(**kw):
    a = dict(dz=A[0], dz_type=0, y=A[1], ys=None, nw=A[2], T=9, H=260, eps=1e-5, dy=A[3],
             dnw=A[4], work=A[5], nbytes=mhc.norm_bwd_work_bytes(9, 260)) | kw
    return mhc.branch_norm_bwd_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(dz_type=1), OK), (dict(ys=A[6]), OK),
    (dict(T=0, dz=None, y=None, work=None, nbytes=0), OK), (dict(T=0, dnw=None), EINVAL),
    (dict(dz_type=2), EINVAL), (dict(H=8196), EUNSUP), (dict(H=258), EALIGN),
    (dict(eps=0.0), EINVAL), (dict(dy=None), EINVAL), (dict(work=None), EINVAL),
    (dict(nbytes=mhc.norm_bwd_work_bytes(9, 260) - 1), EINVAL), (dict(work=A[5] + 4), EALIGN),
    (dict(ys=A[6] + 1), EALIGN), (dict(dy=A[0]), EOVERLAP), (dict(dy=A[1]), EOVERLAP),
    (dict(ys=A[6], dy=A[1] + 9 * 384), OK), (dict(ys=A[6], dy=A[1] + 9 * 384 - 16), EOVERLAP),
    (dict(dnw=A[2]), EOVERLAP), (dict(work=A[3]), EOVERLAP)])
def test_branch_norm_bwd_check(kw, code):
    assert norm_bwd(**kw) == code


def post(**kw):
    a = dict(x=A[0], f=A[1], f_type=0, nw=A[2], gate=A[3], gate_type=0, rows=9, act=1, alpha=0.5,
             post=A[4], comb=A[5], T=9, S=4, H=260, eps=1e-5, out=A[6]) | kw
    return mhc.site_post_norm_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(f_type=1, gate_type=1, rows=1, act=2), OK), (dict(alpha=0.0), OK),
    (dict(gate=None, gate_type=7, rows=5, act=9), OK), (dict(T=0, x=None, rows=0), OK),
    (dict(T=0, x=None, rows=1), OK), (dict(alpha=NAN), EINVAL), (dict(alpha=-INF), EINVAL),
    (dict(gate=None, alpha=NAN), EINVAL), (dict(f_type=2), EINVAL), (dict(gate_type=2), EINVAL),
    (dict(act=3), EINVAL), (dict(act=-1), EINVAL), (dict(rows=2), EINVAL), (dict(rows=0), EINVAL),
    (dict(gate=A[3] + 4), EALIGN), (dict(S=9), EUNSUP), (dict(H=8196), EUNSUP),
    (dict(H=262), EALIGN), (dict(eps=NAN), EINVAL), (dict(comb=None), EINVAL),
    (dict(out=A[0]), EOVERLAP), (dict(out=A[1]), EOVERLAP), (dict(out=A[3] + 9 * 1040 - 16), EOVERLAP),
    (dict(out=A[3] + 9 * 1040), OK), (dict(out=A[3] + 1040, rows=1), OK)])
def test_post_norm_check(kw, code):
    assert post(**kw) == code


def post_bwd(**kw):
    a = dict(g=A[0], x=A[1], xs=None, f=A[2], f_type=0, fs=None, nw=A[3], gate=A[4], gate_type=0,
             rows=9, act=1, alpha=0.5, post=A[5], comb=A[6], T=9, S=4, H=260, eps=1e-5, dx=A[7],
             df=A[8], dpost=A[9], dcomb=A[10], dnw=A[11], dgate=A[12], work=A[13],
             nbytes=mhc.norm_bwd_work_bytes(9, 260)) | kw
    return mhc.site_post_norm_bwd_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(xs=A[14], fs=A[15], f_type=9), OK), (dict(f_type=9), EINVAL),
    (dict(gate=None, dgate=None), OK), (dict(gate=None), EINVAL), (dict(dgate=None), EINVAL),
    (dict(rows=1), OK), (dict(rows=3), EINVAL), (dict(act=3), EINVAL), (dict(alpha=INF), EINVAL),
    (dict(T=0, rows=1, g=None, dx=None, work=None, nbytes=0), OK),
    (dict(T=0, rows=1, dgate=None), EINVAL), (dict(T=0, rows=0, dgate=None), OK),
    (dict(T=0, dnw=None), EINVAL), (dict(dnw=None), EINVAL), (dict(dcomb=None), EINVAL),
    (dict(nbytes=64), EINVAL), (dict(S=9), EUNSUP), (dict(H=8196), EUNSUP),
    (dict(xs=A[14] + 8), EALIGN), (dict(dgate=A[12] + 8), EALIGN), (dict(dx=A[0]), EOVERLAP),
    (dict(df=A[2]), EOVERLAP), (dict(dgate=A[4]), EOVERLAP), (dict(dnw=A[3]), EOVERLAP),
    (dict(dgate=A[11]), EOVERLAP), (dict(work=A[8]), EOVERLAP),
    (dict(T=0, rows=1, dgate=A[11]), EOVERLAP)])
def test_post_norm_bwd_check(kw, code):
    assert post_bwd(**kw) == code


def enc(**kw):
    a = dict(w=A[0], w_type=0, N=10, K=160, group=64, codes=A[1], scales=A[2], zeros=A[3]) | kw
    return mhc.q4_encode_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(w_type=1, zeros=None), OK), (dict(group=32), OK), (dict(group=128), OK),
    (dict(group=16), EINVAL), (dict(group=0), EINVAL), (dict(N=0), EINVAL), (dict(K=0), EINVAL),
    (dict(K=100), EALIGN), (dict(w_type=2), EINVAL), (dict(K=(1 << 20) + 32), EUNSUP),
    (dict(N=(1 << 24) + 1), EUNSUP), (dict(w=None), EINVAL), (dict(scales=None), EINVAL),
    (dict(codes=A[1] + 8), EALIGN), (dict(zeros=A[3] + 1), EALIGN), (dict(codes=A[0]), EOVERLAP),
    (dict(scales=A[1] + 10 * 80 - 16), EOVERLAP), (dict(scales=A[1] + 10 * 80), OK),
    (dict(zeros=A[2]), EOVERLAP)])
def test_q4_encode_check(kw, code):
    assert enc(**kw) == code


def mm(**kw):
    a = dict(a=A[0], a_type=0, a_s=None, codes=A[1], scales=A[2], scale_type=1, zeros=A[3], M=7,
             N=10, K=160, group=64, out=A[4], out_type=0) | kw
    return mhc.q4_matmul_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(a_type=1, scale_type=2, zeros=None, out_type=1), OK),
    (dict(a_type=3, a_s=A[5]), OK), (dict(a_type=3), EINVAL), (dict(a_s=A[5]), EINVAL),
    (dict(a_type=2), EINVAL), (dict(scale_type=0), EINVAL), (dict(out_type=2), EINVAL),
    (dict(M=0, a=None, out=None), OK), (dict(M=-1), EINVAL), (dict(N=0), EINVAL),
    (dict(K=48), EALIGN), (dict(group=256), EINVAL), (dict(M=(1 << 20) + 1), EUNSUP),
    (dict(M=1 << 20, N=1 << 11), EUNSUP), (dict(a=None), EINVAL), (dict(a=A[0] + 2), EALIGN),
    (dict(out=A[4] + 4), EALIGN), (dict(out=A[0]), EOVERLAP), (dict(out=A[3]), EOVERLAP),
    (dict(out=A[1] + 10 * 80 - 16), EOVERLAP), (dict(out=A[1] + 10 * 80), OK)])
def test_q4_matmul_check(kw, code):
    assert mm(**kw) == code


def test_calls_refuse_before_any_gpu_work(lib):
    assert lib.mhc_branch_norm(A[0], A[1], 4, 6, 1e-5, A[2], 0, None) == EALIGN
    assert lib.mhc_branch_norm(A[0], A[1], 0, 8, 1e-5, A[2], 0, None) == OK
    assert lib.mhc_branch_norm_bwd(A[0], 0, A[1], None, A[2], 9, 8, 1e-5, A[3], A[4], A[5], 8,
                                   None) == EINVAL
    assert lib.mhc_site_post_norm(A[0], A[1], 0, A[2], None, 0, 1, 0, 1.0, A[3], A[4], 4, 4, 128,
                                  0.0, A[5], None) == EINVAL
    assert lib.mhc_q4_encode(A[0], 0, 4, 33, 32, A[1], A[2], None, None) == EALIGN
    assert lib.mhc_q4_decode(A[0], A[1], 0, None, 4, 32, 32, A[2], None) == EINVAL
    assert lib.mhc_q4_decode(A[0], A[1], 1, None, 4, 32, 32, A[1], None) == EOVERLAP
    assert lib.mhc_q4_decode(A[0], A[1], 1, A[3] + 1, 4, 32, 32, A[2], None) == EALIGN
    assert lib.mhc_q4_matmul(A[0], 0, None, A[1], A[2], 1, None, 0, 4, 32, 32, A[3], 0, None) == OK


def test_work_bytes():
    assert mhc.norm_bwd_work_bytes(0, 4096) == 0
    assert mhc.norm_bwd_work_bytes(4, 4098) == 0
    assert mhc.norm_bwd_work_bytes(4, 8196) == 0
    assert mhc.norm_bwd_work_bytes(4, 1024) == 0  # a few short rows need none
    assert 0 < mhc.norm_bwd_work_bytes(5, 4) <= mhc.norm_bwd_work_bytes(5000, 4)
    assert norm_bwd(T=4, work=None, nbytes=0) == OK and post_bwd(T=4, rows=4, work=None, nbytes=0) == OK
    # less than the row's own tensor at the production site
    assert mhc.norm_bwd_work_bytes(4096, 4096) < 4096 * 4096 * 4


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(4, 128), torch.zeros(128)
    codes = torch.zeros(4, 64, dtype=torch.uint8)
    scales = torch.zeros(4, 1, dtype=torch.bfloat16)
    for call in (lambda: mhc.branch_norm(x, w), lambda: mhc.branch_norm_bwd(x, x, w),
                 lambda: mhc.site_post_norm(x[:, None], x, w, x, x),
                 lambda: mhc.site_post_norm_bwd(x[:, None], x, x, w, x, x),
                 lambda: mhc.q4_encode(x), lambda: mhc.q4_decode(codes, scales, cols=128),
                 lambda: mhc.q4_matmul(x, codes, scales),
                 lambda: mhc.q4_matmul((x, x), codes, scales)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call, text in (
            (lambda: mhc.branch_norm(x[0], w), "y must be"),
            (lambda: mhc.branch_norm(x, w, dtype=torch.float16), "float32 or bfloat16"),
            (lambda: mhc.branch_norm_bwd(x.half(), x, w), "float32 or bfloat16"),
            (lambda: mhc.site_post_norm(x, x, w, x, x), "x must be"),
            (lambda: mhc._gate(x, "tanh", 4, 128), "gate_act"),
            (lambda: mhc._gate(None, "silu", 4, 128), "without a gate"),
            (lambda: mhc._gate(x[0].half(), None, 4, 128), "float32 or bfloat16"),
            (lambda: mhc.q4_encode(x, group=16), "32, 64 or 128"),
            (lambda: mhc.q4_encode(x[0]), "w must be"),
            (lambda: mhc.q4_encode(x.double()), "float32 or bfloat16"),
            (lambda: mhc.q4_decode(codes, scales, cols=100), "multiple of 32"),
            (lambda: mhc.q4_decode(codes, scales, cols=1024), "groups"),
            (lambda: mhc.q4_decode(codes, scales.float(), cols=128), "bfloat16 or float16"),
            (lambda: mhc.q4_matmul(x[0], codes, scales), "a must be"),
            (lambda: mhc.q4_matmul(x, codes, scales, dtype=torch.float16), "float32 or bfloat16")):
        with pytest.raises(ValueError, match=text):
            call()


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 1056, 4096])
def test_group_size_follows_from_the_scales(K, monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(mhc, "_gpu", lambda t, name, dtype, shape=None: 0)
    for group in (32, 64, 128):
        kg = -(-K // group)
        got = mhc._q4_weight(torch.zeros(3, 64), torch.zeros(3, kg, dtype=torch.float16), None, K)
        # where two sizes give as many groups there is one, and they are the same weight
        assert got[5] == group or (kg == 1 and got[5] >= K)


def test_plain_packing_is_the_documented_one():
    c = np.arange(256, dtype=np.uint8).reshape(1, 256) % 16
    b = bf.pack(c)
    assert b.shape == (1, 128)
    for s in range(8):
        for j in range(16):
            assert b[0, 16 * s + j] == c[0, 32 * s + j] | c[0, 32 * s + 16 + j] << 4
    np.testing.assert_array_equal(bf.unpack(b, 256), c)
