"""Host-side argument checks of the 8-bit blocks and the backward passes (no GPU work)."""
import numpy as np
import pytest

import mhc_hyper_connection_token_amd as mhc
import plain_forms as pf

OK, EINVAL, EALIGN, EUNSUP, EHIP, EOVERLAP, ECAPTURE = range(7)
A = [(k + 1) << 36 for k in range(24)]  # aligned addresses far apart, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(mhc.LIB_PATH):
        pytest.skip("libmhc.so not built")
    return mhc.load_library()


def enc(**kw):
    a = dict(x=A[0], x_type=0, rows=300, cols=1028, square=0, codes=A[1], scales=A[2],
             codes_t=A[3], scales_t=A[4]) | kw
    return mhc.f8_encode_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(x_type=1), OK), (dict(square=1), OK), (dict(codes=None, scales=None), OK),
    (dict(codes_t=None, scales_t=None), OK), (dict(rows=0, x=None), OK),
    (dict(x_type=2), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL),
    (dict(cols=1030), EALIGN), (dict(x=A[0] + 4), EALIGN), (dict(scales_t=A[4] + 1), EALIGN),
    (dict(x=None), EINVAL), (dict(scales=None), EINVAL), (dict(codes_t=None), EINVAL),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), EINVAL),
    (dict(cols=(1 << 28) + 4), EUNSUP), (dict(rows=1 << 26, cols=516), EUNSUP),
    (dict(codes=A[0] + 16), EOVERLAP), (dict(scales=A[1] + 300 * 1152 - 16), EOVERLAP),
    (dict(scales=A[1] + 300 * 1152), OK), (dict(scales_t=A[3] + 1028 * 384), OK),
    (dict(scales_t=A[3] + 1028 * 384 - 16), EOVERLAP)])
def test_encode_check(kw, code):
    assert enc(**kw) == code


def mm(**kw):
    a = dict(a=A[0], a_s=A[1], b=A[2], b_s=A[3], square=1, M=300, N=1028, K=512, out=A[4],
             out_type=0) | kw
    return mhc.f8_matmul_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(out_type=1), OK), (dict(M=0, a=None, out=None), OK),
    (dict(K=0, a=None, a_s=None, b=None, b_s=None), OK), (dict(K=0, out=None), EINVAL),
    (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=-128), EINVAL), (dict(out_type=3), EINVAL),
    (dict(N=1030), EALIGN), (dict(K=100), EALIGN), (dict(b=None), EINVAL),
    (dict(a_s=A[1] + 8), EALIGN), (dict(M=1 << 21, N=1 << 10), EUNSUP),
    (dict(out=A[0] + 512), EOVERLAP), (dict(out=A[3]), EOVERLAP)])
def test_matmul_check(kw, code):
    assert mm(**kw) == code


def post(**kw):
    a = dict(g=A[0], x=A[1], xs=A[2], f=A[3], fs=None, post=A[4], comb=A[5], T=9, S=4, H=260,
             dx=A[6], df=A[7], dpost=A[8], dcomb=A[9]) | kw
    return mhc.site_post_bwd_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(xs=None), OK), (dict(fs=A[10]), OK), (dict(T=0, g=None), OK),
    (dict(S=0), EINVAL), (dict(T=-1), EINVAL), (dict(S=9), EUNSUP), (dict(H=262), EALIGN),
    (dict(T=1 << 23), EUNSUP), (dict(g=None), EINVAL), (dict(dcomb=None), EINVAL),
    (dict(xs=A[2] + 2), EALIGN), (dict(df=A[7] + 4), EALIGN), (dict(dx=A[0]), EOVERLAP),
    (dict(dx=A[1] + 36 * 384 - 16), EOVERLAP), (dict(dx=A[1] + 36 * 384), OK),
    (dict(dx=A[1] + 36 * 384, xs=None), EOVERLAP), (dict(dpost=A[6] + 64), EOVERLAP)])
def test_post_bwd_check(kw, code):
    assert post(**kw) == code


def pre(**kw):
    a = dict(x=A[0], xs=A[1], w=A[2], scale=A[3], base=A[4], T=9, S=4, H=260, iters=20, eps=1e-6,
             dy=A[5], dpre=A[6], dpost=A[7], dcomb=A[8], dx_in=A[9], dx=A[10], dw=A[11],
             ds=A[12], db=A[13], work=A[14], nbytes=mhc.site_pre_bwd_work_bytes(9, 4, 260)) | kw
    return mhc.site_pre_bwd_check(*a.values())


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(xs=None, dpre=None, dx_in=None), OK), (dict(dx_in=A[10]), OK),
    (dict(T=0, x=None, dy=None, work=None, nbytes=0), OK), (dict(T=0, dw=None), EINVAL),
    (dict(iters=0), EINVAL), (dict(iters=120), OK), (dict(iters=121), EUNSUP),
    (dict(eps=0.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(eps=float("inf")), EINVAL),
    (dict(S=9), EUNSUP), (dict(H=258), EALIGN), (dict(T=1, S=8, H=1 << 24), EUNSUP),
    (dict(dy=None), EINVAL), (dict(work=None), EINVAL), (dict(nbytes=64), EINVAL),
    (dict(work=A[14] + 8), EALIGN), (dict(dx_in=A[9] + 4), EALIGN),
    (dict(dx_in=A[10] + 16), EOVERLAP), (dict(dx=A[0]), EOVERLAP), (dict(work=A[10]), EOVERLAP),
    (dict(dw=A[2]), EOVERLAP), (dict(db=A[12]), EOVERLAP)])
def test_pre_bwd_check(kw, code):
    assert pre(**kw) == code


def test_calls_refuse_before_any_gpu_work(lib):
    assert lib.mhc_f8_encode(A[0], 0, 4, 6, 0, A[1], A[2], None, None, None) == EALIGN
    assert lib.mhc_f8_repack(A[0], A[1], 4, 128, A[0], A[3], None) == EOVERLAP
    assert lib.mhc_f8_repack(A[0], None, 4, 128, A[2], A[3], None) == EINVAL
    assert lib.mhc_f8_repack(None, None, 0, 128, None, None, None) == OK
    assert lib.mhc_f8_decode(A[0], A[1], 4, 128, A[2] + 4, None) == EALIGN
    assert lib.mhc_f8_decode(A[0], A[1], -1, 128, A[2], None) == EINVAL
    assert lib.mhc_f8_decode(A[0], A[1], 4, 128, A[1], None) == EOVERLAP
    assert lib.mhc_f8_matmul(A[0], A[1], A[2], A[3], 1, 4, 4, 100, A[4], 0, None) == EALIGN
    assert lib.mhc_site_post_bwd(*[None] * 7, 4, 4, 128, *[None] * 5) == EINVAL
    assert lib.mhc_site_pre_bwd(*A[:5], 4, 4, 128, 0, 1e-6, *A[5:15], 1 << 30, None) == EINVAL


def test_work_bytes():
    assert mhc.site_pre_bwd_work_bytes(0, 4, 4096) == 0
    assert mhc.site_pre_bwd_work_bytes(4, 9, 4096) == 0
    assert mhc.site_pre_bwd_work_bytes(4, 4, 4098) == 0
    assert mhc.site_pre_bwd_work_bytes(1, 1, 4) > 0
    # within a few per cent of the state itself at the production site
    assert mhc.site_pre_bwd_work_bytes(4096, 4, 4096) < 4096 * 4 * 4096


def test_binding_refuses_what_is_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128)
    codes, scales = x.to(torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        mhc.f8_encode(x)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        mhc.f8_encode(x.half())
    with pytest.raises(ValueError, match="rows, cols"):
        mhc.f8_encode(x[0])
    with pytest.raises(ValueError, match="GPU"):
        mhc.f8_decode(codes, scales, 128)
    with pytest.raises(ValueError, match="GPU"):
        mhc.f8_repack(codes, scales, 128)
    with pytest.raises(ValueError, match="GPU"):
        mhc.f8_matmul(codes, scales, codes, scales)
    with pytest.raises(ValueError, match="b \\[N, K\\]"):
        mhc.f8_matmul(codes, scales, codes[:, :0], scales)
    with pytest.raises(ValueError, match="GPU"):
        mhc.site_post_bwd(torch.zeros(4, 2, 128), torch.zeros(4, 2, 128), x, x, x)


def test_plain_code_table_matches_torch():
    """The tests' own e4m3 rounding against torch's on the CPU, ties and ends included."""
    torch = pytest.importorskip("torch")
    g = np.random.default_rng(0)
    v = np.concatenate([pf.E4M3, (pf.E4M3[1:] + pf.E4M3[:-1]) / 2,
                        g.standard_normal(5000) * 2.0 ** g.integers(-12, 8, 5000)])
    v = np.concatenate([v, -v]).astype(np.float32)
    v = v[np.abs(v) <= 448]
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(pf.e4m3_codes(v.astype(np.float64)), want)


def test_first_calls_from_two_threads(lib, monkeypatch):
    """A second thread's call while the first one's is still being prepared: neither meets
    a half-prepared state (no GPU: the entry is a stand-in that counts its calls)."""
    import threading
    torch = pytest.importorskip("torch")
    calls, errors = [], []
    monkeypatch.setattr(mhc, "_entry", {})
    monkeypatch.setattr(mhc, "_gpus", None)
    monkeypatch.setattr(mhc, "load_library", lambda: type("L", (), {
        "mhc_f8_decode": staticmethod(lambda *a: calls.append(a) or 0)}))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    second = threading.Event()

    def call():
        try:
            mhc._call("mhc_f8_decode", 0, (1, 2), ())
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    def count():
        if not second.is_set():  # the first thread, between its two steps
            second.set()
            t = threading.Thread(target=call)
            t.start()
            t.join(30)
        return 1

    monkeypatch.setattr(torch.cuda, "device_count", count)
    call()
    assert errors == [] and calls == [(1, 2, 0), (1, 2, 0)]
