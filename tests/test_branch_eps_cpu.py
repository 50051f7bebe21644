"""The smallest epsilon of the norms around a branch: 2^-126, the smallest normal number.  (With a
smaller one a row of zeros would get 0 * inf.)"""
import pytest

import mhc_hyper_connection_token_amd as mhc

OK, EINVAL = 0, 1
A = [(k + 1) << 36 for k in range(16)]  # aligned addresses far apart, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def lib():
    import os
    if not os.path.exists(mhc.LIB_PATH):
        pytest.skip("libmhc.so not built")
    return mhc.load_library()


@pytest.mark.parametrize("eps,code", [(2.0 ** -126, OK), (1e-30, OK), (1.0, OK), (1.1e-38, EINVAL),
                                      (1e-45, EINVAL), (0.0, EINVAL), (-1e-5, EINVAL)])
def test_smallest_epsilon(eps, code):
    n = mhc.norm_bwd_work_bytes(9, 260)
    assert mhc.branch_norm_check(A[0], A[1], 9, 260, eps, A[2], 0) == code
    assert mhc.branch_norm_bwd_check(A[0], 0, A[1], None, A[2], 9, 260, eps, A[3], A[4], A[5],
                                     n) == code
    assert mhc.site_post_norm_check(A[0], A[1], 0, A[2], None, 0, 1, 0, 1.0, A[3], A[4], 9, 4, 260,
                                    eps, A[5]) == code
    assert mhc.site_post_norm_bwd_check(A[0], A[1], None, A[2], 0, None, A[3], None, 0, 1, 0, 1.0,
                                        A[4], A[5], 9, 4, 260, eps, A[6], A[7], A[8], A[9], A[10],
                                        None, A[11], n) == code
