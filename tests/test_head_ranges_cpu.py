"""The output head's entry points without a GPU: the ends of the ranges of their arguments."""
import numpy as np
import pytest


@pytest.fixture(scope="module")
def nq():
    from binary_rank_linear_02_b200 import build

    build.build()
    from binary_rank_linear_02_b200 import nq as mod

    return mod


@pytest.fixture(scope="module")
def ptrs():
    buf = np.zeros(1 << 16, dtype=np.uint8)
    base = (buf.ctypes.data + 255) // 256 * 256
    return [base + 4096 * i for i in range(8)], buf


def test_distill_temperature_range(nq, ptrs):
    """Below the normal fp32 numbers 1 / temperature overflows: refused, as infinity is; the largest
    and the smallest normal number are taken (host memory is what is wrong with these calls)."""
    p, _ = ptrs

    def both(t):
        f = nq.lib().nq_distill_topk_fwd(p[0], nq.NQ_F32, 64, p[1], p[2], 0, 2, 64, 4, t, p[3], 0)
        b = nq.lib().nq_distill_topk_bwd(p[0], nq.NQ_F32, 64, p[1], p[2], 0, p[4], 2, 64, 4, t, p[3], p[5], nq.NQ_F32, 0)
        assert f == b
        return f

    tiny, huge = float(np.finfo(np.float32).tiny), float(np.finfo(np.float32).max)
    for t in (tiny / 2, 2.0 ** -149, 1e-40, -tiny, float("inf"), 2 * huge):
        assert both(t) == nq.NQ_ERR_VALUE
    for t in (tiny, 1e-30, 1e30, huge):
        assert both(t) == nq.NQ_ERR_PTRKIND


def test_head_wait_limit_range(nq):
    for bad in (-1, 10**10 + 1):
        assert nq.nq_selftest_head_wait_limit(bad) == nq.NQ_ERR_VALUE
    for good in (1, 10**10, 0):  # (0, the last one, is the usual limit)
        assert nq.nq_selftest_head_wait_limit(good) == nq.NQ_OK
