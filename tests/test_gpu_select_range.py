"""Block selection where scores are small, or small beside |q|_1 max|m|: lists are those of scores summed in 64
bits, equal to the plain form's.  The scores of different blocks differ by far more than the sums' last bits.
"""
import numpy as np
import pytest

from test_gpu_paged_kv import sv  # noqa: F401
from test_gpu_sparse import check_select, select_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["mean", "bounds"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,blocks", [(1, 90), (80, 90), (2, 2100)])  # few lists, many, long ones
@pytest.mark.parametrize("of_q,of_m", [(-60, -60), (-66, -60), (-80, -80), (-100, -20), (-20, -110), (-30, -64),
                                       (-130, 40), (40, -130)])  # (numbers below 2^-126 among them)
def test_small_magnitudes(sv, kind, shared, B, blocks, of_q, of_m):  # noqa: F811
    """Products near the lower end of fp32 and far below it."""
    rng = np.random.default_rng(3)
    q, summary, table, base, _ = select_case(rng, B, 2, 4, 1, 64, 16, blocks, kind == "bounds")
    base[:] = blocks * 16
    q *= 2.0 ** of_q
    summary *= 2.0 ** of_m
    assert q.any() and summary.any()
    for top in (4, 60):
        check_select(sv, q, summary, table, base, None, 16, top, kind, 1, 1, shared)
    summary.zero_()  # and true zeros are all alike
    check_select(sv, q, summary, table, base, None, 16, 12, kind, 1, 1, shared)


@pytest.mark.parametrize("kind", ["mean", "bounds"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,Q,blocks", [(1, 2, 90), (1, 9, 90), (80, 2, 90), (2, 2, 2100)])
@pytest.mark.parametrize("far", [30, 60, 90])
def test_large_elements_that_meet_zeros(sv, kind, shared, B, Q, blocks, far):  # noqa: F811
    """An element of the queries, or of the summaries, far above the others whose partner is zero: |q|_1 max|m| is
    2 ** far times what the scores are, and they keep their order."""
    rng = np.random.default_rng(4)
    for side in ("query", "summary"):
        q, summary, table, base, _ = select_case(rng, B, Q, 4, 1, 64, 16, blocks, kind == "bounds")
        base[:] = blocks * 16
        q[..., 0] = 2.0 ** far if side == "query" else 0
        summary[..., 0::64] = 0 if side == "query" else 2.0 ** far
        for top in (4, 33, 60):
            check_select(sv, q, summary, table, base, None, 16, top, kind, 1, 1, shared)
