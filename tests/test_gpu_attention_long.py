"""Attention over a context of hundreds of millions of positions that is not split: one CTA walks
it for seconds, longer than any single wait may last, and every wait counts the work before it."""
import numpy as np
import pytest

from test_gpu_paged_kv import ints, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def test_an_unsplit_context_of_seconds(sv):  # noqa: F811
    """426 million positions (one page of 65536 zero keys and values, in the table 6500 times), then
    17 new tokens whose values are as large as the context is long.  All scores are 0, so the sums
    are whole numbers: query i gets (i + 1) n / (n + i + 1), lse ln(n + i + 1)."""
    import torch
    D, ps, Q, pages = 64, 65536, 17, 6500
    n = pages * ps
    k = torch.zeros((2, 1, ps, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    v[1, 0, :Q] = float(n)                       # 6500 * 2^16 has 11 significant bits: rounded below
    big = v[1, 0, 0, 0].double().item()
    table = np.zeros((1, pages + 1), np.int32)
    table[0, pages] = 1
    q = torch.ones((1, Q, 1, D), dtype=torch.bfloat16, device="cuda")
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t, b = ints(table), ints([n])
    start.record()
    o, l = sv.spec_paged_attention(q, k, v, t, b, workspace=None, want_lse=True)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) > 1000.0      # longer than a wait's quarter of a second by far
    seen = np.arange(1, Q + 1)
    want = seen * big / (n + seen)
    assert (np.abs(o[0, :, 0].double().cpu().numpy() - want[:, None]) <= 2.0 ** -8 * want[:, None] + 1e-6).all()
    want = np.log(n + seen)
    assert (np.abs(l[0, :, 0].double().cpu().numpy() - want) <= 2.0 ** -21 * (1 + want)).all()
