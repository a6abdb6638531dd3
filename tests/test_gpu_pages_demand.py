"""Rows that together lack more pages than 31 bits count, against a short stack: none of them is served,
and none is reported as served.  Whole numbers, equal.
"""
import pytest

from test_gpu_paged_kv import ints, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,width,N", [(6, 1 << 30, 4), (40, 1 << 26, 4), (40, 1 << 26, 1200)])
def test_demand_beyond_31_bits(sv, B, width, N):  # noqa: F811
    """B rows of one-token pages.  The first takes its page; then rows lack all of `width`, until the last three:
    one lacks two pages, one lacks none, one gives a page back."""
    import torch
    if torch.cuda.mem_get_info()[0] < 8 * B * width + (4 << 30):
        pytest.skip("needs memory for two copies of the table")
    table = torch.full((B, width), -7, dtype=torch.int32, device="cuda")
    pages, length = [0] * B, [width] * B
    length[0] = 1
    pages[-3], length[-3] = 3, 5
    pages[-2], length[-2] = 3, 3
    pages[-1], length[-1] = 3, 2
    for at, b in enumerate((B - 3, B - 2, B - 1)):
        table[b, :3] = ints([3 * at, 3 * at + 1, 3 * at + 2])
    before = table[:, :8].clone()
    t_pages, stack, count = ints(pages), ints([9, 10, 11] + [-1] * 9), ints([3])
    base = [n - 2 for n in length]
    ok, slots = sv.spec_page_resize(table, t_pages, ints(length), stack, count, 1, base=ints(base), num_tokens=N)
    served = [0, B - 2, B - 1]
    assert ok.tolist() == [int(b in served) for b in range(B)]
    assert t_pages.tolist() == [1] + [0] * (B - 4) + [3, 3, 2]
    # page 8 was pushed on 9, 10, 11 and taken by row 0
    assert count.tolist() == [3] and stack[:3].tolist() == [9, 10, 11]
    before[0, 0], before[B - 1, 2] = 8, -1
    assert torch.equal(table[:, :8], before)
    assert bool((table[:B - 3, 8:] == -7).all())
    want = torch.full((B, N), -1, dtype=torch.int64)
    want[0, 1] = 8  # base -1
    want[B - 2, :2], want[B - 1, :2] = torch.tensor([4, 5]), torch.tensor([6, 7])
    assert torch.equal(slots.cpu(), want)
