"""Page tables that grow and shrink on the GPU against their plain form: whole numbers, equal."""
import numpy as np
import pytest

from oracle import context
from test_gpu_paged_kv import ints, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def state(rng, B, width, ps, spare):
    """A shuffled table that holds random numbers of pages, and the stack of the others."""
    pages = rng.integers(0, width + 1, B)
    P = int(pages.sum()) + spare
    perm = rng.permutation(P)
    table = np.full((B, width), -1)
    at = 0
    for b in range(B):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
    stack = np.full(P, -7)
    stack[:P - at] = perm[at:]
    return table, pages, stack, P - at


def check(sv, table, pages, length, stack, count, ps, base=None, N=0):  # noqa: F811
    import torch
    want = context.page_resize(table, pages, length, stack, count, ps, base, N)
    t = [ints(x) for x in (table, pages, length, stack, [count])]
    ok, slots = sv.spec_page_resize(t[0], t[1], t[2], t[3], t[4], ps, base=None if base is None else ints(base),
                                    num_tokens=None if base is None else N)
    torch.cuda.synchronize()
    for got, exp, name in zip((t[0], t[1], t[3], t[4], ok), (want[0], want[1], want[2], [want[3]], want[4]),
                              ("table", "pages", "stack", "count", "ok")):
        assert np.array_equal(got.cpu().numpy(), exp), name
    if base is None:
        assert slots is None
    else:
        assert np.array_equal(slots.cpu().numpy(), want[5])
    return want


@pytest.mark.parametrize("B,width,ps,spare,N", [(1, 1, 1, 0, 1), (1, 9, 16, 3, 5), (3, 40, 8, 30, 13), (17, 300, 16, 900, 1),
                                                (40, 33, 64, 10, 700), (200, 70, 24, 9000, 37), (700, 5, 128, 2, 3),
                                                (16384, 2, 3, 5000, 2), (2, 20000, 1, 5000, 20000), (5, 600, 16, 99, 9000)])
def test_matches_the_plain_form(sv, B, width, ps, spare, N):  # noqa: F811
    for seed in range(3):
        rng = np.random.default_rng([B, width, seed])
        table, pages, stack, count = state(rng, B, width, ps, spare)
        length = rng.integers(0, width * ps + 1, B)
        if seed == 1:  # only a few rows change
            length = np.where(rng.random(B) < 0.9, pages * ps, length)
        base = np.clip(length - rng.integers(0, N + 3, B), -2, None)
        check(sv, table, pages, length, stack, count, ps, base, N)
        check(sv, table, pages, length, stack, count, ps)


def test_rows_that_cannot_be_served(sv):  # noqa: F811
    """Bad lengths and page counts leave rows as they are; the first row that finds too few pages stops later ones."""
    table = np.array([[0, 1, -1], [2, -1, -1], [3, 4, 5], [6, -1, -1], [7, -1, -1], [8, 9, -1]])
    stack = np.array([10, 11, 12, -1, -1, -1, -1, -1, -1, -1, -1, -1, -1])
    pages = np.array([2, 1, 3, 1, 1, 2])
    for length in ([-1, 13, 4, 12, 12, 8], [0, 4, 0, 12, 12, 12], [8, 8, 12, 8, 8, 12], [8, 12, 12, 12, 1, 9], [2 ** 31 - 1] * 6):
        check(sv, table, pages, np.array(length), stack, 3, 4, np.zeros(6, int), 14)
    for bad in (-1, 4, 2 ** 31 - 1):
        check(sv, table, np.where(np.arange(6) == 2, bad, pages), np.array([0, 4, 0, 12, 12, 12]), stack, 3, 4, np.zeros(6, int), 14)
    for count in (-5, 0, 13, 14, 1 << 30):  # a count outside the stack is read as if within it
        check(sv, table, pages, np.array([0, 8, 1, 0, 12, 12]), stack, count, 4)


def test_holes_are_not_given_back(sv):  # noqa: F811
    """A row whose early pages were dropped (a sliding window): its holes do not reach the stack."""
    table = np.array([[-1, -1, 5, 1, 99, 3], [7, 0, -1, -1, -1, -1]])
    stack = np.full(9, -1)
    stack[0] = 8
    check(sv, table, [6, 2], [0, 24], stack, 1, 4, [0, 3], 24)
    check(sv, table, [6, 2], [12, 9], stack, 1, 4, [-3, 3], 24)


@pytest.mark.parametrize("B,N", [(8, 6), (128, 40), (64, 2000)])
def test_captured_and_replayed(sv, B, N):  # noqa: F811
    """A graph that grows the rows and takes the growth back, replayed on new lengths, on two streams in turn."""
    import torch
    rng = np.random.default_rng(N)
    ps, width = 16, 40 + N // 16 + 1
    held = rng.integers(0, 640, B)
    need = -(-held // ps)
    P = B * width
    table = np.full((B, width), -1)
    perm = rng.permutation(P)
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    stack = np.concatenate([perm[at:], np.full(at, -1)])
    t = [ints(x) for x in (table, need, held, stack, [P - at])]
    longer, base = ints(held), ints(held)
    ok = torch.zeros((2, B), dtype=torch.int32, device="cuda")
    slots = torch.zeros((B, N), dtype=torch.int64, device="cuda")

    def step():
        sv.spec_page_resize(t[0], t[1], longer, t[3], t[4], ps, base=base, out_slots=slots, out_ok=ok[0])
        sv.spec_page_resize(t[0], t[1], t[2], t[3], t[4], ps, out_ok=ok[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    state_now = (table, need, stack, P - at)
    w = context.page_resize(*state_now[:2], held, state_now[2], state_now[3], ps)
    w = context.page_resize(w[0], w[1], held, w[2], w[3], ps)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        new = held + rng.integers(0, N + 1, B)
        longer.copy_(ints(new))
        graph.replay()
        w = context.page_resize(w[0], w[1], new, w[2], w[3], ps, held, N)
        want = w[5]
        w = context.page_resize(w[0], w[1], held, w[2], w[3], ps)
        torch.cuda.synchronize()
        assert np.array_equal(slots.cpu().numpy(), want)
        for got, exp in zip((t[0], t[1], t[3], t[4]), (w[0], w[1], w[2], [w[3]])):
            assert np.array_equal(got.cpu().numpy(), exp)
        assert ok.min() == 1


def test_refusals(sv):  # noqa: F811
    import torch
    good = dict(page_table=ints(np.zeros((2, 3))), pages=ints([0, 0]), length=ints([0, 0]), free_pages=ints(np.arange(6)),
                free_count=ints([6]), page_size=16)
    sv.spec_page_resize(**good)
    for bad in (dict(pages=ints([0])), dict(length=ints([0, 0, 0])), dict(free_count=ints([1, 2])),
                dict(page_table=ints(np.zeros(6))), dict(page_table=ints(np.zeros((2, 6)))[:, ::2]), dict(base=ints([0, 0])),
                dict(num_tokens=4), dict(out_slots=torch.zeros((2, 4), dtype=torch.int64, device="cuda")),
                dict(base=ints([0, 0]), num_tokens=-1), dict(pages=torch.zeros(2, dtype=torch.int32)),
                dict(base=ints([0, 0]), num_tokens=4, out_slots=torch.zeros((2, 3), dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            sv.spec_page_resize(**{**good, **bad})
    with pytest.raises(TypeError):
        sv.spec_page_resize(**{**good, "length": torch.zeros(2, dtype=torch.int64, device="cuda")})
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_page_resize(**{**good, "page_size": 0})
    ok, slots = sv.spec_page_resize(**good, base=ints([0, 0]), num_tokens=0)
    assert slots.shape == (2, 0) and ok.tolist() == [1, 1]
    empty = sv.spec_page_resize(ints(np.zeros((0, 3))), ints([]), ints([]), ints(np.arange(6)), ints([6]), 16)[0]
    assert empty.shape == (0,)
