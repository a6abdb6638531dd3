"""What a query does not see never moves its output, not by a bit.

A new token's key, value and scales change, from far below to far above those around it and
through the whole range in which the e4m3 kernel keeps room for it (2^12 times the largest value
scale that every query sees); the queries that do not see it return the very same bits, and
match the plain form with a tolerance that takes its scales from what they do see."""
import numpy as np
import pytest

from test_gpu_attention import case, check, run
from test_gpu_paged_kv import host, sv  # noqa: F401

pytestmark = pytest.mark.gpu

SHAPES = [  # Q, Hq, D, page_size, ctx
    (3, 4, 128, 16, 300), (20, 4, 128, 16, 300), (30, 2, 64, 16, 1500), (61, 4, 128, 64, 700), (61, 4, 128, 24, 2500),
    (40, 4, 128, 16, 0), (40, 1, 128, 16, 130), (40, 4, 256, 16, 500), (33, 2, 64, 8, 60)]


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_hidden_tokens_move_no_bit(sv, shape, tree, cache):  # noqa: F811
    import torch
    Q, Hq, D, ps, ctx = shape
    rng = np.random.default_rng([*shape, tree])
    c = case(rng, 1, Q, Hq, 1, D, ps, ctx, cache, tree, False, ragged=False)
    q, k, v, ks, vs, table, base, new_len, mask = c
    clean, clean_l = run(sv, c)
    node = Q // 2 - 1                             # token node + 1
    sees = np.array([False] + [(bool((int(mask[0, i, node // 32]) >> (node % 32)) & 1) if tree else i >= node)
                               for i in range(Q - 1)])
    assert sees.any() and not sees.all()
    pos = int(base[0]) + node + 1
    page, row = int(table[0, pos // ps]), pos % ps
    held = host(vs) if cache == "e4m3" else None
    top = held[np.isfinite(held)].max() if cache == "e4m3" else 1.0
    for step in range(14):
        if cache == "e4m3":
            factor = 2.0 ** [-40, -3, 0.5, 2, 3.3, 5, 7.1, 8, 9, 10.2, 11, 11.9, 12.5, 60][step]
            vs[page, 0, row], ks[page, 0, row] = float(top * factor), float(rng.uniform(1e-3, 1e3))
            for t in (k, v):
                t[page, 0, row].view(torch.uint8).copy_(torch.from_numpy(rng.integers(0, 127, D, dtype=np.uint8)))
        else:
            for t in (k, v):
                t[page, 0, row] = torch.from_numpy(rng.normal(size=D) * 10.0 ** (4 * step - 20)).to(t.dtype)
        o, l = run(sv, c)
        assert torch.equal(o[0, ~sees], clean[0, ~sees]) and torch.equal(l[0, ~sees], clean_l[0, ~sees]), step
    if cache == "e4m3":  # the last one 2^60 above: out of the sums of the tolerance
        ks[page, 0, row] = float("nan")
        check(clean, clean_l, q, k, v, ks, vs, table, base, new_len, mask, D ** -0.5, 5.0, 6.0, ~sees, top)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("first", ["zero", "hole"])
@pytest.mark.parametrize("shape", [(20, 4, 128, 16, 0), (150, 4, 64, 16, 0), (300, 1, 128, 64, 0), (61, 4, 128, 24, 0),
                                   (40, 4, 256, 16, 0), (200, 4, 128, 16, 600), (30, 4, 64, 16, 700)])
def test_no_value_scale_to_go_by(sv, shape, first, tree):  # noqa: F811
    """Nothing that every query sees has a value of any size: a prompt (or a context of zeros and new
    tokens) whose first values are zeros of the smallest scale, or lie in a hole.  All other new
    tokens' values are then left to the end."""
    import torch
    Q, Hq, D, ps, ctx = shape
    rng = np.random.default_rng([*shape, tree])
    c = case(rng, 2, Q, Hq, 1, D, ps, ctx, "e4m3", tree, False, ragged=False)
    q, k, v, ks, vs, table, base, new_len, mask = c
    for b in range(2):
        for pos in range(ctx + 1):
            page, row = int(table[b, pos // ps]), pos % ps
            vs[page, 0, row] = 2.0 ** -126
            v[page, 0, row].view(torch.uint8).fill_(0)
        if first == "hole":
            table[b, :ctx // ps + 1] = -1
    o, l = run(sv, c)
    check(o, l, *c[:9], D ** -0.5, 5.0, 6.0)


@pytest.mark.parametrize("workspace", ["auto", None])
@pytest.mark.parametrize("Q,ctx", [(1, 40), (3, 1500), (20, 300), (30, 1500), (61, 2500), (61, 0)])
def test_scores_of_minus_infinity_alone_give_zero(sv, Q, ctx, workspace):  # noqa: F811
    """Every key holds -inf: no position has any weight, whatever the values hold."""
    import torch
    rng = np.random.default_rng([Q, ctx])
    c = case(rng, 1, Q, 4, 1, 128, 16, ctx, "bf16", Q == 61, False, ragged=False)
    q, k, v, ks, vs, table, base, new_len, mask = c
    q.abs_().clamp_(min=0.1)
    k[..., 7].masked_fill_(~k[..., 7].isnan(), float("-inf"))
    for pos in (ctx // 2, ctx, ctx + Q // 2):
        v[int(table[0, pos // 16]), 0, pos % 16, 3:9] = float("nan")
        v[int(table[0, pos // 16]), 0, pos % 16, 9:12] = float("inf")
    o, l = run(sv, c, workspace=workspace)
    assert (o == 0).all() and torch.isneginf(l).all()
