"""Block summaries, block selection and attention over selected blocks on the GPU against their
plain forms in 64 bits.

Summaries: bounds are values of the cache (e4m3: code x scale, rounded by 2^-24) rounded to bf16, half a step 2^-8; a mean
of n values is off by n 2^-24 of the mean magnitude and by two fp32 roundings besides that.
Selection: whole numbers, equal: the order is that of sums in 64 bits, which bf16 products of
these magnitudes reach exactly in any order of summation.
Attention: the tolerance of the paged attention's own tests, over the listed positions.
"""
import math

import numpy as np
import pytest

import oracle
from oracle import context, paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_paged_kv import host, ints, make_cache, sv, values  # noqa: F401

pytestmark = pytest.mark.gpu


def decoded(pages, scales):
    v = values(pages)
    return v if scales is None else v * host(scales)[..., None]


def make_table(rng, B, width, spare=2):
    P = B * width + spare
    return rng.permutation(P)[:B * width].reshape(B, width), P


# ---------------------------------------------------------------- summaries

@pytest.mark.parametrize("kind", ["mean", "bounds"])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N,H,D,ps,ctx,nhd", [(1, 1, 1, 64, 16, 3, False), (3, 6, 8, 128, 64, 500, True),
                                                (2, 700, 3, 96, 24, 40, False), (2, 33, 2, 256, 5, 60, True),
                                                (1, 40, 2, 20, 16, 9, False), (2, 9, 1, 33, 1, 4, True),
                                                (2, 3000, 8, 128, 16, 100, False), (1, 2000, 1, 64, 4096, 5000, False)])
def test_summary(sv, kind, cache, B, N, H, D, ps, ctx, nhd):  # noqa: F811
    import torch
    rng = np.random.default_rng([N, D, ps])
    base, new = rng.integers(0, ctx + 1, B), rng.integers(0, N + 1, B)
    new[0] = N
    width = (ctx + N + ps - 1) // ps
    table, P = make_table(rng, B, width)
    if B > 1:
        table[1, int(base[1]) // ps] = P + 5  # a hole
    k, _, ks, _ = make_cache(rng, P, H, ps, D, cache, nhd)
    bounds = kind == "bounds"
    shape = (P, H, D * (1 + bounds))
    out = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got = sv.spec_block_summary(k, ints(table), ints(base), N, kind=kind, new_len=ints(new), k_scale=ks, summary=out)
    assert got is out
    v = decoded(k, ks)
    want = context.block_summary(v, table, base, new, N, bounds, np.full(shape, 7.0))
    size = context.block_summary(np.abs(v), table, base, new, N, False, np.zeros((P, H, D)))
    if bounds:
        tol = (2.0 ** -8 + 2.0 ** -23) * np.abs(want)
    else:
        tol = 2.0 ** -8 * np.abs(want) + (ps + 3) * 2.0 ** -24 * size
    assert (np.abs(host(out) - want) <= tol + 1e-37).all()
    new_out = sv.spec_block_summary(k, ints(table), ints(base), N, kind=kind, new_len=ints(new), k_scale=ks)
    touched = torch.from_numpy((want != 7).any((1, 2))).cuda()
    assert torch.equal(new_out[touched], out[touched]) and (new_out[~touched] == 0).all()


@pytest.mark.parametrize("kind", ["mean", "bounds"])
def test_summary_of_numbers_that_are_not_finite(sv, kind):  # noqa: F811
    """NaN makes its element NaN, infinities are values; the others of the block do not change."""
    import torch
    k = torch.from_numpy(np.random.default_rng(1).normal(size=(3, 2, 16, 64))).to(torch.bfloat16).cuda()
    # zeros between values of both signs: neither the largest nor the smallest, whose loss would show in the other bound
    k[1, 0, 5, 7] = k[1, 1, 3, 9] = k[2, 0, 0, 1] = k[2, 0, 9, 1] = 0
    table, base = ints([[0, 1, 2]]), ints([0])
    clean = sv.spec_block_summary(k, table, base, 48, kind=kind)
    k[1, 0, 5, 7], k[1, 1, 3, 9], k[2, 0, 0, 1], k[2, 0, 9, 1] = math.nan, math.inf, math.inf, -math.inf
    got = sv.spec_block_summary(k, table, base, 48, kind=kind)
    changed = (got != clean).nonzero().tolist()
    if kind == "mean":
        assert changed == [[1, 0, 7], [1, 1, 9], [2, 0, 1]]
        assert torch.isnan(got[1, 0, 7]) and got[1, 1, 9] == math.inf and torch.isnan(got[2, 0, 1])
    else:
        assert changed == [[1, 0, 7], [1, 0, 71], [1, 1, 9], [2, 0, 1], [2, 0, 65]]
        assert torch.isnan(got[1, 0, [7, 71]]).all() and got[2, 0, 1] == math.inf and got[2, 0, 65] == -math.inf
    # hidden behind the row's end: not read
    k[2, :, 10:] = math.nan
    short = sv.spec_block_summary(k, table, ints([40]), 2, kind=kind)
    assert torch.equal(short[2, 1], sv.spec_block_summary(torch.where(torch.isnan(k), 0, k), table, ints([40]), 2, kind=kind)[2, 1])


# ---------------------------------------------------------------- selection

def select_case(rng, B, Q, Hq, H, D, ps, blocks, bounds, spread=1.0):
    import torch
    base = rng.integers(0, blocks * ps + 1, B)
    base[0] = blocks * ps + min(ps - 1, 3)
    new = rng.integers(0, Q + 1, B)
    new[0] = Q
    width = blocks + 1 + (Q + ps - 1) // ps
    table, P = make_table(rng, B, width)
    m = rng.normal(size=(P, H, D)) * spread
    if bounds:
        m = np.concatenate([m + rng.uniform(0, 1, m.shape), m - rng.uniform(0, 1, m.shape)], -1)
    summary = torch.from_numpy(m).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.normal(size=(B, Q, Hq + 2, D))).to(torch.bfloat16).cuda()[:, :, 1:Hq + 1]
    return q, summary, table, base, new


def check_select(sv, q, summary, table, base, new, ps, top, kind, sink, recent, shared):  # noqa: F811
    got = sv.spec_block_select(q, summary, ints(table), ints(base), ps, top, kind=kind, sink=sink, recent=recent, shared=shared,
                               new_len=None if new is None else ints(new))
    want = context.block_select(host(q), host(summary), table, base, new, ps, top, kind == "bounds", sink, recent, shared)
    assert np.array_equal(got.cpu().numpy(), want)
    return got


@pytest.mark.parametrize("kind", ["mean", "bounds"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,Q,Hq,H,D,ps,blocks,top,sink,recent", [
    (1, 1, 4, 1, 64, 16, 40, 8, 1, 1), (2, 6, 8, 2, 128, 16, 300, 32, 1, 2), (2, 5, 7, 1, 96, 8, 100, 17, 0, 0),
    (2, 3, 24, 1, 72, 4, 70, 5, 2, 3), (1, 2, 40, 1, 128, 4, 50, 9, 1, 0), (3, 61, 8, 2, 128, 64, 130, 20, 1, 1),
    (2, 4, 6, 2, 256, 16, 77, 12, 0, 4), (1, 17, 16, 1, 64, 32, 33, 32, 1, 1), (2, 9, 3, 3, 8, 1, 500, 4, 4, 0),
    (1, 3, 2, 1, 64, 16, 3000, 700, 5, 9), (2, 2, 2, 2, 64, 16, 1, 4, 1, 1), (1, 130, 12, 3, 128, 16, 40, 10, 1, 1)])
def test_select(sv, kind, shared, B, Q, Hq, H, D, ps, blocks, top, sink, recent):  # noqa: F811
    rng = np.random.default_rng([Q, D, blocks])
    q, summary, table, base, new = select_case(rng, B, Q, Hq, H, D, ps, blocks, kind == "bounds")
    check_select(sv, q, summary, table, base, new, ps, top, kind, sink, recent, shared)
    check_select(sv, q, summary, table, base, None, ps, top, kind, sink, recent, shared)


@pytest.mark.parametrize("kind", ["mean", "bounds"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("same", [3, 60, 200])
@pytest.mark.parametrize("B,Q,blocks", [(2, 3, 260), (27, 3, 260), (80, 1, 260), (2, 3, 2100)])  # few lists, many, long ones
def test_select_among_equals(sv, kind, shared, same, B, Q, blocks):  # noqa: F811
    """Equal scores go to the lower blocks: few of them, as many as fit the short paths, and more; scores that
    differ by less than fp32 resolves keep their order."""
    rng = np.random.default_rng(same)
    q, summary, table, base, new = select_case(rng, B, Q, 4, 2, 64, 16, blocks, kind == "bounds")
    base[:] = blocks * 16
    for b in range(B):
        for h in range(2):
            at = np.sort(rng.permutation(250)[:same] + 5)
            summary[table[b, at], h] = summary[table[b, at[0]], h]
    for top in (4, 30, 120):
        check_select(sv, q, summary, table, base, None, 16, top, kind, 1, 1, shared)
    # one element far above the others: it hides in fp32 what 64 bits still tell apart
    q[..., 0] = 1.0
    for x in (0, 64) if kind == "bounds" else (0,):
        summary[..., x] = 2.0 ** 18
    for top in (4, 30, 120):
        check_select(sv, q, summary, table, base, None, 16, top, kind, 1, 1, shared)
    summary[:] = 0
    check_select(sv, q, summary, table, base, None, 16, 30, kind, 1, 1, shared)
    summary.normal_()
    q.zero_()
    check_select(sv, q, summary, table, base, None, 16, 30, kind, 1, 1, shared)


@pytest.mark.parametrize("kind", ["mean", "bounds"])
@pytest.mark.parametrize("B", [1, 80])  # few lists, and many
def test_select_numbers_that_are_not_finite(sv, kind, B):  # noqa: F811
    """NaN ranks below everything but holes; infinities rank where they belong; large numbers overflow nothing."""
    rng = np.random.default_rng(2)
    for case in range(5):
        q, summary, table, base, _ = select_case(rng, B, 2, 4, 1, 64, 16, 90, kind == "bounds")
        base[:] = 90 * 16
        pages = table[:, :90].T  # [block][row]
        if case == 0:
            summary[pages[10:80], 0, 5] = math.nan
        elif case == 1:
            summary[pages[20], 0, 5], summary[pages[30], 0, 6] = math.inf, -math.inf
        elif case == 2:
            q[0, 0, 1, 3] = math.nan
            q[0, 1, 2, 3] = math.inf
        elif case == 3:
            summary *= 2.0 ** 120
            q *= 2.0 ** 100
        else:
            table[:, 3:85] = -1  # holes: fewer blocks left than are wanted
            table[0, 50] = 10 ** 6
        for top in (4, 12, 60):
            check_select(sv, q, summary, table, base, None, 16, top, kind, 1, 1, False)


def test_select_many_blocks(sv):  # noqa: F811
    """65536 blocks, the most there can be; lists that hold all of a row's blocks, and untouched rows."""
    import torch
    rng = np.random.default_rng(8)
    width = 65536
    table = np.stack([rng.permutation(width + 3)[:width] for _ in range(2)])
    summary = torch.from_numpy(rng.normal(size=(width + 3, 1, 64))).to(torch.bfloat16).cuda()
    q = torch.from_numpy(rng.normal(size=(2, 2, 2, 64))).to(torch.bfloat16).cuda()
    base = np.array([width - 2, -1])
    check_select(sv, q, summary, table, base, None, 1, 4096, "mean", 1, 1, False)
    check_select(sv, q, summary, table, np.array([4096, 4097]), None, 1, 4096, "mean", 1, 1, True)
    check_select(sv, q, summary, table, np.array([width - 1, 0]), None, 1, 33, "mean", 30, 3, True)


def test_select_captured(sv):  # noqa: F811
    """A graph of summary and selection on a stream of its own, with its own scratch, replayed on new data."""
    import torch
    rng = np.random.default_rng(12)
    q, _, table, base, _ = select_case(rng, 2, 4, 8, 2, 64, 16, 120, False)
    base = np.array([1900, 900])
    k = make_cache(rng, table.size + 2, 2, 16, 64, "bf16", False)[0]
    q, t_table, t_base, zero, length = q.clone(), ints(table), ints(base), ints([0, 0]), ints(base)
    summary = torch.zeros((table.size + 2, 2, 128), dtype=torch.bfloat16, device="cuda")

    def step():
        sv.spec_block_summary(k, t_table, zero, 1950, kind="bounds", new_len=length, summary=summary)
        return sv.spec_block_select(q, summary, t_table, t_base, 16, 24, kind="bounds")

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lists = step()
    for _ in range(2):
        k.normal_()
        q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        want_m = context.block_summary(values(k), table, np.zeros(2, int), base, 1950, True, np.zeros(summary.shape))
        assert np.array_equal(host(summary), want_m)  # bf16 bounds are exact
        want = context.block_select(host(q), want_m, table, base, None, 16, 24, True, 1, 1, False)
        assert np.array_equal(lists.cpu().numpy(), want)


# ---------------------------------------------------------------- attention

def check_attention(got, lse, q, k, v, ks, vs, table, base, new, mask, blocks, scale, keep):
    """As the paged attention's tests, over the listed blocks."""
    B, Q, Hq, D = q.shape
    kv, vv, qh = decoded(k, ks), decoded(v, vs), host(q)
    args = (table, base, new, mask, blocks, scale)
    full, full_lse = np.full((B, Q, Hq, D), keep), np.full((B, Q, Hq), keep)
    want, want_lse = context.sparse_attention(qh, kv, vv, *args, full, full_lse)
    size, _ = context.sparse_attention(qh, kv, np.abs(vv), *args, full, full_lse)
    H = kv.shape[1]
    ka = np.where(np.isfinite(kv), np.abs(kv), 0).transpose(1, 0, 2, 3).reshape(H, -1, D)
    qa = np.abs(qh).reshape(B * Q, H, Hq // H, D).transpose(1, 0, 2, 3).reshape(H, -1, D)
    e = (D + 16) * 2.0 ** -22 * abs(scale) * max((qa[h] @ ka[h].T).max() for h in range(H))
    tol = (2.0 ** -8 + 4 * e) * np.abs(size) + 2.0 ** -8 * np.abs(want) + 1e-30
    if vs is not None and Q * Hq // H > 16:  # multiplied as fp16
        s = host(vs)
        n = blocks.shape[3] * kv.shape[2] + Q + kv.shape[2]
        tol = tol + n * 2.0 ** -31 * 448 * s[np.isfinite(s)].max()
    g, gl = host(got), host(lse)
    assert np.isfinite(g).all()
    worst = (np.abs(g - want) / tol).max()
    assert worst <= 1, f"output off by {worst:.3g} tolerances"
    assert np.array_equal(np.isneginf(gl), np.isneginf(want_lse))
    f = np.isfinite(want_lse)
    assert (np.abs(gl[f] - want_lse[f]) <= 2 * e + 2.0 ** -21 * (1 + np.abs(want_lse[f]))).all()


def attention_case(rng, B, Q, Hq, H, D, ps, ctx, n, cache, tree, nhd, shared):
    import torch
    base = rng.integers(0, ctx + 1, B)
    base[0] = ctx
    new = rng.integers(0, Q + 1, B)
    new[0] = Q
    width = (ctx + Q + ps - 1) // ps
    table, P = make_table(rng, B, width)
    k, v, ks, vs = make_cache(rng, P, H, ps, D, cache, nhd)
    if cache == "e4m3":
        for t in (k, v):
            t.view(torch.uint8).bitwise_xor_(torch.randint(0, 2, t.shape, device="cuda", dtype=torch.uint8) << 7)
        ks *= 0.05
    blocks = np.full((B, 1 if shared else Q, H, n), -1)
    for idx in np.ndindex(blocks.shape[:3]):
        full = int(base[idx[0]]) // ps
        m = int(rng.integers(0, min(full, n) + 1))
        blocks[idx][:m] = np.sort(rng.permutation(full)[:m])
    q = torch.from_numpy(rng.normal(size=(B, Q, Hq + 3, D))).to(torch.bfloat16).cuda()[:, :, 1:Hq + 1]
    mask = None
    if tree and Q > 1:
        mask = oracle.tree_mask(synth.random_parents(int(rng.integers(1 << 20)), B, Q - 1, max_depth=9))["mask"]
    return q, k, v, ks, vs, table, base, new, mask, blocks


def run(sv, c, **kw):  # noqa: F811
    import torch
    q, k, v, ks, vs, table, base, new, mask, blocks = c
    B, Q, Hq, D = q.shape
    out = torch.full((B, Q, Hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, Q, Hq), 3.0, device="cuda")
    words = None if mask is None else torch.from_numpy(np.ascontiguousarray(mask).view(np.int32)).cuda()
    return sv.spec_sparse_attention(q, k, v, ints(table), ints(base), ints(blocks), new_len=ints(new), tree_mask=words,
                                    k_scale=ks, v_scale=vs, out=out, out_lse=lse, **kw)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("B,Q,Hq,H,D,ps,ctx,n,tree,nhd", [
    (1, 1, 4, 1, 64, 16, 500, 8, False, False), (2, 6, 8, 2, 128, 16, 1000, 20, False, True),
    (2, 5, 7, 1, 96, 8, 300, 9, True, False), (2, 3, 20, 1, 64, 24, 400, 5, True, False),
    (2, 4, 6, 2, 256, 16, 333, 7, False, False), (2, 30, 8, 2, 128, 64, 1500, 6, True, False),
    (1, 2, 40, 1, 128, 32, 700, 9, False, False), (2, 17, 2, 2, 64, 1, 90, 33, False, True),
    (2, 9, 4, 4, 8, 5, 77, 4, True, False), (1, 130, 4, 1, 128, 16, 260, 3, False, False),
    (2, 7, 4, 2, 128, 128, 2600, 40, False, False), (2, 4, 4, 2, 64, 16, 100, 0, True, False),
    (1, 3, 64, 1, 64, 4096, 9000, 2, False, False)])
def test_attention(sv, cache, shared, B, Q, Hq, H, D, ps, ctx, n, tree, nhd):  # noqa: F811
    rng = np.random.default_rng([Q, D, n])
    c = attention_case(rng, B, Q, Hq, H, D, ps, ctx, n, cache, tree, nhd, shared)
    if cache == "e4m3" and D % 16:  # rows of 8 bytes: refused, as spec_paged_attention does
        with pytest.raises(sv.SpecVerifyError):
            run(sv, c)
        return
    got, lse = run(sv, c)
    check_attention(got, lse, *c, D ** -0.5, 3.0)


@pytest.mark.parametrize("shared", [False, True])
def test_all_blocks_are_the_paged_attention(sv, shared):  # noqa: F811
    """Lists of every context block: the sums of spec_paged_attention, within both tolerances."""
    import torch
    rng = np.random.default_rng(4)
    c = attention_case(rng, 3, 6, 8, 2, 128, 16, 640, 40, "bf16", True, False, shared)
    q, k, v, ks, vs, table, base, new, mask, blocks = c
    for b in range(3):
        blocks[b] = np.where(np.arange(40) < base[b] // 16, np.arange(40), -1)
    got, lse = run(sv, c)
    dense, dense_lse = sv.spec_paged_attention(q, k, v, ints(table), ints(base), new_len=ints(new),
                                               tree_mask=torch.from_numpy(mask.view(np.int32)).cuda(), want_lse=True)
    for b in range(3):
        a, d = host(got[b, :new[b]]), host(dense[b, :new[b]])
        # two results off by (2^-8 + 2^-8) of a weighted mean of |v| each, |v| <= 6
        assert (np.abs(a - d) <= 2.0 ** -6 * 6).all()
        assert (np.abs(host(lse[b, :new[b]]) - host(dense_lse[b, :new[b]])) <= 1e-3).all()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shared", [False, True])
def test_lists_out_of_order(sv, cache, shared):  # noqa: F811
    """Entries that do not ascend, repeat, lie outside the context, or name holes."""
    rng = np.random.default_rng(6)
    c = attention_case(rng, 3, 5, 8, 2, 64, 16, 900, 37, cache, False, False, shared)
    table, base, blocks = c[5], c[6], c[9]
    base[:] = [900, 40, -1]
    blocks[...] = rng.integers(-3, 70, blocks.shape)
    blocks[0, 0, 0, :6] = [5, 5, 4, 2 ** 31 - 1, 6, -2 ** 31]
    blocks[0, -1, 1] = 7
    table[0, [3, 6, 9, 12]] = [-1, 10 ** 6, -5, 2 ** 31 - 1]
    table[1, 2] = -1
    got, lse = run(sv, c)
    check_attention(got, lse, *c, 64 ** -0.5, 3.0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shared,Q", [(False, 5), (True, 5), (True, 40)])
def test_hidden_positions_do_not_matter(sv, cache, shared, Q):  # noqa: F811
    """NaN and infinities in blocks that no list names, behind the rows' ends, and at tokens that a query
    does not see change no bit of its output."""
    import torch
    rng = np.random.default_rng(7)
    c = attention_case(rng, 2, Q, 8, 2, 64, 16, 700, 12, cache, True, False, shared)
    q, k, v, ks, vs, table, base, new, mask, blocks = c
    new[:] = Q - 1
    first = [x.clone() for x in run(sv, c)]
    P = k.shape[0]
    named = np.zeros((P, 2), bool)
    for b in range(2):
        for i in range(blocks.shape[1]):
            for h in range(2):
                for e in blocks[b, i, h]:
                    if e >= 0:
                        named[table[b, e], h] = True
        for j in range(int(base[b]) // 16, (int(base[b]) + Q + 15) // 16):
            named[table[b, j]] = True
    hide = torch.from_numpy(~named).cuda()[:, :, None, None]
    bad = 0x7f if cache == "e4m3" else math.nan
    for t in (k, v):
        (t.view(torch.uint8) if cache == "e4m3" else t).masked_fill_(hide, bad)
    for b in range(2):  # the row that is not real
        p, r = paged.place(table, b, int(base[b]) + Q - 1, P, 16)
        for t in (k, v):
            (t.view(torch.uint8) if cache == "e4m3" else t)[p, :, r] = bad
    again = run(sv, c)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # a node that only its descendants see: the others' bits stay
    leaf = Q - 3  # node index of token Q - 2
    b = 0
    p, r = paged.place(table, b, int(base[b]) + leaf + 1, P, 16)
    (v.view(torch.uint8) if cache == "e4m3" else v)[p, :, r] = bad
    third = run(sv, c)
    words = mask[b].view(np.uint32)
    for i in range(Q - 1):
        sees = i > 0 and bool((int(words[i - 1, leaf // 32]) >> (leaf % 32)) & 1)
        assert torch.equal(third[0][b, i], again[0][b, i]) != sees
        if sees:
            assert torch.isnan(third[0][b, i]).all()


def test_rows_whose_scores_are_all_minus_infinity(sv):  # noqa: F811
    """They give zero and lse -infinity, as the paged attention does."""
    rng = np.random.default_rng(9)
    c = attention_case(rng, 1, 3, 4, 2, 64, 16, 200, 5, "bf16", False, False, False)
    q, k = c[0], c[1]
    q[..., 0] = 1.0
    k[..., 0] = -math.inf
    got, lse = run(sv, c)
    assert (got == 0).all() and (lse == -math.inf).all()


def test_workspace_streams_and_graphs(sv):  # noqa: F811
    """A given scratch, two graphs that share it and run in turn, and a call on another stream."""
    import torch
    rng = np.random.default_rng(10)
    cases = [attention_case(rng, 2, 5, 8, 2, 128, 16, 2000, 50, "bf16", False, False, s) for s in (False, True)]
    wants = [[x.clone() for x in run(sv, c)] for c in cases]
    sizes = [sv.spec_sparse_attention_workspace_size(2, 5, 8, 2, 128, torch.bfloat16, 16, 50, s) for s in (False, True)]
    scratch = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    tensors, graphs, outs = [], [], []
    for c in cases:
        q, k, v, _, _, table, base, new, _, blocks = c
        tensors.append((q, k, v, ints(table), ints(base), ints(blocks)))
        lens = ints(new)
        out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(q.shape[:3], 3.0, device="cuda")
        call = lambda t=tensors[-1], n=lens, o=out, z=lse: sv.spec_sparse_attention(*t, new_len=n, out=o, out_lse=z, workspace=scratch)  # noqa: E731
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
        outs.append((out, lse))
        tensors.append(lens)
    for k in (0, 1, 0, 1):
        for o in outs[k]:
            o.fill_(3.0)
        scratch.fill_(0xff)
        graphs[k].replay()
        assert torch.equal(outs[k][0], wants[k][0]) and torch.equal(outs[k][1], wants[k][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [run_on(sv, c, side) for c in cases]
    side.synchronize()
    for (o, z), w, c in zip(got, wants, cases):
        for b in range(2):
            n = c[7][b]
            assert torch.equal(o[b, :n], w[0][b, :n]) and torch.equal(z[b, :n], w[1][b, :n])


def run_on(sv, c, stream):  # noqa: F811
    import torch
    q, k, v, _, _, table, base, new, _, blocks = c
    args = [ints(x) for x in (table, base, blocks, new)]
    torch.cuda.synchronize()
    return sv.spec_sparse_attention(q, k, v, *args[:3], new_len=args[3], want_lse=True, stream=stream)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shared,Q", [(False, 5), (True, 5), (True, 70)])
def test_rows_that_see_nothing_and_short_rows(sv, cache, shared, Q):  # noqa: F811
    """Tables of holes alone, no context, no real query, a context of less than a block."""
    rng = np.random.default_rng(11)
    c = attention_case(rng, 5, Q, 8, 2, 64, 16, 400, 6, cache, True, False, shared)
    table, base, new = c[5], c[6], c[7]
    base[:], new[:] = [400, 0, 300, 7, 16], [Q, Q, 0, 1, 2]
    c[9][1:] = -1
    c[9][4, :, :, 0] = 0
    table[0] = -1
    got, lse = run(sv, c)
    check_attention(got, lse, *c, 64 ** -0.5, 3.0)
    assert (got[0] == 0).all() and (lse[0] == -math.inf).all() and (got[2] == 3).all()


def test_offsets_beyond_32_bits(sv):  # noqa: F811
    """Pages that lie more than 4 GB into the cache, against the same pages in a small one."""
    import torch
    P, H, ps, D, B, Q, n = 40000, 8, 64, 128, 2, 5, 9  # 131 KB a page: 5.2 GB of keys
    if torch.cuda.mem_get_info()[0] < 24e9:
        pytest.skip("needs 24 GB")
    k, v = (torch.zeros((P, H, ps, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    summary = torch.zeros((P, H, 2 * D), dtype=torch.bfloat16, device="cuda")
    used = torch.arange(P - 40, P, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    k[used], v[used] = (torch.randn((40, H, ps, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in "kv")
    small = [k[used].clone(), v[used].clone(), torch.zeros((40, H, 2 * D), dtype=torch.bfloat16, device="cuda")]
    table = ints(np.random.default_rng(1).permutation(40).reshape(2, 20))
    base, qkv = ints([1100, 700]), torch.randn((B, Q, 48, D), generator=gen, device="cuda").to(torch.bfloat16)
    freq = sv.rotary_frequencies(D, device="cuda")
    got = []
    for kk, vv, mm, t in ((k, v, summary, table + (P - 40)), (*small, table)):
        q = sv.spec_rotary_append(qkv[:, :, :32], qkv[:, :, 32:40], qkv[:, :, 40:], freq, kk, vv, t, base)
        sv.spec_block_summary(kk, t, ints([0, 0]), 1105, kind="bounds", new_len=base + Q, summary=mm)
        blocks = sv.spec_block_select(q, mm, t, base, ps, n, kind="bounds")
        got.append((q, blocks, *sv.spec_sparse_attention(q, kk, vv, t, base, blocks, want_lse=True),
                    *sv.spec_sparse_attention(q, kk, vv, t, base, blocks[:, :1].contiguous(), want_lse=True)))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    for big, few in zip((k, v, summary), small):
        assert torch.equal(big[used], few)


def test_refusals(sv):  # noqa: F811
    import torch
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros((6, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    table, base, blocks = ints(np.zeros((2, 3))), ints([40, 40]), ints(np.zeros((2, 3, 2, 2)))
    good = dict(q=q, k_pages=pages, v_pages=pages, page_table=table, base=base, blocks=blocks)
    sv.spec_sparse_attention(**good)
    for bad in (dict(blocks=blocks[:, :2]), dict(blocks=blocks[0]), dict(blocks=blocks[:, :, :1]), dict(base=ints([1])),
                dict(q=q[:, :0]), dict(q=torch.zeros((2, 3, 5, 64), dtype=torch.bfloat16, device="cuda")),
                dict(tree_mask=ints(np.zeros((2, 3, 1)))), dict(k_scale=torch.ones((6, 2, 16), device="cuda")),
                dict(blocks=blocks.cpu()), dict(out=q[:1]), dict(blocks=ints(np.zeros((2, 3, 2, 4)))[..., ::2])):
        with pytest.raises(ValueError):
            sv.spec_sparse_attention(**{**good, **bad})
    with pytest.raises(TypeError):
        sv.spec_sparse_attention(**{**good, "blocks": blocks.long()})
    for bad in (dict(workspace=None), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
                dict(scale=math.nan), dict(q=torch.zeros((2, 3, 4, 72), dtype=torch.bfloat16, device="cuda")[..., 4:68])):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_sparse_attention(**{**good, **bad})
    summary = torch.zeros((6, 2, 64), dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, summary=summary, page_table=table, base=base, page_size=16, top_k=2)
    assert sv.spec_block_select(**good).tolist() == [[[[0, 1]] * 2] * 3] * 2
    for bad in (dict(summary=summary[..., :32]), dict(kind="bounds"), dict(kind="sum"), dict(base=ints([1])),
                dict(page_table=table[0]), dict(out=ints(np.zeros((2, 3, 2, 3)))), dict(q=q[:, :, :3])):
        with pytest.raises(ValueError):
            sv.spec_block_select(**{**good, **bad})
    for bad in (dict(top_k=1), dict(sink=2), dict(workspace=None), dict(page_size=0), dict(top_k=4097),
                dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(sv.SpecVerifyError):
            sv.spec_block_select(**{**good, **bad})
    with pytest.raises(ValueError):
        sv.spec_block_summary(pages, table, base, 4, summary=summary[:5])
    with pytest.raises(ValueError):
        sv.spec_block_summary(pages, table, base, -1)
    assert sv.spec_block_summary(pages, table, base, 0, kind="bounds").shape == (6, 2, 128)
