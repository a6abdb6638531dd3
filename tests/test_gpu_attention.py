"""Paged attention on the GPU against its plain float64 form.

Tolerance of an output: each probability enters the second product rounded to bf16 (half a
step, 2^-8 of itself), and a score is off by at most e = (D + 16) 2^-22 scale sum|q k| (fp32
products and sums, the tensor cores' own rounding included; the exponential's 2^-22 is far
below), which moves a weight by at most 2e + the same for the sum.  So with A the weighted
mean of |v|, |out - want| <= (2^-8 + 4 e) A, plus the output's own half step 2^-8 |want|.
lse moves by at most 2 e, plus fp32 roundings of its own value.

e4m3 calls of more than 16 query rows per cache head multiply in fp16, half step 2^-11: an
element of a value and a probability are rounded once each, together below bf16's 2^-8.
Probabilities are held times 2^7, where fp16 steps by 2^-24 below 2^-14: a position whose weight
is tiny is off by up to 2^-32 of the largest weight, and the sum they are divided by is at
least 1: n positions add at most n 2^-32 V, V = 448 vmax the largest |v| that the scales allow.  A value element far below V is
off by up to 2^-25 2^E with 2^E <= 2^-5 vmax, below 2^-38 V (both are within n 2^-31 V); a hidden
scale of up to 2^12 vmax takes that to 2^-26 V, which the test of such scales adds.
"""
import numpy as np
import pytest

import oracle
from oracle import paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_paged_kv import host, ints, make_cache, sv, values  # noqa: F401

pytestmark = pytest.mark.gpu


def check(got, lse, q, k, v, ks, vs, table, base, new_len, mask, scale, keep_out, keep_lse, rows=None, vmax=None):
    """Compares whole outputs, or the queries `rows`, for which `vmax` is the largest value scale;
    keep_out and keep_lse fill what must not be written."""
    B, Q, Hq, D = q.shape
    kv, vv = values(k), values(v)
    if ks is not None:
        kv, vv = kv * host(ks)[..., None], vv * host(vs)[..., None]
    qh, zo = host(q), np.full((B, Q, Hq, D), keep_out)
    want, want_lse = paged.attention(qh, kv, vv, None, None, table, base, new_len, mask, scale, zo,
                                     np.full((B, Q, Hq), keep_lse))
    size, _ = paged.attention(qh, kv, np.abs(vv), None, None, table, base, new_len, mask, scale, zo,
                              np.zeros((B, Q, Hq)))
    H = kv.shape[1]
    ka = np.where(np.isfinite(kv), np.abs(kv), 0).transpose(1, 0, 2, 3).reshape(H, -1, D)
    qa = np.abs(qh).reshape(B * Q, H, Hq // H, D).transpose(1, 0, 2, 3).reshape(H, -1, D)
    reach = abs(scale) * max((qa[h] @ ka[h].T).max() for h in range(H))  # largest sum |q k|
    half = vs is not None and Q * Hq // H > 16  # multiplied as fp16
    e = (D + 16) * 2.0 ** -22 * reach
    g, gl = host(got), host(lse)
    tol = (2.0 ** -8 + 4 * e) * np.abs(size) + 2.0 ** -8 * np.abs(want) + 1e-30
    if half:
        scales = host(vs)
        vmax = scales[np.isfinite(scales)].max() if vmax is None else vmax
        tol = tol + (int(base.max()) + Q) * 2.0 ** -31 * 448 * vmax
        if rows is not None:
            tol = tol + 2.0 ** -26 * 448 * vmax
    if rows is not None:
        g, gl, want, want_lse, tol = (x[:, rows] for x in (g, gl, want, want_lse, tol))
    assert np.isfinite(g).all()
    worst = (np.abs(g - want) / tol).max()
    assert worst <= 1, f"output off by {worst:.3g} tolerances"
    assert np.array_equal(np.isneginf(gl), np.isneginf(want_lse))
    f = np.isfinite(want_lse)
    gl, want_lse = gl[f], want_lse[f]
    assert (np.abs(gl - want_lse) <= 2 * e + 2.0 ** -21 * (1 + np.abs(want_lse))).all()


def case(rng, B, Q, Hq, H, D, ps, ctx, cache, tree, nhd, ragged=True, spread=1.0):
    """Random call: ragged contexts, every page that no row owns filled with NaN."""
    import torch
    base = rng.integers(0, ctx + 1, B) if ragged else np.full(B, ctx)
    new_len = rng.integers(0 if B > 1 else 1, Q + 1, B) if ragged else np.full(B, Q)
    new_len[0] = Q
    mp = (ctx + Q + ps - 1) // ps
    P = B * mp + 2
    table = rng.permutation(P)[:B * mp].reshape(B, mp)
    k, v, ks, vs = make_cache(rng, P, H, ps, D, cache, nhd)
    if cache == "e4m3":  # all codes that are numbers
        for t in (k, v):
            t.view(torch.uint8).bitwise_xor_(torch.randint(0, 2, t.shape, device="cuda", dtype=torch.uint8) << 7)
        ks *= 0.05
    poison(k, v, ks, vs, table, base, new_len, ps)
    q = torch.from_numpy(spread * rng.normal(size=(B, Q, Hq + 3, D))).to(torch.bfloat16).cuda()[:, :, 1:Hq + 1]
    mask = None
    if tree and Q > 1:
        par = synth.random_parents(int(rng.integers(1 << 20)), B, Q - 1, max_depth=9)
        mask = oracle.tree_mask(par)["mask"]
    return q, k, v, ks, vs, table, base, new_len, mask


def poison(k, v, ks, vs, table, base, new_len, ps):
    """NaN in every cache row that holds no real position."""
    import torch
    held = np.zeros((k.shape[0], ps), bool)
    for b in range(len(base)):
        for pos in range(max(0, int(base[b])) + int(new_len[b])):
            p = table[b, pos // ps] if pos // ps < table.shape[1] else -1
            if 0 <= p < len(held):
                held[p, pos % ps] = True
    free = torch.from_numpy(~held).cuda()[:, None, :, None]
    for t in (k, v):
        if t.dtype == torch.bfloat16:
            t.masked_fill_(free, float("nan"))
        else:
            t.view(torch.uint8).masked_fill_(free, 0x7f)
    for s in (ks, vs):
        if s is not None:
            s.masked_fill_(free[..., 0], float("nan"))


def run(sv, c, scale=None, workspace="auto", max_len=None, **kw):
    import torch
    q, k, v, ks, vs, table, base, new_len, mask = c
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:3], 6.0, device="cuda")
    m = None if mask is None else ints(mask.view(np.int32))
    o, l = sv.spec_paged_attention(q, k, v, ints(table), ints(base), new_len=ints(new_len), tree_mask=m, scale=scale,
                                   k_scale=ks, v_scale=vs, out=out, out_lse=lse, workspace=workspace, max_len=max_len,
                                   **kw)
    assert o is out and l is lse
    return o, l


def both(sv, c, **kw):
    q = c[0]
    o, l = run(sv, c, **kw)
    check(o, l, *c[:5], c[5], c[6], c[7], c[8], q.shape[3] ** -0.5, 5.0, 6.0)


CASES = [  # B, Q, Hq, H, D, page_size, ctx
    (1, 1, 1, 1, 64, 16, 0), (1, 1, 8, 1, 128, 16, 1), (3, 1, 8, 2, 128, 16, 777), (2, 6, 8, 2, 128, 24, 300),
    (3, 6, 7, 1, 64, 1, 130), (2, 2, 16, 2, 96, 64, 500), (2, 17, 4, 2, 128, 16, 129), (2, 61, 4, 1, 128, 32, 200),
    (1, 130, 2, 2, 64, 8, 70), (2, 5, 3, 3, 256, 16, 260), (1, 33, 2, 1, 200, 128, 90), (2, 64, 1, 1, 128, 64, 0),
    (1, 9, 8, 1, 16, 5, 63), (2, 20, 8, 4, 128, 16, 640), (1, 70, 8, 2, 128, 48, 150), (1, 300, 2, 1, 128, 64, 100), (2, 30, 4, 1, 64, 16, 300), (1, 25, 8, 2, 128, 16, 500),
    (2, 40, 4, 2, 96, 16, 130), (1, 61, 4, 1, 128, 16, 2500), (1, 150, 1, 1, 64, 8, 900), (2, 33, 7, 1, 128, 64, 40)]


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", CASES)
def test_matches_the_plain_form(sv, shape, cache, tree):  # noqa: F811
    rng = np.random.default_rng([*shape, cache == "e4m3", tree])
    if cache == "e4m3" and shape[4] % 16:
        pytest.skip("rows of codes would not be 16-byte aligned")
    both(sv, case(rng, *shape, cache, tree, nhd=sum(shape) % 2 == 1))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Q,Hq", [(1, 2), (7, 4), (61, 4)])
def test_peaked_scores_and_other_scales(sv, cache, Q, Hq):  # noqa: F811
    """Scores of several tens: the running maximum moves from tile to tile."""
    rng = np.random.default_rng([Q, Hq])
    c = case(rng, 2, Q, Hq, 1, 128, 16, 500, cache, Q > 7, False, spread=6.0)
    for scale in (0.2, -0.05, 0.0):
        o, l = run(sv, c, scale=scale)
        check(o, l, *c[:9], scale, 5.0, 6.0)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Q", [1, 6, 61])
def test_split_and_unsplit_agree_with_the_plain_form(sv, cache, Q):  # noqa: F811
    """The automatic split, none, and bounds that are too small or far too large."""
    rng = np.random.default_rng(Q)
    c = case(rng, 3, Q, 8, 2, 128, 16, 1500, cache, Q == 61, False)
    for kw in (dict(), dict(workspace=None), dict(max_len=1), dict(max_len=200), dict(max_len=1 << 30)):
        both(sv, c, **kw)


@pytest.mark.parametrize("Q,ps", [(6, 16), (61, 16), (61, 24), (30, 64)])
def test_e4m3_scales_of_very_different_sizes(sv, Q, ps):  # noqa: F811
    """Value scales over a factor of 2^18 that grow and shrink along the context, key scales over
    2^6, a row of zeros (the smallest scale there is), queries from tiny to large."""
    import torch
    rng = np.random.default_rng([Q, ps])
    c = case(rng, 2, Q, 4, 1, 128, ps, 700, "e4m3", Q > 7, False, ragged=False)
    q, k, v, ks, vs, table, base, new_len, mask = c
    P, H, _ = vs.shape
    vs.copy_(torch.from_numpy(2.0 ** rng.uniform(-9, 9, (P, H, ps))).float())
    ks.copy_(torch.from_numpy(0.01 * 2.0 ** rng.uniform(-3, 3, (P, H, ps))).float())
    page, row = int(table[0, 5]), 3
    vs[page, :, row] = 2.0 ** -126
    v[page, :, row] = 0
    poison(k, v, ks, vs, table, base, new_len, ps)
    q *= torch.from_numpy(2.0 ** rng.uniform(-20, 3, (2, Q, 4, 1))).cuda()
    both(sv, c)


@pytest.mark.parametrize("cache,D,width", [("e4m3", 72, 80), ("e4m3", 40, 48), ("e4m3", 128, 144), ("bf16", 72, 80), ("bf16", 128, 136),
                                           ("e4m3", 200, 208)])
@pytest.mark.parametrize("Q", [2, 9, 61])
def test_rows_that_are_slices_of_wider_ones(sv, cache, D, width, Q):  # noqa: F811
    """Cache rows of a fused tensor: what lies beside a row is never read as part of it."""
    import torch
    rng = np.random.default_rng([D, Q])
    q, k, v, ks, vs, table, base, new_len, mask = case(rng, 2, Q, 8, 2, D, 16, 150, cache, False, False)
    wide = []
    for t in (k, v):
        w = torch.full((*t.shape[:3], width), float("nan"), dtype=torch.bfloat16, device="cuda") if cache == "bf16" else \
            torch.full((*t.shape[:3], width), 0x7f, dtype=torch.uint8, device="cuda").view(t.dtype)
        bits = torch.int16 if cache == "bf16" else torch.uint8
        w.view(bits)[..., :D].copy_(t.view(bits))
        wide.append(w[..., :D])
    both(sv, (q, *wide, ks, vs, table, base, new_len, mask))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,Q,ctx", [(2, 3, 2600), (5, 6, 1300), (32, 5, 700), (33, 5, 700), (7, 70, 1500)])
def test_unequal_contexts_of_many_rows(sv, cache, B, Q, ctx):  # noqa: F811
    """Split calls of one to 33 batch rows whose contexts differ, empty and invalid rows among them."""
    rng = np.random.default_rng([B, Q, ctx])
    c = list(case(rng, B, Q, 8, 2, 64, 16, ctx, cache, Q == 70, False))
    c[6] = c[6].copy()
    c[6][1], c[7][-1] = -5, 0                  # a row that is invalid, and one without tokens
    both(sv, c)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shape", [(2, 9, 8, 2, 256, 16, 300), (1, 61, 4, 1, 256, 64, 2500), (2, 20, 2, 1, 136, 24, 100),
                                   (1, 150, 2, 1, 192, 16, 40), (3, 40, 3, 3, 256, 1, 140), (1, 17, 1, 1, 248, 128, 0)])
def test_wide_heads(sv, shape, cache, tree):  # noqa: F811
    if cache == "e4m3" and shape[4] % 16:
        pytest.skip("rows of codes would not be 16-byte aligned")
    both(sv, case(np.random.default_rng([*shape, tree]), *shape, cache, tree, nhd=sum(shape) % 2 == 1))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Q", [3, 20, 80])
def test_a_bad_query_harms_its_own_row_only(sv, cache, Q):  # noqa: F811
    import torch
    rng = np.random.default_rng(Q)
    c = case(rng, 1, Q, 4, 1, 128, 16, 700, cache, False, False, ragged=False)
    want, want_l = run(sv, c)
    q = c[0].clone()
    q[0, 1, 2, 5] = float("nan")
    q[0, Q - 1, 0, 0] = float("inf")
    o, l = run(sv, (q, *c[1:]))
    bad = torch.zeros(o.shape[:3], dtype=torch.bool, device="cuda")
    bad[0, 1, 2] = bad[0, Q - 1, 0] = True
    assert torch.equal(o[~bad], want[~bad]) and torch.equal(l[~bad], want_l[~bad])
    assert not o[bad].isfinite().any()


@pytest.mark.parametrize("Q", [1, 8, 60])
def test_rows_that_share_pages(sv, Q):  # noqa: F811
    """A common prefix whose pages are in every row's table."""
    rng = np.random.default_rng(Q + 5)
    c = list(case(rng, 4, Q, 8, 2, 128, 16, 640, "bf16", False, False, ragged=False))
    c[5][1:, :40] = c[5][0, :40]               # 640 positions, 40 pages
    both(sv, c)


def test_rows_that_see_nothing_holes_and_invalid_rows(sv):  # noqa: F811
    import torch
    rng = np.random.default_rng(11)
    c = list(case(rng, 6, 5, 4, 2, 64, 8, 60, "bf16", False, False, ragged=False))
    c[6] = np.array([0, 30, -1, 60, 20, 44])
    c[7] = np.array([5, 5, 5, 6, 0, 3])      # row 2: negative base; 3: new_len over Q; 4: no token
    c[5][0] = -1                               # row 0: nothing but holes
    c[5][1, 1:3] = [10 ** 6, -7]               # row 1: two pages of holes
    c[5][5, 44 // 8] = -1                      # row 5: its own first tokens in a hole
    poison(c[1], c[2], None, None, c[5], np.clip(c[6], 0, 60), [5, 5, 0, 0, 0, 3], 8)
    both(sv, c)
    o, l = run(sv, c)
    assert (o[0] == 0).all() and torch.isneginf(l[0]).all()
    for b in (2, 3, 4):
        assert (o[b] == 5).all() and (l[b] == 6).all()
    assert (o[5, 3:] == 5).all() and (o[5, :3] != 5).any()


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Q", [6, 40, 200])
def test_bad_values_reach_only_who_sees_them(sv, cache, Q):  # noqa: F811
    """NaN and infinities in a drafted token's key or value leave the other branches alone."""
    import torch
    rng = np.random.default_rng([Q, 3])
    c = case(rng, 1, Q, 4, 1, 128, 16, 100, cache, True, False, ragged=False)
    q, k, v, ks, vs, table, base, new_len, mask = c
    clean, clean_l = run(sv, c)
    node = 3                                     # token 4
    pos = int(base[0]) + node + 1
    sees = np.array([False] + [bool((int(mask[0, i, 0]) >> node) & 1) for i in range(Q - 1)])
    assert sees.any() and not sees.all()
    page, row = int(table[0, pos // 16]), pos % 16
    for which, bads in ((v, ["nan", "inf"] if cache == "bf16" else ["nan", "scale"]), (k, ["nan"])):
        for bad in bads:
            keep = which[page, 0, row].clone(), None if vs is None else vs[page, 0, row].item()
            if bad == "scale":
                vs[page, 0, row] = float("inf")
            elif cache == "bf16":
                which[page, 0, row, 7:9] = float(bad)
            else:
                which[page, 0, row].view(torch.uint8)[7:9] = 0x7f
            o, l = run(sv, c)
            assert torch.equal(o[0, ~sees], clean[0, ~sees]) and torch.equal(l[0, ~sees], clean_l[0, ~sees])
            hit = o[0, sees].float()
            if which is k:
                assert hit.isnan().all()
            elif bad == "scale":
                assert (~hit.isfinite()).all()
            else:
                assert (~hit[..., 7:9].isfinite()).all() and (hit[..., 7:9].isinf().all() or bad == "nan")
                assert torch.equal(hit[..., 9:], clean[0, sees][..., 9:].float())
                assert torch.equal(l, clean_l)
            which[page, 0, row].copy_(keep[0]) if which.dtype == torch.bfloat16 else \
                which[page, 0, row].view(torch.uint8).copy_(keep[0].view(torch.uint8))
            if vs is not None:
                vs[page, 0, row] = keep[1]
    again, _ = run(sv, c)
    assert torch.equal(again, clean)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("Q,ctx", [(3, 0), (3, 90), (4, 700), (6, 100), (40, 0), (40, 128), (61, 700), (200, 20), (300, 600)])
def test_large_values_reach_only_who_sees_them(sv, cache, tree, Q, ctx):  # noqa: F811
    """Finite but huge drafted values and keys, and what a page holds behind the last token."""
    import torch
    rng = np.random.default_rng([Q, ctx, tree])
    c = case(rng, 2, Q, 4, 1, 128, 16, ctx, cache, tree, False, ragged=False)
    q, k, v, ks, vs, table, base, new_len, mask = c
    node = Q // 2 - 1                             # token node + 1
    last = int(base[0]) + Q                       # behind the last token
    for pos in (int(base[0]) + node + 1, last):
        page, row = (int(table[0, pos // 16]), pos % 16) if pos // 16 < table.shape[1] else (None, None)
        if page is None:
            continue
        if cache == "e4m3":
            vs[page, 0, row] = 1e30
            v[page, 0, row].view(torch.uint8).fill_(0x55)
        else:
            v[page, 0, row] = 1e30
        if pos == last:
            k[page, 0, row].view(torch.uint8).fill_(0x55) if cache == "e4m3" else k[page, 0, row].fill_(1e30)
            if cache == "e4m3":
                ks[page, 0, row] = 1e30
    sees = np.array([False] + [(bool((int(mask[0, i, node // 32]) >> (node % 32)) & 1) if tree else i >= node)
                               for i in range(Q - 1)])
    o, l = run(sv, c)
    scale = q.shape[3] ** -0.5
    vmax = None
    if cache == "e4m3":
        f = host(vs)
        vmax = f[np.isfinite(f) & (f < 1e29)].max()
        ks = ks.clone()
        ks[ks == 1e30] = float("nan")             # no query reaches it: out of the tolerance's sums
    else:
        k = k.clone()
        k[k > 1e29] = float("nan")
    def some(rows, vmax):
        check(o[:1], l[:1], q[:1], k, v, ks, vs, table[:1], base[:1], new_len[:1], None if mask is None else mask[:1],
              scale, 5.0, 6.0, rows, vmax)
    some(~sees, vmax)
    some(sees, None)
    check(o[1:], l[1:], q[1:], k, v, ks, vs, table[1:], base[1:], new_len[1:], None if mask is None else mask[1:],
          scale, 5.0, 6.0, None, vmax)


def test_a_long_context_in_pages_beyond_32_bits(sv):  # noqa: F811
    """A pool of more than 2^32 bytes, and one peaked score far back in a long context."""
    import torch
    P, H, ps, D, n = 140000, 1, 128, 128, 100000   # 4.6 GB of bf16 pages
    k = torch.zeros((P, H, ps, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((P, H, ps, D), dtype=torch.bfloat16, device="cuda")
    mp = (n + 6 + ps - 1) // ps
    table = torch.arange(P - 1, P - 1 - mp, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    at = 54321
    k[P - 1 - at // ps, 0, at % ps] = 1.0
    v[P - 1 - at // ps, 0, at % ps] = 3.0
    q = torch.ones((1, 6, 4, D), dtype=torch.bfloat16, device="cuda")
    o, l = sv.spec_paged_attention(q, k, v, table, ints([n]), scale=1.0, want_lse=True)
    w = np.exp(128.0) / (np.exp(128.0) + n)
    assert (o.float() == np.float32(3.0 * w)).all() and (l - 128).abs().max() < 1e-3
    del k, v
    torch.cuda.empty_cache()


def test_results_repeat_bit_for_bit_and_two_graphs_share_nothing(sv):  # noqa: F811
    """Two captured calls replayed in turn on two streams, each on its own inputs."""
    import torch
    rng = np.random.default_rng(17)
    a, b = (case(rng, 2, 6, 8, 2, 128, 16, 900, x, False, False) for x in ("bf16", "e4m3"))
    want = [run(sv, c) for c in (a, b)]
    torch.cuda.synchronize()
    graphs, outs, keep = [], [], []
    for c in (a, b):
        q, k, v, ks, vs, table, base, new_len, mask = c
        dev = [ints(table), ints(base), ints(new_len)]
        keep.append(dev)
        o = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full(q.shape[:3], 6.0, device="cuda")
        sv.spec_paged_attention(q, k, v, dev[0], dev[1], new_len=dev[2], k_scale=ks, v_scale=vs, out=o, out_lse=l)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.spec_paged_attention(q, k, v, dev[0], dev[1], new_len=dev[2], k_scale=ks, v_scale=vs, out=o, out_lse=l)
        graphs.append(g)
        outs.append((o, l))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for (o, l) in outs:
            o.fill_(5.0)
            l.fill_(6.0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for (o, l), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(l, wl)


def test_refusals(sv):  # noqa: F811
    import torch
    rng = np.random.default_rng(1)
    k, v, _, _ = make_cache(rng, 4, 2, 16, 64, "bf16", False)
    q = torch.zeros((1, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    t, b = ints([[0, 1]]), ints([4])
    f = sv.spec_paged_attention
    for bad, err in ((dict(q=q.float()), TypeError), (dict(q=q[:, :, :3]), ValueError), (dict(q=q[..., :32]), ValueError),
                     (dict(q=q[:, :0]), ValueError), (dict(base=b.long()), TypeError), (dict(base=ints([1, 2])), ValueError),
                     (dict(page_table=ints([[0], [1]])), ValueError), (dict(tree_mask=ints([[[0]]])), ValueError),
                     (dict(out=q[:, :2]), ValueError), (dict(out_lse=torch.zeros(1, 3, 4)), ValueError),
                     (dict(k_scale=torch.zeros(4, 2, 16, device="cuda")), ValueError),
                     (dict(workspace=torch.zeros(8, 2, device="cuda").t()), ValueError)):
        kw = dict(q=q, k_pages=k, v_pages=v, page_table=t, base=b)
        kw.update(bad)
        with pytest.raises(err):
            f(kw.pop("q"), kw.pop("k_pages"), kw.pop("v_pages"), kw.pop("page_table"), kw.pop("base"), **kw)
    for kw, code in ((dict(scale=float("nan")), sv.SV_ERR_INVALID_ARG), (dict(max_len=0), sv.SV_ERR_INVALID_ARG)):
        with pytest.raises(sv.SpecVerifyError) as e:
            f(q, k, v, t, b, **kw)
        assert e.value.status == code
    k8, v8, ks, vs = make_cache(rng, 4, 2, 16, 72, "e4m3", False)  # rows of 72 codes: not 16-byte aligned
    with pytest.raises(sv.SpecVerifyError) as e:
        f(torch.zeros((1, 3, 4, 72), dtype=torch.bfloat16, device="cuda"), k8, v8, t, b, k_scale=ks, v_scale=vs)
    assert e.value.status == sv.SV_ERR_UNSUPPORTED
    with pytest.raises(sv.SpecVerifyError) as e:  # a query tensor that starts off a 16-byte boundary
        f(torch.zeros(1 * 3 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(1, 3, 4, 64), k, v, t, b)
    assert e.value.status == sv.SV_ERR_UNSUPPORTED
    o, l = f(q[:0], k, v, t[:0], b[:0])
    assert o.shape == (0, 3, 4, 64) and l is None
