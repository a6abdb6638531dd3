"""Rotary positions on the GPU against their plain form in 64 bits.

Tolerance of an element x' = a (x c - y s): the angle is within 2^-24 of a turn (1.6 times fp32's
half step of the fraction, 2^-25), which moves cosine and sine by at most 2 pi 2^-24; both are
rounded (2^-23 with CUDA's own error of about an ulp), multiplied by the amplitude (2^-24), and the two products and their sum round
by 2^-24 each.  So |error| <= (2 pi 2^-24 + 2^-22) a (|x| + |y|), plus half a step of the type, 2^-8 for
bf16 and 2^-24 for fp32, of the result.  Positions up to 2^24, frequencies up to one radian.
"""
import math

import numpy as np
import pytest

from oracle import context, paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_paged_kv import _torch_dtype, host, ints, make_cache, sv, values  # noqa: F401

pytestmark = pytest.mark.gpu

ANGLE = 2 * math.pi * 2.0 ** -24 + 2.0 ** -22


def reach(x, R, interleaved):
    """|x| + |y| of each element's pair, 0 for elements that are copied."""
    a = np.zeros_like(x)
    first = slice(0, 2 * R, 2) if interleaved else slice(0, R)
    second = slice(1, 2 * R, 2) if interleaved else slice(R, 2 * R)
    a[..., first] = a[..., second] = np.abs(x[..., first]) + np.abs(x[..., second])
    return a


def close(got, want, size, dtype, angle=ANGLE):
    half = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}[dtype]
    tol = angle * size + half * np.abs(want) + 1e-37
    worst = (np.abs(got - want) / tol).max() if got.size else 0
    assert worst <= 1, f"off by {worst:.3g} tolerances"


def make(rng, B, N, heads, D, dtype):
    """A slice of wider rows, as a fused projection's output."""
    import torch
    x = torch.from_numpy(rng.normal(size=(B, N, heads + 2, D)) * np.exp(rng.normal(size=(heads + 2, 1))))
    return x.to(_torch_dtype(dtype)).cuda()[:, :, 1:heads + 1]


SHAPES = [  # B, N, q heads, k heads, D, R, dtype, interleaved, tree, far
    (1, 1, 32, 8, 128, 64, "bf16", False, False, 130000), (2, 5, 4, 2, 64, 32, "bf16", True, False, 100),
    (3, 61, 8, 1, 128, 64, "fp32", False, True, 9000), (2, 7, 3, 3, 96, 48, "bf16", False, False, 50),
    (2, 9, 5, 1, 96, 10, "fp32", False, True, 1000000), (1, 300, 6, 2, 256, 128, "bf16", True, False, 16000000),
    (2, 3, 1, 1, 33, 7, "bf16", False, False, 10), (2, 3, 1, 2, 33, 16, "fp32", True, False, 10),
    (2, 4, 2, 1, 64, 0, "bf16", False, False, 10), (1, 2, 1, 1, 2, 1, "bf16", True, False, 10),
    (1, 1, 1, 1, 1, 0, "fp32", False, False, 10), (5, 1000, 2, 1, 64, 16, "bf16", False, False, 70000),
    (9, 700, 7, 1, 128, 32, "fp32", True, False, 5000), (2, 4, 2, 1, 256, 124, "bf16", False, False, 3000),
]


@pytest.mark.parametrize("shape", SHAPES)
def test_matches_the_plain_form(sv, shape):  # noqa: F811
    import torch
    B, N, Hq, Hk, D, R, dtype, interleaved, tree, far = shape
    rng = np.random.default_rng([B, N, D, R])
    q, k = make(rng, B, N, Hq, D, dtype), make(rng, B, N, Hk, D, dtype)
    freq = 10000.0 ** (-np.arange(R) / max(R, 1))
    base = rng.integers(0, far + 1, B)
    depth = rng.integers(1, 9, (B, N - 1)) if tree else None
    f, t_base = torch.from_numpy(freq).cuda(), ints(base)
    pos = context.positions(base, N, depth)
    kw = dict(interleaved=interleaved, tree_depth=None if depth is None else ints(depth))
    for inverse, amplitude in ((False, 1.0), (True, 1.25)):
        out, out_k = sv.spec_rotary(q, f, t_base, key=k, inverse=inverse, amplitude=amplitude, **kw)
        for x, got in ((q, out), (k, out_k)):
            want = context.rotary(host(x), freq, pos, interleaved, inverse, amplitude)
            close(host(got), want, amplitude * reach(host(x), R, interleaved), dtype)
            assert torch.equal(got[..., 2 * R:], x[..., 2 * R:])
    # queries alone, and in place on the slices of the wider rows
    alone, none = sv.spec_rotary(q, f, t_base, **kw)
    assert none is None
    first, first_k = sv.spec_rotary(q, f, t_base, key=k, **kw)
    assert torch.equal(alone, first)
    q2, k2 = q.clone(), k.clone()
    wide = torch.zeros((B, N, Hq + Hk, D), dtype=q.dtype, device="cuda")
    wide[:, :, :Hq], wide[:, :, Hq:] = q2, k2
    a, b = sv.spec_rotary(wide[:, :, :Hq], f, t_base, key=wide[:, :, Hq:], out=wide[:, :, :Hq], out_key=wide[:, :, Hq:], **kw)
    assert a.data_ptr() == wide.data_ptr() and torch.equal(wide[:, :, :Hq], first) and torch.equal(wide[:, :, Hq:], first_k)


@pytest.mark.parametrize("B,N,Hq,Hk,D,R,interleaved", [
    (5, 4001, 3, 1, 64, 32, False), (7, 2801, 2, 1, 128, 20, True), (5, 4001, 1, 2, 256, 128, False),
    (19999, 1, 9, 0, 96, 16, False), (3, 7000, 32, 0, 40, 8, True)])
def test_many_tokens_of_few_rows(sv, B, N, Hq, Hk, D, R, interleaved):  # noqa: F811
    """A warp takes several tokens (but for the last two shapes, whose rows are too many), across batch rows, some of which are
    not written; alike in place."""
    import torch
    rng = np.random.default_rng([B, N, D])
    q, k = make(rng, B, N, Hq, D, "bf16"), make(rng, B, N, Hk, D, "bf16") if Hk else None
    freq = 10000.0 ** (-np.arange(R) / R)
    base, new = rng.integers(0, 100000, B), rng.integers(0, N + 1, B)
    base[1], new[0], new[2] = -1, N, 0
    f, kw = torch.from_numpy(freq).cuda(), dict(interleaved=interleaved, new_len=ints(new))
    live = (np.arange(N) < new[:, None]) & (base >= 0)[:, None]
    pos = context.positions(base, N)
    outs = [torch.full(x.shape, 9.0, dtype=x.dtype, device="cuda") if x is not None else None for x in (q, k)]
    sv.spec_rotary(q, f, ints(base), key=k, out=outs[0], out_key=outs[1], **kw)
    for x, out in zip((q, k), outs):
        if x is None:
            continue
        got, want = host(out), context.rotary(host(x), freq, pos, interleaved)
        assert (got[~live] == 9).all()
        close(got[live], want[live], reach(host(x), R, interleaved)[live], "bf16")
        assert torch.equal(out[..., 2 * R:][torch.from_numpy(live).cuda()], x[..., 2 * R:][torch.from_numpy(live).cuda()])
    q2 = q.clone()
    sv.spec_rotary(q2, f, ints(base), key=k, out=q2, out_key=k, **kw)
    keep = torch.from_numpy(live).cuda()[..., None, None]
    assert torch.equal(q2, torch.where(keep, outs[0], q))


def test_turning_back(sv):  # noqa: F811
    """The inverse is the transpose: <turn(x), y> = <x, turn back(y)> for every x and y, as a gradient needs."""
    import torch
    rng = np.random.default_rng(5)
    freq = torch.from_numpy(10000.0 ** (-np.arange(32) / 32)).cuda()
    x, y = make(rng, 2, 9, 3, 64, "fp32"), make(rng, 2, 9, 3, 64, "fp32")
    base = ints([7, 40000])
    a = host(sv.spec_rotary(x, freq, base, amplitude=0.7)[0]) * host(y)
    b = host(x) * host(sv.spec_rotary(y, freq, base, amplitude=0.7, inverse=True)[0])
    # every element of a turned row is off by (ANGLE + 2^-24) (|x| + |y|) at most, times the other's
    tol = (ANGLE + 2.0 ** -24) * (reach(host(x), 32, False) * np.abs(host(y)) + reach(host(y), 32, False) * np.abs(host(x))).sum()
    assert abs(a.sum() - b.sum()) <= tol


def test_far_positions(sv):  # noqa: F811
    """Up to 2^30 the angle is within 2^-19 of a turn, so cosine and sine within 2 pi 2^-19."""
    import torch
    freq = np.array([1.0, 0.7391, 0.1, 1e-3, 1e-6, 0.0])
    x = np.zeros((4, 1, 1, 12))
    x[..., :6] = 1
    base = np.array([2 ** 24 - 1, 2 ** 24 + 1, 2 ** 30 - 3, 2 ** 30])
    q = torch.from_numpy(x.astype(np.float32)).cuda()
    got = host(sv.spec_rotary(q, torch.from_numpy(freq).cuda(), ints(base))[0])
    want = context.rotary(x, freq, context.positions(base, 1))
    close(got[:1], want[:1], reach(x[:1], 6, False), "fp32")
    close(got, want, reach(x, 6, False), "fp32", angle=2 * math.pi * 2.0 ** -19)


def test_rows_left_untouched(sv):  # noqa: F811
    import torch
    rng = np.random.default_rng(3)
    q = make(rng, 6, 4, 2, 64, "bf16")
    base, new = np.array([5, -1, 2 ** 30 + 1, 6, 7, 8]), np.array([4, 4, 4, 5, -1, 2])
    freq = 100.0 ** (-np.arange(16) / 16)
    out = torch.full(q.shape, 9.0, dtype=q.dtype, device="cuda")
    sv.spec_rotary(q, torch.from_numpy(freq).cuda(), ints(base), new_len=ints(new), out=out)
    want = np.full(q.shape, 9.0)
    turned = context.rotary(host(q), freq, context.positions(base, 4))
    want[0], want[5, :2] = turned[0], turned[5, :2]
    got = host(out)
    assert (got[1:5] == 9).all() and (got[5, 2:] == 9).all()
    close(got[[0, 5]], want[[0, 5]], reach(host(q), 16, False)[[0, 5]], "bf16")


def test_numbers_that_are_not_finite(sv):  # noqa: F811
    """They stay in their pair, and elements behind the turned ones are copied bit for bit."""
    import torch
    q = torch.ones((1, 2, 3, 64), device="cuda")
    q[0, 0, 1, 3], q[0, 1, 2, 20], q[0, 0, 0, 40], q[0, 0, 0, 41] = math.inf, math.nan, math.nan, -0.0
    out = sv.spec_rotary(q, torch.linspace(0.1, 1, 16, dtype=torch.float64, device="cuda"), ints([3]))[0]
    bad = ~torch.isfinite(out)
    want = torch.zeros_like(bad)
    want[0, 0, 1, [3, 19]] = want[0, 1, 2, [4, 20]] = want[0, 0, 0, 40] = True
    assert torch.equal(bad, want)
    assert torch.equal(out[..., 32:].view(torch.int32), q[..., 32:].view(torch.int32))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,N,Hq,H,D,R,ps,dtype,interleaved,tree,nhd", [
    (1, 1, 4, 2, 64, 32, 16, "bf16", False, False, False), (3, 61, 8, 2, 128, 64, 64, "bf16", False, True, False),
    (4, 30, 3, 1, 96, 24, 8, "fp32", True, False, True), (2, 6, 0, 3, 128, 32, 16, "bf16", False, False, False),
    (2, 11, 5, 2, 36, 9, 5, "fp32", False, True, True), (2, 700, 7, 1, 64, 32, 24, "bf16", False, False, True),
    (2, 9, 2, 2, 256, 128, 1, "fp32", False, False, False)])
def test_append(sv, cache, B, N, Hq, H, D, R, ps, dtype, interleaved, tree, nhd):  # noqa: F811
    """Turned keys in the cache: those that spec_kv_append would write of the turned keys, in fp32; pages
    and rows of tokens that are not real, in holes or untouched rows stay as they are."""
    import torch
    rng = np.random.default_rng([N, D])
    q = make(rng, B, N, Hq, D, dtype) if Hq else None
    kv = make(rng, B, N, 2 * H, D, dtype)
    key, value = kv[:, :, :H], kv[:, :, H:]
    base = rng.integers(0, 200, B)
    new = rng.integers(0, N + 1, B)
    new[0] = N
    if B > 2:
        base[2] = -4
    width = (200 + N + ps - 1) // ps
    P = B * width + 2
    table = rng.permutation(P)[:B * width].reshape(B, width)
    table[-1, (base[-1] + max(int(new[-1]) - 1, 0)) // ps] = -1  # a hole
    freq = 10000.0 ** (-np.arange(R) / R)
    depth = rng.integers(1, 6, (B, N - 1)) if tree else None
    kp, vp, ks, vs = make_cache(rng, P, H, ps, D, cache, nhd)
    before = [t.clone() if t is not None else None for t in (kp, vp, ks, vs)]
    args = dict(tree_depth=None if depth is None else ints(depth), interleaved=interleaved, amplitude=1.5)
    f = torch.from_numpy(freq).cuda()
    out = sv.spec_rotary_append(q, key, value, f, kp, vp, ints(table), ints(base), new_len=ints(new), k_scale=ks,
                                v_scale=vs, **args)
    pos = context.positions(base, N, depth)
    real = np.zeros((B, N), bool)
    for b in range(B):
        real[b, :new[b]] = base[b] >= 0
    if Hq:
        want = context.rotary(host(q), freq, pos, interleaved, False, 1.5)
        close(host(out)[real], want[real], 1.5 * reach(host(q), R, interleaved)[real], dtype)
    else:
        assert out is None
    # the same through fp32 keys and the plain append
    turned = torch.zeros(key.shape, device="cuda")
    sv.spec_rotary(key.float(), f, ints(base), out=turned, **args)
    held = np.zeros((P, ps), bool)
    for b in range(B):
        for i in range(N):
            p, r = paged.place(table, b, int(base[b]) + i, P, ps) if real[b, i] else (-1, 0)
            if p >= 0:
                held[p, r] = True
    by = before
    sv.spec_kv_append(turned, torch.zeros_like(turned).copy_(value), by[0], by[1], ints(table), ints(base), new_len=ints(new),
                      k_scale=by[2], v_scale=by[3])
    for got, exp in zip((kp, vp, ks, vs), by):
        if got is not None:
            got, exp = (x.contiguous().view(torch.uint8 if x.dtype == torch.float8_e4m3fn else x.dtype) for x in (got, exp))
            assert torch.equal(got, exp)
    if cache == "bf16":  # and against the formula itself
        want = context.rotary(host(key), freq, pos, interleaved, False, 1.5)
        got, size = values(kp), 1.5 * reach(host(key), R, interleaved)
        for b in range(B):
            for i in np.nonzero(real[b])[0]:
                p, r = paged.place(table, b, int(base[b]) + int(i), P, ps)
                if p >= 0:
                    close(got[p, :, r], want[b, i], size[b, i], "bf16")


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("shape", [
    (5, 4001, 3, 1, 64, 32, 16, "bf16", False, True, True), (7, 2801, 1, 1, 128, 20, 24, "bf16", True, False, False),
    (3, 7000, 0, 1, 256, 128, 32, "bf16", False, False, True), (9, 2300, 5, 2, 40, 8, 8, "bf16", False, False, False)])
def test_append_many_tokens_of_few_rows(sv, cache, shape):  # noqa: F811
    """A warp takes several tokens; the last shape's rows are as many as one does not."""
    test_append(sv, cache, *shape)


def test_captured(sv):  # noqa: F811
    """One graph of both entries on a stream of its own, replayed after inputs and positions changed."""
    import torch
    rng = np.random.default_rng(1)
    B, N, Hq, H, D, ps = 3, 25, 4, 2, 64, 16
    x = make(rng, B, N, Hq + 2 * H, D, "bf16").contiguous()
    freq = 10000.0 ** (-np.arange(32) / 32)
    f = torch.from_numpy(freq).cuda()
    parent = synth.random_parents(4, B, N - 1, "bfs", max_depth=5)
    base, t_parent = ints([0, 17, 60]), ints(parent)
    table = ints(rng.permutation(B * 6).reshape(B, 6))
    kp, vp, _, _ = make_cache(rng, B * 6, H, ps, D, "bf16", False)
    out = torch.zeros((B, N, Hq, D), dtype=torch.bfloat16, device="cuda")

    def step():
        _, depth, _ = sv.spec_tree_mask(t_parent)
        sv.spec_rotary_append(x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:], f, kp, vp, table, base, tree_depth=depth, out=out)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(make(rng, B, N, Hq + 2 * H, D, "bf16"))
    base.copy_(ints([5, 40, 0]))
    parent = synth.random_parents(9, B, N - 1, "bfs", max_depth=5)
    t_parent.copy_(ints(parent))
    graph.replay()
    depth = np.zeros((B, N - 1), np.int64)
    for b in range(B):
        for i in range(N - 1):
            depth[b, i] = 1 + (depth[b, parent[b, i]] if parent[b, i] >= 0 else 0)
    pos = context.positions([5, 40, 0], N, depth)
    q = host(x[:, :, :Hq])
    close(host(out), context.rotary(q, freq, pos), reach(q, 32, False), "bf16")
    k, got, t = host(x[:, :, Hq:Hq + H]), values(kp), table.cpu().numpy()
    want, size = context.rotary(k, freq, pos), reach(k, 32, False)
    for b, s in enumerate([5, 40, 0]):
        for i in range(N):
            close(got[t[b, (s + i) // ps], :, (s + i) % ps], want[b, i], size[b, i], "bf16")


def test_refusals(sv):  # noqa: F811
    import torch
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    f = torch.ones(32, dtype=torch.float64, device="cuda")
    base = ints([0, 0])
    for bad in (dict(freq=torch.ones(33, dtype=torch.float64, device="cuda")), dict(freq=f[None]), dict(base=ints([0])),
                dict(tree_depth=ints(np.zeros((2, 3)))), dict(key=q[:, :2]), dict(key=q.float()), dict(out=q[:1]),
                dict(out=q.float()), dict(out_key=q), dict(q=q[0]), dict(q=q.transpose(2, 3)), dict(freq=f.cpu()),
                dict(key=q, out_key=q[..., :32])):
        with pytest.raises(ValueError):
            sv.spec_rotary(**{**dict(q=q, freq=f, base=base), **bad})
    for bad in (dict(freq=f.float()), dict(q=q.half()), dict(base=base.long())):
        with pytest.raises(TypeError):
            sv.spec_rotary(**{**dict(q=q, freq=f, base=base), **bad})
    with pytest.raises(sv.SpecVerifyError):
        sv.spec_rotary(q, f, base, amplitude=math.nan)
    pages = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, key=q[:, :, :2], value=q[:, :, 2:], freq=f, k_pages=pages, v_pages=pages.clone(), page_table=ints([[0], [1]]), base=base)
    sv.spec_rotary_append(**good)
    for bad in (dict(q=q[:, :2]), dict(q=q.float()), dict(key=q), dict(value=q[:, :, 1:2]), dict(q=None, out=q),
                dict(page_table=ints([[0]])), dict(k_scale=torch.ones((4, 2, 16), device="cuda"))):
        with pytest.raises(ValueError):
            sv.spec_rotary_append(**{**good, **bad})
