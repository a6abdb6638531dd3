"""Paged-cache writing, reading and compaction on the GPU against their plain float64 forms.

Tolerances: a rounding is off by at most half a step of its type, relative to the value
2^-8 for bf16, 2^-24 for fp32.  An e4m3 code must be a nearest value, up to the 2^-22 by
which fp32's x / scale may differ from the quotient in 64 bits (its own rounding and the
scale's, 2^-24 each, doubled); one test asks for the very code of the fp32 quotient.
"""
import numpy as np
import pytest

from oracle import paged
from speculative_decoding_verification_53_gb300 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_verification_53_gb300 import build
    build.build()
    import speculative_decoding_verification_53_gb300 as m
    m.lib()
    return m


def _torch_dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def make_cache(rng, P, H, ps, D, cache, nhd):
    """(k_pages, v_pages, k_scale, v_scale) on the GPU, with random contents."""
    import torch

    def pages():
        if cache == "bf16":
            x = torch.from_numpy(rng.normal(size=(P, ps, H, D) if nhd else (P, H, ps, D))).to(torch.bfloat16)
        else:
            x = torch.from_numpy(rng.integers(0, 127, (P, ps, H, D) if nhd else (P, H, ps, D), dtype=np.uint8))
            x = x.view(torch.float8_e4m3fn)
        x = x.cuda()
        return x.permute(0, 2, 1, 3) if nhd else x

    k, v = pages(), pages()
    if cache == "bf16":
        return k, v, None, None
    return k, v, *(torch.from_numpy(rng.uniform(0.001, 0.1, (P, H, ps)).astype(np.float32)).cuda() for _ in "kv")


def values(pages):
    import torch
    if pages.dtype == torch.float8_e4m3fn:
        return paged.e4m3_values()[pages.contiguous().view(torch.uint8).cpu().numpy()]
    return pages.double().cpu().numpy()


def host(t):
    return None if t is None else t.double().cpu().numpy()


def ints(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


CODES = None


def nearest_gap(y):
    """Distance from each y to the nearest finite code value."""
    global CODES
    if CODES is None:
        v = paged.e4m3_values()
        CODES = np.unique(v[np.isfinite(v)])
    i = np.clip(np.searchsorted(CODES, y), 1, len(CODES) - 1)
    return np.minimum(np.abs(y - CODES[i - 1]), np.abs(y - CODES[i]))


SHAPES = [  # B, N, H, D, page_size, max_pages
    (1, 1, 1, 128, 16, 1), (3, 6, 8, 128, 16, 4), (2, 133, 3, 64, 24, 8), (4, 5, 2, 96, 1, 12), (2, 9, 5, 256, 64, 1),
    (2, 17, 2, 7, 5, 6), (1, 70, 1, 1, 32, 3), (2, 8, 2, 200, 16, 2), (3, 4, 1, 80, 128, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("nhd", [False, True])
def test_append_and_read(sv, shape, cache, dtype, nhd):
    """Ragged rows, a hole, an invalid row, strided sources: every element of the cache and
    of the outputs, written or not."""
    import torch
    B, N, H, D, ps, mp = shape
    rng = np.random.default_rng([B, N, H, D, ps])
    P = B * mp + 2
    table = rng.permutation(P)[:B * mp].reshape(B, mp)
    new_len = rng.integers(0, N + 1, B)
    new_len[0] = N
    base = np.array([rng.integers(0, mp * ps - n + 1) for n in new_len])
    if B > 1:
        table[1, base[1] // ps] = -1 if B % 2 else P   # holes, either side
    if B > 2:
        base[2] = [-1, mp * ps - new_len[2] + 1][B % 2]  # the row stays untouched
    k, v, ks, vs = make_cache(rng, P, H, ps, D, cache, nhd)
    before = [values(k), values(v), host(ks), host(vs)]
    fused = rng.normal(size=(B, N, 2 * H + 1, D)) * np.exp(2 * rng.normal(size=(B, N, 2 * H + 1, 1)))
    fused[0, 0, :, 0] = 0
    fused = torch.from_numpy(fused).to(_torch_dtype(dtype)).cuda()
    key, value = fused[:, :, :H], fused[:, :, H:2 * H]
    sv.spec_kv_append(key, value, k, v, ints(table), ints(base), new_len=ints(new_len), k_scale=ks, v_scale=vs)
    for x, pages, scales, was, was_s in ((key, k, ks, before[0], before[2]), (value, v, vs, before[1], before[3])):
        want, want_s = paged.append(host(x), was, was_s, table, base, new_len)
        got = values(pages)
        written = paged.append(np.full_like(host(x), np.nan), was, None, table, base, new_len)[0]
        kept = ~np.isnan(written)
        assert np.array_equal(got[kept], was[kept])
        if cache == "bf16":
            assert np.array_equal(got, torch.from_numpy(want).to(torch.bfloat16).double().numpy())
        else:
            gap = np.abs(got - want)[~kept]
            y = want[~kept]
            assert (gap <= nearest_gap(y) + 2.0 ** -21 * np.abs(y)).all()
            s = host(scales)
            assert (np.abs(s - want_s) <= 2.0 ** -23 * want_s).all()
            untouched = kept.all(-1)
            assert np.array_equal(s[untouched], was_s[untouched])
    # read back what was written, into both types
    for out in ("bf16", "fp32"):
        o = [torch.full((B, N, H, D), 3.0, dtype=_torch_dtype(out), device="cuda") for _ in "kv"]
        a, b = sv.spec_kv_read(k, v, ints(table), ints(base), N, new_len=ints(new_len), k_scale=ks, v_scale=vs,
                               out_key=o[0], out_value=o[1])
        assert a is o[0] and b is o[1]
        for got, pages, scales in ((a, k, ks), (b, v, vs)):
            want = paged.read(values(pages), host(scales), table, base, new_len, N, np.full((B, N, H, D), 3.0))
            tol = (2.0 ** -8 + 2.0 ** -20 if out == "bf16" else 2.0 ** -23) * np.abs(want)
            if cache == "bf16":
                tol = 0
            assert (np.abs(host(got) - want) <= tol).all()


def test_append_special_values(sv):
    """Zeros, infinities, NaN, the largest and the smallest numbers of both source types."""
    import torch
    big, tiny = 3.3e38, 1e-40
    rows = np.array([[0] * 8, [np.inf, 1, -2, 0, 0, 0, 0, 0], [-np.inf, np.nan, 1, 3, 0, 0, 0, 0], [np.nan] * 8,
                     [big, -big, big / 2, 1, 0, 0, 0, 0], [tiny, -tiny, 0, 0, 0, 0, 0, 0], [448, 0.5, -447, 1e-3, 1, 2, 3, 4],
                     [np.inf, -np.inf, 0, 0, 0, 0, 0, 0]], np.float32)
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.from_numpy(rows).to(dtype).cuda().view(1, 8, 1, 8)
        k = torch.zeros((1, 1, 8, 8), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        v, ks, vs = k.clone(), torch.zeros((1, 1, 8), device="cuda"), torch.zeros((1, 1, 8), device="cuda")
        sv.spec_kv_append(x, x, k, v, ints([[0]]), ints([0]), k_scale=ks, v_scale=vs)
        y, s = paged.quantise(host(x)[0, :, 0])
        got, got_s = values(k)[0, 0], host(ks)[0, 0]
        assert (np.abs(got_s - s) <= 2.0 ** -23 * s).all()
        assert np.array_equal(np.isnan(got), np.isnan(y))
        fine = ~np.isnan(y)
        assert (np.abs(got - y)[fine] <= nearest_gap(y[fine]) + 2.0 ** -21 * np.abs(y[fine])).all()
        assert np.array_equal(values(k), values(v), equal_nan=True) and torch.equal(ks, vs)
        a, _ = sv.spec_kv_read(k, v, ints([[0]]), ints([0]), 8, k_scale=ks, v_scale=vs, dtype=torch.float32)
        a = host(a)[0, :, 0]
        assert np.isnan(a[3]).all() and (a[0] == 0).all() and a[6, 0] == 448


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D,amp", [(128, 1.0), (64, 1e30), (120, 1e-20), (7, 1e-30), (256, 1e-37)])
def test_codes_are_of_the_rounded_quotient(sv, dtype, D, amp):
    """Every code is e4m3 of x / scale rounded to fp32, with the scale that is stored: bf16 elements
    over their row's largest often lie next to the middle of two codes, where x * (1 / scale) takes
    the other one for 5 in 10000."""
    import torch
    rng = np.random.default_rng([D, int(amp > 1)])
    n = 3000
    x = rng.normal(size=(1, n, 1, D)) * np.exp(2 * rng.normal(size=(1, n, 1, 1))) * amp
    x = torch.from_numpy(np.clip(x, -3e38, 3e38)).to(_torch_dtype(dtype))
    x[0, 5] = 0
    x[0, 17, 0, D // 2] = float("inf")
    x[0, 18, 0, D // 2] = float("nan")
    k = torch.zeros((1, 1, n, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v, ks, vs = k.clone(), torch.zeros((1, 1, n), device="cuda"), torch.zeros((1, 1, n), device="cuda")
    sv.spec_kv_append(x.cuda(), x.cuda(), k, v, ints([[0]]), ints([0]), k_scale=ks, v_scale=vs)
    f = x[0, :, 0].float().numpy()
    a = np.where(np.isfinite(f), np.abs(f), 0).max(-1)
    s = np.maximum(a / np.float32(448), np.float32(2.0 ** -126))
    assert np.array_equal(ks[0, 0].cpu().numpy(), s) and torch.equal(ks, vs)
    y = np.clip(f / s[:, None], np.float32(-448), np.float32(448))
    assert y.dtype == np.float32
    want = torch.from_numpy(y).to(torch.float8_e4m3fn)
    for pages in (k, v):
        got = pages[0, 0].cpu()
        assert np.array_equal(got.float().numpy(), want.float().numpy(), equal_nan=True)


def test_read_new_outputs_are_zero_behind_the_tokens(sv):
    import torch
    rng = np.random.default_rng(4)
    k, v, _, _ = make_cache(rng, 4, 2, 8, 16, "bf16", False)
    a, b = sv.spec_kv_read(k, v, ints([[1, 3]]), ints([2]), 9, new_len=ints([5]))
    assert a.dtype == torch.bfloat16 and a.shape == (1, 9, 2, 16) and (a[0, 5:] == 0).all() and (b[0, 5:] == 0).all()
    assert torch.equal(a[0, :5], k[1, :, 2:7].transpose(0, 1))


def test_offsets_beyond_32_bits(sv):
    """A pool of more than 2^32 bytes: the last page is written and read where it lies."""
    import torch
    P, H, ps, D = 70000, 8, 64, 128   # 4.6 GB of codes
    k = torch.zeros((P, H, ps, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ks = torch.ones((P, H, ps), device="cuda")
    x = torch.randn((1, 3, H, D), device="cuda")
    t = ints([[P - 1, 12]])
    sv.spec_kv_append(x, x, k, k, t, ints([62]), k_scale=ks, v_scale=ks)
    a, _ = sv.spec_kv_read(k, k, t, ints([62]), 3, k_scale=ks, v_scale=ks, dtype=torch.float32)
    err = (a - x).abs().amax(-1) / x.abs().amax(-1)
    assert err.max() <= 2.0 ** -4  # half a step of the largest element
    raw = k.view(torch.uint8)
    assert raw[P - 1, :, 62:].any() and raw[12, :, 0].any() and not raw[13:P - 1].any() and not raw[:12].any()
    del k, raw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("width,dtype", [(128, "bf16"), (12, "u8"), (5, "u8"), (1, "fp32"), (64, "e4m3")])
@pytest.mark.parametrize("ps,nhd", [(16, False), (24, True), (1, False)])
def test_compact_paged_matches_the_plain_form(sv, width, dtype, ps, nhd):
    import torch
    B, N, D, H, n_buf = 12, 40, 6, 3, 5
    rng = np.random.default_rng([width, ps])
    mp = (N + 20 + ps - 1) // ps
    P = B * mp + 1
    table = rng.permutation(P)[:B * mp].reshape(B, mp).astype(np.int32)
    par = synth.random_parents(31, B, N, max_depth=D)
    path, count = synth.accepted_paths(31, par, D)
    base = rng.integers(0, mp * ps - N + 1, B).astype(np.int32)
    count[0] = 0                                   # an invalid verify row
    path[1, 1] = 0
    count[1] = max(count[1], 3)                    # path[1] < 1
    path[2, :2], count[2] = [1, 3], 3
    table[2, (base[2] + 3) // ps] = -1             # a hole among the sources
    base[3] = -4
    count[4] = D + 2
    base[5] = mp * ps - 2
    path[5, :2], count[5] = [0, 2], 3              # beyond the table
    shape = (P, ps, H, width) if nhd else (P, H, ps, width)
    es = {"bf16": 2, "u8": 1, "fp32": 4, "e4m3": 1}[dtype]
    raw = [rng.integers(0, 256, shape[:3] + (width * es,), dtype=np.uint8) for _ in range(n_buf)]
    td = {"bf16": torch.bfloat16, "u8": torch.uint8, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[dtype]
    dev = [torch.from_numpy(r).cuda().view(td) for r in raw]
    views = [t.permute(0, 2, 1, 3) if nhd else t for t in dev]
    sv.spec_kv_compact_paged(views, ints(table), ints(path), ints(count), ints(base))
    for t, r in zip(dev, raw):
        want = paged.compact(r.transpose(0, 2, 1, 3) if nhd else r, table, path, count, base)
        got = t.view(torch.uint8).cpu().numpy()
        assert (got == (want.transpose(0, 2, 1, 3) if nhd else want)).all()
    # the same through one stacked tensor
    one = torch.stack([torch.from_numpy(r).cuda() for r in raw]).view(td)
    sv.spec_kv_compact_paged(one.permute(0, 1, 3, 2, 4) if nhd else one, ints(table), ints(path), ints(count), ints(base))
    for t, o in zip(dev, one):
        assert torch.equal(t.view(torch.uint8), o.view(torch.uint8))


def test_compact_paged_without_base_and_at_its_limits(sv):
    """No base; 256 buffers; paths of 64 with gaps; the largest batch."""
    import torch
    rng = np.random.default_rng(8)
    B, ps, mp, W = 3, 16, 13, 16
    table = rng.permutation(B * mp).reshape(B, mp)
    path = np.full((B, 64), -1)
    count = np.array([65, 41, 1])
    for b, L in enumerate(count - 1):
        path[b, :L] = np.sort(rng.choice(200, L, replace=False))
    raw = rng.integers(0, 256, (256, B * mp, 1, ps, W), dtype=np.uint8)
    dev = torch.from_numpy(raw).cuda()
    sv.spec_kv_compact_paged(dev, ints(table), ints(path), ints(count))
    for t, r in zip(dev, raw):
        assert (t.cpu().numpy() == paged.compact(r, table, path, count, None)).all()
    B = 65535
    table = np.arange(2 * B).reshape(B, 2)
    path, count = np.tile([0, 2, 5], (B, 1)), np.full(B, 4)
    raw = rng.integers(0, 256, (2 * B, 1, 4, 4), dtype=np.uint8)
    dev = torch.from_numpy(raw).cuda()
    sv.spec_kv_compact_paged([dev], ints(table), ints(path), ints(count))
    flat = raw.reshape(B, 8, 4)
    flat[:, 1], flat[:, 2] = flat[:, 2].copy(), flat[:, 5]
    assert (dev.cpu().numpy().reshape(B, 8, 4) == flat).all()


def test_captured_append_and_read_replay_on_new_contents(sv):
    """One graph of append, read and compaction replays on what its tensors then hold."""
    import torch
    rng = np.random.default_rng(5)
    k, v, ks, vs = make_cache(rng, 6, 2, 4, 64, "e4m3", False)
    table, base, new_len = ints([[4, 0, 5]]), ints([1]), ints([6])
    x = torch.randn((1, 6, 2, 64), device="cuda")
    out = [torch.zeros((1, 6, 2, 64), device="cuda") for _ in "kv"]
    path, count, after = ints([[1, 3, -1]]), ints([3]), ints([2])

    def step():
        sv.spec_kv_append(x, x, k, v, table, base, new_len=new_len, k_scale=ks, v_scale=vs)
        for p in ([k, v], [ks[..., None], vs[..., None]]):
            sv.spec_kv_compact_paged(p, table, path, count, after)
        sv.spec_kv_read(k, v, table, base, 6, k_scale=ks, v_scale=vs, out_key=out[0], out_value=out[1])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    for seed in (1, 2):
        torch.manual_seed(seed)
        x.copy_(torch.randn_like(x))
        base.fill_(seed)
        after.fill_(seed + 1)
        g.replay()
        torch.cuda.synchronize()
        want = x[:, [0, 2, 4, 3, 4, 5]]  # rows base+1 and base+2 hold nodes 1 and 3 (tokens 2 and 4)
        assert ((out[0] - want).abs().amax(-1) <= 2.0 ** -4 * want.abs().amax(-1)).all()
        assert torch.equal(out[0], out[1])


def test_given_stream_is_the_one_used(sv):
    """Inputs written on a side stream are read there in order, without any other wait."""
    import torch
    s = torch.cuda.Stream()
    k = torch.zeros((1, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    x = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device="cuda")
    table, base = ints([[0]]), ints([3])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x.fill_(2.0)
    sv.spec_kv_append(x, x, k, v, table, base, stream=s)
    a, b = sv.spec_kv_read(k, v, table, base, 4, stream=s)
    s.synchronize()
    assert (a == 2).all() and (b == 2).all() and (k[0, 0, 3:7] == 2).all() and (k[0, 0, 7:] == 0).all()
