"""Refusals of the paged-cache entry points, and their plain forms' own pins (no GPU needed)."""
import ctypes
import os
import shutil

import numpy as np
import pytest

import oracle
from oracle import paged
from speculative_decoding_verification_53_gb300 import synth


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_verification_53_gb300 import build
    build.build()
    import speculative_decoding_verification_53_gb300 as sv
    return sv.lib()


def _cache(**kw):
    import speculative_decoding_verification_53_gb300 as sv
    d = dict(k_pages=256, v_pages=256, k_scale=None, v_scale=None, page_table=256, page_stride=8 * 16 * 256,
             head_stride=16 * 256, row_stride=256, dtype=sv.SV_CACHE_BF16, num_pages=4, page_size=16, max_pages=2,
             num_heads=8, head_dim=128)
    d.update(kw)
    return sv.PagedCache(**d)


BAD_CACHES = [dict(dtype=2), dict(num_pages=0), dict(page_size=0), dict(page_size=65537), dict(max_pages=0),
              dict(page_size=65536, max_pages=16385), dict(num_heads=0), dict(num_heads=1025), dict(head_dim=0),
              dict(head_dim=257, row_stride=1024), dict(row_stride=254), dict(row_stride=257), dict(page_stride=-2),
              dict(k_pages=None), dict(v_pages=None), dict(page_table=None), dict(k_pages=257),
              dict(dtype=1), dict(dtype=1, k_scale=256)]


@pytest.mark.parametrize("bad", range(len(BAD_CACHES)))
def test_bad_caches_are_refused(lib, bad):
    vp = ctypes.c_void_p(256)  # never dereferenced: the checks come first
    st = (ctypes.c_int64 * 3)(0, 0, 0)
    c = _cache(**BAD_CACHES[bad])
    assert lib.spec_kv_append(vp, vp, 1, st, c, vp, None, 1, 1, None) == 1
    assert lib.spec_kv_read(c, vp, None, 1, 1, vp, vp, 1, None) == 1


def test_append_and_read_arguments(lib):
    vp = ctypes.c_void_p(256)
    st = (ctypes.c_int64 * 3)(0, 0, 0)
    c = _cache()
    a, r = lib.spec_kv_append, lib.spec_kv_read
    assert a(vp, vp, 2, st, c, vp, None, 1, 1, None) == 1           # unknown dtype
    assert a(vp, vp, 1, st, None, vp, None, 1, 1, None) == 1        # no cache
    assert a(vp, vp, 1, st, c, vp, None, -1, 1, None) == 1
    assert a(vp, vp, 1, st, c, vp, None, 65536, 1, None) == 1
    assert a(vp, vp, 1, st, c, vp, None, 1, -1, None) == 1
    assert a(vp, vp, 1, st, c, vp, None, 1, 1 << 28, None) == 1     # N * heads beyond 2^31
    assert a(None, vp, 1, st, c, vp, None, 1, 1, None) == 1
    assert a(vp, vp, 1, None, c, vp, None, 1, 1, None) == 1
    assert a(vp, vp, 1, st, c, None, None, 1, 1, None) == 1
    assert a(ctypes.c_void_p(257), vp, 1, st, c, vp, None, 1, 1, None) == 1  # misaligned element
    assert a(None, None, 1, None, c, None, None, 0, 4, None) == 0   # an empty batch
    assert a(None, None, 1, None, c, None, None, 4, 0, None) == 0   # no tokens
    assert r(c, vp, None, 1, 1, vp, vp, 3, None) == 1
    assert r(c, None, None, 1, 1, vp, vp, 1, None) == 1
    assert r(c, vp, None, 1, 1, None, vp, 1, None) == 1
    assert r(c, vp, None, 1, 1, vp, ctypes.c_void_p(258), 0, None) == 1      # misaligned fp32
    assert r(c, None, None, 0, 1, None, None, 1, None) == 0
    assert r(_cache(page_table=None), None, None, 0, 1, None, None, 1, None) == 0


def test_compact_paged_arguments(lib):
    vp = ctypes.c_void_p(256)
    arr = (ctypes.c_void_p * 257)(*([256] * 257))
    f = lib.spec_kv_compact_paged

    def call(n=1, planes=1, row_stride=16, row_bytes=16, table=vp, pages=4, ps=16, mp=2, path=vp, count=vp, B=1, D=4,
             bufs=arr, page_stride=256, plane_stride=256):
        return f(bufs, n, page_stride, plane_stride, planes, row_stride, row_bytes, table, pages, ps, mp, path, count,
                 None, B, D, None)

    for bad in (dict(n=0), dict(n=257), dict(planes=0), dict(row_stride=8), dict(row_bytes=0), dict(table=None),
                dict(pages=0), dict(ps=0), dict(ps=65537), dict(mp=0), dict(ps=65536, mp=16385), dict(path=None),
                dict(count=None), dict(B=-1), dict(B=65536), dict(D=0), dict(D=65), dict(bufs=None),
                dict(page_stride=-1), dict(plane_stride=-16), dict(planes=1 << 30, n=256),
                dict(bufs=(ctypes.c_void_p * 2)(256, None), n=2)):
        assert call(**bad) == 1, bad
    assert call(B=0, table=None, path=None, count=None) == 0


def test_binding_checks_before_the_library():
    """Shapes, dtypes and devices are refused in Python, before any pointer is passed."""
    import torch
    import speculative_decoding_verification_53_gb300 as sv
    t = torch.zeros((1, 1, 1, 8))
    pages = torch.zeros((2, 1, 4, 8), dtype=torch.bfloat16)
    ints = torch.zeros((1, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv_append(t, t, pages, pages, ints, ints[0])
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv_read(pages, pages, ints, ints[0], 1)
    with pytest.raises(ValueError, match="empty"):
        sv.spec_kv_compact_paged([], ints, ints, ints[0])
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv_compact_paged([pages], ints, ints, ints[0])
    for bad, err in ((dict(k_pages=pages[0]), ValueError), (dict(v_pages=pages[:1]), ValueError),
                     (dict(k_pages=pages.float(), v_pages=pages.float()), TypeError),
                     (dict(k_scale=t), ValueError), (dict(page_table=ints[0]), ValueError),
                     (dict(page_table=ints.long()), TypeError), (dict(B=2), ValueError),
                     (dict(k_pages=pages.transpose(2, 3), v_pages=pages.transpose(2, 3)), ValueError),
                     (dict(k_pages=pages.to(torch.float8_e4m3fn), v_pages=pages.to(torch.float8_e4m3fn)), ValueError)):
        a = dict(k_pages=pages, v_pages=pages, page_table=ints, k_scale=None, v_scale=None, B=1)
        a.update(bad)
        with pytest.raises(err):
            sv._paged_cache(**a)


# ------------------------------------------------------------- pins of the plain forms

def test_e4m3_values_and_quantisation():
    v = paged.e4m3_values()
    assert v[0x7e] == 448 and v[0x01] == 2.0 ** -9 and v[0x38] == 1 and v[0xb8] == -1 and np.isnan(v[0x7f])
    torch = pytest.importorskip("torch")
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(got, v, equal_nan=True)
    y, s = paged.quantise(np.array([[0.5, -1.75, np.inf, np.nan, -np.inf], [0, 0, 0, 0, 0]]))
    assert s[0] == 1.75 / 448 and s[1] == 2.0 ** -126
    assert y[0, 1] == -448 and y[0, 0] == 128 and y[0, 2] == 448 and np.isnan(y[0, 3]) and y[0, 4] == -448
    assert (y[1] == 0).all()


def test_plain_append_then_read_is_the_identity():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(2, 5, 3, 8))
    pages, table = np.zeros((6, 3, 4, 8)), np.array([[5, 0, 2], [1, -1, 3]])
    base, new_len = np.array([3, 2]), np.array([5, 4])
    got, _ = paged.append(x, pages, None, table, base, new_len)
    back = paged.read(got, None, table, base, new_len, 5, np.full_like(x, 7.0))
    assert (back[0] == x[0]).all()
    assert (back[1, :2] == x[1, :2]).all() and (back[1, 2:4] == 0).all() and (back[1, 4] == 7).all()  # hole, rest
    assert (got[4] == 0).all()


def test_plain_attention_pins():
    """One visible position: its value, lse its score.  Equal keys: the mean.  A chain tree: the chain."""
    rng = np.random.default_rng(2)
    H, Hq, D, ps = 2, 4, 8, 4
    kp, vp = rng.normal(size=(4, H, ps, D)), rng.normal(size=(4, H, ps, D))
    table = np.array([[2, 0, 3]])
    q = rng.normal(size=(1, 3, Hq, D))
    z, zl = np.zeros((1, 3, Hq, D)), np.zeros((1, 3, Hq))
    o, l = paged.attention(q, kp, vp, None, None, table, [0], None, None, 0.5, z, zl)
    for h in range(Hq):
        assert np.allclose(o[0, 0, h], vp[2, h // 2, 0])
        assert np.isclose(l[0, 0, h], 0.5 * q[0, 0, h] @ kp[2, h // 2, 0])
    o, l = paged.attention(q, np.zeros_like(kp), vp, None, None, table, [5], None, None, 1.0, z, zl)
    flat = np.concatenate([vp[2], vp[0], vp[3]], 1)  # [H][12][D]
    assert np.allclose(o[0, 1, 3], flat[1, :7].mean(0)) and np.isclose(l[0, 1, 3], np.log(7))
    m = oracle.tree_mask(np.array([[-1, 0]]))["mask"]
    a = paged.attention(q, kp, vp, None, None, table, [5], None, m, 0.5, z, zl)
    c = paged.attention(q, kp, vp, None, None, table, [5], None, None, 0.5, z, zl)
    assert np.allclose(a[0], c[0]) and np.allclose(a[1], c[1])
    o, l = paged.attention(q, kp, vp, None, None, np.array([[-1, 9, -3]]), [5], None, None, 0.5, z + 1, zl)
    assert (o == 0).all() and np.isneginf(l).all()  # nothing but holes


def test_plain_compact_matches_the_dense_one():
    rng = np.random.default_rng(3)
    B, N, D, H, ps, W = 5, 20, 4, 2, 8, 6
    par = synth.random_parents(9, B, N, max_depth=D)
    path, count = synth.accepted_paths(9, par, D)
    base = rng.integers(0, 10, B).astype(np.int32)
    mp = 4
    table = rng.permutation(B * mp).reshape(B, mp).astype(np.int32)
    pages = rng.integers(0, 256, (B * mp, H, ps, W), dtype=np.uint8)
    dense = pages[table].transpose(0, 2, 1, 3, 4).reshape(B * H, mp * ps, W)
    want = oracle.kv_compact(np.ascontiguousarray(dense), np.repeat(path, H, axis=0), np.repeat(count, H),
                             np.repeat(base, H))
    got = paged.compact(pages, table, path, count, base)
    got = got[table].transpose(0, 2, 1, 3, 4).reshape(B * H, mp * ps, W)
    assert (got == want).all()


def test_attention_arguments(lib):
    vp = ctypes.c_void_p(256)
    st = (ctypes.c_int64 * 3)(0, 0, 0)
    f = lib.spec_paged_attention

    def call(q=vp, stride=st, Hq=8, cache=None, base=vp, scale=1.0, B=1, Q=6, max_len=32, out=vp, cache_kw={}):
        c = cache if cache is not None else _cache(**cache_kw)
        return f(q, stride, Hq, c, base, None, None, scale, B, Q, max_len, out, None, None, 0, None)

    for bad in BAD_CACHES:
        assert call(cache_kw=bad) == 1, bad
    for bad in (dict(q=None), dict(stride=None), dict(Hq=0), dict(Hq=7), dict(Hq=12), dict(base=None),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(B=-1), dict(B=65536), dict(Q=0),
                dict(Q=65537), dict(max_len=0), dict(out=None), dict(Hq=65544)):
        assert call(**bad) == 1, bad
    for odd in (dict(cache_kw=dict(head_dim=100)), dict(q=ctypes.c_void_p(264)), dict(out=ctypes.c_void_p(258)),
                dict(cache_kw=dict(row_stride=264)), dict(cache_kw=dict(k_pages=264)),
                dict(stride=(ctypes.c_int64 * 3)(4, 0, 0))):
        assert call(**odd) == 2, odd
    assert call(B=0, q=None, base=None, out=None) == 0
    size = lib.spec_paged_attention_workspace_size
    assert size(0, 1, 8, 8, 128, 0, 100) == 0 and size(1, 1, 8, 3, 128, 0, 100) == 0
    assert size(1, 1, 8, 8, 128, 5, 100) == 0 and size(1, 1, 8, 8, 128, 0, 0) == 0


def test_compaction_refuses_a_buffer_named_twice():
    import torch
    import speculative_decoding_verification_53_gb300 as sv
    t = torch.zeros(2, 1, 4, 8)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for bufs in ([t, t], t[None].expand(2, 2, 1, 4, 8)):
        with pytest.raises(ValueError, match="twice"):
            sv.spec_kv_compact_paged(bufs, i, i, i[0])
