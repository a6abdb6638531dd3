"""Refusals of the long-context operators, and pins of their plain forms (no GPU needed)."""
import ctypes
import math
import os
import shutil

import numpy as np
import pytest

from oracle import context, paged
from test_paged_args import BAD_CACHES, _cache


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from speculative_decoding_verification_53_gb300 import build
    build.build()
    import speculative_decoding_verification_53_gb300 as sv
    return sv.lib()


VP = ctypes.c_void_p(256)  # never dereferenced: the checks come first
ODD = ctypes.c_void_p(257)
ST = (ctypes.c_int64 * 3)(0, 0, 0)


def test_page_resize_arguments(lib):
    def call(table=VP, pages=VP, length=VP, free=VP, count=VP, P=4, ps=16, mp=2, base=None, slots=None, ok=VP, B=1, N=0):
        return lib.spec_page_resize(table, pages, length, free, count, P, ps, mp, base, slots, ok, B, N, None)

    for bad in (dict(table=None), dict(pages=None), dict(length=None), dict(free=None), dict(count=None), dict(ok=None),
                dict(P=-1), dict(P=(1 << 30) + 1), dict(ps=0), dict(ps=65537), dict(mp=0), dict(ps=65536, mp=16385),
                dict(B=-1), dict(B=16385), dict(N=-1), dict(N=(1 << 30) + 1), dict(base=VP), dict(slots=VP),
                dict(base=VP, slots=VP, B=1024, N=1 << 30)):
        assert call(**bad) == 1, bad
    assert call(B=0, table=None, ok=None) == 0


def _rot(freq=256, depth=None, amplitude=1.0, n=32):
    import speculative_decoding_verification_53_gb300 as sv
    return sv.Rotary(freq, depth, amplitude, n, 0, 0)


def test_rotary_arguments(lib):
    def call(q=VP, qs=ST, Hq=4, k=VP, ks=ST, Hk=2, dt=1, rot=None, base=VP, B=1, N=3, D=64, oq=VP, oqs=ST, ok=VP, oks=ST):
        return lib.spec_rotary(q, qs, Hq, k, ks, Hk, dt, rot or _rot(), base, None, B, N, D, oq, oqs, ok, oks, None)

    for bad in (dict(q=None), dict(qs=None), dict(Hq=0), dict(Hq=65537), dict(k=None), dict(ks=None), dict(Hk=-1),
                dict(dt=2), dict(rot=_rot(freq=None)), dict(rot=_rot(n=33)), dict(rot=_rot(n=-1)),
                dict(rot=_rot(amplitude=math.inf)), dict(rot=_rot(amplitude=math.nan)), dict(base=None), dict(B=-1),
                dict(B=65536), dict(N=-1), dict(N=(1 << 20) + 1), dict(B=4096, N=1 << 20), dict(D=0), dict(D=257),
                dict(oq=None), dict(oqs=None), dict(ok=None), dict(oks=None), dict(q=ODD), dict(ok=ODD)):
        assert call(**bad) == 1, bad
    assert lib.spec_rotary(VP, ST, 4, None, None, 0, 1, None, VP, None, 1, 3, 64, VP, ST, None, None, None) == 1
    assert call(B=0, q=None) == 0 and call(N=0, q=None) == 0


@pytest.mark.parametrize("bad", range(len(BAD_CACHES)))
def test_bad_caches_are_refused(lib, bad):
    c = _cache(**BAD_CACHES[bad])
    assert lib.spec_rotary_append(VP, ST, 8, VP, VP, ST, 1, _rot(), c, VP, None, 1, 1, VP, ST, None) == 1
    if BAD_CACHES[bad] != dict(v_pages=None):
        assert lib.spec_block_summary(c, VP, None, 0, 1, 1, VP, None) == 1
    assert lib.spec_sparse_attention(VP, ST, 8, c, VP, None, None, VP, 4, 0, 0.1, 1, 1, VP, None, VP, 1 << 40, None) == 1


def test_rotary_append_arguments(lib):
    c = _cache()

    def call(q=VP, qs=ST, Hq=8, k=VP, v=VP, ks=ST, dt=1, rot=None, base=VP, B=1, N=3, oq=VP, oqs=ST):
        return lib.spec_rotary_append(q, qs, Hq, k, v, ks, dt, rot or _rot(), c, base, None, B, N, oq, oqs, None)

    for bad in (dict(q=None), dict(qs=None), dict(Hq=-1), dict(k=None), dict(v=None), dict(ks=None), dict(dt=3),
                dict(rot=_rot(n=65)), dict(base=None), dict(B=65536), dict(N=-1), dict(oq=None), dict(oqs=None),
                dict(v=ODD)):
        assert call(**bad) == 1, bad
    assert call(B=0, k=None) == 0


def test_summary_and_select_arguments(lib):
    c = _cache()
    s = lib.spec_block_summary
    assert s(c, VP, None, 2, 1, 1, VP, None) == 1
    assert s(c, VP, None, 0, -1, 1, VP, None) == 1
    assert s(c, VP, None, 0, 1, -1, VP, None) == 1
    assert s(c, None, None, 0, 1, 1, VP, None) == 1
    assert s(c, VP, None, 0, 1, 1, None, None) == 1
    assert s(c, VP, None, 0, 1, 1, ODD, None) == 1
    assert s(c, VP, None, 0, 1, 1, ctypes.c_void_p(258), None) == 2  # 16 bytes at a time
    assert s(c, None, None, 0, 0, 1, None, None) == 0

    def call(q=VP, qs=ST, Hq=8, m=VP, kind=0, table=VP, P=4, ps=16, mp=8, H=4, D=64, base=VP, shared=0, top=4, sink=1,
             recent=1, B=1, Q=2, out=VP, ws=VP, size=1 << 40):
        return lib.spec_block_select(q, qs, Hq, m, kind, table, P, ps, mp, H, D, base, None, shared, top, sink, recent, B, Q,
                                     out, ws, size, None)

    need = lib.spec_block_select_workspace_size(1, 2, 8, 4, 8, 0)
    assert need > 0
    for bad in (dict(q=None), dict(qs=None), dict(Hq=9), dict(Hq=0), dict(m=None), dict(kind=2), dict(table=None),
                dict(P=0), dict(ps=0), dict(mp=0), dict(mp=65537), dict(H=0), dict(D=0), dict(D=264), dict(base=None),
                dict(top=0), dict(top=4097), dict(sink=-1), dict(recent=-1), dict(sink=3, recent=2), dict(B=-1),
                dict(B=65536), dict(Q=0), dict(Q=65537), dict(out=None), dict(ws=None), dict(size=need - 1),
                dict(ws=ctypes.c_void_p(264)), dict(ps=65536, mp=16385)):
        assert call(**bad) == 1, bad
    assert call(D=60) == 2 and call(q=ctypes.c_void_p(264)) == 2
    assert call(qs=(ctypes.c_int64 * 3)(0, 4, 0)) == 2
    assert call(B=0, q=None) == 0


def test_sparse_attention_arguments(lib):
    c = _cache()

    def call(q=VP, qs=ST, Hq=8, cache=c, base=VP, blocks=VP, n=4, shared=0, scale=0.1, B=1, Q=2, out=VP, ws=VP, size=1 << 40):
        return lib.spec_sparse_attention(q, qs, Hq, cache, base, None, None, blocks, n, shared, scale, B, Q, out, None, ws,
                                         size, None)

    for bad in (dict(q=None), dict(qs=None), dict(Hq=9), dict(base=None), dict(blocks=None), dict(n=-1), dict(n=4097),
                dict(scale=math.nan), dict(B=-1), dict(B=65536), dict(Q=0), dict(out=None), dict(ws=None)):
        assert call(**bad) == 1, bad
    assert call(q=ctypes.c_void_p(264)) == 2
    assert call(cache=_cache(head_dim=60)) == 2
    assert call(B=0, q=None) == 0
    assert lib.spec_sparse_attention_workspace_size(0, 2, 8, 4, 64, 0, 16, 4, 0) == 0
    assert lib.spec_sparse_attention_workspace_size(1, 2, 8, 3, 64, 0, 16, 4, 0) == 0


def test_page_resize_by_hand():
    table = np.array([[7, 3, 5, -1], [1, -1, -1, -1], [0, 2, -1, -1]])
    t, p, s, n, ok, slots = context.page_resize(table, [3, 1, 2], [4, 9, 20], [6, 4, -1, -1, -1, -1, -1, -1], 2, 4,
                                                base=[3, 7, 0], N=3)
    # row 0 gives back 3 then 5; rows 1 and 2 lack two and three pages of the four
    assert s[:4].tolist() == [6, 4, 3, 5] and n == 2
    assert t.tolist() == [[7, -1, -1, -1], [1, 5, 3, -1], [0, 2, -1, -1]]
    assert p.tolist() == [1, 3, 2] and ok.tolist() == [1, 1, 0]
    assert slots.tolist() == [[31, -1, -1], [23, 12, -1], [-1, -1, -1]]


def test_rotary_frequencies():
    import torch
    import speculative_decoding_verification_53_gb300 as sv
    f = sv.rotary_frequencies(8, 100.0)
    assert torch.allclose(f, torch.tensor([1, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    assert torch.equal(sv.rotary_frequencies(8, 100.0, scaling="linear", factor=4.0), f / 4)
    base = sv.rotary_frequencies(8, 100.0, scaling="base", factor=4.0)
    assert base[0] == 1 and abs(float(base[-1] / f[-1]) * 4 - 1) < 1e-14
    parts = sv.rotary_frequencies(64, 10000.0, scaling="parts", factor=8.0, original_len=4096, low=1, high=32)
    whole = sv.rotary_frequencies(64, 10000.0)
    turns = 4096 * whole / (2 * math.pi)
    assert torch.equal(parts[turns >= 32], whole[turns >= 32])
    assert torch.allclose(parts[turns <= 1], whole[turns <= 1] / 8, rtol=1e-15)
    between = (turns > 1) & (turns < 32)
    assert between.any() and ((parts < whole) & (parts > whole / 8))[between].all()
    for bad in (dict(dim=7), dict(dim=0), dict(dim=8, factor=0.0), dict(dim=8, scaling="other"),
                dict(dim=8, low=2.0, high=2.0), dict(dim=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            sv.rotary_frequencies(**bad)


def test_plain_forms_by_hand():
    x = np.array([[[[1.0, 2.0, 3.0, 4.0, 9.0]]]])
    quarter = np.array([math.pi / 2, 0.0])
    assert np.allclose(context.rotary(x, quarter, np.array([[1]]))[0, 0, 0], [-3, 2, 1, 4, 9])
    assert np.allclose(context.rotary(x, quarter, np.array([[1]]), interleaved=True)[0, 0, 0], [-2, 1, 3, 4, 9])
    assert np.allclose(context.rotary(x, quarter, np.array([[1]]), inverse=True, amplitude=2)[0, 0, 0], [6, 4, -2, 8, 9])
    assert context.positions([5], 3, [[1, 2]]).tolist() == [[5, 6, 7]]
    # scores: one head at a time, the largest of the group's; ties to the lower block; holes last
    q = np.array([[[[1.0, -1.0], [0.0, 0.0]]]])
    m = np.zeros((5, 1, 2))
    m[:, 0, 0] = [0, 3, 3, -1, 9]
    table = np.array([[0, 1, 2, 3, 7, 4]])
    pick = lambda **kw: context.block_select(q, m, table, [11], None, 2, **{**dict(top=3, bounds=False, sink=1, recent=1, shared=False), **kw})[0, 0, 0].tolist()  # noqa: E731
    assert pick() == [0, 1, 4]
    assert pick(sink=0, recent=0) == [0, 1, 2]
    assert pick(top=4, sink=0, recent=0) == [0, 1, 2, 3]
    assert pick(top=5) == [0, 1, 2, 3, 4]
    assert pick(top=6) == [0, 1, 2, 3, 4, -1]
    low_high = np.array([[[2.0, 5.0, 1.0, -4.0]]])
    assert context.block_scores(q[0, 0, 0], low_high[:, 0], True).tolist() == [2 + 4]
    # lists: entries that do not ascend or are no context block are passed over
    k = np.zeros((5, 1, 2, 2))
    v = np.arange(5.0)[:, None, None, None] + np.zeros_like(k)
    out, _ = context.sparse_attention(q, k, v, np.array([[0, 1, 2, 3, 4]]), [6], None, None,
                                      np.array([[[[-1, 2, 1, 2, 3, 9]]]]), 1.0, np.zeros((1, 1, 2, 2)), np.zeros((1, 1, 2)))
    assert np.allclose(out, (2 + 2 + 3) / 3)
