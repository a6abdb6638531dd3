"""The attention's scratch: how much a call asks for, a caller's own buffer of every kind, and that
nothing behind it is touched."""
import numpy as np
import pytest

from test_gpu_attention import both, case, check, run
from test_gpu_paged_kv import sv  # noqa: F401

pytestmark = pytest.mark.gpu


def need(sv, c, max_len=None):  # noqa: F811
    q, k = c[0], c[1]
    B, Q, Hq, D = q.shape
    return sv.spec_paged_attention_workspace_size(B, Q, Hq, k.shape[1], D, k.dtype, max_len or c[5].shape[1] * k.shape[2])


@pytest.mark.parametrize("cache", ["bfloat16", "float8_e4m3fn"])
def test_scratch_does_not_grow_with_the_batch(sv, cache):  # noqa: F811
    """Partial results are kept for real rows only, and where every row tile is one CTA's for none."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    size = lambda B, Q, n: sv.spec_paged_attention_workspace_size(B, Q, 32, 8, 128, getattr(torch, cache), n)  # noqa: E731
    for B in (64, 512, 4096):
        assert size(B, 6, 4096) == 0 and size(B, 6, 512) == 0 and size(B, 6, 1 << 20) == 0
    for B in (1, 2, 8, 16):
        assert 0 < size(B, 6, 65536) <= 3 * sms * 24 * 129 * 4
        assert size(B, 6, 65536) % (24 * 129 * 4) == 0
    for B in (1, 8, 64, 4096):  # one token: the kernel for few rows, about four CTAs an SM
        assert size(B, 1, 2000) <= (4 * sms + 8 * B) * 4 * 129 * 4
    assert size(4096, 1, 2000) == 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,Q,D,ps,ctx", [(300, 6, 64, 16, 600), (155, 30, 128, 16, 500), (160, 5, 64, 24, 1200)])
def test_large_batches(sv, B, Q, D, ps, ctx, tree, cache):  # noqa: F811
    """One or two CTAs a row: unequal rows, some shorter than a stretch, one invalid."""
    import torch
    rng = np.random.default_rng([B, Q, tree])
    c = list(case(rng, B, Q, 4, 1, D, ps, ctx, cache, tree, False, ragged=False))
    c[6], c[7] = rng.integers(0, ctx + 1, B), rng.integers(0, Q + 1, B)
    c[6][1:8], c[7][0] = [0, 1, 100, 127, 128, -3, 260], Q
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert need(sv, c, 1 << 16) <= (0 if 2 * B > 3 * sms else 3 * sms * Q * 4 * (D + 1) * 4)
    both(sv, c)
    both(sv, c, workspace=None)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("Q,Hq,H,D,ctx", [(1, 8, 2, 128, 900), (5, 2, 2, 64, 700), (6, 8, 2, 128, 1500), (61, 4, 1, 128, 3000),
                                          (20, 4, 1, 256, 2500), (33, 7, 1, 128, 2000)])
def test_a_workspace_of_the_callers(sv, Q, Hq, H, D, ctx, cache):  # noqa: F811
    """Fitting, larger, of another type, too small, off a 16-byte boundary, empty, none."""
    import torch
    rng = np.random.default_rng([Q, Hq, D])
    c = case(rng, 2, Q, Hq, H, D, 16, ctx, cache, Q > 7, False, ragged=False)
    n = need(sv, c)
    assert n > 0
    want, want_l = run(sv, c)
    held = torch.full((n + 4096,), 0xff, dtype=torch.uint8, device="cuda")  # NaN, whatever it is read as
    for ws in (held[:n], held[:n + 1024], held[:n + 8 & ~7].view(torch.int64)):
        held.fill_(0xff)
        o, l = run(sv, c, workspace=ws)
        assert torch.equal(o, want) and torch.equal(l, want_l)
        assert (held[n:] == 0xff).all()
    for ws in (held[:n - 1], held[8:n + 8], held[:0], None):  # not split: the same to the tolerance
        held.fill_(0xff)
        o, l = run(sv, c, workspace=ws)
        assert (held == 0xff).all()
        check(o, l, *c[:9], D ** -0.5, 5.0, 6.0)
    both(sv, c)
