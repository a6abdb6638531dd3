"""Keys that only one query sees do not move a bit of what the other queries get from attention over
selected blocks: a block that only its list names, a draft node or a chain's token that only it sees.
No tolerance: outputs and lse are compared bit for bit.
"""
import numpy as np
import pytest

from oracle import context, paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_paged_kv import ints, make_cache, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def put_large_key(k, ks, page, row, head, q):
    """The key at a page's row becomes 4 q: its score for the query q is far above all others."""
    import torch
    key = 4 * q.float()
    if ks is None:
        k[page, head, row] = key.to(k.dtype)
        return
    scale = key.abs().max() / 448
    ks[page, head, row] = scale
    k.view(torch.uint8)[page, head, row] = (key / scale).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("shared,Q,Hq,D,n", [
    (False, 5, 8, 64, 12), (False, 8, 8, 128, 40), (False, 7, 2, 128, 12), (False, 40, 8, 128, 12), (False, 6, 8, 256, 12),
    (True, 5, 8, 64, 12), (True, 8, 8, 128, 40), (True, 12, 8, 128, 12), (True, 6, 8, 256, 12), (True, 70, 8, 128, 40)])
def test_a_key_that_one_query_sees(sv, cache, tree, shared, Q, Hq, D, n):  # noqa: F811
    import torch
    rng = np.random.default_rng([Q, D, n, tree])
    B, H, ps, full = 2, 2, 16, 200
    g = Hq // H
    base = np.array([full * ps + 5, full * ps])
    width = full + 1 + (Q + ps) // ps
    P = B * width
    table = rng.permutation(P).reshape(B, width)
    k, v, ks, vs = make_cache(rng, P, H, ps, D, cache, False)
    if cache == "e4m3":
        for t in (k, v):
            t.view(torch.uint8).bitwise_xor_(torch.randint(0, 2, t.shape, device="cuda", dtype=torch.uint8) << 7)
        ks *= 0.05
    q = torch.from_numpy(rng.normal(size=(B, Q, Hq, D))).to(torch.bfloat16).cuda()
    # lists: n - 1 even blocks in common, and an odd block of each query's own
    blocks = np.empty((B, 1 if shared else Q, H, n), np.int32)
    for b, i, h in np.ndindex(blocks.shape[:3]):
        common = np.sort(np.random.default_rng([b, h]).permutation(full // 2)[:n - 1]) * 2
        blocks[b, i, h] = np.sort(np.append(common, 2 * i + 1))
    mask = words = None
    if tree:
        mask, _, _ = sv.spec_tree_mask(ints(synth.random_parents(Q, B, Q - 1, "random")))
        words = mask.cpu().numpy().view(np.uint32)
    args = (ints(table), ints(base), ints(blocks))
    call = lambda: sv.spec_sparse_attention(q, k, v, *args, tree_mask=mask, k_scale=ks, v_scale=vs, want_lse=True)  # noqa: E731
    out, lse = (t.clone() for t in call())
    keep = k.clone(), None if ks is None else ks.clone()
    places = []  # (row, position, the one query that sees it)
    for b in range(B):
        if not shared:
            places += [(b, (2 * i + 1) * ps + 3, i) for i in (0, Q // 2)]
        sees = [[paged.visible(i, int(base[b]) + j, int(base[b]), Q, None if mask is None else words[b]) for j in range(Q)]
                for i in range(Q)]
        places += [(b, int(base[b]) + j, j) for j in range(1, Q) if sum(s[j] for s in sees) == 1][:2]
    assert len(places) >= B
    for b, pos, i in places:
        k.view(torch.uint8).copy_(keep[0].view(torch.uint8))
        if ks is not None:
            ks.copy_(keep[1])
        page, row = paged.place(table, b, pos, P, ps)
        for h in range(H):
            put_large_key(k, ks, page, row, h, q[b, i, h * g])
        got, got_lse = call()
        same = ((got == out).all(-1) & (got_lse == lse)).cpu().numpy()
        assert not same[b, i, ::g].any(), "the key is seen"
        others = np.ones((B, Q), bool)
        others[b, i] = False
        assert same[others].all(), (b, pos, i, np.argwhere(~same & others[..., None]).tolist())
