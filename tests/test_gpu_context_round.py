"""Whole verification rounds over a long context, as a serving loop runs them: page tables grow,
tree nodes' keys are turned by depth and written, summaries follow, blocks are selected and attended
to, the accepted nodes' rows move, and pages that are no longer needed go back.  No length leaves
the device.  Each step is compared with its plain form on what the step before it left.
"""
import numpy as np
import pytest

import oracle
from oracle import context, paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_paged_kv import host, ints, make_cache, sv, values  # noqa: F401
from test_gpu_rotary import close, reach
from test_gpu_sparse import check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree,shared", [(False, False), (True, True), (True, False)])
def test_rounds(sv, cache, tree, shared):  # noqa: F811
    import torch
    rng = np.random.default_rng([tree, shared, cache == "e4m3"])
    B, HQ, H, D, PS, Q, TOP, R, V = 3, 8, 2, 64, 16, 7, 6, 24, 64
    N, rounds, depth_max = Q - 1, 3, 4 if tree else Q - 1
    held = np.array([150, 16 * 9, 300])
    width = (300 + (rounds + 1) * Q) // PS + 2
    P = B * width
    k, v, ks, vs = make_cache(rng, P, H, PS, D, cache, False)
    freq = sv.rotary_frequencies(2 * R, scaling="parts", factor=4.0, original_len=128, device="cuda")
    stack = rng.permutation(P)
    t_table, t_pages, t_stack, t_count = ints(np.full((B, width), -1)), ints(np.zeros(B)), ints(stack), ints([P])
    base = ints(held)
    summary = torch.zeros((P, H, 2 * D), dtype=torch.bfloat16, device="cuda")
    # the prompts: pages for them, and their summaries
    ok, _ = sv.spec_page_resize(t_table, t_pages, base, t_stack, t_count, PS)
    assert ok.tolist() == [1] * B
    sv.spec_block_summary(k, t_table, ints([0] * B), 300, kind="bounds", new_len=base, k_scale=ks, summary=summary)
    temperature = torch.tensor([1.0, 0.0, 0.7], device="cuda")
    head = torch.from_numpy(0.4 * rng.normal(size=(HQ * D, V))).to(torch.bfloat16).cuda()
    moved = 0
    for step in range(rounds):
        b_now = base.cpu().numpy()
        parent = synth.random_parents(50 + step, B, N, "bfs" if tree else "chain", max_depth=depth_max)
        t_parent = ints(parent)
        before = [x.cpu().numpy() for x in (t_table, t_pages, t_stack, t_count)]
        ok, slots = sv.spec_page_resize(t_table, t_pages, base + Q, t_stack, t_count, PS, base=base, num_tokens=Q)
        want = context.page_resize(before[0], before[1], b_now + Q, before[2], before[3][0], PS, b_now, Q)
        assert np.array_equal(t_table.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[5])
        assert ok.tolist() == [1] * B
        table = want[0]
        mask, depth, _ = sv.spec_tree_mask(t_parent)
        qkv = torch.from_numpy(rng.normal(size=(B, Q, HQ + 2 * H, D))).to(torch.bfloat16).cuda()
        q, key, value = qkv[:, :, :HQ], qkv[:, :, HQ:HQ + H], qkv[:, :, HQ + H:]
        kw = dict(tree_depth=depth if tree else None)
        turned = sv.spec_rotary_append(q, key, value, freq, k, v, t_table, base, k_scale=ks, v_scale=vs, **kw)
        pos = context.positions(b_now, Q, depth.cpu().numpy() if tree else None)
        f = freq.cpu().numpy()
        close(host(turned), context.rotary(host(q), f, pos), reach(host(q), R, False), "bf16")
        # slots are where the keys went
        got = values(k) if ks is None else values(k) * host(ks)[..., None]
        exp = context.rotary(host(key), f, pos)
        flat = slots.cpu().numpy()
        half = 2.0 ** -8 if cache == "bf16" else 2.0 ** -4
        for b in range(B):
            for i in range(Q):
                row, want_row = got[flat[b, i] // PS, :, flat[b, i] % PS], exp[b, i]
                small = 0 if cache == "bf16" else 2.0 ** -10 * np.abs(want_row).max() / 448
                assert (np.abs(row - want_row) <= half * (1 + 2.0 ** -10) * np.abs(want_row) + small + 1e-5).all()
        blocks = sv.spec_block_select(turned, summary, t_table, base, PS, TOP, kind="bounds", shared=shared)
        assert np.array_equal(blocks.cpu().numpy(), context.block_select(host(turned), host(summary), table, b_now, None, PS,
                                                                         TOP, True, 1, 1, shared))
        out, lse = sv.spec_sparse_attention(turned, k, v, t_table, base, blocks, tree_mask=mask if tree else None, k_scale=ks,
                                            v_scale=vs, want_lse=True)
        check_attention(out, lse, turned, k, v, ks, vs, table, b_now, None, mask.cpu().numpy().view(np.uint32) if tree else None,
                        blocks.cpu().numpy(), D ** -0.5, 0.0)
        logits = (out.reshape(B, Q, HQ * D) @ head).contiguous()
        draft = torch.from_numpy(rng.normal(size=(B, Q, V))).to(torch.bfloat16).cuda()
        tokens = ints(rng.integers(0, V, (B, N)))
        _, count, path = sv.spec_verify_tree(logits, draft, tokens, t_parent, temperature, depth_max, 7, step, draft_kind="logits")
        old = values(k)
        bufs = [k.view(torch.uint8), v.view(torch.uint8)] if cache == "e4m3" else [k, v]
        sv.spec_kv_compact_paged(bufs, t_table, path, count, base + 1)
        if ks is not None:
            sv.spec_kv_compact_paged([ks[..., None], vs[..., None]], t_table, path, count, base + 1)
        assert np.array_equal(values(k), paged.compact(old, table, path.cpu().numpy(), count.cpu().numpy(), b_now + 1), equal_nan=True)
        moved += int(count.sum())
        # the accepted tokens stay; summaries of the blocks that they touch, and pages behind them go back
        sv.spec_block_summary(k, t_table, base, Q, kind="bounds", new_len=count, k_scale=ks, summary=summary)
        base = base + count
        end = base.cpu().numpy()
        kd = values(k) if ks is None else values(k) * host(ks)[..., None]
        exp = context.block_summary(kd, table, b_now, end - b_now, Q, True, host(summary))
        assert (np.abs(host(summary) - exp) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(exp)).all()
        before = [x.cpu().numpy() for x in (t_table, t_pages, t_stack, t_count)]
        sv.spec_page_resize(t_table, t_pages, base, t_stack, t_count, PS)
        want = context.page_resize(before[0], before[1], end, before[2], before[3][0], PS)
        for x, y in zip((t_table, t_pages, t_stack, t_count), (want[0], want[1], want[2], [want[3]])):
            assert np.array_equal(x.cpu().numpy(), y)
    assert moved >= B * rounds
    # everybody leaves: every page is free again, once
    sv.spec_page_resize(t_table, t_pages, ints([0] * B), t_stack, t_count, PS)
    assert t_count.tolist() == [P] and sorted(t_stack.tolist()) == list(range(P)) and t_pages.tolist() == [0] * B


FIRST = """
import torch
import speculative_decoding_verification_53_gb300 as sv
B, Q, H, HQ, D, P, ps = 40, 5, 2, 8, 64, 900, 16
torch.manual_seed(1)
f = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
k, v, qkv = f(P, H, ps, D), f(P, H, ps, D), f(B, Q, HQ + 2 * H, D)
table, base = torch.randperm(P, device="cuda").int()[:B * 22].view(B, 22), i([320 - 5 * b for b in range(B)])
held, stack, top = (base + 15) // ps, i(list(range(P))), i([0])
summary, freq, zero = torch.zeros((P, H, D), dtype=torch.bfloat16, device="cuda"), sv.rotary_frequencies(D, device="cuda"), i([0] * B)
state = [k, v, table, held, stack, top, summary]
start = [t.clone() for t in state]
def go():
    sv.spec_page_resize(table, held, base - 16, stack, top, ps)
    ok, slots = sv.spec_page_resize(table, held, base + Q, stack, top, ps, base=base, num_tokens=Q)
    out, key = sv.spec_rotary(qkv[:, :, :HQ], freq, base, key=qkv[:, :, HQ:HQ + H])
    q = sv.spec_rotary_append(qkv[:, :, :HQ], qkv[:, :, HQ:HQ + H], qkv[:, :, HQ + H:], freq, k, v, table, base)
    sv.spec_block_summary(k, table, zero, 330, new_len=base, summary=summary)
    lists = sv.spec_block_select(q, summary, table, base, ps, 6)
    one = sv.spec_block_select(q, summary, table, base, ps, 6, shared=True)
    return [ok, slots, out, key, q, lists, one, *sv.spec_sparse_attention(q, k, v, table, base, lists, want_lse=True),
            *sv.spec_sparse_attention(q, k, v, table, base, one, want_lse=True)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = go()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got + state]
for t, s in zip(state, start):
    t.copy_(s)
want = go() + state
assert all(torch.equal(a, b) for a, b in zip(got, want))
# and on a stream of its own, again and again, while the current one is idle
torch.cuda.synchronize()
side = torch.cuda.Stream()
for _ in range(10):
    q = sv.spec_rotary(qkv[:, :, :HQ], freq, base, stream=side)[0]
    one = sv.spec_block_select(q, summary, table, base, ps, 6, shared=True, stream=side)
    o = sv.spec_sparse_attention(q, k, v, table, base, one, stream=side)[0]
    m = sv.spec_block_summary(k, table, zero, 330, new_len=base, stream=side)
    side.synchronize()
    assert torch.equal(q, want[2]) and torch.equal(one, want[6]) and torch.equal(o, want[9]) and m.shape == summary.shape
print("same")
"""


def test_the_first_calls_of_a_process_can_be_captured(sv):  # noqa: F811
    """Nothing that a first call sets up is refused while a stream is captured; calls on another stream."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
