"""Whole verification rounds on a paged cache: the new tokens' keys and values written, their
attention under the chain's or the tree's mask, logits, penalties and masks on them, the verify,
and the accepted nodes' cache rows moved, several rounds in a row.  Each step is compared with
its plain form on what the step before it left, at the tolerance of that step's own tests.
"""
import numpy as np
import pytest

import oracle
from _harness import compare as compare_verify
from oracle import paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_attention import check as check_attention
from test_gpu_logits import compare as check_logits
from test_gpu_logits import floats
from test_gpu_paged_kv import host, ints, make_cache, sv, values  # noqa: F401

pytestmark = pytest.mark.gpu

B, HQ, H, D, V, PS, HIST = 3, 8, 2, 64, 96, 16, 40


def start(cache, Q, rounds, seed):
    """(cache tensors, table, base): a shuffled page table with room for the rounds."""
    rng = np.random.default_rng(seed)
    base = np.array([0, 37, 130])
    mp = (130 + Q * (rounds + 1) + PS - 1) // PS
    table = rng.permutation(B * mp + 3)[:B * mp].reshape(B, mp)
    return rng, make_cache(rng, B * mp + 3, H, PS, D, cache, False), table, base


def appended(before, after, x, table, base, cache):
    """The cache rows of x [B][Q][H][D] hold it to half a step, all others what they held."""
    got, scales = after
    new = np.zeros(got.shape[:1] + got.shape[2:3], bool)
    for b in range(B):
        for i in range(x.shape[1]):
            p, r = paged.place(table, b, int(base[b]) + i, len(got), PS)
            new[p, r] = True
            v = got[p, :, r] * (1 if scales is None else scales[p, :, r, None])
            w = x[b, i]
            if cache == "bf16":
                assert np.array_equal(v, w)
            else:  # half a step, 2^-10 scales where codes are subnormal; 2^-22 for fp32's x (1 / s)
                assert (np.abs(v - w) <= 2.0 ** -4 * np.abs(w) * (1 + 2.0 ** -18) + 2.0 ** -10 * scales[p, :, r, None]).all()
    old = ~new[:, None, :, None] & np.ones(got.shape, bool)
    assert np.array_equal(got[old], before[old], equal_nan=True)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("N", [4, 24])
def test_rounds_match_the_plain_forms(sv, cache, tree, N):  # noqa: F811
    import torch
    Q, depth, rounds = N + 1, 5 if tree else N, 3
    rng, (k, v, ks, vs), table, base = start(cache, Q, rounds, [N, tree, cache == "e4m3"])
    t_table, t_base = ints(table), ints(base)
    head = torch.from_numpy(0.4 * rng.normal(size=(HQ * D, V))).to(torch.bfloat16).cuda()
    history = np.full((B, HIST), -1)
    history[:, :4] = rng.integers(0, V, (B, 4))
    length = np.full(B, 4)
    penalties = dict(repetition=np.array([1.2, 1.0, 0.8], np.float32), presence=np.array([0.1, 0.0, 0.5], np.float32),
                     frequency=np.array([0.0, 0.3, 0.2], np.float32))
    temperature = np.array([1.0, 0.0, 0.7], np.float32)
    moved = 0
    for step in range(rounds):
        # what the target's layer would have computed for the chunk
        x, y, q = (torch.from_numpy(rng.normal(size=(B, Q, n, D))).to(torch.bfloat16).cuda() for n in (H, H, HQ))
        parent = synth.random_parents(10 * step + N, B, N, "bfs" if tree else "chain", max_depth=depth)
        mask = None
        if tree:
            mask = sv.spec_tree_mask(ints(parent))[0]
            assert np.array_equal(mask.cpu().numpy().view(np.uint32), oracle.tree_mask(parent)["mask"])

        was = values(k), values(v)
        sv.spec_kv_append(x, y, k, v, t_table, t_base, k_scale=ks, v_scale=vs)
        appended(was[0], (values(k), host(ks)), host(x), table, base, cache)
        appended(was[1], (values(v), host(vs)), host(y), table, base, cache)
        for got, z, s in zip(sv.spec_kv_read(k, v, t_table, t_base, Q, k_scale=ks, v_scale=vs, dtype=torch.float32),
                             (k, v), (ks, vs)):
            want = paged.read(values(z), host(s), table, base, None, Q, np.zeros((B, Q, H, D)))
            assert (np.abs(host(got) - want) <= 2.0 ** -24 * np.abs(want)).all()

        out, lse = sv.spec_paged_attention(q, k, v, t_table, t_base, tree_mask=mask, k_scale=ks, v_scale=vs,
                                           want_lse=True)
        check_attention(out, lse, q, k, v, ks, vs, table, base, np.full(B, Q), None if mask is None else
                        mask.cpu().numpy().view(np.uint32), D ** -0.5, 0.0, 0.0)

        logits = (out.view(B, Q, HQ * D) @ head).contiguous()
        # a drafter that is not far from the target, and the likeliest tokens of its rows
        draft = (logits.float() + 0.5 * torch.from_numpy(rng.normal(size=(B, Q, V))).float().cuda()).to(torch.bfloat16)
        order = np.argsort(-host(draft), -1, kind="stable")
        rank = [[int((parent[b, :i] == parent[b, i]).sum()) for i in range(N)] for b in range(B)]
        tokens = np.array([[order[b, parent[b, i] + 1, rank[b][i]] for i in range(N)] for b in range(B)])
        allowed = rng.integers(0, 1 << 32, (B, Q, (V + 31) // 32), dtype=np.uint64).astype(np.uint32) | 0x11111111
        c = dict(history=history, history_len=length, prompt_len=np.full(B, 4), draft_tokens=tokens, allowed=allowed,
                 **penalties)
        if tree:
            c["tree_mask"] = mask.cpu().numpy().view(np.uint32)
        adjusted = sv.spec_adjust_logits(
            logits, history=ints(history), history_len=ints(length), prompt_len=ints(np.full(B, 4)),
            draft_tokens=ints(tokens), tree_mask=mask, allowed=ints(allowed.view(np.int32)),
            **{n: floats(p) for n, p in penalties.items()})
        check_logits(adjusted, host(logits), c, "bf16")

        if not tree:
            draft = draft[:, :N].contiguous()
        seed, offset = 77, 1000 * step
        bits = lambda t: t.view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        if tree:
            ot, oc, op = sv.spec_verify_tree(adjusted, draft, ints(tokens), ints(parent), floats(temperature), depth, seed,
                                             offset, draft_kind="logits")
            want = oracle.verify_tree(bits(adjusted), bits(draft), tokens, parent, temperature, depth, seed, offset)
            got = dict(tokens=ot.cpu().numpy(), count=oc.cpu().numpy(), path=op.cpu().numpy())
            compare_verify(got, want, keys=("tokens", "count", "path"))
        else:
            ot, oc = sv.spec_verify_chain(adjusted, draft, ints(tokens), floats(temperature), seed, offset,
                                          draft_kind="logits")[:2]
            want = oracle.verify_chain(bits(adjusted), bits(draft), tokens, temperature, seed, offset)
            got = dict(tokens=ot.cpu().numpy(), count=oc.cpu().numpy())
            compare_verify(got, want)
        assert (got["count"] >= 1).all()

        if tree:  # a chain's accepted rows lie where they belong
            node0 = ints(base + 1)
            for bufs in ([k, v],) if ks is None else ([k.view(torch.uint8), v.view(torch.uint8)],
                                                      [ks[..., None], vs[..., None]]):
                before = [t.clone() for t in bufs]
                sv.spec_kv_compact_paged(bufs, t_table, op, oc, node0)
                for t, w in zip(bufs, before):
                    as_int = lambda z: (z.view(torch.int16) if z.dtype == torch.bfloat16 else z).cpu().numpy()  # noqa: E731
                    assert np.array_equal(as_int(t), paged.compact(as_int(w), table, got["path"], got["count"], base + 1))
            moved += int((got["path"][np.arange(depth)[None] < got["count"][:, None] - 1] >
                          np.concatenate([np.arange(n - 1) for n in got["count"]])).sum())
        for b in range(B):
            n = int(got["count"][b])
            history[b, length[b]:length[b] + n] = got["tokens"][b, :n]
        length, base = length + got["count"], base + got["count"]
        t_base = ints(base)
    if tree:
        assert moved > 0


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_a_captured_round_replays_as_it_ran(sv, cache):  # noqa: F811
    """One tree round captured into a graph: each replay on restored inputs, on another stream than
    the capture's, leaves the bits that the eager calls left; two rounds side by side too."""
    import torch
    N, depth = 20, 5
    Q = N + 1

    def make(seed):
        rng, (k, v, ks, vs), table, base = start(cache, Q, 1, seed)
        x, y, q = (torch.from_numpy(rng.normal(size=(B, Q, n, D))).to(torch.bfloat16).cuda() for n in (H, H, HQ))
        parent = ints(synth.random_parents(seed, B, N, max_depth=depth))
        tokens = ints(np.stack([rng.permutation(V)[:N] for _ in range(B)]))
        head = torch.from_numpy(0.4 * rng.normal(size=(HQ * D, V))).to(torch.bfloat16).cuda()
        draft = torch.from_numpy(rng.normal(size=(B, Q, V))).to(torch.bfloat16).cuda()
        temp, rep = floats(np.ones(B)), floats(np.full(B, 1.1))
        t, b, b1 = ints(table), ints(base), ints(base + 1)
        state = [z for z in (k, v, ks, vs) if z is not None]

        def go():
            mask = sv.spec_tree_mask(parent)[0]
            sv.spec_kv_append(x, y, k, v, t, b, k_scale=ks, v_scale=vs)
            out, _ = sv.spec_paged_attention(q, k, v, t, b, tree_mask=mask, k_scale=ks, v_scale=vs)
            logits = (out.view(B, Q, HQ * D) @ head).contiguous()
            logits = sv.spec_adjust_logits(logits, draft_tokens=tokens, tree_mask=mask, repetition=rep, out=logits)
            ot, oc, op = sv.spec_verify_tree(logits, draft, tokens, parent, temp, depth, 5, 9, draft_kind="logits")
            sv.spec_kv_compact_paged([k.view(torch.uint8), v.view(torch.uint8)] if ks is not None else [k, v], t, op, oc, b1)
            if ks is not None:
                sv.spec_kv_compact_paged([ks[..., None], vs[..., None]], t, op, oc, b1)
            return out, logits, ot, oc, op
        return go, state

    raw = lambda z: z.contiguous().view(torch.uint8)  # noqa: E731
    runs = []
    for seed in (3, 4):
        go, state = make(seed)
        fresh = [z.clone() for z in state]
        want = [raw(z).clone() for z in go()] + [raw(z).clone() for z in state]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = go()
        runs.append((graph, state, fresh, res, want, go))  # go holds the inputs that the graph reads
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for _, state, fresh, *_ in runs:
            for z, f in zip(state, fresh):
                z.copy_(f)
        torch.cuda.synchronize()
        for s, (graph, *_) in zip(streams, runs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, state, _, res, want, _ in runs:
            for z, w in zip([*res, *state], want):
                assert torch.equal(raw(z), w)


def test_side_stream_calls(sv):  # noqa: F811
    """Calls on a stream that is not the current one, outputs and workspace allocated for it."""
    import torch
    rng, (k, v, _, _), table, base = start("bf16", 6, 1, 8)
    x, y, q = (torch.from_numpy(rng.normal(size=(B, 6, n, D))).to(torch.bfloat16).cuda() for n in (H, H, HQ))
    t, b = ints(table), ints(base)
    logits = torch.from_numpy(rng.normal(size=(B, 6, V))).float().cuda()
    toks = ints(rng.integers(0, V, (B, 5)))
    k0, v0 = k.clone(), v.clone()
    sv.spec_kv_append(x, y, k, v, t, b)
    want = sv.spec_paged_attention(q, k, v, t, b)[0]
    want_l = sv.spec_adjust_logits(logits, draft_tokens=toks, frequency=floats(np.ones(B)))
    fr = floats(np.ones(B))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        sv.spec_kv_append(x, y, k0, v0, t, b, stream=s)
        out = sv.spec_paged_attention(q, k0, v0, t, b, stream=s)[0]
        got_l = sv.spec_adjust_logits(logits, draft_tokens=toks, frequency=fr, stream=s)
        back = sv.spec_kv_read(k0, v0, t, b, 6, stream=s)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(got_l, want_l)
        assert torch.equal(back[0], x) and torch.equal(back[1], y)


FIRST = """
import torch
import speculative_decoding_verification_53_gb300 as sv
B, Q, H, D, P, ps, V = 2, 9, 2, 64, 40, 16, 300
torch.manual_seed(1)
f = lambda *s: torch.randn(*s, device="cuda").to(torch.bfloat16)
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
k, v, x, y, q, lg = f(P, H, ps, D), f(P, H, ps, D), f(B, Q, H, D), f(B, Q, H, D), f(B, Q, 8, D), f(B, Q, V)
table, base = torch.randperm(P, device="cuda").int().view(B, 20), i([200, 37])
toks, path, count, rep = i([list(range(8))] * B), i([[1, 4]] * B), i([3, 1]), torch.full((B,), 1.2, device="cuda")
k0, v0 = k.clone(), v.clone()
def go():
    sv.spec_kv_append(x, y, k, v, table, base)
    o, l = sv.spec_paged_attention(q, k, v, table, base, want_lse=True)
    a = sv.spec_adjust_logits(lg, draft_tokens=toks, repetition=rep)
    sv.spec_kv_compact_paged([k, v], table, path, count, base)
    return [o, l, a, *sv.spec_kv_read(k, v, table, base, Q)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = go()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got] + [k.clone(), v.clone()]
k.copy_(k0); v.copy_(v0)
want = go() + [k, v]
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("same")
"""


def test_the_first_calls_of_a_process_can_be_captured(sv):  # noqa: F811
    """Nothing that a first call sets up is refused while a stream is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
