"""Logit penalties, biases and masks on the GPU against their plain float64 form.

Tolerance: the fp32 steps (a division or product, a product and three sums) each round by
at most 2^-24 of what they hold, at most S = |x| max(rep, 1 / rep) + c freq + pres + |bias|
in magnitude: 6 x 2^-24 S; then half a step of the output's type, 2^-8 (bf16) of its value.
"""
import numpy as np
import pytest

import oracle
from oracle import paged
from speculative_decoding_verification_53_gb300 import synth
from test_gpu_paged_kv import host, ints, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def floats(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def make(rng, B, R, V, H, M, tree, grammar, drafts=True):
    c = dict(logits=4 * rng.normal(size=(B, R, V)))
    few = min(V, 50)                               # tokens repeat
    if H:
        c["history"] = np.where(rng.random((B, H)) < 0.5, rng.integers(0, few, (B, H)), rng.integers(-2, V + 2, (B, H)))
        c["history_len"] = rng.integers(-1, H + 3, B)
        c["prompt_len"] = rng.integers(-1, H + 2, B)
        c["history_len"][0], c["prompt_len"][0] = H, H // 2
    if R > 1 and drafts:
        c["draft_tokens"] = rng.integers(-1, few + 1, (B, R - 1))
        if tree:
            c["tree_mask"] = oracle.tree_mask(synth.random_parents(int(rng.integers(1 << 20)), B, R - 1, max_depth=40))["mask"]
    c["repetition"] = rng.uniform(0.5, 2, B).astype(np.float32)
    c["presence"] = rng.uniform(-1, 1, B).astype(np.float32)
    c["frequency"] = rng.uniform(-0.5, 0.5, B).astype(np.float32)
    if M:
        c["bias_tokens"] = rng.integers(-1, V + 1, (B, M))
        c["bias_values"] = (3 * rng.normal(size=(B, M))).astype(np.float32)
    if grammar:
        W = (V + 31) // 32
        words = rng.integers(0, 1 << 32, (B, R, W), dtype=np.uint64)
        pick = rng.random((B, R, W))
        c["allowed"] = np.where(pick < 0.4, 0, np.where(pick < 0.7, 0xffffffff, words)).astype(np.uint32)
        c["allowed"][0, 0] = 0                     # a row that allows nothing
    return c


def device(c, dtype):
    import torch
    d = {}
    for k, v in c.items():
        if k == "logits":
            d[k] = torch.from_numpy(v).to(torch.bfloat16 if dtype == "bf16" else torch.float32).cuda()
        elif k in ("repetition", "presence", "frequency", "bias_values"):
            d[k] = floats(v)
        else:
            d[k] = ints(np.asarray(v).astype(np.int64).astype(np.uint32).view(np.int32) if k in ("tree_mask", "allowed") else v)
    return d


def compare(got, x, c, dtype):
    want = paged.adjust_logits(x, **{k: v for k, v in c.items() if k != "logits"})
    got = host(got)
    rep = c.get("repetition", np.ones(len(x)))[:, None, None].astype(np.float64)
    count = (c["history"].shape[1] if "history" in c else 0) + x.shape[1]
    S = np.abs(x) * np.maximum(rep, 1 / rep)
    for k, m in (("frequency", count), ("presence", 1)):
        if k in c:
            S = S + m * np.abs(c[k].astype(np.float64))[:, None, None]
    if "bias_values" in c:
        S = S + np.abs(c["bias_values"]).max()
    assert np.array_equal(np.isneginf(got), np.isneginf(want)) and np.array_equal(np.isnan(got), np.isnan(want))
    f = np.isfinite(want)
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    tol = 6 * 2.0 ** -24 * S[f] * (1 + half) + half * np.abs(want[f])
    assert (np.abs(got[f] - want[f]) <= tol).all()
    same = f & (want == x)                         # tokens of no list pass through bit for bit
    assert np.array_equal(got[same], x[same])


CASES = [  # B, R, V, H, M, tree, grammar
    (1, 1, 1, 0, 0, False, False), (2, 1, 7, 5, 3, False, True), (3, 6, 4099, 200, 9, False, True),
    (2, 9, 5000, 0, 0, False, False), (2, 13, 2048, 700, 0, True, False), (1, 61, 20001, 300, 40, True, True),
    (2, 33, 3000, 90, 1, True, True), (1, 4, 40000, 3000, 300, False, False), (4, 5, 31, 64, 2, False, True),
    (1, 129, 100, 20, 0, True, True), (300, 2, 333, 30, 5, False, True)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", CASES)
def test_matches_the_plain_form(sv, shape, dtype, in_place):  # noqa: F811
    rng = np.random.default_rng([*shape])
    c = make(rng, *shape)
    d = device(c, dtype)
    x = host(d["logits"])
    logits = d.pop("logits")
    before = logits.clone()
    out = sv.spec_adjust_logits(logits, **d, out=logits if in_place else None)
    assert (out is logits) == in_place
    compare(out, x, c, dtype)
    if not in_place:
        import torch
        assert torch.equal(logits, before)


@pytest.mark.parametrize("in_place", [False, True])
def test_each_part_alone(sv, in_place):  # noqa: F811
    """Every argument may be missing."""
    rng = np.random.default_rng(3)
    full = make(rng, 2, 6, 3001, 150, 12, True, True)
    for keep in ((), ("allowed",), ("bias_tokens", "bias_values"), ("history", "history_len", "frequency"),
                 ("history", "history_len", "prompt_len", "repetition"), ("draft_tokens", "presence"),
                 ("draft_tokens", "tree_mask", "repetition"), ("repetition", "presence", "frequency")):
        c = {k: full[k] for k in ("logits", *keep)}
        d = device(c, "bf16")
        logits = d.pop("logits")
        x = host(logits)
        compare(sv.spec_adjust_logits(logits, **d, out=logits if in_place else None), x, c, "bf16")


@pytest.mark.parametrize("in_place", [False, True])
def test_special_values_and_repeated_entries(sv, in_place):  # noqa: F811
    """NaN and infinities in place and in masked places; a token listed many times everywhere."""
    V, R = 70, 40
    x = np.zeros((1, R, V))
    x[0, :, 3], x[0, :, 4], x[0, :, 5], x[0, :, 6] = np.nan, np.inf, -np.inf, np.nan
    c = dict(history=np.full((1, 500), 4), history_len=np.array([500]), prompt_len=np.array([2]),
             draft_tokens=np.full((1, R - 1), 9), repetition=np.array([1.5], np.float32),
             frequency=np.array([0.25], np.float32), presence=np.array([0.5], np.float32),
             bias_tokens=np.array([[9, 11, 9, 12, 11, -1]]), bias_values=np.array([[5, 1, -2, -np.inf, 3, 9]], np.float32))
    ok = np.full((1, R, 3), 0xffffffff, np.uint32)
    ok[:, :, 0] &= ~np.uint32(1 << 6)
    c["allowed"] = ok
    d = device(c | dict(logits=x), "fp32")
    logits = d.pop("logits")
    out = host(sv.spec_adjust_logits(logits, **d, out=logits if in_place else None))
    want = paged.adjust_logits(x, **c)
    assert np.array_equal(out, want.astype(np.float32), equal_nan=True)  # quarters: exact in fp32
    assert np.isnan(out[0, 0, 3]) and np.isneginf(out[0, :, 6]).all() and np.isneginf(out[0, :, 12]).all()
    assert out[0, 1, 9] == -0.25 - 0.5 - 2 and out[0, 39, 9] == -39 * 0.25 - 0.5 - 2 and out[0, 0, 11] == 3


def test_long_chain_shaped_tree_of_one_token(sv):  # noqa: F811
    """1024 nodes below one another, all the same token: row r counts it r times."""
    import torch
    N, V = 1024, 600
    mask = sv.spec_tree_mask(ints(np.arange(-1, N - 1)[None]))[0]
    for in_place in (False, True):
        x = torch.zeros((1, N + 1, V), device="cuda")
        out = sv.spec_adjust_logits(x, draft_tokens=ints(np.full((1, N), 77)), tree_mask=mask,
                                    frequency=floats([1.0]), out=x if in_place else None)
        assert torch.equal(out[0, :, 77], -torch.arange(N + 1, device="cuda", dtype=torch.float32))
        out[0, :, 77] = 0
        assert not out.any()


def test_odd_alignments_of_input_and_output(sv):  # noqa: F811
    """Rows that start anywhere, and outputs that start elsewhere than their inputs."""
    import torch
    rng = np.random.default_rng(6)
    c = make(rng, 2, 3, 4097, 60, 5, False, True)
    for dtype, es in (("bf16", 8), ("fp32", 4)):
        d = device(c, dtype)
        logits = d.pop("logits")
        x = host(logits)
        for a, z in ((0, 1), (3, 3), (1, 2)):
            src = torch.zeros(logits.numel() + es, dtype=logits.dtype, device="cuda")
            dst = torch.full((logits.numel() + es,), 7.0, dtype=logits.dtype, device="cuda")
            src[a:a + logits.numel()] = logits.reshape(-1)
            out = sv.spec_adjust_logits(src[a:a + logits.numel()].view(logits.shape), **d,
                                        out=dst[z:z + logits.numel()].view(logits.shape))
            compare(out, x, c, dtype)
            assert (dst[:z] == 7).all() and (dst[z + logits.numel():] == 7).all()


def test_a_vocabulary_at_the_limit_and_more_than_32_bits_of_bytes(sv):  # noqa: F811
    import torch
    V, R = 1 << 24, 65                              # 4.4 GB of fp32
    x = torch.zeros((1, R, V), device="cuda")
    last = V - 1
    ok = torch.full((1, R, V // 32), -1, dtype=torch.int32, device="cuda")
    ok[0, R - 1, -1] = 0x7fffffff                   # the last token of the last row is not allowed
    out = sv.spec_adjust_logits(x, history=ints([[last, 5]]), frequency=floats([2.0]), bias_tokens=ints([[last - 1]]),
                                bias_values=floats([[3.0]]), allowed=ok, out=x)
    assert out[0, R - 2, last] == -2 and torch.isneginf(out[0, R - 1, last]) and (out[0, :, last - 1] == 3).all()
    assert (out[0, :, 5] == -2).all() and int((out[0, R - 1] != 0).sum()) == 3
    del x, out
    torch.cuda.empty_cache()


def test_captured_and_replayed_on_new_lists(sv):  # noqa: F811
    import torch
    rng = np.random.default_rng(9)
    c = make(rng, 2, 5, 6000, 100, 8, False, True)
    d = device(c, "bf16")
    logits = d.pop("logits")
    out = torch.empty_like(logits)
    sv.spec_adjust_logits(logits, **d, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.spec_adjust_logits(logits, **d, out=out)
    for seed in (1, 2):
        n = make(np.random.default_rng(seed), 2, 5, 6000, 100, 8, False, True)
        e = device(n, "bf16")
        x = e.pop("logits")
        logits.copy_(x)
        for k in d:
            d[k].copy_(e[k])
        g.replay()
        compare(out, host(x), n, "bf16")


def test_refusals(sv):  # noqa: F811
    import torch
    x = torch.zeros((2, 3, 10), device="cuda")
    f = sv.spec_adjust_logits
    i, fl = torch.zeros((2, 2), dtype=torch.int32, device="cuda"), torch.zeros((2,), device="cuda")
    for kw, err in ((dict(history=i.long()), TypeError), (dict(history_len=i[:, 0].contiguous()), ValueError),
                    (dict(draft_tokens=i[:, :1]), ValueError), (dict(tree_mask=i[..., None].contiguous()), ValueError),
                    (dict(repetition=fl[:1]), ValueError), (dict(repetition=fl.double()), TypeError),
                    (dict(bias_tokens=i), ValueError), (dict(bias_tokens=i, bias_values=fl), ValueError),
                    (dict(allowed=i), ValueError), (dict(out=x[:, :2]), ValueError), (dict(out=x.bfloat16()), TypeError),
                    (dict(history=i.cpu()), ValueError), (dict(history=i[:, 0]), ValueError)):
        with pytest.raises(err):
            f(x, **kw)
    with pytest.raises(TypeError):
        f(x.half())
    with pytest.raises(ValueError):
        f(x[:, :, ::2])
    flat = torch.zeros(61, device="cuda")
    with pytest.raises(sv.SpecVerifyError) as e:
        f(flat[:60].view(2, 3, 10), out=flat[1:].view(2, 3, 10))
    assert e.value.status == sv.SV_ERR_INVALID_ARG
    assert f(x[:0]).shape == (0, 3, 10)
