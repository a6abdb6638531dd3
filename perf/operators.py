"""Cases of a verification round on a paged key/value cache, for timing and comparison.

Five operators of one round: new tokens' keys and values written into cache pages (bf16, or e4m3 with one scale per
token and head), pages read back, attention of the new tokens over the cache, the logits' penalties, biases and
grammar masks, and the move of the accepted tree nodes' cache rows.  ``run`` computes each in plain torch
operations, or through the package where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one conversation, five drafts verified against a large vocabulary: latency counts
        dict(name="adjust one chain", op="adjust", B=1, R=6, V=128256, H=1500, bias=0, grammar=False, tree=False,
             dtype="bf16"),
        # a batch of draft trees with a grammar each: every row of the tree is written
        dict(name="adjust trees", op="adjust", B=16, R=61, V=128256, H=6000, bias=64, grammar=True, tree=True,
             dtype="bf16"),
        # a chain's six new tokens enter a quantised cache, one layer
        dict(name="append chain", op="append", B=8, N=6, Hkv=8, D=128, page=16, ctx=2000, cache="e4m3", dtype="bf16",
             ragged=True, nhd=False),
        # prompts enter the cache in chunks
        dict(name="append prompts", op="append", B=16, N=2048, Hkv=8, D=128, page=64, ctx=1000, cache="e4m3",
             dtype="bf16", ragged=True, nhd=True),
        # a short odd stretch handed to a drafter with its own small cache
        dict(name="read stretch", op="read", B=3, N=133, Hkv=4, D=64, page=16, ctx=40, cache="e4m3", dtype="bf16",
             ragged=True, nhd=False),
        # whole contexts read back
        dict(name="read contexts", op="read", B=8, N=8192, Hkv=8, D=128, page=64, ctx=0, cache="e4m3", dtype="bf16",
             ragged=True, nhd=False),
        # one conversation, one new token: the smallest call
        dict(name="attention one token", op="attention", B=1, Q=1, Hq=32, Hkv=8, D=128, page=16, ctx=777, cache="bf16",
             tree=False, ragged=False, nhd=False),
        # chains of five drafts and the last token over long ragged contexts
        dict(name="attention chains", op="attention", B=8, Q=6, Hq=32, Hkv=8, D=128, page=16, ctx=32768, cache="bf16",
             tree=False, ragged=True, nhd=False),
        # 60-node trees and their roots over a quantised cache
        dict(name="attention trees", op="attention", B=16, Q=61, Hq=32, Hkv=8, D=128, page=64, ctx=8192, cache="e4m3",
             tree=True, ragged=True, nhd=False),
        # a chunk of a prompt behind a context: bound by its products
        dict(name="attention chunk", op="attention", B=2, Q=2048, Hq=32, Hkv=8, D=128, page=64, ctx=6001, cache="bf16",
             tree=False, ragged=False, nhd=True),
        # the accepted nodes of one tree, every layer's keys and values
        dict(name="compact one tree", op="compact", B=1, N=60, L=4, bufs=64, Hkv=8, D=128, page=16, cache="bf16"),
        # a batch of trees
        dict(name="compact trees", op="compact", B=64, N=60, L=5, bufs=64, Hkv=8, D=128, page=64, cache="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(("adjust", "append", "read", "attention", "attention", "attention", "compact"))
    if op == "adjust":
        tree = rng.random() < 0.4
        R = _log_int(rng, 2, 129) if tree else _log_int(rng, 1, 17)
        V = _log_int(rng, 1000, 160000)
        B = _log_int(rng, 1, max(1, min(256, 100_000_000 // (R * V))))
        return dict(op=op, B=B, R=R, V=V, H=_log_int(rng, 1, 20000), bias=rng.choice((0, 1, 37, 300)),
                    grammar=rng.random() < 0.5, tree=tree, dtype=rng.choice(("bf16", "fp32")))
    Hkv = rng.choice((1, 2, 3, 4, 8, 8, 16))
    D = rng.choice((64, 64, 96, 128, 128, 128, 256))
    page = rng.choice((1, 8, 16, 16, 24, 32, 64, 64, 128))
    cache = rng.choice(("bf16", "e4m3"))
    nhd = rng.random() < 0.5
    if op in ("append", "read"):
        B = _log_int(rng, 1, 128)
        N = _log_int(rng, 1, max(1, min(8192, 60_000_000 // (B * Hkv * D))))
        return dict(op=op, B=B, N=N, Hkv=Hkv, D=D, page=page, ctx=_log_int(rng, 1, 4000), cache=cache,
                    dtype=rng.choice(("bf16", "fp32")), ragged=rng.random() < 0.7, nhd=nhd)
    if op == "compact":
        bufs, L = _log_int(rng, 1, 128), rng.randint(1, 8)
        B = _log_int(rng, 1, max(1, min(256, 1_000_000_000 // (bufs * Hkv * D * 3 * max(page, 64)))))
        return dict(op=op, B=B, N=rng.randint(L + 1, 128), L=L, bufs=bufs, Hkv=Hkv, D=D, page=page, cache=cache)
    g = rng.choice((1, 2, 4, 4, 7, 8))
    kind = rng.choice(("token", "chain", "chain", "tree", "tree", "chunk"))
    Q = {"token": 1, "chain": rng.randint(2, 17), "tree": _log_int(rng, 3, 129), "chunk": _log_int(rng, 64, 1500)}[kind]
    B = _log_int(rng, 1, 8 if kind == "chunk" else 64)
    most = min(131072, 3_000_000_000 // (B * Hkv * g * Q), 500_000_000 // (B * Hkv * D))
    return dict(op=op, B=B, Q=Q, Hq=Hkv * g, Hkv=Hkv, D=D, page=page, ctx=_log_int(rng, 1, max(2, most)), cache=cache,
                tree=kind == "tree", ragged=rng.random() < 0.7, nhd=nhd)


# ------------------------------------------------------------------ inputs

def _spread(B, hi, ragged):
    """Lengths of the batch rows: all `hi`, or spread evenly from `hi` down to about a quarter of it."""
    if not ragged or B == 1:
        return [hi] * B
    return [hi - (b * (hi - (hi + 3) // 4)) // (B - 1) for b in range(B)]


def _torch_dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def _tree_words(rng, B, N):
    """Ancestor-or-self bits int32 [B][N][ceil(N/32)] of random draft trees (children of one of the few nodes before)."""
    W = (N + 31) // 32
    bits = np.zeros((B, N, W * 32), np.uint8)
    for i in range(N):
        parent = rng.integers(-1 if i < 4 else max(-1, i // 2 - 3), i, B)
        has = parent >= 0
        bits[has, i] = bits[np.nonzero(has)[0], parent[has]]
        bits[:, i, i] = 1
    return torch.from_numpy(np.packbits(bits, axis=2, bitorder="little").view(np.int32)).cuda()


def _cache(c, seed, gen, lens, most):
    """A pool of pages for rows of up to `most` positions, its scales, and a shuffled page table that holds `lens[b]`
    positions of row b."""
    page, H, D = c["page"], c["Hkv"], c["D"]
    need = [(n + page - 1) // page for n in lens]
    width = (most + page - 1) // page
    P = len(lens) * width + 3 if c["op"] != "attention" else sum(need) + 3
    perm = np.random.default_rng([seed, 11]).permutation(P).astype(np.int32)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    shape = (P, page, H, D) if c.get("nhd") else (P, H, page, D)

    def pages():
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        if c["cache"] == "e4m3":
            x = (x * 110).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return x.permute(0, 2, 1, 3) if c.get("nhd") else x

    s = dict(k_pages=pages(), v_pages=pages(), page_table=torch.from_numpy(table).cuda(), k_scale=None, v_scale=None,
             max_len=max(lens))
    if c["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = ((0.5 + torch.rand((P, H, page), generator=gen, device="cuda")) / 110 for _ in "kv")
    return s


def prepare(case, seed):
    c = case
    rng = np.random.default_rng([seed, 7])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "adjust":
        B, R, V, H = c["B"], c["R"], c["V"], c["H"]
        s["logits"] = (3 * torch.randn((B, R, V), generator=gen, device="cuda")).to(_torch_dtype(c["dtype"]))

        def tokens(*shape):  # frequent tokens come first, as in a vocabulary ordered by frequency
            return (V * torch.rand(shape, generator=gen, device="cuda") ** 4).to(torch.int32).clamp_(max=V - 1)

        s["history"] = tokens(B, H)
        n = _spread(B, H, True)
        rng.shuffle(n)
        s["history_len"] = _ints(n)
        s["prompt_len"] = _ints([x // 2 for x in n])
        s["draft_tokens"] = tokens(B, R - 1) if R > 1 else None
        s["tree_mask"] = _tree_words(rng, B, R - 1) if c["tree"] and R > 1 else None
        u = torch.rand((3, B), generator=gen, device="cuda")
        s["repetition"], s["presence"], s["frequency"] = (1 + 0.5 * u[0], 0.8 * u[1], 0.3 * u[2])
        s["bias_tokens"] = s["bias_values"] = s["allowed"] = None
        if c["bias"]:
            m = min(c["bias"], V)
            s["bias_tokens"] = torch.stack([torch.randperm(V, generator=gen, device="cuda")[:m] for _ in range(B)]).int()
            s["bias_values"] = 4 * torch.randn((B, m), generator=gen, device="cuda")
        if c["grammar"]:  # a grammar allows runs of the vocabulary here, single tokens there
            W = (V + 31) // 32
            r = torch.randint(-2 ** 31, 2 ** 31, (B, R, W), generator=gen, device="cuda", dtype=torch.int64)
            pick = torch.rand((B, R, W), generator=gen, device="cuda")
            r = torch.where(pick < 0.6, torch.zeros_like(r), torch.where(pick < 0.8, torch.full_like(r, -1), r))
            s["allowed"] = r.to(torch.int32)
        s["out"] = torch.empty_like(s["logits"])
        return s
    if c["op"] == "compact":
        B, N, L, page = c["B"], c["N"], c["L"], c["page"]
        base = rng.integers(0, page + 40, B)
        width = (page + 40 + N + page - 1) // page
        P = B * width
        s["page_table"] = torch.from_numpy(rng.permutation(P).astype(np.int32).reshape(B, width)).cuda()
        kv = torch.randn((c["bufs"], P, c["Hkv"], page, c["D"]), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["kv"] = kv if c["cache"] == "bf16" else kv.to(torch.float8_e4m3fn)
        path = np.stack([np.sort(rng.choice(np.arange(1, N), L, replace=False)) for _ in range(B)]).astype(np.int32)
        s["path"] = torch.from_numpy(np.concatenate([path, np.full((B, 2), -1, np.int32)], 1)).cuda()
        s["count"] = _ints([L + 1] * B)
        s["base"] = torch.from_numpy(base.astype(np.int32)).cuda()
        return s
    n_new = c["Q"] if c["op"] == "attention" else c["N"]
    B, H, D = c["B"], c["Hkv"], c["D"]
    if c["op"] == "attention":
        base = _spread(B, c["ctx"], c["ragged"])
        rng.shuffle(base)
        s["new_len"], new = None, [n_new] * B
    else:
        base = [int(x) for x in rng.integers(0, c["ctx"] + 1, B)]
        new = _spread(B, n_new, c["ragged"])
        rng.shuffle(new)
        s["new_len"] = _ints(new) if c["ragged"] else None
    s |= _cache(c, seed, gen, [b + n_new for b in base], c["ctx"] + n_new)
    s["base"] = _ints(base)
    if c["op"] == "attention":
        # the queries are a slice of the fused projection's output
        qkv = torch.randn((B, n_new, c["Hq"] + 2 * H, D), generator=gen, device="cuda", dtype=torch.bfloat16)
        s["q"] = (2 * qkv)[:, :, :c["Hq"]]
        s["scale"] = 1 / math.sqrt(D)
        s["tree_mask"] = _tree_words(rng, B, n_new - 1) if c["tree"] and n_new > 1 else None
        s["out"] = torch.empty((B, n_new, c["Hq"], D), dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] == "append":
        amp = torch.exp(torch.randn((H, 1), generator=gen, device="cuda"))
        kv = (torch.randn((B, n_new, 2 * H, D), generator=gen, device="cuda") * amp.repeat(2, 1)).to(_torch_dtype(c["dtype"]))
        s["key"], s["value"] = kv[:, :, :H], kv[:, :, H:]
        return s
    s["N"], s["dtype"] = n_new, _torch_dtype(c["dtype"])
    s["out_key"], s["out_value"] = (torch.zeros((B, n_new, H, D), dtype=s["dtype"], device="cuda") for _ in "kv")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["case"]["op"]
    if own:
        import speculative_decoding_verification_53_gb300 as sv
        if op == "adjust":
            return sv.spec_adjust_logits(
                s["logits"], history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"],
                draft_tokens=s["draft_tokens"], tree_mask=s["tree_mask"], repetition=s["repetition"],
                presence=s["presence"], frequency=s["frequency"], bias_tokens=s["bias_tokens"],
                bias_values=s["bias_values"], allowed=s["allowed"], out=s["out"])
        if op == "compact":
            sv.spec_kv_compact_paged(s["kv"], s["page_table"], s["path"], s["count"], s["base"])
            return s["kv"]
        if op == "append":
            sv.spec_kv_append(s["key"], s["value"], s["k_pages"], s["v_pages"], s["page_table"], s["base"],
                              new_len=s["new_len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
            return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
        if op == "read":
            return sv.spec_kv_read(s["k_pages"], s["v_pages"], s["page_table"], s["base"], s["N"],
                                   new_len=s["new_len"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                   out_key=s["out_key"], out_value=s["out_value"])
        return sv.spec_paged_attention(
            s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["base"], max_len=s["max_len"],
            tree_mask=s["tree_mask"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"],
            want_lse=True)
    return {"adjust": _adjust, "compact": _compact, "append": _append, "read": _read, "attention": _attention}[op](s)


def _bits(words, n):
    """The first n bits of each row of int32 words, as truth values."""
    b = (words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    return b.flatten(-2)[..., :n] != 0


def _adjust(s):
    logits = s["logits"]
    B, R, V = logits.shape
    H = s["history"].shape[1]
    at = torch.arange(H, device="cuda")[None]
    inside = at < s["history_len"][:, None]
    output = inside & (at >= s["prompt_len"][:, None])
    hist = s["history"].long()
    zero = torch.zeros((B, V), device="cuda")
    counts = zero.scatter_add(1, hist, output.float())[:, None]
    seen = zero.scatter_add(1, hist, inside.float())[:, None] > 0
    if R > 1:
        N = R - 1
        see = torch.zeros((B, R, N), device="cuda")
        if s["tree_mask"] is not None:
            see[:, 1:] = _bits(s["tree_mask"], N).float()
        else:
            see[:] = (torch.arange(N, device="cuda")[None] < torch.arange(R, device="cuda")[:, None]).float()
        drafted = torch.zeros((B, R, V), device="cuda")
        drafted.scatter_add_(2, s["draft_tokens"].long()[:, None].expand(B, R, N), see)
        counts = counts + drafted
    seen = seen | (counts > 0)
    rep, pres, freq = (s[k][:, None, None] for k in ("repetition", "presence", "frequency"))
    x = logits.float()
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * counts - pres * (counts > 0).float()
    if s["bias_tokens"] is not None:
        x = x + zero.scatter(1, s["bias_tokens"].long(), s["bias_values"])[:, None]
    if s["allowed"] is not None:
        x = x.masked_fill(~_bits(s["allowed"], V), -math.inf)
    s["out"].copy_(x)
    return s["out"]


def _places(s, pos):
    """Page and slot of each position [B][N]."""
    page = s["k_pages"].shape[2]
    return s["page_table"].gather(1, pos // page).long(), pos % page


def _as_bytes(pages):
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def _append(s):
    B, N = s["key"].shape[:2]
    at = torch.arange(N, device="cuda")[None]
    page, slot = _places(s, s["base"].long()[:, None] + at)
    held = (at < s["new_len"][:, None])[:, :, None] if s["new_len"] is not None else torch.ones((1, N, 1), dtype=torch.bool, device="cuda")

    def write(x, pages, scales):
        flat = _as_bytes(pages)
        if scales is None:
            new = x.to(pages.dtype)
        else:
            x = x.float()
            scale = (x.abs().amax(-1) / E4M3_MAX).clamp(min=SCALE_MIN)
            new = (x / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(pages.dtype).view(torch.uint8)
            scales[page, :, slot] = torch.where(held, scale, scales[page, :, slot])
        flat[page, :, slot] = torch.where(held[..., None], new, flat[page, :, slot])

    write(s["key"], s["k_pages"], s["k_scale"])
    write(s["value"], s["v_pages"], s["v_scale"])
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _values(pages, scales, page, slot):
    """fp32 values [B][n][heads][dim] of the positions in the given pages and slots."""
    x = _as_bytes(pages)[page, :, slot].view(pages.dtype).float()
    return x if scales is None else x * scales[page, :, slot][..., None]


def _read(s):
    at = torch.arange(s["N"], device="cuda")[None]
    page, slot = _places(s, s["base"].long()[:, None] + at)
    for pages, scales, out in ((s["k_pages"], s["k_scale"], s["out_key"]), (s["v_pages"], s["v_scale"], s["out_value"])):
        x = _values(pages, scales, page, slot).to(out.dtype)
        out.copy_(x if s["new_len"] is None else torch.where((at < s["new_len"][:, None])[:, :, None, None], x, out))
    return s["out_key"], s["out_value"]


def _visible(s, n):
    """[B][Q][n]: whether query i sees position p."""
    B, Q = s["q"].shape[:2]
    new = torch.arange(n, device="cuda")[None] - s["base"].long()[:, None]  # index among the new tokens
    if s["tree_mask"] is None:
        return new[:, None] <= torch.arange(Q, device="cuda")[None, :, None]
    tree = torch.zeros((B, Q, Q), dtype=torch.bool, device="cuda")
    tree[:, :, 0] = True
    tree[:, 1:, 1:] = _bits(s["tree_mask"], Q - 1)
    inside = (new >= 0) & (new < Q)
    own_part = tree.gather(2, new.clamp(0, Q - 1)[:, None].expand(B, Q, n))
    return (new < 0)[:, None] | (inside[:, None] & own_part)


def _attention(s):
    q, n = s["q"], s["max_len"]
    B, Q, Hq, D = q.shape
    H = s["k_pages"].shape[1]
    pos = torch.arange(n, device="cuda")[None].expand(B, n)
    held = pos < (s["base"].long()[:, None] + Q)
    page, slot = _places(s, torch.where(held, pos, torch.zeros_like(pos)))
    k = _values(s["k_pages"], s["k_scale"], page, slot)
    v = _values(s["v_pages"], s["v_scale"], page, slot)
    x = q.float().view(B, Q, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    scores = (x @ k.permute(0, 2, 3, 1)).view(B, H, Hq // H, Q, n).mul_(s["scale"])
    scores.masked_fill_(~(_visible(s, n) & held[:, None])[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    weight = scores.sub_(top).exp_()
    total = weight.sum(-1, keepdim=True)
    out = (weight.view(B, H, -1, n) @ v.permute(0, 2, 1, 3)).view(B, H, Hq // H, Q, D) / total
    lse = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(B, Q, Hq)
    s["out"].copy_(out.permute(0, 3, 1, 2, 4).reshape(B, Q, Hq, D))
    return s["out"], lse


def _compact(s):
    L, page = s["case"]["L"], s["kv"].shape[3]
    kv = _as_bytes(s["kv"])

    def places(rows):
        pos = s["base"].long()[:, None] + rows
        return s["page_table"].gather(1, pos // page).long(), pos % page

    p, t = places(s["path"][:, :L].long())
    moved = kv[:, p, :, t]
    p, t = places(torch.arange(L, device="cuda")[None])
    kv[:, p, :, t] = moved
    return s["kv"]


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    if c["op"] == "adjust":
        es = 2 if c["dtype"] == "bf16" else 4
        rows = c["B"] * c["R"]
        hist = sum(_spread(c["B"], c["H"], True))
        bits = rows * ((c["V"] + 31) // 32) * 4 if c["grammar"] else 0
        return {"bytes": 2 * rows * c["V"] * es + bits + 4 * hist + 8 * c["B"] * c["bias"], "flops": rows * c["V"]}
    row = c["Hkv"] * c["D"]
    if c["op"] == "compact":
        return {"bytes": 2 * c["B"] * c["L"] * c["bufs"] * row * (2 if c["cache"] == "bf16" else 1), "flops": 0}
    held = 2 * (row * 2 if c["cache"] == "bf16" else row + 4 * c["Hkv"])  # bytes of one position's key and value
    if c["op"] in ("append", "read"):
        n = sum(_spread(c["B"], c["N"], c["ragged"]))
        return {"bytes": n * (held + 2 * row * (2 if c["dtype"] == "bf16" else 4)), "flops": 2 * n * row}
    base, Q = _spread(c["B"], c["ctx"], c["ragged"]), c["Q"]
    pairs = sum(b * Q + Q * (Q + 1) // 2 for b in base)
    return {"bytes": sum(b + Q for b in base) * held + c["B"] * Q * c["Hq"] * (4 * c["D"] + 4),
            "flops": 4 * c["D"] * c["Hq"] * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    return {"adjust": _exact_adjust, "append": _exact_append, "read": _exact_read, "attention": _exact_attention,
            "compact": _exact_compact}[case["op"]](s)


def _exact_adjust(s):
    """Row by row in float64 on the host, from the token lists."""
    x = s["logits"].double().cpu().numpy()
    B, R, V = x.shape
    hist, n, pl = (s[k].cpu().numpy() for k in ("history", "history_len", "prompt_len"))
    rep, pres, freq = (s[k].double().cpu().numpy() for k in ("repetition", "presence", "frequency"))
    drafts = s["draft_tokens"].cpu().numpy() if R > 1 else None
    mask = s["tree_mask"].cpu().numpy().view(np.uint32) if s["tree_mask"] is not None else None
    words = s["allowed"].cpu().numpy().view(np.uint8) if s["allowed"] is not None else None
    for b in range(B):
        once = np.bincount(hist[b, pl[b]:n[b]], minlength=V)
        prompt = set(hist[b, :pl[b]].tolist())
        for r in range(R):
            if r == 0:
                nodes = []
            elif mask is None:
                nodes = list(range(r))
            else:
                nodes = [j for j in range(R - 1) if mask[b, r - 1, j // 32] >> np.uint32(j % 32) & 1]
            c = once.copy()
            for j in nodes:
                c[drafts[b, j]] += 1
            t = np.array(sorted(prompt | set(np.nonzero(c)[0].tolist())), np.int64)
            row = x[b, r]
            if t.size:
                row[t] = np.where(row[t] > 0, row[t] / rep[b], row[t] * rep[b])
                row[t] -= freq[b] * c[t] + pres[b] * (c[t] > 0)
        if s["bias_tokens"] is not None:
            x[b][:, s["bias_tokens"][b].cpu().numpy()] += s["bias_values"][b].double().cpu().numpy()
        if words is not None:
            ok = np.unpackbits(words[b], axis=-1, bitorder="little")[:, :V]
            x[b][ok == 0] = -np.inf
    return x


def _each_position(s, count):
    """(b, positions, pages, slots) of the first count[b] positions from the base, by the page table."""
    table, base, page = s["page_table"].cpu().numpy(), s["base"].cpu().numpy(), s["k_pages"].shape[2]
    for b in range(len(base)):
        pos = np.arange(base[b], base[b] + count[b])
        yield b, torch.from_numpy(table[b, pos // page].astype(np.int64)).cuda(), torch.from_numpy(pos % page).cuda()


def _counts(s, n):
    return [n] * len(s["base"]) if s["new_len"] is None else s["new_len"].tolist()


def _exact_append(s):
    quantised = s["k_scale"] is not None
    got = [t.double() if t is not None else None for t in (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])]
    n = _counts(s, s["key"].shape[1])
    for b, p, t in _each_position(s, n):
        for k, x in enumerate((s["key"], s["value"])):
            x = x[b, :n[b]].double()
            if quantised:
                scale = torch.amax(torch.abs(x), -1) / E4M3_MAX
                got[2 + k].index_put_((p[:, None], torch.arange(x.shape[1], device="cuda")[None], t[:, None]), scale)
                x = x / scale[..., None]
            got[k].index_put_((p[:, None], torch.arange(x.shape[1], device="cuda")[None], t[:, None]), x)
    return tuple(got)


def _wide(pages, scales, p, t):
    """float64 values [heads][n][dim]."""
    x = torch.stack([pages[:, h].double()[p, t] for h in range(pages.shape[1])])
    return x if scales is None else x * torch.stack([scales[:, h].double()[p, t] for h in range(pages.shape[1])])[..., None]


def _exact_read(s):
    got = [torch.zeros(t.shape, dtype=torch.float64, device="cuda") for t in (s["out_key"], s["out_value"])]
    n = _counts(s, s["N"])
    for b, p, t in _each_position(s, n):
        for k, (pages, scales) in enumerate(((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"]))):
            got[k][b, :n[b]] = _wide(pages, scales, p, t).transpose(0, 1)
    return tuple(got)


def _exact_attention(s):
    c = s["case"]
    B, Q, Hq, D = s["q"].shape
    g = Hq // c["Hkv"]
    out = torch.zeros((B, Q, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Q, Hq), dtype=torch.float64, device="cuda")
    base = s["base"].tolist()
    zero = dict(s, base=torch.zeros_like(s["base"]), new_len=None)
    for b, p, t in _each_position(zero, [x + Q for x in base]):
        n = base[b] + Q
        see = torch.ones((Q, n), dtype=torch.bool, device="cuda")
        if s["tree_mask"] is None:
            see[:, base[b]:] = torch.tril(torch.ones((Q, Q), device="cuda")) > 0
        else:
            words = s["tree_mask"][b].cpu().numpy().view(np.uint8)
            tree = np.zeros((Q, Q), bool)
            tree[:, 0] = True
            tree[1:, 1:] = np.unpackbits(words, axis=-1, bitorder="little")[:, :Q - 1] != 0
            see[:, base[b]:] = torch.from_numpy(tree).cuda()
        for h in range(c["Hkv"]):
            k, v = (_wide(x[:, h:h + 1], None if y is None else y[:, h:h + 1], p, t)[0]
                    for x, y in ((s["k_pages"], s["k_scale"]), (s["v_pages"], s["v_scale"])))
            for j in range(h * g, (h + 1) * g):
                z = (s["q"][b, :, j].double() @ k.T) * s["scale"]
                z = torch.where(see, z, torch.full_like(z, -math.inf))
                lse[b, :, j] = torch.logsumexp(z, -1)
                out[b, :, j] = torch.exp(z - lse[b, :, j][:, None]) @ v
    return out, lse


def _exact_compact(s):
    """The copies in path order, one after the other."""
    kv, page = s["kv"].clone(), s["kv"].shape[3]
    table, path, base = (s[k].cpu().numpy() for k in ("page_table", "path", "base"))
    raw = _as_bytes(kv)
    for b in range(len(base)):
        for d in range(s["case"]["L"]):
            a, z = base[b] + path[b, d], base[b] + d
            raw[:, table[b, z // page], :, z % page] = raw[:, table[b, a // page], :, a % page]
    return kv
