"""Cases of long contexts on a paged key/value cache, for timing and comparison.

Six operators around a verification round: page tables that grow and shrink with their rows and the slots of new
tokens, rotary positions of queries and keys (chains, or draft trees by depth), the same with the keys and values
written into cache pages, summaries of the pages' keys, the pages that a cheap score against those summaries selects,
and attention over the selected pages.  ``run`` computes each in plain torch operations, or through the package where
``own`` is true.
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
        # a batch of chains: each grows by six tokens, what was not accepted is given back: latency counts
        dict(name="pages chains", op="pages", B=8, N=6, page=16, ctx=4000, turn=0.0, short=False),
        # prompts enter a large pool while other rows leave it
        dict(name="pages prompts", op="pages", B=128, N=8192, page=16, ctx=20000, turn=0.3, short=False),
        # one token of one conversation: the smallest call
        dict(name="rotary one token", op="rotary", B=1, N=1, Hq=32, Hkv=8, D=128, rot=128, far=130000, dtype="bf16",
             tree=False, interleaved=False, scaled=True),
        # chunks of prompts, part of each head, neighbouring elements paired
        dict(name="rotary prompts", op="rotary", B=4, N=6001, Hq=32, Hkv=8, D=128, rot=64, far=8000, dtype="bf16",
             tree=False, interleaved=True, scaled=False),
        # a batch of draft trees enters a quantised cache, one layer
        dict(name="rotary append trees", op="rotary_append", B=16, N=61, Hq=32, Hkv=8, D=128, rot=128, page=64,
             far=30000, cache="e4m3", dtype="bf16", tree=True, interleaved=False, scaled=True, ragged=False, nhd=False),
        # prompts enter the cache in chunks
        dict(name="rotary append prompts", op="rotary_append", B=16, N=2048, Hq=32, Hkv=8, D=128, rot=128, page=64,
             far=1000, cache="bf16", dtype="bf16", tree=False, interleaved=False, scaled=False, ragged=True, nhd=True),
        # the pages that a round of chains has written to
        dict(name="summary chains", op="summary", B=8, N=6, Hkv=8, D=128, page=64, ctx=4000, cache="bf16",
             kind="mean", ragged=False, nhd=False),
        # whole contexts of a quantised cache, bounds of every element
        dict(name="summary contexts", op="summary", B=8, N=8192, Hkv=8, D=128, page=64, ctx=0, cache="e4m3",
             kind="bounds", ragged=True, nhd=False),
        # one conversation of 100 thousand tokens, one new token
        dict(name="select one token", op="select", B=1, Q=1, Hq=32, Hkv=8, D=128, page=64, ctx=100001, kind="mean",
             top=64, shared=False, ragged=False),
        # chains of five drafts and the last token: each query selects for itself, by bounds
        dict(name="select chains", op="select", B=32, Q=6, Hq=32, Hkv=8, D=128, page=32, ctx=32768, kind="bounds",
             top=64, shared=False, ragged=True),
        # the same chains' attention, every query over its own pages
        dict(name="sparse chains", op="sparse", B=8, Q=6, Hq=32, Hkv=8, D=128, page=64, ctx=32768, top=32,
             cache="bf16", tree=False, shared=False, ragged=True, nhd=False),
        # 60-node trees whose queries share the selected pages of a quantised cache
        dict(name="sparse trees", op="sparse", B=16, Q=61, Hq=32, Hkv=8, D=128, page=64, ctx=32768, top=64,
             cache="e4m3", tree=True, shared=True, ragged=True, nhd=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(("pages", "rotary", "rotary_append", "summary", "select", "select", "sparse", "sparse"))
    page = rng.choice((8, 16, 16, 24, 32, 64, 64, 128))
    if op == "pages":
        B = _log_int(rng, 1, 256)
        return dict(op=op, B=B, N=_log_int(rng, 1, max(1, min(16384, 1_000_000 // B))), page=page,
                    ctx=_log_int(rng, 1, 30000), turn=rng.choice((0.0, 0.1, 0.5)), short=rng.random() < 0.15)
    Hkv = rng.choice((1, 2, 3, 4, 8, 8, 16))
    g = rng.choice((1, 2, 4, 4, 7, 8))
    D = rng.choice((64, 64, 96, 128, 128, 128, 256))
    cache = rng.choice(("bf16", "e4m3"))
    nhd = rng.random() < 0.5
    ragged = rng.random() < 0.7
    kind = rng.choice(("mean", "bounds"))
    if op in ("rotary", "rotary_append"):
        tree = rng.random() < 0.4
        B = _log_int(rng, 1, 64)
        N = _log_int(rng, 2, 129) if tree else _log_int(rng, 1, max(1, min(8192, 100_000_000 // (B * Hkv * (g + 2) * D))))
        c = dict(op=op, B=B, N=N, Hq=Hkv * g, Hkv=Hkv, D=D, rot=rng.choice((D, D, D // 2, D // 4, 20)),
                 far=_log_int(rng, 1, 1_000_000 if op == "rotary" else 30000), dtype=rng.choice(("bf16", "bf16", "fp32")),
                 tree=tree, interleaved=rng.random() < 0.4, scaled=rng.random() < 0.5)
        return c if op == "rotary" else c | dict(page=page, cache=cache, ragged=ragged, nhd=nhd)
    if op == "summary":
        B = _log_int(rng, 1, 64)
        return dict(op=op, B=B, N=_log_int(rng, 1, max(1, min(16384, 60_000_000 // (B * Hkv * D)))), Hkv=Hkv, D=D,
                    page=page, ctx=_log_int(rng, 1, 4000), cache=cache, kind=kind, ragged=ragged, nhd=nhd)
    shared = rng.random() < 0.5
    Q = rng.choice((1, 1, rng.randint(2, 9), rng.randint(2, 17), _log_int(rng, 3, 129 if shared else 33)))
    top = _log_int(rng, 2, 128)
    if op == "select":
        B = _log_int(rng, 1, 32)
        blocks = _log_int(rng, 32, max(32, min(8192, 400_000_000 // (B * Q * Hkv * g * D), 20_000_000 // (B * Hkv * D))))
        return dict(op=op, B=B, Q=Q, Hq=Hkv * g, Hkv=Hkv, D=D, page=page, ctx=blocks * page + rng.randrange(page),
                    kind=kind, top=_log_int(rng, 6, min(128, blocks // 4)), shared=shared, ragged=ragged)
    B = _log_int(rng, 1, 16)
    lists = B * Hkv * (1 if shared else Q)
    top = max(2, min(top, 100_000_000 // (lists * page * D), 130_000_000 // (B * Hkv * g * Q * page)))
    ctx = _log_int(rng, 1, max(2, min(200_000, 500_000_000 // (B * Hkv * D))))
    return dict(op=op, B=B, Q=Q, Hq=Hkv * g, Hkv=Hkv, D=D, page=page, ctx=ctx, top=top, cache=cache,
                tree=Q > 2 and rng.random() < 0.5, shared=shared, ragged=ragged, nhd=nhd)


# ------------------------------------------------------------------ inputs

def _spread(B, hi, ragged):
    """Lengths of the batch rows: all `hi`, or spread evenly from `hi` down to about a quarter of it."""
    if not ragged or B == 1:
        return [hi] * B
    return [hi - (b * (hi - (hi + 3) // 4)) // (B - 1) for b in range(B)]


def _torch_dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}[name]


def _ints(v, dtype=torch.int32):
    return torch.tensor(np.asarray(v), dtype=dtype, device="cuda")


def _trees(rng, B, N):
    """Parents of random draft trees (children of one of the few nodes before) int64 [B][N]."""
    parent = np.zeros((B, N), np.int64)
    for i in range(N):
        parent[:, i] = rng.integers(-1 if i < 4 else max(-1, i // 2 - 3), i, B)
    return parent


def _tree_depth(parent):
    depth = np.zeros(parent.shape, np.int32)
    for i in range(parent.shape[1]):
        p = parent[:, i]
        depth[:, i] = 1 + np.where(p >= 0, depth[np.arange(len(p)), np.maximum(p, 0)], 0)
    return depth


def _tree_words(parent):
    """Ancestor-or-self bits int32 [B][N][ceil(N/32)]."""
    B, N = parent.shape
    bits = np.zeros((B, N, (N + 31) // 32 * 32), np.uint8)
    for i in range(N):
        p = parent[:, i]
        has = p >= 0
        bits[has, i] = bits[np.nonzero(has)[0], p[has]]
        bits[:, i, i] = 1
    return torch.from_numpy(np.packbits(bits, axis=2, bitorder="little").view(np.int32)).cuda()


def _table(rng, need, width, P):
    """A shuffled page table that holds need[b] pages of row b."""
    perm = rng.permutation(P).astype(np.int32)
    table = np.full((len(need), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return torch.from_numpy(table).cuda()


def _cache(c, rng, gen, lens, most):
    """A pool of pages for rows of up to `most` positions, its scales, and a page table that holds lens[b] positions of
    row b."""
    page, H, D = c["page"], c["Hkv"], c["D"]
    need = [(n + page - 1) // page for n in lens]
    width = (most + page - 1) // page
    P = (sum(need) if c["op"] == "sparse" else len(lens) * width) + 3
    shape = (P, page, H, D) if c.get("nhd") else (P, H, page, D)

    def pages():
        x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
        if c["cache"] == "e4m3":
            x = (x * 110).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return x.permute(0, 2, 1, 3) if c.get("nhd") else x

    s = dict(k_pages=pages(), v_pages=pages(), page_table=_table(rng, need, width, P - 1), k_scale=None, v_scale=None)
    if c["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = ((0.5 + torch.rand((P, H, page), generator=gen, device="cuda")) / 110 for _ in "kv")
    return s


def _lists(c, rng, full):
    """Lists of blocks int32 [B][Q or 1][H][top], ascending, -1 behind; full[b]: blocks before the new tokens.  The
    first and the last block are always there; queries of a row share three quarters of the others."""
    B, H, top, Q = c["B"], c["Hkv"], c["top"], 1 if c["shared"] else c["Q"]
    out = np.full((B, Q, H, top), -1, np.int32)
    for b, n in enumerate(full):
        if n <= top:
            out[b, :, :, :n] = np.arange(n)
            continue
        for h in range(H):
            perm = rng.permutation(n - 2) + 1
            free = top - 2
            common = _common(free)
            for i in range(Q):
                rest = perm[common:]
                mine = rest[rng.choice(len(rest), free - common, replace=False)] if Q > 1 else rest[:free - common]
                out[b, i, h] = np.sort(np.concatenate([[0, n - 1], perm[:common], mine]))
    return torch.from_numpy(out).cuda()


def _common(free):
    return free - free // 4


def _angles(c):
    """Radians per position of each pair, in 64 bits; by parts interpolated for long contexts where scaled."""
    rot = c["rot"]
    f = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
    if c["scaled"]:  # slow pairs go four times slower, fast ones stay, what is between is blended
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1) / (32 - 1), 0, 1)
        f = f * keep + f / 4 * (1 - keep)
    return torch.from_numpy(f).cuda()


def prepare(case, seed):
    c = case
    rng = np.random.default_rng([seed, 7])
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    B = c["B"]
    if c["op"] == "pages":
        page, N = c["page"], c["N"]
        held = rng.permutation(_spread(B, c["ctx"], True))
        new = rng.integers((N + 1) // 2, N + 1, B)
        gone = rng.random(B) < c["turn"]  # rows that end
        need = (held + page - 1) // page
        grown = np.where(gone, 0, held + new)
        width = int((c["ctx"] + N + page - 1) // page)
        P = int(need.sum()) + B * N // (2 * page) + 1 if c["short"] else B * width + 5
        table = _table(rng, need, width, P)
        free = np.setdiff1d(np.arange(P), table.cpu().numpy())
        rng.shuffle(free)
        s["page_table"], s["pages"] = table, _ints(need)
        s["free_pages"] = _ints(np.concatenate([free, np.full(P - len(free), -1)]))
        s["free_count"] = _ints([len(free)])
        s["held"], s["grown"], s["base"] = _ints(held), _ints(grown), _ints(held)
        s["ok"] = [torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(2)]
        s["slots"] = torch.zeros((B, N), dtype=torch.int64, device="cuda")
        return s
    Hkv, D = c["Hkv"], c["D"]
    if c["op"] in ("rotary", "rotary_append"):
        N, Hq, dt = c["N"], c["Hq"], _torch_dtype(c["dtype"])
        # queries, keys and values are slices of the fused projection's output
        amp = torch.exp(0.5 * torch.randn((Hq + 2 * Hkv, 1), generator=gen, device="cuda"))
        qkv = (torch.randn((B, N, Hq + 2 * Hkv, D), generator=gen, device="cuda") * amp).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
        s["freq"] = _angles(c)
        s["amplitude"] = 1.1 if c["scaled"] else 1.0
        s["depth"] = _ints(_tree_depth(_trees(rng, B, N - 1))) if c["tree"] and N > 1 else None
        base = rng.integers(0, c["far"] + 1, B)
        s["base"] = _ints(base)
        s["out"] = torch.zeros((B, N, Hq, D), dtype=dt, device="cuda")
        if c["op"] == "rotary":
            s["out_k"] = torch.zeros((B, N, Hkv, D), dtype=dt, device="cuda")
            return s
        new = _spread(B, N, c["ragged"])
        rng.shuffle(new)
        s["new_len"] = _ints(new) if c["ragged"] else None
        # a pool that holds the new tokens' pages; those of the positions before are not touched
        page = c["page"]
        first, last = base // page, (base + new + page - 1) // page
        P = B * ((N + page - 1) // page + 1) + 3
        table = np.full((B, (c["far"] + N + page - 1) // page), -1, np.int32)
        perm, at = rng.permutation(P - 1), 0
        for b in range(B):
            table[b, first[b]:last[b]] = perm[at:at + last[b] - first[b]]
            at += last[b] - first[b]
        s |= _cache(c, rng, gen, [page * (P - 3)], page * (P - 3))
        s["page_table"] = torch.from_numpy(table).cuda()
        return s
    if c["op"] == "summary":
        base = rng.integers(0, c["ctx"] + 1, B)
        new = _spread(B, c["N"], c["ragged"])
        rng.shuffle(new)
        s["new_len"] = _ints(new) if c["ragged"] else None
        s |= _cache(c, rng, gen, [int(b) + n for b, n in zip(base, new)], c["ctx"] + c["N"])
        s["base"] = _ints(base)
        P = s["k_pages"].shape[0]
        s["summary"] = torch.zeros((P, Hkv, D * (2 if c["kind"] == "bounds" else 1)), dtype=torch.bfloat16, device="cuda")
        return s
    base = _spread(B, c["ctx"], c["ragged"])
    rng.shuffle(base)
    s["base"] = _ints(base)
    qkv = torch.randn((B, c["Q"], c["Hq"] + 2 * Hkv, D), generator=gen, device="cuda", dtype=torch.bfloat16)
    s["q"] = (2 * qkv)[:, :, :c["Hq"]]
    page = c["page"]
    if c["op"] == "select":
        need = [(n + c["Q"] + page - 1) // page for n in base]
        P = sum(need) + 3
        s["page_table"] = _table(rng, need, max(need), P)
        x = 0.3 * torch.randn((P, Hkv, D), generator=gen, device="cuda")
        if c["kind"] == "bounds":
            x = torch.cat([x + 2 + 0.5 * torch.rand(x.shape, generator=gen, device="cuda"),
                           x - 2 - 0.5 * torch.rand(x.shape, generator=gen, device="cuda")], -1)
        s["summary"] = x.to(torch.bfloat16)
        s["blocks"] = torch.zeros((B, 1 if c["shared"] else c["Q"], Hkv, c["top"]), dtype=torch.int32, device="cuda")
        return s
    s |= _cache(c, rng, gen, [n + c["Q"] for n in base], c["ctx"] + c["Q"])
    s["blocks"] = _lists(c, rng, [n // page for n in base])
    s["scale"] = 1 / math.sqrt(D)
    s["tree_mask"] = _tree_words(_trees(rng, B, c["Q"] - 1)) if c["tree"] and c["Q"] > 1 else None
    s["out"] = torch.empty((B, c["Q"], c["Hq"], D), dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    c = s["case"]
    op = c["op"]
    if own:
        import speculative_decoding_verification_53_gb300 as sv
        if op == "pages":
            sv.spec_page_resize(s["page_table"], s["pages"], s["grown"], s["free_pages"], s["free_count"], c["page"],
                                base=s["base"], out_slots=s["slots"], out_ok=s["ok"][0])
            sv.spec_page_resize(s["page_table"], s["pages"], s["held"], s["free_pages"], s["free_count"], c["page"],
                                out_ok=s["ok"][1])
            return s["ok"], s["slots"], s["page_table"], s["pages"], s["free_pages"], s["free_count"]
        if op == "rotary":
            return sv.spec_rotary(s["q"], s["freq"], s["base"], key=s["k"], tree_depth=s["depth"],
                                  interleaved=c["interleaved"], amplitude=s["amplitude"], out=s["out"], out_key=s["out_k"])
        if op == "rotary_append":
            sv.spec_rotary_append(s["q"], s["k"], s["v"], s["freq"], s["k_pages"], s["v_pages"], s["page_table"],
                                  s["base"], tree_depth=s["depth"], new_len=s["new_len"], k_scale=s["k_scale"],
                                  v_scale=s["v_scale"], interleaved=c["interleaved"], amplitude=s["amplitude"], out=s["out"])
            return s["out"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
        if op == "summary":
            return sv.spec_block_summary(s["k_pages"], s["page_table"], s["base"], c["N"], kind=c["kind"],
                                         new_len=s["new_len"], k_scale=s["k_scale"], summary=s["summary"])
        if op == "select":
            return sv.spec_block_select(s["q"], s["summary"], s["page_table"], s["base"], c["page"], c["top"],
                                        kind=c["kind"], shared=c["shared"], out=s["blocks"])
        return sv.spec_sparse_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["base"], s["blocks"],
                                        tree_mask=s["tree_mask"], scale=s["scale"], k_scale=s["k_scale"],
                                        v_scale=s["v_scale"], out=s["out"], want_lse=True)
    return {"pages": _pages, "rotary": _rotary, "rotary_append": _rotary_append, "summary": _summary,
            "select": _select, "sparse": _sparse}[op](s)


def _resize(s, length, ok):
    """Every row holds the pages of its length: those too many go onto the stack of free pages, row by row, then rows
    take what they lack from its top, in their order, until one finds too few; that row and later ones that need
    pages stay as they are."""
    table, pages, stack, count, page = s["page_table"], s["pages"], s["free_pages"], s["free_count"], s["case"]["page"]
    P, width = stack.shape[0], table.shape[1]
    need = (length + page - 1) // page
    at = torch.arange(width, device="cuda")[None]
    back = (at >= need[:, None]) & (at < pages[:, None])
    place = (count.long() + back.flatten().cumsum(0) - 1).view(table.shape)
    spare = torch.cat([stack, stack[:1]])  # a last entry that takes what does not count
    spare.scatter_(0, torch.where(back, place, P).flatten(), table.flatten())
    stack.copy_(spare[:P])
    top = count.long() + back.sum()
    lack = (need - pages).clamp(min=0).long()
    ahead = lack.cumsum(0)
    fine = (lack == 0) | (ahead <= top)
    want = (at < need[:, None]) & (at >= pages[:, None]) & fine[:, None]
    index = top - 1 - (ahead - lack)[:, None] - (at - pages[:, None])
    table.copy_(torch.where(want, stack[torch.where(want, index, 0)], torch.where(back, -1, table)))
    taken = torch.where(fine, lack, 0).sum()
    count.copy_(top - taken)
    pages.copy_(torch.where(fine, need, pages))
    ok.copy_(fine)


def _pages(s):
    page, N = s["case"]["page"], s["case"]["N"]
    _resize(s, s["grown"], s["ok"][0])
    pos = s["base"].long()[:, None] + torch.arange(N, device="cuda")[None]
    there = (pos < s["grown"][:, None]) & (s["ok"][0] != 0)[:, None]
    p = s["page_table"].gather(1, torch.where(there, pos // page, 0)).long()
    s["slots"].copy_(torch.where(there, p * page + pos % page, -1))
    _resize(s, s["held"], s["ok"][1])
    return s["ok"], s["slots"], s["page_table"], s["pages"], s["free_pages"], s["free_count"]


def _turned(s, x):
    """fp32 elements of x [B][N][heads][D], the first 2 R of each head turned by their position."""
    N, R = x.shape[1], s["freq"].shape[0]
    step = torch.arange(N, device="cuda")[None].expand(x.shape[0], N)
    if s["depth"] is not None:
        step = torch.cat([torch.zeros_like(step[:, :1]), s["depth"].long()], 1)
    angle = (s["base"].long()[:, None] + step)[..., None].double() * s["freq"]  # far positions need 64 bits
    cos, sin = ((f(angle) * s["amplitude"]).float()[:, :, None] for f in (torch.cos, torch.sin))
    x = x.float()
    part, rest = x[..., :2 * R], x[..., 2 * R:]
    if s["case"]["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = part[..., :R], part[..., R:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _rotary(s):
    s["out"].copy_(_turned(s, s["q"]))
    s["out_k"].copy_(_turned(s, s["k"]))
    return s["out"], s["out_k"]


def _places(s, pos):
    """Page and slot of each position [B][N]."""
    page = s["k_pages"].shape[2]
    index = pos // page
    inside = index < s["page_table"].shape[1]
    p = s["page_table"].gather(1, torch.where(inside, index, 0)).long()
    return torch.where(inside, p, -1), pos % page


def _as_bytes(pages):
    return pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages


def _rotary_append(s):
    B, N = s["k"].shape[:2]
    at = torch.arange(N, device="cuda")[None]
    held = (at < s["new_len"][:, None])[:, :, None] if s["new_len"] is not None else torch.ones((1, N, 1), dtype=torch.bool, device="cuda")
    page, slot = _places(s, s["base"].long()[:, None] + at)
    page = torch.where(held[..., 0], page, s["k_pages"].shape[0] - 1)  # the last page is nobody's

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

    s["out"].copy_(torch.where(held[..., None], _turned(s, s["q"]), s["out"].float()))
    write(_turned(s, s["k"]), s["k_pages"], s["k_scale"])
    write(s["v"], s["v_pages"], s["v_scale"])
    return s["out"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _values(pages, scales, page, head, slot):
    """fp32 values of the given pages, heads and slots (one shape)."""
    x = _as_bytes(pages)[page, head, slot].view(pages.dtype).float()
    return x if scales is None else x * scales[page, head, slot][..., None]


def _summary(s):
    B, N, page = s["base"].shape[0], s["case"]["N"], s["case"]["page"]
    H = s["k_pages"].shape[1]
    first = s["base"].long() // page
    new = s["new_len"].long() if s["new_len"] is not None else torch.full((B,), N, device="cuda")
    end = s["base"].long() + new
    block = first[:, None] + torch.arange((N + 2 * page - 2) // page, device="cuda")[None]
    real = (block * page < end[:, None]) & (new > 0)[:, None]
    pg = s["page_table"].gather(1, torch.where(real, block, 0)).long()  # [B][blocks]
    at = torch.arange(page, device="cuda")
    held = (block[..., None] * page + at < end[:, None, None])[:, :, None, :, None]  # [B][blocks][1][page][1]
    heads = torch.arange(H, device="cuda")[:, None]
    x = _values(s["k_pages"], s["k_scale"], pg[:, :, None, None], heads, at)
    if s["case"]["kind"] == "mean":
        got = torch.where(held, x, 0).sum(3) / held.sum(3).clamp(min=1)
    else:
        got = torch.cat([torch.where(held, x, -math.inf).amax(3), torch.where(held, x, math.inf).amin(3)], -1)
    spare = s["summary"].shape[0] - 1  # the last page is nobody's
    pg = torch.where(real, pg, spare)
    s["summary"][pg] = torch.where(real[..., None, None], got, 0).to(torch.bfloat16)
    return s["summary"]


def _select(s):
    c, q, table = s["case"], s["q"], s["page_table"]
    B, Q, Hq, D = q.shape
    H, top = c["Hkv"], c["top"]
    full = s["base"].long() // c["page"]  # blocks before the new tokens
    n = table.shape[1]
    at = torch.arange(n, device="cuda")[None]
    cand = at < full[:, None]
    # scores next to the border decide: 64 bits
    m = s["summary"].double()[torch.where(cand, table.long(), 0)]  # [B][n][H][D or 2 D]
    x = q.double().view(B, Q, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    if c["kind"] == "bounds":
        x = torch.cat([x.clamp(min=0), x.clamp(max=0)], -1)
    score = (x @ m.permute(0, 2, 3, 1)).view(B, H, Q, Hq // H, n).amax(3).permute(0, 2, 1, 3)  # [B][Q][H][n]
    if c["shared"]:
        score = score.amax(1, keepdim=True)
    always = ((at < 1) | (at >= (full - 1)[:, None]))[:, None, None]
    score = torch.where(always, math.inf, score)
    score = torch.where(cand[:, None, None], score, -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :top]
    order = torch.where(torch.arange(order.shape[-1], device="cuda") < full[:, None, None, None], order, n)
    order = torch.sort(order, -1)[0]
    s["blocks"].fill_(-1)
    s["blocks"][..., :order.shape[-1]] = torch.where(order < n, order, -1).int()
    return s["blocks"]


def _bits(words, n):
    """The first n bits of each row of int32 words, as truth values."""
    b = (words[..., None] >> torch.arange(32, device=words.device, dtype=torch.int32)) & 1
    return b.flatten(-2)[..., :n] != 0


def _sparse(s):
    c, q, page = s["case"], s["q"], s["case"]["page"]
    B, Q, Hq, D = q.shape
    H, g = c["Hkv"], Hq // c["Hkv"]
    base = s["base"].long()
    at = torch.arange(page, device="cuda")
    # positions of the listed blocks, then from the block in which the new tokens begin
    lists = s["blocks"].long()  # [B][Q or 1][H][top]
    QL = lists.shape[1]
    front = (lists[..., None] * page + at).flatten(-2)
    first = (base // page * page)[:, None, None, None]
    tail = first + torch.arange(page + Q, device="cuda")
    pos = torch.cat([front, tail.expand(B, QL, H, page + Q)], -1)  # [B][QL][H][n]
    n = pos.shape[-1]
    held = (pos >= 0) & (pos < (base + Q)[:, None, None, None])
    pos = torch.where(held, pos, 0)
    pg = s["page_table"].gather(1, (pos // page).view(B, -1)).view(pos.shape).long()
    head = torch.arange(H, device="cuda")[:, None]
    k = _values(s["k_pages"], s["k_scale"], pg, head, pos % page)  # [B][QL][H][n][D]
    v = _values(s["v_pages"], s["v_scale"], pg, head, pos % page)
    new = pos - base[:, None, None, None]
    i = torch.arange(Q, device="cuda")[None, :, None, None]
    if s["tree_mask"] is None:
        see = new <= i  # [B][Q][H][n]
    else:
        tree = torch.zeros((B, Q, Q), dtype=torch.bool, device="cuda")
        tree[:, :, 0] = True
        tree[:, 1:, 1:] = _bits(s["tree_mask"], Q - 1)
        j = new.clamp(0, Q - 1)
        see = tree[torch.arange(B, device="cuda")[:, None, None, None], i, j] | (new < 0)
    see = (see & held).expand(B, Q, H, n)
    x = q.float().view(B, Q, H, g, D)
    if QL == 1:
        x = x.permute(0, 2, 1, 3, 4).reshape(B, 1, H, Q * g, D)
    scores = ((x @ k.transpose(-1, -2)) * s["scale"]).view(B, QL, H, Q // QL, g, n)
    see = see.reshape(B, QL, Q // QL, H, n).transpose(2, 3)[:, :, :, :, None]
    scores = torch.where(see, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    weight = torch.exp(scores - top)
    total = weight.sum(-1, keepdim=True)
    out = (weight.reshape(B, QL, H, -1, n) @ v).view(B, QL, H, Q // QL, g, D) / total
    lse = (top + total.log())[..., 0]
    s["out"].copy_(out.transpose(2, 3).reshape(B, Q, Hq, D))
    return s["out"], lse.transpose(2, 3).reshape(B, Q, Hq)


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    B = c["B"]
    if c["op"] == "pages":
        # the slots, and the pages of half to all of the new tokens taken and given back: table and stack
        moved = int(B * 0.75 * c["N"] / c["page"]) + 1
        return {"bytes": 8 * B * c["N"] + 4 * 4 * moved + 40 * B, "flops": 0}
    H, D = c["Hkv"], c["D"]
    if c["op"] in ("rotary", "rotary_append"):
        es = 2 if c["dtype"] == "bf16" else 4
        tokens = sum(_spread(B, c["N"], c.get("ragged", False)))
        if c["op"] == "rotary":
            moved = 2 * (c["Hq"] + H) * D * es
        else:
            moved = 2 * c["Hq"] * D * es + 2 * H * D * es + 2 * H * (2 * D if c["cache"] == "bf16" else D + 4)
        return {"bytes": tokens * moved, "flops": 3 * tokens * (c["Hq"] + H) * c["rot"]}
    if c["op"] == "summary":
        es = 2 * D if c["cache"] == "bf16" else D + 4
        tokens = sum(_spread(B, c["N"], c["ragged"]))
        out = (tokens // c["page"] + B) * H * D * (4 if c["kind"] == "bounds" else 2)
        return {"bytes": tokens * H * es + out, "flops": tokens * H * D * (2 if c["kind"] == "bounds" else 1)}
    Q, base = c["Q"], _spread(B, c["ctx"], c["ragged"])
    lists = 1 if c["shared"] else Q
    full = [n // c["page"] for n in base]
    if c["op"] == "select":
        width = 2 * D if c["kind"] == "bounds" else D
        return {"bytes": sum(full) * H * width * 2 + B * Q * c["Hq"] * D * 2 + 4 * B * lists * H * c["top"],
                "flops": 2 * sum(full) * Q * c["Hq"] * D}
    held = 2 * (2 * D if c["cache"] == "bf16" else D + 4)  # bytes of one position's key and value of one head
    free = c["top"] - 2
    common = 2 + _common(free)
    blocks = sum(min(n, common + lists * (c["top"] - common)) for n in full)  # about as many different ones
    new = B * (c["page"] // 2 + Q)
    pairs = sum(Q * (min(n, c["top"]) * c["page"] + c["page"] // 2) + Q * (Q + 1) // 2 for n in full)
    return {"bytes": (blocks * c["page"] + new) * H * held + B * Q * c["Hq"] * (4 * D + 4) + 4 * B * lists * H * c["top"],
            "flops": 4 * D * c["Hq"] * pairs}


def exact(case, seed):
    if case["op"] in ("pages", "select"):
        return None  # whole numbers
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "rotary_append": _exact_rotary_append, "summary": _exact_summary,
            "sparse": _exact_sparse}[case["op"]](s)


def _exact_turn(s, x):
    """Pairs as complex numbers, times a unit number's amplitude."""
    B, N = x.shape[:2]
    R = s["freq"].shape[0]
    depth = np.arange(N)[None].repeat(B, 0)
    if s["depth"] is not None:
        depth = np.concatenate([np.zeros((B, 1), np.int64), s["depth"].cpu().numpy()], 1)
    pos = s["base"].cpu().numpy().astype(np.float64)[:, None] + depth
    turn = torch.from_numpy(pos[..., None] * s["freq"].cpu().numpy()).cuda()
    by = torch.polar(torch.full_like(turn, s["amplitude"]), turn)[:, :, None]
    y = x.double()
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(y[..., :2 * R].reshape(*y.shape[:-1], R, 2)) * by
        first = torch.view_as_real(z).reshape(*y.shape[:-1], 2 * R)
    else:
        z = torch.complex(y[..., :R], y[..., R:2 * R]) * by
        first = torch.cat([z.real, z.imag], -1)
    return torch.cat([first, y[..., 2 * R:]], -1)


def _exact_rotary(s):
    return _exact_turn(s, s["q"]), _exact_turn(s, s["k"])


def _each_position(s, count):
    """(b, pages, slots) of the first count[b] positions from the base, by the page table."""
    table, base, page = s["page_table"].cpu().numpy(), s["base"].cpu().numpy(), s["k_pages"].shape[2]
    for b in range(len(base)):
        pos = np.arange(base[b], base[b] + count[b])
        yield b, torch.from_numpy(table[b, pos // page].astype(np.int64)).cuda(), torch.from_numpy(pos % page).cuda()


def _counts(s, n):
    return [n] * len(s["base"]) if s["new_len"] is None else s["new_len"].tolist()


def _exact_rotary_append(s):
    q = _exact_turn(s, s["q"])
    key = _exact_turn(s, s["k"])
    got = [t.double() if t is not None else None for t in (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])]
    n = _counts(s, key.shape[1])
    out = torch.zeros_like(q)
    for b, p, t in _each_position(s, n):
        out[b, :n[b]] = q[b, :n[b]]
        for i, x in enumerate((key[b, :n[b]], s["v"][b, :n[b]].double())):
            at = (p[:, None], torch.arange(x.shape[1], device="cuda")[None], t[:, None])
            if s["k_scale"] is not None:
                scale = torch.amax(torch.abs(x), -1) / E4M3_MAX
                got[2 + i].index_put_(at, scale)
                x = x / scale[..., None]
            got[i].index_put_(at, x)
    return (out, *got)


def _exact_summary(s):
    c, page = s["case"], s["case"]["page"]
    table, base = s["page_table"].cpu().numpy(), s["base"].cpu().numpy()
    out = torch.zeros(s["summary"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_counts(s, c["N"])):
        end = int(base[b]) + n
        for j in range(base[b] // page, (end + page - 1) // page if n else 0):
            p, m = int(table[b, j]), min(page, end - j * page)
            x = s["k_pages"][p, :, :m].double()
            if s["k_scale"] is not None:
                x = x * s["k_scale"][p, :, :m].double()[..., None]
            out[p] = x.mean(1) if c["kind"] == "mean" else torch.cat([x.max(1)[0], x.min(1)[0]], -1)
    return out


def _exact_sparse(s):
    """List by list, over the positions that it names and those from the block of the first new token on."""
    c, page = s["case"], s["case"]["page"]
    B, Q, Hq, D = s["q"].shape
    g = Hq // c["Hkv"]
    table, base, lists = (s[k].cpu().numpy() for k in ("page_table", "base", "blocks"))
    if lists.shape[0] * lists.shape[1] * lists.shape[2] > 8000:
        return None
    out = torch.zeros((B, Q, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, Q, Hq), dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(base[b]) + Q
        see = np.tril(np.ones((Q, Q), bool))
        if s["tree_mask"] is not None:
            see = np.zeros((Q, Q), bool)
            see[:, 0] = True
            see[1:, 1:] = np.unpackbits(s["tree_mask"][b].cpu().numpy().view(np.uint8), axis=-1, bitorder="little")[:, :Q - 1] != 0
        start = int(base[b]) // page * page
        for y in range(lists.shape[1]):
            rows = range(Q) if lists.shape[1] == 1 else range(y, y + 1)
            for h in range(c["Hkv"]):
                mine = lists[b, y, h]
                pos = np.concatenate([(j * page + np.arange(page)) for j in mine[mine >= 0]] + [np.arange(start, n)])
                p = torch.from_numpy(table[b, pos // page].astype(np.int64)).cuda()
                t = torch.from_numpy(pos % page).cuda()
                k, v = (x.view(torch.uint8 if s["k_scale"] is not None else x.dtype)[:, h][p, t].view(x.dtype).double()
                        for x in (s["k_pages"], s["v_pages"]))
                if s["k_scale"] is not None:
                    k, v = k * s["k_scale"][p, h, t].double()[:, None], v * s["v_scale"][p, h, t].double()[:, None]
                mask = np.ones((len(rows), len(pos)), bool)
                mask[:, len(pos) - Q:] = see[list(rows)]
                x = s["q"][b, list(rows), h * g:(h + 1) * g].double() @ k.T * s["scale"]
                x = x.masked_fill(torch.from_numpy(~mask).cuda()[:, None], -math.inf)
                z = torch.logsumexp(x, -1)
                lse[b, list(rows), h * g:(h + 1) * g] = z
                out[b, list(rows), h * g:(h + 1) * g] = torch.exp(x - z[..., None]) @ v
    return out, lse
