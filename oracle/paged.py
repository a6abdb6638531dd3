"""Plain float64 forms of a verification round on a paged cache (test infrastructure).

Written from the definitions in ``include/spec_paged_kv.h`` and ``include/spec_logits.h``
with numpy on the host, token by token where that keeps them obvious.  They share no code
with the CUDA library.  Cache pages are arrays [pages][heads][page_size][head_dim] of
values (codes already decoded), scales [pages][heads][page_size].
"""
import numpy as np

E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126


def e4m3_values():
    """The value of each of the 256 codes: sign, 4 bits of exponent (bias 7), 3 of mantissa."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v[(c & 127) == 127] = np.nan
    return np.where(c >= 128, -v, v)


def place(table, b, pos, num_pages, page_size):
    """(page, row) of a position; page -1 in a hole."""
    p = int(table[b, pos // page_size])
    return (p if 0 <= p < num_pages else -1), pos % page_size


def row_ok(table, base, new_len, b, N, page_size):
    n = N if new_len is None else int(new_len[b])
    return base[b] >= 0 and 0 <= n <= N and int(base[b]) + n <= table.shape[1] * page_size, n


def quantise(x):
    """(x / scale before rounding, scale) of rows [..., D]; infinities count as the largest code."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    s = np.maximum(a / E4M3_MAX, SCALE_MIN)
    return np.clip(x / s[..., None], -E4M3_MAX, E4M3_MAX), s


def append(x, pages, scales, table, base, new_len):
    """Copies of pages (and scales) with the unrounded elements of x [B][N][H][D] written in."""
    B, N = x.shape[:2]
    P, _, ps, _ = pages.shape
    pages = np.array(pages, np.float64)
    scales = None if scales is None else np.array(scales, np.float64)
    for b in range(B):
        ok, n = row_ok(table, base, new_len, b, N, ps)
        for i in range(n if ok else 0):
            p, r = place(table, b, int(base[b]) + i, P, ps)
            if p < 0:
                continue
            if scales is None:
                pages[p, :, r] = x[b, i]
            else:
                pages[p, :, r], scales[p, :, r] = quantise(x[b, i])
    return pages, scales


def read(pages, scales, table, base, new_len, N, out):
    """out [B][N][H][D] with the positions' values; the rest of out as it was."""
    P, _, ps, _ = pages.shape
    out = np.array(out, np.float64)
    for b in range(len(base)):
        ok, n = row_ok(table, base, new_len, b, N, ps)
        for i in range(n if ok else 0):
            p, r = place(table, b, int(base[b]) + i, P, ps)
            if p < 0:
                out[b, i] = 0
            else:
                out[b, i] = pages[p, :, r] if scales is None else pages[p, :, r] * scales[p, :, r, None]
    return out


def visible(i, pos, base, n, mask):
    """Whether query i (of n real ones) sees a position; mask: this row's tree words or None."""
    if pos < base:
        return True
    j = pos - base
    if j >= n:
        return False
    if mask is None:
        return j <= i
    return j == 0 or (i > 0 and bool((int(mask[i - 1, (j - 1) // 32]) >> ((j - 1) % 32)) & 1))


def attention(q, k_pages, v_pages, k_scale, v_scale, table, base, new_len, tree_mask, scale, out, lse):
    """(out, lse) with the real queries' rows written; only visible positions enter any sum."""
    B, Q, Hq, D = q.shape
    P, H, ps, _ = k_pages.shape
    out, lse, q = np.array(out, np.float64), np.array(lse, np.float64), np.asarray(q, np.float64)
    for b in range(B):
        ok, n = row_ok(table, base, new_len, b, Q, ps)
        if not ok or n == 0:
            continue
        L = int(base[b]) + n
        at = [place(table, b, pos, P, ps) for pos in range(L)]
        pg, rw = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        k = np.asarray(k_pages, np.float64)[pg, :, rw]  # [L][H][D]
        v = np.asarray(v_pages, np.float64)[pg, :, rw]
        if k_scale is not None:
            k = k * np.asarray(k_scale, np.float64)[pg, :, rw][..., None]
            v = v * np.asarray(v_scale, np.float64)[pg, :, rw][..., None]
        mask = None if tree_mask is None else np.asarray(tree_mask[b]).view(np.uint32)
        for i in range(n):
            see = np.array([pg[pos] >= 0 and visible(i, pos, int(base[b]), n, mask) for pos in range(L)], bool)
            for h in range(Hq):
                kh, vh = k[see, h // (Hq // H)], v[see, h // (Hq // H)]
                if not len(kh):
                    out[b, i, h], lse[b, i, h] = 0, -np.inf
                    continue
                s = kh @ q[b, i, h] * scale
                m = s.max()
                w = np.exp(s - m)
                out[b, i, h], lse[b, i, h] = w @ vh / w.sum(), m + np.log(w.sum())
    return out, lse


def compact(pages, table, path, count, base):
    """In-order copies through the table on a copy of pages [P][H][page_size][W]."""
    pages = np.array(pages)
    P, _, ps, _ = pages.shape
    rows = table.shape[1] * ps
    for b in range(len(count)):
        L, at = int(count[b]) - 1, 0 if base is None else int(base[b])
        if L < 0 or L > path.shape[1] or at < 0:
            continue
        moves = [(int(path[b, d]), d) for d in range(L)]
        if any(s < d or at + s >= rows for s, d in moves):
            continue
        where = [(place(table, b, at + s, P, ps), place(table, b, at + d, P, ps)) for s, d in moves if s != d]
        if any(a[0] < 0 or z[0] < 0 for a, z in where):
            continue
        for (p, r), (g, t) in where:
            pages[g, :, t] = pages[p, :, r]
    return pages


def adjust_logits(logits, history=None, history_len=None, prompt_len=None, draft_tokens=None, tree_mask=None,
                  repetition=None, presence=None, frequency=None, bias_tokens=None, bias_values=None, allowed=None):
    """Penalties, biases and masks of logits [B][R][V], token by token from the lists."""
    x = np.array(logits, np.float64)
    B, R, V = x.shape
    for b in range(B):
        n = 0 if history is None else min(max(int(history_len[b]), 0), history.shape[1])
        start = 0 if prompt_len is None else int(prompt_len[b])
        prompt = {int(t) for t in (history[b, :n][:max(start, 0)] if n else []) if 0 <= t < V}
        output = [int(t) for t in (history[b, :n][max(start, 0):] if n else []) if 0 <= t < V]
        bias = {}
        if bias_tokens is not None:
            for t, v in zip(bias_tokens[b], bias_values[b]):
                if 0 <= t < V:
                    bias[int(t)] = float(v)
        for r in range(R):
            count = {}
            for t in output:
                count[t] = count.get(t, 0) + 1
            for j in range(R - 1 if draft_tokens is not None else 0):
                if tree_mask is None:
                    follows = j < r
                else:
                    follows = r > 0 and bool((int(np.asarray(tree_mask).view(np.uint32)[b, r - 1, j // 32]) >> (j % 32)) & 1)
                t = int(draft_tokens[b, j])
                if follows and 0 <= t < V:
                    count[t] = count.get(t, 0) + 1
            for t in prompt | set(count):
                v, c = x[b, r, t], count.get(t, 0)
                if repetition is not None:
                    v = v / repetition[b] if v > 0 else v * repetition[b]
                if frequency is not None:
                    v -= c * frequency[b]
                if presence is not None and c:
                    v -= presence[b]
                x[b, r, t] = v
            for t, v in bias.items():
                x[b, r, t] += v
            if allowed is not None:
                bits = np.unpackbits(np.ascontiguousarray(allowed[b, r]).view(np.uint8), bitorder="little")[:V]
                x[b, r, bits == 0] = -np.inf
    return x
