"""Plain float64 forms of the operators for long contexts on a paged cache (test infrastructure).

Written from the definitions in ``include/spec_pages.h``, ``include/spec_rotary.h`` and
``include/spec_sparse.h`` with numpy on the host, entry by entry where that keeps them obvious.
They share no code with the CUDA library.  Cache pages are arrays [pages][heads][page_size][head_dim]
of values (codes already decoded and scaled).
"""
import numpy as np

from oracle import paged


def page_resize(table, pages, length, stack, count, page_size, base=None, N=0):
    """(table, pages, stack, count, ok, slots) after the call, on copies."""
    table, pages, stack = np.array(table), np.array(pages), np.array(stack)
    B, width = table.shape
    P = len(stack)
    count = min(max(int(count), 0), P)
    fine = np.array([0 <= int(n) <= width * page_size and 0 <= int(p) <= width for n, p in zip(length, pages)], bool)
    need = [-(-int(n) // page_size) for n in length]
    for b in range(B):
        if fine[b]:
            for e in range(need[b], pages[b]):
                if 0 <= table[b, e] < P:
                    if count < P:
                        stack[count] = table[b, e]
                        count += 1
                table[b, e] = -1
    short = False
    for b in range(B):
        if not fine[b]:
            continue
        lack = need[b] - int(pages[b])
        if lack > 0:
            short = short or lack > count
            if short:
                fine[b] = False
                continue
            for e in range(int(pages[b]), need[b]):
                count -= 1
                table[b, e] = stack[count]
        pages[b] = need[b]
    slots = np.full((B, N), -1, np.int64)
    for b in range(B):
        for i in range(N if fine[b] and base is not None else 0):
            pos = int(base[b]) + i
            if 0 <= pos < int(length[b]):
                p, r = paged.place(table, b, pos, P, page_size)
                if p >= 0:
                    slots[b, i] = p * page_size + r
    return table, pages, stack, count, fine.astype(np.int32), slots


def positions(base, N, depth=None):
    step = np.arange(N)[None].repeat(len(base), 0)
    if depth is not None and N > 1:
        step = np.concatenate([np.zeros((len(base), 1), np.int64), np.asarray(depth, np.int64)], 1)
    return np.asarray(base, np.int64)[:, None] + step


def rotary(x, freq, pos, interleaved=False, inverse=False, amplitude=1.0):
    """x [B][N][heads][D] with its pairs turned; angles reduced with more digits than float64 has."""
    x = np.array(x, np.float64)
    freq = np.asarray(freq, np.float64)
    R = len(freq)
    angle = pos[..., None].astype(np.longdouble) * freq.astype(np.longdouble)
    c = (np.cos(angle) * amplitude).astype(np.float64)[:, :, None]
    s = (np.sin(angle) * amplitude).astype(np.float64)[:, :, None] * (-1 if inverse else 1)
    first = slice(0, 2 * R, 2) if interleaved else slice(0, R)
    second = slice(1, 2 * R, 2) if interleaved else slice(R, 2 * R)
    a, b = x[..., first].copy(), x[..., second].copy()
    x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def block_summary(k, table, base, new_len, N, bounds, out):
    """out [P][H][D or 2 D] with the touched blocks' summaries."""
    P, H, ps, D = k.shape
    out = np.array(out, np.float64)
    for b in range(len(base)):
        ok, n = paged.row_ok(table, base, new_len, b, N, ps)
        if not ok or n == 0:
            continue
        end = int(base[b]) + n
        for j in range(int(base[b]) // ps, -(-end // ps)):
            p = int(table[b, j])
            if not 0 <= p < P:
                continue
            x = k[p, :, :min(ps, end - j * ps)]
            out[p] = np.concatenate([x.max(1), x.min(1)], -1) if bounds else x.mean(1)
    return out


def block_scores(q, m, bounds):
    """Scores of one query head's row q [D] against summaries m [n][D or 2 D], sums exact to 64 bits."""
    D = len(q)
    with np.errstate(all="ignore"):
        return (np.where(q >= 0, q * m[:, :D], q * m[:, D:]) if bounds else q * m).sum(-1)


def block_select(q, summary, table, base, new_len, page_size, top, bounds, sink, recent, shared):
    """Lists of blocks [B][Q or 1][H][top]."""
    B, Q, Hq, D = q.shape
    P, H, _ = summary.shape
    g = Hq // H
    out = np.full((B, 1 if shared else Q, H, top), -1, np.int32)
    for b in range(B):
        ok, n = paged.row_ok(table, base, new_len, b, Q, page_size)
        if not ok or n == 0:
            continue
        full = int(base[b]) // page_size
        for i in range(1 if shared else n):
            for h in range(H):
                if full <= top:
                    out[b, i, h, :full] = np.arange(full)
                    continue
                chosen = set(range(sink)) | set(range(full - recent, full))
                rank = []
                rows = [(y, h * g + z) for y in (range(n) if shared else [i]) for z in range(g)]
                cand = list(range(sink, full - recent))
                page = np.array([int(table[b, j]) for j in cand])
                hole = (page < 0) | (page >= P)
                m = summary[np.where(hole, 0, page), h]
                with np.errstate(all="ignore"):
                    score = np.max([block_scores(q[b, y, z], m, bounds) for y, z in rows], 0)  # NaN stays
                for j, s, none in zip(cand, score, hole):
                    rank.append((0 if none else 1 if np.isnan(s) else 2, 0.0 if none or np.isnan(s) else s, -j))
                rank.sort(reverse=True)
                chosen |= {-r[2] for r in rank[:top - sink - recent]}
                out[b, i, h] = sorted(chosen)
    return out


def sparse_attention(q, k, v, table, base, new_len, tree_mask, blocks, scale, out, lse):
    """(out, lse) with the real queries' rows written."""
    B, Q, Hq, D = q.shape
    P, H, ps, _ = k.shape
    g = Hq // H
    out, lse = np.array(out, np.float64), np.array(lse, np.float64)
    for b in range(B):
        ok, n = paged.row_ok(table, base, new_len, b, Q, ps)
        if not ok or n == 0:
            continue
        full = int(base[b]) // ps
        mask = None if tree_mask is None else np.asarray(tree_mask[b]).view(np.uint32)
        for i in range(n):
            for h in range(H):
                last, taken = -1, []
                for e in blocks[b, i if blocks.shape[1] > 1 else 0, h]:
                    if last < e < full:
                        taken.append(int(e))
                        last = int(e)
                pos = [j * ps + r for j in taken for r in range(ps)]
                pos += [x for x in range(full * ps, int(base[b]) + n) if paged.visible(i, x, int(base[b]), n, mask)]
                at = [paged.place(table, b, x, P, ps) for x in pos]
                at = [a for a in at if a[0] >= 0]
                for y in range(h * g, (h + 1) * g):
                    if not at:
                        out[b, i, y], lse[b, i, y] = 0, -np.inf
                        continue
                    pg, rw = np.array([a[0] for a in at]), np.array([a[1] for a in at])
                    s = k[pg, h, rw] @ q[b, i, y] * scale
                    m = s.max()
                    if not np.isfinite(m):
                        out[b, i, y], lse[b, i, y] = (0, -np.inf) if m == -np.inf else (np.nan, np.nan)
                        continue
                    w = np.exp(s - m)
                    out[b, i, y], lse[b, i, y] = w @ v[pg, h, rw] / w.sum(), m + np.log(w.sum())
    return out, lse
