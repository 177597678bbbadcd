"""Index, choice of pages and sparse attention over the paged NVFP4 cache (oracle side; test infrastructure only).

The index is computed in whole numbers, scores in the fp32 operations that the definition names, attention in float64.
"""

from __future__ import annotations

import numpy as np

from . import kv_cache as okv


def _span(offsets, lens, r, tokens):
    """(first row, rows, length) of request r; tokens past the last row have no row and are not looked at."""
    a, b = (min(max(int(x), 0), tokens) for x in (offsets[r], offsets[r + 1]))
    return a, b - a, max(int(lens[r]) - (int(offsets[r + 1]) - b), 0)


def index_update(codes, scales, pages, page_size, offsets, lens, table, tokens):
    """Recompute codes [P, H, D] and scales [P, H] (in place) of the pages that a step's rows touch."""
    for r in range(len(lens)):
        _, n, length = _span(offsets, lens, r, tokens)
        if n == 0 or length == 0:
            continue
        for b in range(max(length - n, 0) // page_size, min((length - 1) // page_size + 1, table.shape[1])):
            phys = int(table[r, b])
            if not 0 <= phys < pages.shape[0]:
                continue
            held = min(page_size, length - b * page_size)
            keys = okv.decode(pages, page_size, phys * page_size + np.arange(held), 1.0, False) * 1024.0
            s = keys.astype(np.int64)
            assert np.array_equal(s, keys)
            s = s.sum(0)                                                # [H, D], exact
            top = np.abs(s).max(-1)
            for h in range(s.shape[0]):
                a = int(top[h])
                # 127 s / a to the nearest whole number, ties to even, in whole numbers
                q, rest = np.divmod(127 * np.abs(s[h]), max(a, 1))
                up = (2 * rest > a) | ((2 * rest == a) & (q % 2 == 1))
                codes[phys, h] = np.sign(s[h]) * (q + up) if a else 0
                scales[phys, h] = np.float32(a / (127 * 1024 * held))


def query_codes(q):
    """Rows [T, heads, D] (bf16-exact) -> (8-bit codes, largest magnitudes), zeros for rows outside the range."""
    x = np.asarray(q).astype(np.float32)
    with np.errstate(all="ignore"):
        top = np.abs(x).max(-1)
        use = np.all(np.abs(x) <= np.float32(2.0) ** 100, -1) & (top >= np.float32(2.0) ** -100)
        inv = np.float32(127) / np.where(use, top, np.float32(1))
        codes = np.rint(np.where(use[..., None], x, np.float32(0)) * inv[..., None])
    return codes.astype(np.int64), np.where(use, top, np.float32(0)).astype(np.float32)


def scores(q, codes, scales, table_row, kv_heads):
    """float32 scores [kv_heads, width] of one token's heads q [heads, D] for the pages of a table row."""
    width = len(table_row)
    x8, top = query_codes(q)
    g = q.shape[0] // kv_heads
    out = np.full((kv_heads, width), -np.inf, np.float32)
    for j, phys in enumerate(table_row):
        if not 0 <= phys < codes.shape[0]:
            continue
        for h in range(kv_heads):
            dot = x8[h * g:(h + 1) * g] @ codes[phys, h].astype(np.int64)
            out[h, j] = (dot.astype(np.float32) * top[h * g:(h + 1) * g]).max() * scales[phys, h]
    return out


def select(q, codes, scales, page_size, offsets, lens, table, top_k, first=1, last=1):
    """Chosen pages [T, kv_heads, top_k]."""
    tokens, kv_heads = q.shape[0], codes.shape[1]
    out = np.full((tokens, kv_heads, top_k), -1, np.int32)
    for r in range(len(lens)):
        a, n, length = _span(offsets, lens, r, tokens)
        for t in range(a, a + n):
            pos = length - n + t - a
            if pos < 0:
                continue
            own = pos // page_size
            width = min(own + 1, table.shape[1])
            sc = scores(q[t], codes, scales, table[r, :width], kv_heads)
            forced = {j for j in range(own + 1) if j > own - last or (j < first and j < width)}
            for h in range(kv_heads):
                rest = [j for j in range(width) if j not in forced and 0 <= table[r, j] < codes.shape[0]]
                rest.sort(key=lambda j: (-sc[h, j], j))
                got = sorted(forced | set(rest[:top_k - len(forced)]))
                out[t, h, :len(got)] = got
    return out


def attention(q, pages, page_size, k_gscale, v_gscale, offsets, lens, table, selected, scale):
    """float64 attention of q [T, heads, D] over the listed pages: (out, lse, (terms, plain, mag)) as okv.attention;
    rows outside every request are NaN, rows that see a bad page too."""
    q = np.asarray(q, np.float64)
    tokens, heads, dim = q.shape
    kv_heads = pages.shape[1]
    g = heads // kv_heads
    out, lse = np.full(q.shape, np.nan), np.full((tokens, heads), np.nan)
    terms, plain, mag = np.zeros(q.shape), np.zeros(q.shape), np.zeros((tokens, heads))
    for r in range(len(lens)):
        a, n, length = _span(offsets, lens, r, tokens)
        # the request's keys and values by position; pages that are not in the cache are never looked at
        slots = np.zeros(length, np.int64)
        for b in range(min(-(-length // page_size), table.shape[1])):
            if 0 <= table[r, b] < pages.shape[0]:
                at = np.arange(b * page_size, min((b + 1) * page_size, length))
                slots[at] = int(table[r, b]) * page_size + at % page_size
        keys = okv.decode(pages, page_size, slots, k_gscale, False)
        values = okv.decode(pages, page_size, slots, v_gscale, True)
        for t in range(a, a + n):
            pos = length - n + t - a
            for kh in range(kv_heads):
                seen = sorted({int(b) for b in selected[t, kh] if b >= 0 and int(b) * page_size <= pos})
                if not seen:
                    out[t, kh * g:(kh + 1) * g], lse[t, kh * g:(kh + 1) * g] = 0.0, -np.inf
                    continue
                if any(b >= table.shape[1] or not 0 <= table[r, b] < pages.shape[0] for b in seen):
                    continue
                at = np.concatenate([np.arange(b * page_size, min((b + 1) * page_size, pos + 1)) for b in seen])
                k, v = keys[at, kh], values[at, kh]
                for h in range(kh * g, (kh + 1) * g):
                    s = scale * (k @ q[t, h])
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    out[t, h], lse[t, h] = (p @ v) / l, m + np.log(l)
                    terms[t, h], plain[t, h] = (p @ np.abs(v)) / l, np.abs(v).sum(0) / l
                    mag[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * scale
    return out, lse, (terms, plain, mag)
