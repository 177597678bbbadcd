"""Paged NVFP4 key/value cache and its attention (oracle side; test infrastructure only).

Rows are quantized by oracle.nvfp4.quantize (every decision in fp32); the page layout is the one
stated in include/moe_nvfp4.h, written out here element by element; attention is float64 on the
exact cached values.
"""

from __future__ import annotations

import numpy as np

from . import nvfp4

UNIT = 32


def unit_maps(dim: int, values: bool):
    """(code byte, nibble shift, scale byte) of every (position of a unit, element): [32, dim] each."""
    ns = dim // 32
    byte = np.zeros((UNIT, dim), np.int64)
    shift = np.zeros((UNIT, dim), np.int64)
    scale = np.zeros((UNIT, dim), np.int64)
    for p in range(UNIT):
        b, n = divmod(p, 16)
        q, i = divmod(n, 4)
        for d in range(dim):
            s, rest = divmod(d, 32)
            z = (d // 16) % 2
            if values:
                m = rest // 2
                byte[p, d] = 16 * dim + 1024 * (s // 2) + 16 * (16 * q + m) + 8 * (s % 2) + 4 * b + i
                scale[p, d] = 34 * dim + ((2 * q + z) * ns + s) * 8 + 4 * b + i
            else:
                w = b * ns + s
                byte[p, d] = 1024 * (w // 4) + 16 * (16 * (rest // 8) + n) + 4 * (w % 4) + (d % 8) // 2
                scale[p, d] = 32 * dim + (16 * z + n) * 2 * ns + b * ns + s
            shift[p, d] = 4 * (d % 2)
    return byte, shift, scale


def new_pages(num_pages: int, page_size: int, kv_heads: int, dim: int, fill: int = 0) -> np.ndarray:
    return np.full((num_pages, kv_heads, page_size // UNIT, 36 * dim), fill, np.uint8)


def append(pages: np.ndarray, page_size: int, rows: np.ndarray, slots, gscale: float, values: bool) -> None:
    """Quantize rows [T, heads, dim] (float) into the pages at ``slots``; slots outside are skipped."""
    t, heads, dim = rows.shape
    byte, shift, scale = unit_maps(dim, values)
    rows32 = np.asarray(rows, np.float64).astype(np.float32)
    packed, sc = nvfp4.quantize(rows32.reshape(t * heads, dim), gscale)
    codes = nvfp4.unpack_nibbles(packed).reshape(t, heads, dim)
    sc = sc.reshape(t, heads, dim // 16)
    for i, slot in enumerate(np.asarray(slots)):
        if slot < 0 or slot >= pages.shape[0] * page_size:
            continue
        page, off = divmod(int(slot), page_size)
        u, p = divmod(off, UNIT)
        for h in range(heads):
            unit = pages[page, h, u]
            # even elements in the low nibble of their byte, the odd ones above them
            unit[byte[p, 0::2]] = codes[i, h, 0::2] | (codes[i, h, 1::2] << 4)
            unit[scale[p, 0::16]] = sc[i, h]


def decode(pages: np.ndarray, page_size: int, slots, gscale: float, values: bool) -> np.ndarray:
    """Cached values [n, heads, dim] (float64) at valid slots."""
    dim = pages.shape[3] // 36
    byte, shift, scale = unit_maps(dim, values)
    slots = np.asarray(slots, np.int64)
    page, off = slots // page_size, slots % page_size
    u, p = off // UNIT, off % UNIT
    unit = pages[page, :, u]                                                # [n, heads, 36*dim]
    idx = np.broadcast_to(byte[p][:, None, :], (len(slots), pages.shape[1], dim))
    codes = (np.take_along_axis(unit, idx, 2) >> shift[p][:, None, :]) & 15
    sidx = np.broadcast_to(scale[p][:, None, :], idx.shape)
    return nvfp4.e2m1_decode(codes) * nvfp4.e4m3_decode(np.take_along_axis(unit, sidx, 2)) * float(np.float32(gscale))


def plan(kv_lens, new_lens, table, free_pages, page_size, num_pages, num_tokens):
    """(offsets, lens, positions, slots, used, table after) of a step, token by token."""
    table = np.array(table, np.int32, copy=True)
    r_n, width = table.shape
    top = 2 ** 31 - 1
    offsets, lens, used = [0], [], 0
    positions = np.zeros(num_tokens, np.int32)
    slots = np.full(num_tokens, -1, np.int32)
    t = 0
    for r in range(r_n):
        old, new = max(int(kv_lens[r]), 0), max(int(new_lens[r]), 0)
        have, need = -(-old // page_size), -(-(old + new) // page_size)
        for i in range(min(new, num_tokens - t)):
            pos = old + i
            b = pos // page_size
            page = -1
            if b < width:
                if b < have:
                    page = int(table[r, b])
                elif used + b - have < len(free_pages):
                    page = int(free_pages[used + b - have])
                if not 0 <= page < num_pages:
                    page = -1
                if b >= have:
                    table[r, b] = page
            positions[t + i] = min(pos, top)
            slots[t + i] = -1 if page < 0 else page * page_size + pos % page_size
        t = min(t + new, num_tokens)
        used += need - have
        offsets.append(min(offsets[-1] + new, top))
        lens.append(min(old + new, top))
    return np.array(offsets, np.int32), np.array(lens, np.int32), positions, slots, min(used, top), table


def slots_of(table_row, page_size: int, first: int, last: int) -> np.ndarray:
    """Slots of positions [first, last) of a request."""
    pos = np.arange(first, last)
    return np.asarray(table_row, np.int64)[pos // page_size] * page_size + pos % page_size


def attention(q, pages, page_size, k_gscale, v_gscale, offsets, lens, table, scale, window=0):
    """float64 attention of q [T, heads, dim]: (out, lse, (terms, plain, mag)).

    Rows outside every request are NaN.  What rounding bounds scale with: ``terms`` is
    sum_j p_j |v_j| / sum p and ``plain`` sum_j |v_j| / sum p per output element, with p_j = 1 at the
    largest score, and ``mag`` the largest sum_d |scale q_d k_d| over the positions a row sees.
    """
    q = np.asarray(q, np.float64)
    t_n, heads, dim = q.shape
    g = heads // pages.shape[1]
    out = np.full(q.shape, np.nan)
    lse = np.full((t_n, heads), np.nan)
    terms, plain = np.zeros(q.shape), np.zeros(q.shape)
    mag = np.zeros((t_n, heads))
    for r in range(len(lens)):
        a, b = int(offsets[r]), int(offsets[r + 1])
        length = max(int(lens[r]), 0)
        if a == b:
            continue
        slots = slots_of(table[r], page_size, 0, length)
        k = decode(pages, page_size, slots, k_gscale, False)
        v = decode(pages, page_size, slots, v_gscale, True)
        for t in range(a, min(b, t_n)):
            pos = length - (b - a) + (t - a)
            lo = max(0, pos - window + 1) if window else 0
            if pos < 0:
                out[t], lse[t] = 0.0, -np.inf
                continue
            for h in range(heads):
                kk, vv = k[lo:pos + 1, h // g], v[lo:pos + 1, h // g]
                s = scale * (kk @ q[t, h])
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[t, h] = (p @ vv) / l
                lse[t, h] = m + np.log(l)
                terms[t, h] = (p @ np.abs(vv)) / l
                plain[t, h] = np.abs(vv).sum(0) / l
                mag[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
    return out, lse, (terms, plain, mag)
