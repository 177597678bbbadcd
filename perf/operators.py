"""The paged NVFP4 key/value cache operators, as a serving program calls them, and their plain form.

  kv_plan       block table entries, slot map, positions and offsets of a step from the request lengths
  kv_append     new key/value rows quantized to NVFP4 into the cache pages (read back with kv_gather, so
                that what the cache now holds is the output)
  kv_gather     cache rows dequantized to bf16 by slot
  kv_attention  attention of the step's query rows over the cache pages (decode, drafts, prefill)

``own`` selects the framework's calls; otherwise ``run`` computes the same from elementary torch
operations in fp32.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
GSCALE = 0.0625        # dequant global scale of keys and values (a power of two, as a calibrated 2^k)


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of a batch: every request gets one token, some of them open a page
        dict(name="plan_decode", op="plan", requests=64, max_old=8000, max_new=1, page=64, pad=0),
        # a mixed step: prompts of many lengths next to single tokens and idle requests, a padded batch
        dict(name="plan_mixed", op="plan", requests=512, max_old=20000, max_new=96, page=32, pad=37),
        # the rows of one decode step
        dict(name="append_decode", op="append", tokens=32, kv_heads=8, dim=128, page=64),
        # the rows of a prompt
        dict(name="append_prompt", op="append", tokens=8192, kv_heads=8, dim=128, page=128),
        # a short prefix read back, odd sizes
        dict(name="gather_short", op="gather", tokens=301, kv_heads=3, dim=64, page=32),
        # a long prefix exported to a 16-bit consumer
        dict(name="gather_long", op="gather", tokens=32768, kv_heads=8, dim=128, page=128),
        # one request, one token: latency
        dict(name="decode_single", op="attend", requests=1, new=1, new_min=1, old=1023, old_min=1023, heads=32,
             kv_heads=4, dim=128, page=64, window=0),
        # a decode batch of ragged lengths: bandwidth
        dict(name="decode_batch", op="attend", requests=64, new=1, new_min=1, old=8100, old_min=90, heads=64,
             kv_heads=8, dim=128, page=64, window=0),
        # few requests with long contexts: the keys split over the card
        dict(name="decode_long", op="attend", requests=3, new=1, new_min=1, old=131071, old_min=70001, heads=32,
             kv_heads=8, dim=128, page=128, window=0),
        # drafted tokens checked against their contexts, head dim 64, odd group of heads
        dict(name="verify_drafts", op="attend", requests=33, new=5, new_min=2, old=4100, old_min=10, heads=18,
             kv_heads=3, dim=64, page=32, window=0),
        # a whole prompt: matrix rate
        dict(name="prompt_long", op="attend", requests=1, new=8192, new_min=8192, old=0, old_min=0, heads=32,
             kv_heads=8, dim=128, page=128, window=0),
        # chunks of prompts of ragged lengths on earlier contexts, wide heads, sliding window
        dict(name="chunks_window", op="attend", requests=5, new=1500, new_min=77, old=5000, old_min=0, heads=16,
             kv_heads=2, dim=256, page=64, window=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed ranges: every operator, head layout, page size and length."""
    op = rng.choice(["plan", "append", "gather", "attend", "attend", "attend"])
    page = rng.choice([32, 64, 96, 128, 256])
    kv_heads = rng.choice([1, 2, 3, 4, 8])
    dim = rng.choice([64, 128, 256])
    if op == "plan":
        return dict(op=op, requests=_log(rng, 1, 1024), max_old=_log(rng, 1, 30000), max_new=_log(rng, 1, 128),
                    page=page, pad=rng.randrange(0, 50))
    if op in ("append", "gather"):
        return dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=kv_heads, dim=dim, page=page)
    heads = kv_heads * rng.choice([1, 2, 4, 5, 6, 8, 16])
    window = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
    kind = rng.choice(["decode", "drafts", "prompt"])
    if kind == "decode":
        requests, new, old = _log(rng, 1, 64), 1, _log(rng, 1, 8000)
        if requests <= 4:
            old = _log(rng, 1000, 60000)
    elif kind == "drafts":
        requests, new, old = _log(rng, 1, 32), rng.randrange(2, 9), _log(rng, 1, 4000)
    else:
        requests, new = _log(rng, 1, 6), _log(rng, 9, 1500)
        old = rng.choice([0, _log(rng, 1, 4000)])
        heads = kv_heads * rng.choice([1, 2, 4])
    return dict(op=op, requests=requests, new=new, new_min=rng.randrange(0, new + 1) if requests > 1 else new, old=old,
                old_min=rng.randrange(0, old + 1), heads=heads, kv_heads=kv_heads, dim=dim, page=page, window=window)


def _spread(n, lo, hi):
    """n lengths between lo and hi, hi among them (low-discrepancy, the same for every seed)."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lengths(case):
    """(new tokens, lengths before the step) of the requests of an attention case."""
    r = case["requests"]
    return _spread(r, case["new_min"], case["new"]), list(reversed(_spread(r, case["old_min"], case["old"])))


def _plan_new(case):
    """New tokens of a plan case: every seventh request idle, every third a single token."""
    if case["max_new"] == 1:
        return [1] * case["requests"]
    s = _spread(case["requests"], 1, case["max_new"])
    return [0 if i % 7 == 6 else 1 if i % 3 == 2 else v for i, v in enumerate(s)]


# ----------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(g, nbytes):
    """Bytes of two E2M1 codes each, as quantized normal values have them (codes of N(0, 3^2) values)."""
    out = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    step = 1 << 26
    for i in range(0, nbytes, step):
        n = min(step, nbytes - i)
        x = torch.randn(2 * n, generator=g, device=DEV) * 3.0
        c = torch.bucketize(x.abs(), edges, out_int32=True).to(torch.uint8) | ((x < 0).to(torch.uint8) << 3)
        out[i:i + n] = c[0::2] | (c[1::2] << 4)
    return out


def _make_pages(g, pages, kv_heads, page, dim):
    """Cache pages [pages, kv_heads, page/32, 36*dim] with values of about unit size."""
    units = pages * kv_heads * (page // 32)
    u = torch.empty(units, 36 * dim, dtype=torch.uint8, device=DEV)
    u[:, :32 * dim] = _codes(g, units * 32 * dim).view(units, 32 * dim)
    # E4M3 bytes of scales between 3.5 and 8 (amax / 6 in units of the global scale)
    u[:, 32 * dim:] = torch.randint(0x46, 0x50, (units, 4 * dim), generator=g, device=DEV, dtype=torch.uint8)
    return u.view(pages, kv_heads, page // 32, 36 * dim)


def _table(g, lens, page, spare=3):
    """A block table of shuffled pages for requests of these lengths; (table, number of pages)."""
    need = [-(-n // page) for n in lens]
    width = max(max(need), 1)
    total = sum(need) + spare
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor(np.cumsum([0] + need[:-1]), device=DEV)
    j = torch.arange(width, device=DEV)
    idx = first[:, None] + j[None, :]
    table = perm[idx.clamp(max=total - 1)]
    return torch.where(j[None, :] < torch.tensor(need, device=DEV)[:, None], table, 0).to(torch.int32).contiguous(), total


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "plan":
        new = _plan_new(case)
        old = torch.randint(0, case["max_old"] + 1, (case["requests"],), generator=g, device=DEV, dtype=torch.int32)
        olds = old.tolist()
        page = case["page"]
        have = [-(-o // page) for o in olds]
        need = [-(-(o + n) // page) for o, n in zip(olds, new)]
        width = -(-(case["max_old"] + case["max_new"]) // page)
        total = sum(need) + 8
        perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        table = torch.full((case["requests"], width), -1, dtype=torch.int32, device=DEV)
        j = torch.arange(width, device=DEV)
        first = torch.tensor(np.cumsum([0] + have[:-1]), device=DEV)
        held = j[None, :] < torch.tensor(have, device=DEV)[:, None]
        table = torch.where(held, perm[(first[:, None] + j[None, :]).clamp(max=total - 1)], table).contiguous()
        s.update(old=old, new=_i32(new), table=table, free=perm[sum(have):].contiguous(), pages=total,
                 tokens=sum(new) + case["pad"])
        return s
    kvh, dim, page = case["kv_heads"], case["dim"], case["page"]
    if case["op"] in ("append", "gather"):
        n = case["tokens"]
        total = -(-n // page) + 2
        s["pages"] = _make_pages(g, total, kvh, page, dim)
        # the rows of one request from position 5 on, on shuffled pages
        perm = torch.randperm(total, generator=g, device=DEV)
        pos = torch.arange(n, device=DEV) + 5
        s["slots"] = (perm[pos // page] * page + pos % page).to(torch.int32)
        if case["op"] == "append":
            # key and value rows as slices of a fused projection's output
            qkv = torch.randn(n, 4 * kvh * dim, generator=g, device=DEV).to(torch.bfloat16)
            s["k"] = qkv[:, 2 * kvh * dim:3 * kvh * dim].unflatten(1, (kvh, dim))
            s["v"] = qkv[:, 3 * kvh * dim:].unflatten(1, (kvh, dim))
        return s
    new, old = _lengths(case)
    lens = [a + b for a, b in zip(new, old)]
    s["table"], total = _table(g, lens, page)
    s["pages"] = _make_pages(g, total, kvh, page, dim)
    s["offsets"] = _i32(np.cumsum([0] + new).tolist())
    s["lens"] = _i32(lens)
    s["max_new"] = max(new)
    # query rows as a slice of a fused projection's output
    qkv = torch.randn(sum(new), (case["heads"] + 2 * kvh) * dim, generator=g, device=DEV).to(torch.bfloat16)
    s["q"] = qkv[:, :case["heads"] * dim].unflatten(1, (case["heads"], dim))
    s["scale"] = 1.0 / math.sqrt(dim)
    return s


# ----------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "append": _own_append, "gather": _own_gather, "attend": _own_attend}[op](state)
    return {"plan": _plain_plan, "append": _plain_append, "gather": _plain_gather, "attend": _plain_attend}[op](state)


def _own_cache(s):
    import nvfp4_weight_quantized_amd as moe
    c = s["case"]
    return moe.NvFp4KvCache(s["pages"], c["page"], k_gscale=GSCALE, v_gscale=GSCALE)


def _own_plan(s):
    import nvfp4_weight_quantized_amd as moe
    p = moe.kv_plan(s["old"], s["new"], s["table"], s["free"], s["case"]["page"], s["pages"], s["tokens"])
    return dict(offsets=p.query_offsets, lens=p.seq_lens, positions=p.positions, slots=p.slots, used=p.pages_used,
                table=s["table"])


def _own_append(s):
    import nvfp4_weight_quantized_amd as moe
    cache = _own_cache(s)
    moe.kv_append(cache, s["k"], s["v"], s["slots"])
    k, v = moe.kv_gather(cache, s["slots"])
    return dict(k=k, v=v)


def _own_gather(s):
    import nvfp4_weight_quantized_amd as moe
    k, v = moe.kv_gather(_own_cache(s), s["slots"])
    return dict(k=k, v=v)


def _own_attend(s):
    import nvfp4_weight_quantized_amd as moe
    out, lse = moe.kv_attention(_own_cache(s), s["q"], s["offsets"], s["lens"], s["table"], scale=s["scale"],
                                window=s["case"]["window"], return_lse=True)
    return dict(out=out, lse=lse)


# ----------------------------------------------------------------------------- plain forms

def _plain_plan(s):
    page, tokens, table = s["case"]["page"], s["tokens"], s["table"]
    requests, width = table.shape
    old, new, free = s["old"].long(), s["new"].long(), s["free"]
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    offsets = torch.cat([zero, torch.cumsum(new, 0)])
    have, need = (old + page - 1) // page, (old + new + page - 1) // page
    first_free = torch.cat([zero, torch.cumsum(need - have, 0)])
    t = torch.arange(tokens, device=DEV)
    valid = t < offsets[-1]
    r = torch.searchsorted(offsets[1:].contiguous(), t, right=True).clamp(max=requests - 1)
    pos = old[r] + t - offsets[r]
    b = pos // page
    fresh = b >= have[r]
    fi = first_free[r] + b - have[r]
    pg = torch.where(fresh, free[fi.clamp(0, free.numel() - 1)], table[r, b.clamp(0, width - 1)])
    ok = valid & (b < width) & (~fresh | (fi < free.numel())) & (pg >= 0) & (pg < s["pages"])
    slots = torch.where(ok, pg * page + pos % page, -1).to(torch.int32)
    starts = valid & fresh & (pos % page == 0) & (b < width)
    flat = torch.cat([table.view(-1), table.new_zeros(1)])     # one place more for the tokens that open no page
    flat[torch.where(starts, r * width + b, requests * width)] = torch.where(ok, pg, -1).to(torch.int32)
    table.copy_(flat[:-1].view(requests, width))
    return dict(offsets=offsets.to(torch.int32), lens=(old + new).to(torch.int32),
                positions=torch.where(valid, pos, 0).to(torch.int32), slots=slots,
                used=first_free[-1:].to(torch.int32), table=table)


def _plain_quantize(x):
    """The values NVFP4 holds for bf16 rows [..., dim] (E2M1 x E4M3 per 16 elements x global scale)."""
    v = x.float().unflatten(-1, (-1, 16))
    t = (v.abs().amax(-1, keepdim=True) / (6.0 * GSCALE)).clamp(max=448.0)
    step = torch.ldexp(torch.ones_like(t), torch.frexp(t.clamp(min=2.0 ** -6))[1] - 4)    # E4M3 spacing at t
    sc = torch.round(t / step) * step
    sd = sc * GSCALE
    q = torch.where(sd > 0, v / sd, 0.0)
    a = q.abs()
    st = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    mag = (torch.round(a / st) * st).clamp(max=6.0)
    return (torch.where(q < 0, -mag, mag) * sd).flatten(-2).to(torch.bfloat16)


def _plain_append(s):
    return dict(k=_plain_quantize(s["k"]), v=_plain_quantize(s["v"]))


def _e2m1_pairs():
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    vals = torch.cat([mags, -mags])
    b = torch.arange(256, device=DEV)
    return torch.stack([vals[b & 15], vals[b >> 4]], -1)


def _e4m3_values():
    b = torch.arange(256, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).float()
    mag = torch.where(e == 0, m * 2.0 ** -9, (8.0 + m) * torch.exp2(e.float() - 10.0))
    return torch.where(b >= 128, -mag, mag)


def _plain_decode(units, dim, values):
    """Units [..., 36*dim] of 32 tokens -> fp32 rows [..., 32, dim] of the keys or the values."""
    ns, lead = dim // 32, units.shape[:-1]
    n = len(lead)
    ax = list(range(n))
    if values:
        c = units[..., 16 * dim:32 * dim].reshape(*lead, ns // 2, 4, 16, 2, 2, 4)       # load q n range half key
        c = c.permute(*ax, n + 4, n + 1, n + 5, n, n + 3, n + 2)                        # half q key load range n
        sc = units[..., 34 * dim:].reshape(*lead, 4, 2, ns, 2, 4).permute(*ax, n + 3, n, n + 4, n + 2, n + 1)
    else:
        c = units[..., :16 * dim].reshape(*lead, ns // 2, 4, 16, 4, 4).permute(*ax, n, n + 3, n + 2, n + 1, n + 4)
        c = c.reshape(*lead, 2, ns, 16, 4, 4).permute(*ax, n, n + 2, n + 1, n + 3, n + 4)   # block key step q byte
        sc = units[..., 32 * dim:34 * dim].reshape(*lead, 2, 16, 2, ns).permute(*ax, n + 2, n + 1, n + 3, n)
    x = _e2m1_pairs()[c.reshape(*lead, 32, dim // 16, 8).int()].flatten(-2)             # [..., 32, dim/16, 16]
    return (x * (_e4m3_values()[sc.reshape(*lead, 32, dim // 16).int()] * GSCALE)[..., None]).flatten(-2)


def _plain_gather(s):
    dim, page = s["case"]["dim"], s["case"]["page"]
    slots = s["slots"].long()
    k = _plain_decode(s["pages"], dim, False).flatten(2, 3)[slots // page, :, slots % page]
    v = _plain_decode(s["pages"], dim, True).flatten(2, 3)[slots // page, :, slots % page]
    return dict(k=k.to(torch.bfloat16), v=v.to(torch.bfloat16))


def _plain_attend(s):
    c = s["case"]
    dim, kvh, g = c["dim"], c["kv_heads"], c["heads"] // c["kv_heads"]
    offsets, lens, q = s["offsets"].long(), s["lens"].long(), s["q"]
    requests, tokens, most = lens.numel(), q.shape[0], s["max_new"]
    # keys and values of every request, padded to the longest: [requests, kv_heads, keys, dim]
    units = s["pages"][s["table"].long()].transpose(1, 2)               # [R, kv_heads, blocks, page/32, 36*dim]
    k = _plain_decode(units, dim, False).flatten(2, 4)
    v = _plain_decode(units, dim, True).flatten(2, 4)
    # query rows padded to the longest request: [requests, kv_heads, most * g, dim]
    new = offsets[1:] - offsets[:-1]
    i = torch.arange(most, device=DEV)
    rows = q.float()[(offsets[:-1, None] + i).clamp(max=tokens - 1)]
    rows = rows.view(requests, most, kvh, g, dim).transpose(1, 2).reshape(requests, kvh, most * g, dim)
    scores = torch.matmul(rows, k.transpose(-1, -2)).mul_(s["scale"])
    pos = (lens - new)[:, None] + i                                     # [R, most]
    j = torch.arange(k.shape[2], device=DEV)
    seen = (j <= pos[..., None]) & (j < lens[:, None, None])
    if c["window"]:
        seen &= j > pos[..., None] - c["window"]
    seen = seen[:, None, :, None].expand(-1, 1, -1, g, -1).reshape(requests, 1, most * g, -1)
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[..., 0]
    # back to token rows
    t = torch.arange(tokens, device=DEV)
    r = torch.searchsorted(offsets[1:].contiguous(), t, right=True)
    o = o.view(requests, kvh, most, g, dim)[r, :, t - offsets[r]].reshape(tokens, kvh * g, dim)
    lse = lse.view(requests, kvh, most, g)[r, :, t - offsets[r]].reshape(tokens, kvh * g)
    return dict(out=o.to(torch.bfloat16), lse=lse)


# ----------------------------------------------------------------------------- what a pass cannot do without

def _pairs(case):
    """(visible query-key pairs, cache rows that some query row sees) of an attention case."""
    pairs = rows = 0
    for n, o in zip(*_lengths(case)):
        if n == 0:
            continue
        w = case["window"] or (n + o)
        first = max(0, o - w + 1)
        rows += n + o - first
        pairs += sum(min(o + i + 1, w) for i in range(n))
    return pairs, rows


def work(case):
    if case["op"] == "plan":
        tokens = sum(_plan_new(case))
        r = case["requests"]
        return {"bytes": 4 * (2 * r + 2 * r + 2 * (tokens + case["pad"]) + r + 2 * tokens // case["page"]), "flops": 0}
    kvh, dim = case["kv_heads"], case["dim"]
    row16, row4 = 2 * 2 * kvh * dim, 2 * kvh * dim * 9 // 16
    if case["op"] == "append":
        return {"bytes": case["tokens"] * (2 * row16 + 2 * row4 + 8), "flops": 0}
    if case["op"] == "gather":
        return {"bytes": case["tokens"] * (row16 + row4 + 4), "flops": 0}
    pairs, rows = _pairs(case)
    tokens = sum(_lengths(case)[0])
    return {"bytes": rows * row4 + tokens * case["heads"] * (4 * dim + 4), "flops": 4 * dim * case["heads"] * pairs}


# ----------------------------------------------------------------------------- 64 bits, from the definitions

def _byte_map(dim, values):
    """For each (token of a unit, element): byte offset in the unit, nibble shift, scale byte offset."""
    key = np.arange(32)[:, None]
    d = np.arange(dim)[None, :]
    ns = dim // 32
    if values:
        q, half, low = (key % 16) // 4, key // 16, key % 4
        rng, n = d // 32, (d % 32) // 2
        byte = 16 * dim + (rng // 2) * 1024 + 16 * (16 * q + n) + 8 * (rng % 2) + 4 * half + low
        scale = 34 * dim + ((2 * q + n // 8) * ns + rng) * 8 + 4 * half + low
    else:
        kb, n = key // 16, key % 16
        step, q = d // 32, (d % 32) // 8
        w = kb * ns + step
        byte = (w // 4) * 1024 + 16 * (16 * q + n) + 4 * (w % 4) + (d % 8) // 2
        scale = 32 * dim + ((q // 2) * 16 + n) * 2 * ns + w
    return [torch.tensor(np.broadcast_to(a, (32, dim)).copy(), device=DEV) for a in (byte, 4 * (d % 2), scale)]


def _f64_rows(units, dim, values):
    """Units [n, 36*dim] -> fp64 rows [n, 32, dim], element by element from the format's definition."""
    byte, shift, scale = _byte_map(dim, values)
    code = (units[:, byte].to(torch.int32) >> shift) & 15
    e, m = (code >> 1) & 3, (code & 1).double()
    x = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (e.double() - 1))
    x = torch.where(code >= 8, -x, x)
    b = units[:, scale].to(torch.int32)
    se, sm = (b >> 3) & 15, (b & 7).double()
    return x * torch.where(se == 0, sm / 8 * 2.0 ** -6, (1 + sm / 8) * 2.0 ** (se.double() - 7)) * GSCALE


def _f64_quantize(x):
    """The NVFP4 values of rows: nearest grid values in 64 bits, ties to the even code."""
    mags = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    grid8 = torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)) for e in range(16)
                          for m in range(8)][:127], dtype=torch.float64, device=DEV)

    def nearest(a, grid):
        hi = torch.searchsorted(grid, a).clamp(1, grid.numel() - 1)
        lo = hi - 1
        up, down = grid[hi] - a, a - grid[lo]
        return torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))

    v = x.double().unflatten(-1, (-1, 16))
    t = (v.abs().amax(-1, keepdim=True) / (6 * GSCALE)).clamp(max=448.0)
    sd = grid8[nearest(t, grid8)] * GSCALE
    q = torch.where(sd > 0, v / sd, 0.0)
    mag = mags[nearest(q.abs().clamp(max=6.0), mags)]
    return (torch.sign(q) * mag * sd).flatten(-2)


def exact(case, seed):
    if case["op"] == "plan":
        return None                       # whole numbers only
    s = prepare(case, seed)
    dim, page = case["dim"], case["page"]
    if case["op"] == "append":
        return dict(k=_f64_quantize(s["k"]), v=_f64_quantize(s["v"]))
    if case["op"] == "gather":
        slots, res = s["slots"].long(), {}
        for name, values in (("k", False), ("v", True)):
            parts = []
            for sl in slots.split(2048):
                u = s["pages"][sl // page, :, (sl % page) // 32]
                rows = _f64_rows(u.flatten(0, 1), dim, values).view(*u.shape[:2], 32, dim)
                parts.append(rows[torch.arange(sl.numel(), device=DEV), :, sl % 32])
            res[name] = torch.cat(parts)
        return res
    new, old = _lengths(case)
    g = case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for r, (n, o) in enumerate(zip(new, old)):
        pages = s["table"][r, :-(-(n + o) // page)].long()
        for h in range(case["kv_heads"] if n and n + o else 0):
            u = s["pages"][pages, h].flatten(0, 1)
            k = _f64_rows(u, dim, False).flatten(0, 1)[:n + o]
            v = _f64_rows(u, dim, True).flatten(0, 1)[:n + o]
            for i in range(0, n, 2048):
                m = min(2048, n - i)
                q = s["q"][at + i:at + i + m, h * g:(h + 1) * g].double().reshape(m * g, dim)
                x = (q @ k.T) * s["scale"]
                pos = (o + i + torch.arange(m, device=DEV)).repeat_interleave(g)[:, None]
                j = torch.arange(n + o, device=DEV)[None, :]
                hide = j > pos
                if case["window"]:
                    hide |= j <= pos - case["window"]
                x = x.masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, -1)
                lse[at + i:at + i + m, h * g:(h + 1) * g] = z.view(m, g)
                out[at + i:at + i + m, h * g:(h + 1) * g] = (torch.exp(x - z[:, None]) @ v).view(m, g, dim)
        at += n
    return dict(out=out, lse=lse)
