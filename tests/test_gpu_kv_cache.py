"""GPU parity of the key/value cache's plan, append and gather against the oracle: bit for bit."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_weight_quantized_amd import kv, ops
from oracle import kv_cache as okv
from oracle import moe as omoe
from oracle import nvfp4 as onv
from oracle import w4a4 as oa4

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(v):
    return torch.from_numpy(np.asarray(v, np.int32)).to(DEV)


def _plan_inputs(rng, old, page, width, spare):
    perm = rng.permutation(sum(min(-(-max(o, 0) // page), width) for o in old) + spare).astype(np.int32)
    table = np.full((len(old), width), -1, np.int32)
    at = 0
    for r, o in enumerate(old):
        n = min(-(-max(o, 0) // page), width)
        table[r, :n] = perm[at:at + n]
        at += n
    return table, perm[at:].copy(), len(perm)


@pytest.mark.parametrize("seed,requests,max_old,max_new,page,spare,pad,width_cut", [
    (0, 1, 0, 1, 32, 3, 0, 0),
    (1, 1, 500, 1, 64, 0, 0, 0),             # a page opens and none is free (or none opens)
    (2, 7, 100, 1, 32, 9, 4, 0),
    (3, 64, 4000, 1, 64, 70, 0, 0),
    (4, 65, 300, 90, 32, 400, 11, 0),
    (5, 130, 200, 300, 96, 100, 0, 0),       # shortage, several workgroups
    (6, 1025, 900, 9, 32, 1500, 5, 0),
    (7, 4096, 40, 3, 32, 4500, 1, 0),
    (8, 33, 700, 40, 32, 300, 2, 5),         # tables narrower than some requests
    (9, 3, 70000, 5000, 128, 200, 0, 0),     # page 128, prompts
])
def test_plan_matches_oracle(seed, requests, max_old, max_new, page, spare, pad, width_cut):
    rng = np.random.default_rng(seed)
    old = rng.integers(0, max_old + 1, requests)
    new = rng.integers(0, max_new + 1, requests)
    if requests > 5:
        old[2], new[4] = -9, -2              # negative lengths count as 0
    width = max(1, -(-(max_old + max_new) // page) - width_cut)
    table, free, num_pages = _plan_inputs(rng, old, page, width, spare)
    if len(free) > 6:
        free[5] = num_pages + 3              # a free list entry outside the cache
    tokens = int(np.maximum(new, 0).sum()) + pad
    ref = okv.plan(old, new, table, free, page, num_pages, tokens)
    gtable = _i32(table)
    for _ in range(2):                       # the second call finds its own entries: same answer
        p = kv.kv_plan(_i32(old), _i32(new), gtable, _i32(free), page, num_pages, tokens)
        for got, want in zip((p.query_offsets, p.seq_lens, p.positions, p.slots), ref):
            assert np.array_equal(got.cpu().numpy(), want)
        assert int(p.pages_used) == ref[4]
        assert np.array_equal(gtable.cpu().numpy(), ref[5])


def test_plan_with_fewer_rows_than_tokens_and_with_none():
    old, new, page = np.array([31, 64]), np.array([40, 30]), 32
    table, free, n = _plan_inputs(np.random.default_rng(1), old, page, 4, 6)
    for tokens in (0, 1, 40, 41, 69):
        ref = okv.plan(old, new, table, free, page, n, tokens)
        gtable = _i32(table)
        p = kv.kv_plan(_i32(old), _i32(new), gtable, _i32(free), page, n, tokens)
        for got, want in zip((p.query_offsets, p.seq_lens, p.positions, p.slots), ref):
            assert np.array_equal(got.cpu().numpy(), want)
        assert np.array_equal(gtable.cpu().numpy(), ref[5])
    empty = torch.empty(0, dtype=torch.int32, device=DEV)
    p = kv.kv_plan(empty, empty, torch.empty(0, 4, dtype=torch.int32, device=DEV), empty, 32, 4, 3)
    assert p.query_offsets.tolist() == [0] and p.slots.tolist() == [-1] * 3 and int(p.pages_used) == 0


def test_plan_saturates_lengths_past_31_bits():
    big = 2 ** 31 - 1
    t = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    p = kv.kv_plan(_i32([big, 5]), _i32([big, 2]), t, _i32([0]), 32, 1, 4)
    ref = okv.plan([big, 5], [big, 2], np.full((2, 3), -1, np.int32), [0], 32, 1, 4)
    for got, want in zip((p.query_offsets, p.seq_lens, p.slots), (ref[0], ref[1], ref[3])):
        assert np.array_equal(got.cpu().numpy(), want)


EDGE = np.array([6.0, -3.5, 2.5, 1.25, 0.25, 5.0, 7.5, -1.75, 0.75, -0.75, 3.5, -0.25, 1.75, -5.0, 0.0, -0.0])


def _rows(rng, t, heads, dim):
    x = kh.bf16(rng, (t, heads, dim)) * np.exp2(rng.integers(-9, 9, (t, heads, 1)))
    x[0, 0, :16] = 0.0
    x[0, 0, 16:32] = EDGE                          # ties of both grids under a power-of-two scale
    x[0, 0, 32:48] = rng.normal(0, 1, 16) * 1e-7   # scale in the subnormals or 0
    x[0, 0, 48:64] = rng.normal(0, 1, 16) * 1e6    # scale capped at 448
    return omoe.bf16_to_float(oa4.float_to_bf16_bits(x))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,page,t", [(1, 32, 1), (3, 96, 37), (8, 64, 200), (2, 256, 515), (8, 128, 2051)])
@pytest.mark.parametrize("d_k,d_v", [(1.0, 0.0625), (0.0371, 3.1e-3)])
def test_append_writes_the_oracles_bytes(dim, heads, page, t, d_k, d_v):
    rng = np.random.default_rng(dim + heads + t)
    d_k, d_v = float(np.float32(d_k)), float(np.float32(d_v))
    n_pages = -(-(t + 5) // page) + 2
    # consecutive positions of one request from 5 on, then a shuffled tail, some rows skipped
    slots = (rng.permutation(n_pages)[(np.arange(t) + 5) // page] * page + (np.arange(t) + 5) % page).astype(np.int32)
    tail = t // 3
    slots[t - tail:] = rng.permutation(slots[t - tail:])
    slots[1::29] = -1
    if t > 3:
        slots[3] = n_pages * page                  # outside the cache: skipped
    k, v = _rows(rng, t, heads, dim), _rows(rng, t, heads, dim)
    pages = rng.integers(0, 256, (n_pages, heads, page // 32, 36 * dim)).astype(np.uint8)
    want = pages.copy()
    okv.append(want, page, k, slots, d_k, False)
    okv.append(want, page, v, slots, d_v, True)
    cache = kv.NvFp4KvCache(torch.from_numpy(pages).to(DEV), page, d_k, d_v)
    # rows as slices of a fused projection's output
    qkv = torch.zeros(t, (3 * heads) * dim + 8, dtype=torch.bfloat16, device=DEV)
    gk = qkv[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
    gv = qkv[:, 2 * heads * dim + 8:].unflatten(1, (heads, dim))
    gk.copy_(kh.to_bf16(k))
    gv.copy_(kh.to_bf16(v))
    kv.kv_append(cache, gk, gv, _i32(slots))
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    # the codes and scales are those of the library's activation quantizer
    p_ref, s_ref, _ = ops.quantize_act_nv(kh.to_bf16(k).reshape(t * heads, dim), d_k, values=False)
    pk, sk = onv.quantize(k.reshape(-1, dim).astype(np.float32), d_k)
    assert np.array_equal(p_ref.cpu().numpy(), pk) and np.array_equal(s_ref.cpu().numpy(), sk)


@pytest.mark.parametrize("dim,heads", [(64, 64), (128, 33), (256, 16)])
@pytest.mark.parametrize("runs,page", [([(0, 528)], 96), ([(3, 40), (64, 33), (31, 1), (0, 200), (90, 259)], 64)])
def test_append_of_runs_writes_the_oracles_bytes(dim, heads, runs, page):
    """Enough rows for quads of positions: runs that fill units, begin and end inside units and quads, and
    meet in one window of rows; bytes of other positions stay."""
    rng = np.random.default_rng(dim + len(runs))
    slots, at = [], 0
    for first, n in runs:                          # each run has pages of its own
        pages_of = rng.permutation(-(-(first + n) // page)) + at
        at += len(pages_of)
        pos = first + np.arange(n)
        slots.append(pages_of[pos // page] * page + pos % page)
    slots = np.concatenate(slots).astype(np.int32)
    t = len(slots)
    assert 2 * t * heads * (dim // 16) >= 1 << 18
    k, v = _rows(rng, t, heads, dim), _rows(rng, t, heads, dim)
    pages = rng.integers(0, 256, (at, heads, page // 32, 36 * dim)).astype(np.uint8)
    want = pages.copy()
    okv.append(want, page, k, slots, 0.0625, False)
    okv.append(want, page, v, slots, 0.5, True)
    cache = kv.NvFp4KvCache(torch.from_numpy(pages).to(DEV), page, 0.0625, 0.5)
    kv.kv_append(cache, kh.to_bf16(k), kh.to_bf16(v), _i32(slots))
    assert np.array_equal(cache.pages.cpu().numpy(), want)


@pytest.mark.parametrize("d", [1.0, 2.0 ** -64, 2.0 ** 64, 3.3e-4, 0.0371, 1.0 / 2688.0])
def test_append_of_every_largest_magnitude(d):
    """Groups whose largest element runs over every finite bf16 magnitude, the others random below it or
    on the midpoints of the E2M1 grid: scales and codes bit for bit."""
    d = float(np.float32(d))
    rng = np.random.default_rng(7)
    bits = np.arange(0x7F80, dtype=np.uint16)
    top = omoe.bf16_to_float(bits)
    t, dim, page = len(top) // 4, 64, 256
    x = rng.uniform(-1, 1, (t, 1, dim))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) / 6
    x[::2, 0, 1::2] = rng.choice(ties, (len(x[::2]), dim // 2)) * rng.choice([-1, 1], (len(x[::2]), dim // 2))
    x[:, :, 0::16] = 1.0
    with np.errstate(over="ignore"):
        x = omoe.bf16_to_float(oa4.float_to_bf16_bits(x * np.repeat(top.reshape(t, 4), 16, 1)[:, None, :]))
    n_pages = -(-t // page)
    slots = np.arange(t, dtype=np.int32)
    want = okv.new_pages(n_pages, page, 1, dim)
    with np.errstate(over="ignore", under="ignore"):
        okv.append(want, page, x, slots, d, False)
        okv.append(want, page, x, slots, d, True)
    cache = kv.NvFp4KvCache.allocate(n_pages, page, 1, dim, d, d)
    kv.kv_append(cache, kh.to_bf16(x), kh.to_bf16(x), _i32(slots))
    assert np.array_equal(cache.pages.cpu().numpy(), want)
    assert len(np.unique(want[..., 32 * dim:])) > 100 or d > 1e6 or d < 1e-6


def test_append_of_nonfinite_rows_stays_finite():
    """Infinities saturate, a NaN takes the code of 6: the bytes of the activation quantizer."""
    dim, page = 64, 32
    x = torch.randn(3, 1, dim, dtype=torch.float32).to(torch.bfloat16)
    x[0, 0, 3], x[0, 0, 5], x[0, 0, 20], x[1, 0, 40] = float("inf"), -float("inf"), float("nan"), -float("nan")
    x[2] = float("nan")
    x = x.to(DEV)
    cache = kv.NvFp4KvCache.allocate(1, page, 1, dim, 0.5, 0.25)
    slots = _i32([4, 9, 31])
    kv.kv_append(cache, x, x, slots)
    for d, values in ((0.5, False), (0.25, True)):
        p, s, _ = ops.quantize_act_nv(x.reshape(3, dim), d, values=False)
        want = onv.e2m1_decode(onv.unpack_nibbles(p.cpu().numpy())).reshape(3, dim) * np.repeat(
            onv.e4m3_decode(s.cpu().numpy()), 16, axis=1) * d
        got = okv.decode(cache.pages.cpu().numpy(), page, [4, 9, 31], d, values)[:, 0]
        assert np.all(np.isfinite(got)) and np.array_equal(got, want)


@pytest.mark.parametrize("dim,heads,page,n", [(64, 1, 32, 1), (64, 5, 96, 77), (128, 8, 64, 300), (256, 2, 128, 129),
                                              (64, 2, 64, 29), (64, 1, 256, 31), (128, 3, 32, 61)])
@pytest.mark.parametrize("runs", [False, True])
def test_gather_matches_the_decoded_cache(dim, heads, page, n, runs):
    rng = np.random.default_rng(n)
    pages = rng.integers(0, 256, (5, heads, page // 32, 36 * dim)).astype(np.uint8)
    pages[..., 32 * dim:] &= 0x7E                  # no NaN scale
    slots = rng.integers(0, 5 * page, n).astype(np.int32)   # any order, repeats
    if runs:                                                # positions 5.. of a request, as a prefix is read
        slots = ((np.array([3, 0, 4, 1, 2])[(np.arange(n) + 5) // page % 5]) * page + (np.arange(n) + 5) % page).astype(np.int32)
    d_k, d_v = float(np.float32(0.0371)), 2.0 ** -7
    cache = kv.NvFp4KvCache(torch.from_numpy(pages).to(DEV), page, d_k, d_v)
    k, v = kv.kv_gather(cache, _i32(slots))
    for got, d, values in ((k, d_k, False), (v, d_v, True)):
        # e2m1 * e4m3 is exact; the product with the global scale is rounded to fp32, then to bf16
        ref = (okv.decode(pages, page, slots, 1.0, values).astype(np.float32) * np.float32(d)).astype(np.float64)
        assert np.array_equal(kh.to_bf16(omoe.bf16_to_float(oa4.float_to_bf16_bits(ref))).float().cpu().numpy(),
                              got.float().cpu().numpy())
    bad = slots.copy()
    bad[0] = -1
    if n > 1:
        bad[n // 2] = 5 * page
    k2, v2 = kv.kv_gather(cache, _i32(bad))
    hit = bad != slots
    assert torch.isnan(k2[torch.from_numpy(hit)]).all() and torch.isnan(v2[torch.from_numpy(hit)]).all()
    keep = torch.from_numpy(~hit).to(DEV)
    assert torch.equal(k2[keep], k[keep]) and torch.equal(v2[keep], v[keep])


def test_no_rows_is_a_no_op():
    cache = kv.NvFp4KvCache.allocate(2, 32, 2, 64)
    before = cache.pages.clone()
    z = torch.empty(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    s = torch.empty(0, dtype=torch.int32, device=DEV)
    kv.kv_append(cache, z, z, s)
    k, v = kv.kv_gather(cache, s)
    assert k.shape == v.shape == (0, 2, 64) and torch.equal(cache.pages, before)


def test_wrappers_refuse_before_any_launch():
    cache = kv.NvFp4KvCache.allocate(2, 32, 2, 64)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    s = torch.zeros(3, dtype=torch.int32, device=DEV)
    wide = torch.zeros(3, 2, 132, dtype=torch.bfloat16, device=DEV)
    for bad_k in (k.float(), k.half()):
        with pytest.raises(TypeError):
            kv.kv_append(cache, bad_k, k, s)
    for bad_k in (k[:2], k[:, :1], k[..., :32], wide[..., :64], k.transpose(0, 1), k.cpu(), k[0],
                  torch.zeros(3, 132, dtype=torch.bfloat16, device=DEV)[:, 4:].unflatten(1, (2, 64))):
        with pytest.raises(ValueError):
            kv.kv_append(cache, bad_k, k, s)
    with pytest.raises(TypeError):
        kv.kv_append(cache, k, k, s.long())
    with pytest.raises(ValueError):
        kv.kv_gather(cache, s.cpu())
    for bad in (dict(page_size=64), dict(page_size=32, k_gscale=0.0), dict(page_size=32, v_gscale=float("nan"))):
        with pytest.raises(ValueError):
            kv.NvFp4KvCache(cache.pages, **bad)
    with pytest.raises(ValueError):
        kv.NvFp4KvCache(cache.pages[..., :100], 32)
    z = torch.zeros(2, dtype=torch.int32, device=DEV)
    t = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    for args in ((z, z[:1], t, z, 32, 2, 2), (z, z, t[:1], z, 32, 2, 2), (z, z, t, z, 32, 2, -1), (z, z, t, z.cpu(), 32, 2, 2)):
        with pytest.raises(ValueError):
            kv.kv_plan(*args)
    from nvfp4_weight_quantized_amd import MoeError
    with pytest.raises(MoeError):
        kv.kv_plan(z, z, t, z, 33, 2, 2)
    for args in ((z, z, t, z, 32, 2, 2 ** 31), (z, z, t, z, 2 ** 32 + 32, 2, 2), (z, z, t, z, 32, 2 ** 32 + 2, 2)):
        with pytest.raises(ValueError):
            kv.kv_plan(*args)
    for name in ("pages", "page_size", "k_gscale", "v_gscale"):      # the launches would not see a change
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
