"""Key/value cache, CPU only: the oracle's page layout and plan against independent statements, and the
host-side refusals of the C ABI and of the Python wrappers (nothing is launched)."""

import ctypes

import numpy as np
import pytest
import torch

from nvfp4_weight_quantized_amd import _lib as L
from nvfp4_weight_quantized_amd import kv
from oracle import kv_cache as okv
from oracle import nvfp4 as onv

INV, SMALL = L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_unit_layout_covers_every_byte_once(dim):
    """Keys and values with their scales fill the 36*dim bytes of a unit exactly, 16 elements per scale."""
    count = np.zeros(36 * dim, np.int64)
    for values in (False, True):
        byte, shift, scale = okv.unit_maps(dim, values)
        nib = np.zeros((36 * dim, 2), np.int64)
        np.add.at(nib, (byte, shift // 4), 1)
        used = np.unique(byte)
        assert np.all(nib[used] == 1) and len(used) == 16 * dim
        s_used, s_count = np.unique(scale, return_counts=True)
        assert len(s_used) == 2 * dim and np.all(s_count == 16)
        count[used] += 1
        count[s_used] += 1
    assert np.all(count == 1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_units_are_the_matrix_operands(dim):
    """Lane l = 16u + n of the 16x16x32 key operand reads its words at 16*l; lane 16q + m of the value
    operand finds its eight positions 4q..4q+3, 16+4q..16+4q+3 in consecutive bytes."""
    byte, _, scale = okv.unit_maps(dim, False)
    for p in range(32):
        for s in range(dim // 32):
            for u in range(4):
                w = (p // 16) * (dim // 32) + s
                assert byte[p, 32 * s + 8 * u] == 1024 * (w // 4) + 16 * (16 * u + p % 16) + 4 * (w % 4)
                assert [byte[p, 32 * s + 8 * u + e] for e in range(8)] == [
                    byte[p, 32 * s + 8 * u] + e // 2 for e in range(8)]
    byte, _, scale = okv.unit_maps(dim, True)
    for q in range(4):
        pos = [4 * q + i for i in range(4)] + [16 + 4 * q + i for i in range(4)]
        for d in range(dim):
            b = [byte[p, d] for p in pos]
            assert b == list(range(b[0], b[0] + 8)) and b[0] % 8 == 0
            s = [scale[p, d] for p in pos]
            assert s == list(range(s[0], s[0] + 8)) and s[0] % 8 == 0


def test_oracle_append_and_decode_round_trip():
    rng = np.random.default_rng(5)
    dim, heads, page = 64, 3, 64
    pages = okv.new_pages(3, page, heads, dim, 0xFF)
    rows = rng.normal(0, 1, (70, heads, dim)).astype(np.float32).astype(np.float64)
    slots = rng.permutation(3 * page)[:70]
    for values in (False, True):
        okv.append(pages, page, rows, slots, 0.25, values)
        got = okv.decode(pages, page, slots, 0.25, values)
        p, s = onv.quantize(rows.reshape(-1, dim).astype(np.float32), 0.25)
        assert np.array_equal(got.reshape(-1, dim), onv.dequantize(p, s, 0.25))


def test_oracle_attention_is_softmax():
    """Against a dense statement on one request."""
    rng = np.random.default_rng(6)
    dim, page = 64, 32
    pages = okv.new_pages(3, page, 1, dim)
    table = np.array([[2, 0, 1]], np.int32)
    slots = okv.slots_of(table[0], page, 0, 75)
    k, v = rng.normal(0, 1, (2, 75, 1, dim))
    okv.append(pages, page, k, slots, 0.01, False)
    okv.append(pages, page, v, slots, 0.02, True)
    kd, vd = okv.decode(pages, page, slots, 0.01, False)[:, 0], okv.decode(pages, page, slots, 0.02, True)[:, 0]
    q = rng.normal(0, 1, (4, 2, dim))
    out, lse, _ = okv.attention(q, pages, page, 0.01, 0.02, [0, 4], [75], table, 0.125, window=9)
    for i in range(4):
        for h in range(2):
            s = 0.125 * kd @ q[i, h]
            seen = (np.arange(75) <= 71 + i) & (np.arange(75) > 71 + i - 9)
            e = np.where(seen, np.exp(s), 0.0)
            assert np.allclose(out[i, h], e @ vd / e.sum(), rtol=1e-12)
            assert np.isclose(lse[i, h], np.log(e.sum()), rtol=1e-12)


# ----------------------------------------------------------------------------- the C ABI's refusals

def _cache(p=4, page=64, h=2, d=128, k=1.0, v=1.0, pages=0x1000):
    return L.KvCache(p, page, h, d, k, v, pages)


def _append(cache, k=0x2000, v=0x3000, ks=256, vs=256, slots=0x4000, t=3):
    return L.lib().moe_nvfp4_kv_append(ctypes.byref(cache) if cache else None, k, v, ks, vs, slots, t, None)


BAD_CACHES = [dict(p=0), dict(p=-1), dict(page=0), dict(page=16), dict(page=48), dict(page=65536 + 32), dict(h=0),
              dict(h=1025), dict(d=32), dict(d=96), dict(d=512), dict(p=1 << 20, page=2048), dict(k=0.0), dict(v=-1.0),
              dict(k=float("nan")), dict(v=float("inf")), dict(k=2.0 ** -65), dict(v=2.0 ** 65), dict(pages=None),
              dict(pages=0x1008)]


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_a_bad_cache_is_refused(bad):
    c = _cache(**bad)
    assert _append(c) == INV
    assert L.lib().moe_nvfp4_kv_gather(ctypes.byref(c), 0x4000, 3, 0x2000, 0x3000, None) == INV
    assert _attend(c) == INV


def test_append_and_gather_refusals():
    assert _append(None) == INV
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(k=0x2008), dict(v=0x3002), dict(slots=0x4002),
                dict(ks=255), dict(vs=248), dict(ks=260), dict(t=-1)):
        assert _append(_cache(), **bad) == INV, bad
    assert _append(_cache(), t=0) == L.MOE_OK
    g = L.lib().moe_nvfp4_kv_gather
    c = _cache()
    assert g(None, 0x4000, 3, 0x2000, 0x3000, None) == INV
    assert g(ctypes.byref(c), 0x4000, -1, 0x2000, 0x3000, None) == INV
    assert g(ctypes.byref(c), None, 3, 0x2000, 0x3000, None) == INV
    assert g(ctypes.byref(c), 0x4000, 3, 0x2008, 0x3000, None) == INV
    assert g(ctypes.byref(c), 0x4000, 3, 0x2000, None, None) == INV
    assert g(ctypes.byref(c), None, 0, None, None, None) == L.MOE_OK


def _plan(r=2, page=64, pages=8, nf=4, width=3, t=5, kv_lens=0x1000, new=0x1100, free=0x1200, table=0x1300, qo=0x1400,
          lens=0x1500, pos=0x1600, slots=0x1700, used=0x1800):
    return L.lib().moe_kv_plan(kv_lens, new, r, page, pages, free, nf, table, width, t, qo, lens, pos, slots, used, None)


@pytest.mark.parametrize("bad", [dict(r=-1), dict(r=4097), dict(page=0), dict(page=40), dict(page=65568), dict(pages=0),
                                 dict(pages=1 << 26), dict(nf=-1), dict(width=-1), dict(t=-1), dict(kv_lens=None),
                                 dict(new=None), dict(free=None), dict(table=None), dict(qo=None), dict(lens=None),
                                 dict(pos=None), dict(slots=None), dict(used=None), dict(r=4096, width=1 << 20)])
def test_plan_refusals(bad):
    assert _plan(**bad) == INV


def _attend(cache, q=0x2000, stride=512, t=3, heads=4, off=0x3000, lens=0x3100, r=2, table=0x3200, width=4, scale=0.1,
            window=0, out=0x4000, lse=None, ws=0x100000, ws_bytes=1 << 40):
    return L.lib().moe_nvfp4_kv_attention(ctypes.byref(cache) if cache else None, q, stride, t, heads, off, lens, r,
                                          table, width, scale, window, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=0x2008), dict(stride=511), dict(stride=504), dict(stride=516),
                                 dict(t=-1), dict(heads=0), dict(heads=3), dict(heads=2 * 65), dict(off=None),
                                 dict(lens=None), dict(r=-1), dict(r=4097), dict(table=None), dict(width=-1),
                                 dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")),
                                 dict(scale=1e-39), dict(scale=2.0 ** 101), dict(window=-1), dict(out=None), dict(out=0x4008),
                                 dict(t=1 << 30), dict(r=4096, width=1 << 20)])
def test_attention_refusals(bad):
    assert _attend(_cache(), **bad) == INV


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=0x2008), dict(stride=511), dict(t=-1), dict(heads=3), dict(off=None),
                                 dict(lens=None), dict(r=4097), dict(table=None), dict(scale=0.0), dict(window=-1),
                                 dict(out=None), dict(out=0x4008), dict(out=None, r=0), dict(out=0x4008, r=0),
                                 dict(ws=0x100008, width=1000)])
def test_attention_fill_refusals(bad, monkeypatch):
    """The entry that also fills the rows of no request refuses what the other one does, and without requests
    (where every row is filled) outputs that cannot be written."""
    monkeypatch.setattr(L.lib(), "moe_nvfp4_kv_attention", L.lib().moe_nvfp4_kv_attention_fill)
    assert _attend(_cache(), **bad) == INV
    assert _attend(_cache(), t=0) == L.MOE_OK


def test_steps_past_one_launch_are_refused():
    """More rows than a launch of 2^32 work-items holds."""
    assert _append(_cache(), t=(1 << 28) + 1) == INV
    g = L.lib().moe_nvfp4_kv_gather
    assert g(ctypes.byref(_cache()), 0x4000, (1 << 29) - 31, 0x2000, 0x3000, None) == INV
    assert g(ctypes.byref(_cache()), 0x4000, 2 ** 31 - 1, 0x2000, 0x3000, None) == INV
    big = dict(heads=128, stride=128 * 128, t=(1 << 24) - 1)
    assert _attend(_cache(), **big) == INV
    assert _attend(_cache(), **{**big, "t": 1 << 21, "width": 1000}, ws=None) == SMALL      # 2^28 rows: accepted so far


def test_attention_no_ops_and_sizes():
    assert _attend(None) == INV
    assert _attend(_cache(), t=0) == L.MOE_OK
    assert _attend(_cache(), r=0) == L.MOE_OK
    size = L.lib().moe_nvfp4_kv_attention_workspace_size
    for bad in ((-1, 1, 4, 2, 128), (1, -1, 4, 2, 128), (1, 4097, 4, 2, 128), (1, 1, 5, 2, 128), (1, 1, 130, 2, 128),
                (1, 1, 4, 2, 96), (1 << 30, 1, 4, 2, 128)):
        assert size(*bad) == 0
    need = size(3, 2, 4, 2, 128)
    assert need > 0
    for wide in (dict(width=1000), dict(width=1000, t=400)):      # a narrow table may need none
        need = size(wide.get("t", 3), 2, 4, 2, 128)
        assert _attend(_cache(), ws=None, ws_bytes=0, **wide) == SMALL
        assert _attend(_cache(), ws=None, **wide) == SMALL
        assert _attend(_cache(), ws=0x100008, **wide) == INV
    assert _attend(_cache(), ws_bytes=size(3, 2, 4, 2, 128) - 1, width=1000) == SMALL
    cb = L.lib().moe_nvfp4_kv_cache_bytes
    assert cb(10, 64, 8, 128) == 10 * 64 * 8 * 128 * 2 * 9 // 16
    assert cb(0, 64, 8, 128) == cb(10, 40, 8, 128) == cb(10, 64, 0, 128) == cb(10, 64, 8, 80) == 0


# ----------------------------------------------------------------------------- the wrappers' refusals

def test_wrappers_refuse_cpu_tensors_and_wrong_types():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        kv.kv_plan(z, z, torch.zeros(4, 2, dtype=torch.int32), z, 64, 8, 4)
    with pytest.raises(ValueError):
        kv.NvFp4KvCache(torch.zeros(2, 1, 2, 36 * 64, dtype=torch.uint8), 64)
    with pytest.raises(TypeError):
        kv.NvFp4KvCache(torch.zeros(2, 1, 2, 36 * 64), 64)
    with pytest.raises(ValueError):
        kv.NvFp4KvCache.allocate(2, 64, 1, 80, device="cpu")
    with pytest.raises(ValueError):
        kv.NvFp4KvCache.allocate(2, 50, 1, 64, device="cpu")


@pytest.mark.parametrize("old,new,free,width", [
    ([0, 31, 32, 33, 0], [1, 1, 1, 0, 70], 6, 4),
    ([5, 0], [0, 0], 0, 1),
    ([100, -3, 7], [3, 4, -5], 3, 4),
    ([0, 60], [40, 10], 1, 2),      # shortage
    ([90], [20], 5, 3),             # beyond the table
])
def test_oracle_plan_properties(old, new, free, width):
    """Slots of one step are distinct, positions consecutive, and a request's slots follow its table."""
    page, num_pages = 32, 64
    rng = np.random.default_rng(len(old))
    perm = rng.permutation(num_pages)
    table = np.full((len(old), width), -1, np.int32)
    at = 0
    for r, o in enumerate(old):
        n = min(-(-max(o, 0) // page), width)
        table[r, :n] = perm[at:at + n]
        at += n
    tokens = sum(max(n, 0) for n in new) + 3
    off, lens, pos, slots, used, after = okv.plan(old, new, table, perm[at:at + free], page, num_pages, tokens)
    good = slots[slots >= 0]
    assert len(set(good.tolist())) == len(good)
    for r in range(len(old)):
        for t in range(off[r], off[r + 1]):
            assert pos[t] == max(old[r], 0) + t - off[r]
            b = pos[t] // page
            if slots[t] >= 0:
                assert after[r, b] * page + pos[t] % page == slots[t]
    assert np.all(slots[off[-1]:] == -1)
    assert used == sum(-(-(max(o, 0) + max(n, 0)) // page) - -(-max(o, 0) // page) for o, n in zip(old, new))
