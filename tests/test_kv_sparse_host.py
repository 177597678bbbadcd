"""Sparse attention over the cache, CPU only: the oracle against independent statements, and the host-side refusals of
the C ABI and of the Python wrappers (nothing is launched)."""

import ctypes

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_weight_quantized_amd import _lib as L
from nvfp4_weight_quantized_amd import kv_sparse
from oracle import kv_cache as okv
from oracle import kv_sparse as osp

INV = L.MOE_ERR_INVALID_ARGUMENT


def test_oracle_index_is_the_mean_of_the_keys():
    c = kh.Case(1, 64, 2, 1, 64, [(5, 100), (130, 0)])
    total = c.pages.shape[0]
    codes, scales = np.zeros((total, 2, 64), np.int8), np.zeros((total, 2), np.float32)
    offsets = np.concatenate([[0], np.cumsum(c.lens)]).astype(np.int32)          # whole lengths
    osp.index_update(codes, scales, c.pages, c.page, offsets, c.lens, c.table, int(offsets[-1]))
    for r in range(2):
        for b in range(-(-int(c.lens[r]) // c.page)):
            at = np.arange(b * c.page, min((b + 1) * c.page, int(c.lens[r])))
            k = okv.decode(c.pages, c.page, okv.slots_of(c.table[r], c.page, at[0], at[-1] + 1), c.d_k, False).mean(0)
            phys = c.table[r, b]
            got = codes[phys].astype(np.float64) * scales[phys][:, None] * c.d_k
            step = np.abs(k).max(-1, keepdims=True) / 127
            assert np.all(np.abs(got - k) <= step * (0.5 + 1e-5)) and np.abs(codes[phys]).max() == 127


def test_oracle_choice_takes_the_highest_products():
    rng = np.random.default_rng(2)
    codes = rng.integers(-127, 128, (40, 1, 64)).astype(np.int8)
    scales = rng.uniform(0.1, 1, (40, 1)).astype(np.float32)
    table = rng.permutation(40)[None, :].astype(np.int32)
    q = kh.bf16(rng, (1, 2, 64))
    got = osp.select(q, codes, scales, 32, [0, 1], [40 * 32 - 3], table, 7, 2, 3)[0, 0]
    assert list(got[:2]) == [0, 1] and list(got[-3:]) == [37, 38, 39] and np.all(np.diff(got) > 0)
    means = codes[table[0], 0].astype(np.float64) * scales[table[0]]
    s = (means @ q[0].T).max(-1)[2:37]
    assert set(got[2:4]) <= set(2 + np.argsort(-s)[:4])          # 8 bits of q move a score by little
    few = osp.select(q, codes, scales, 32, [0, 1], [70], table, 7, 2, 3)[0, 0]
    assert list(few) == [0, 1, 2, -1, -1, -1, -1]


def test_oracle_sparse_attention_over_all_pages_is_attention():
    c = kh.Case(3, 64, 2, 2, 32, [(3, 90), (40, 0), (0, 5)])
    width = c.table.shape[1]
    every = np.broadcast_to(np.arange(width, dtype=np.int32), (c.tokens, 2, width))
    out, lse, _ = osp.attention(c.q, c.pages, c.page, c.d_k, c.d_v, c.offsets, c.lens, c.table, every, c.scale)
    ref, ref_lse, _ = c.reference()
    assert np.allclose(out, ref, rtol=1e-12, equal_nan=True) and np.allclose(lse, ref_lse, rtol=1e-12, equal_nan=True)


# ----------------------------------------------------------------------------- the C ABI's refusals

def _cache(p=4, page=64, h=2, d=128, k=1.0, v=1.0, pages=0x10000):
    return L.KvCache(p, page, h, d, k, v, pages)


def _index(p=4, page=64, h=2, d=128, codes=0x20000, scales=0x30000):
    return L.KvIndex(p, page, h, d, codes, scales)


def _update(cache, index, off=0x3000, lens=0x3100, r=2, table=0x3200, width=4, t=3):
    return L.lib().moe_nvfp4_kv_index_update(ctypes.byref(cache) if cache else None,
                                             ctypes.byref(index) if index else None, off, lens, r, table, width, t, None)


def _select(index, q=0x2000, stride=512, t=3, heads=4, off=0x3000, lens=0x3100, r=2, table=0x3200, width=4, top_k=3,
            first=1, last=1, out=0x4000):
    return L.lib().moe_nvfp4_kv_select(ctypes.byref(index) if index else None, q, stride, t, heads, off, lens, r, table,
                                       width, top_k, first, last, out, None)


def _attend(cache, q=0x2000, stride=512, t=3, heads=4, off=0x3000, lens=0x3100, r=2, table=0x3200, width=4,
            selected=0x5000, top_k=3, scale=0.1, out=0x4000, lse=None, fill=False, ws=0x100000, ws_bytes=1 << 40):
    f = L.lib().moe_nvfp4_kv_sparse_attention_fill if fill else L.lib().moe_nvfp4_kv_sparse_attention
    return f(ctypes.byref(cache) if cache else None, q, stride, t, heads, off, lens, r, table, width, selected, top_k,
             scale, out, lse, ws, ws_bytes, None)


STEP = [dict(off=None), dict(off=0x3002), dict(lens=None), dict(lens=0x3101), dict(r=-1), dict(r=4097), dict(table=None),
        dict(table=0x3203), dict(width=-1), dict(r=4096, width=1 << 20), dict(t=-1)]


@pytest.mark.parametrize("bad", [dict(p=0), dict(page=40), dict(page=65568), dict(h=0), dict(h=1025), dict(d=96),
                                 dict(codes=None), dict(codes=0x20008), dict(scales=None), dict(scales=0x30002)])
def test_a_bad_index_is_refused(bad):
    assert _update(_cache(), _index(**bad)) == INV
    assert _select(_index(**bad)) == INV


@pytest.mark.parametrize("bad", STEP + [dict(t=1 << 30), dict(r=4096, width=8, t=1 << 29)])
def test_index_update_refusals(bad):
    assert _update(_cache(), _index(), **bad) == INV


def test_index_update_needs_a_cache_of_its_sizes():
    assert _update(None, _index()) == _update(_cache(), None) == INV
    for other in (dict(p=5), dict(page=32), dict(h=1), dict(d=64)):
        assert _update(_cache(), _index(**other)) == INV
    for none in (dict(t=0), dict(r=0), dict(width=0)):
        assert _update(_cache(), _index(), **none) == L.MOE_OK


@pytest.mark.parametrize("bad", STEP + [dict(q=None), dict(q=0x2008), dict(stride=511), dict(stride=504), dict(heads=0),
                                        dict(heads=3), dict(heads=130), dict(width=16385), dict(top_k=0), dict(top_k=1),
                                        dict(top_k=1025), dict(first=-1), dict(last=0), dict(first=3), dict(last=3),
                                        dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(out=None), dict(out=0x4002),
                                        dict(t=1 << 23)])
def test_select_refusals(bad):
    assert _select(_index(), **bad) == INV


@pytest.mark.parametrize("fill", [False, True])
@pytest.mark.parametrize("bad", STEP + [dict(q=None), dict(q=0x2008), dict(stride=511), dict(stride=504), dict(heads=0),
                                        dict(heads=3), dict(heads=130), dict(selected=None), dict(selected=0x5001),
                                        dict(top_k=0), dict(top_k=1025), dict(scale=0.0), dict(scale=float("nan")),
                                        dict(scale=float("inf")), dict(scale=1e-39), dict(scale=2.0 ** 101),
                                        dict(out=None), dict(out=0x4008), dict(lse=0x6002), dict(t=1 << 29),
                                        dict(t=1 << 24, heads=64)])
def test_sparse_attention_refusals(bad, fill):
    assert _attend(_cache(), fill=fill, **bad) == INV


def test_no_ops():
    assert _select(None) == _attend(None) == INV
    assert _select(_index(), t=0) == _attend(_cache(), t=0) == _attend(_cache(), r=0) == L.MOE_OK
    assert _attend(_cache(), r=0, fill=True, out=None) == INV
    for bad in (dict(d=96), dict(page=40), dict(k=0.0), dict(pages=None)):
        assert _attend(_cache(**bad)) == INV


def test_workspace_sizes():
    size = L.lib().moe_nvfp4_kv_sparse_attention_workspace_size
    for bad in ((-1, 1, 4, 2, 128, 64, 3), (1, -1, 4, 2, 128, 64, 3), (1, 4097, 4, 2, 128, 64, 3), (1, 1, 5, 2, 128, 64, 3),
                (1, 1, 130, 2, 128, 64, 3), (1, 1, 4, 2, 96, 64, 3), (1, 1, 4, 2, 128, 40, 3), (1, 1, 4, 2, 128, 64, 0),
                (1, 1, 4, 2, 128, 64, 1025), (1 << 30, 1, 4, 2, 128, 64, 3)):
        assert size(*bad) == 0
    assert size(0, 1, 4, 2, 128, 64, 300) == size(1, 0, 4, 2, 128, 64, 300) == 0
    long = dict(t=1, top_k=300)
    need = size(1, 2, 4, 2, 128, 64, 300)
    assert need > 0
    for fill in (False, True):
        assert _attend(_cache(), ws=None, fill=fill, **long) == _attend(_cache(), ws_bytes=need - 1, fill=fill,
                                                                        **long) == L.MOE_ERR_WORKSPACE_TOO_SMALL
        assert _attend(_cache(), ws=0x100008, fill=fill, **long) == INV


def test_wrappers_refuse_cpu_tensors():
    with pytest.raises(ValueError):
        kv_sparse.NvFp4KvIndex(torch.zeros(2, 1, 64, dtype=torch.int8), torch.zeros(2, 1), 64)
    with pytest.raises(TypeError):
        kv_sparse.NvFp4KvIndex(torch.zeros(2, 1, 64), torch.zeros(2, 1), 64)
