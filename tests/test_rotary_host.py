"""Rotary positions, CPU only: the oracle against an independent statement, and the host-side refusals of the C ABI and
of the Python wrappers (nothing is launched)."""

import ctypes

import numpy as np
import pytest
import torch

import nvfp4_weight_quantized_amd as moe
from nvfp4_weight_quantized_amd import _lib as L
from oracle import rotary as orot

INV = L.MOE_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_is_a_complex_product_and_keeps_relative_positions(interleaved):
    rng = np.random.default_rng(0)
    n, dim = 8, 32
    freq = 10000.0 ** (-np.arange(n) / n)
    x, y = rng.normal(size=(2, 1, 1, dim))
    first = 2 * np.arange(n) if interleaved else np.arange(n)
    second = first + (1 if interleaved else n)
    out, _ = orot.rotate(x, [7], freq, interleaved=interleaved)
    z = (x[0, 0, first] + 1j * x[0, 0, second]) * np.exp(7j * freq)
    assert np.allclose(out[0, 0, first], z.real, atol=1e-14) and np.allclose(out[0, 0, second], z.imag, atol=1e-14)
    assert np.array_equal(out[..., 2 * n:], x[..., 2 * n:])
    dots = [float(np.sum(orot.rotate(x, [a], freq, interleaved=interleaved)[0][..., :2 * n] *
                         orot.rotate(y, [a - 5], freq, interleaved=interleaved)[0][..., :2 * n])) for a in (5, 100, 3000)]
    assert np.allclose(dots, dots[0], atol=1e-10)


def _rot(dim=128, pairs=64, axes=1, interleaved=0, scale=1.0, freq=0x1000, axis=None):
    return L.RotaryStruct(dim, pairs, axes, interleaved, scale, freq, axis)


def _rotary(rot, x=0x2000, xs=256, t=3, heads=2, pos=0x3000, ps=3, out=0x4000, os_=256):
    return L.lib().moe_rotary(ctypes.byref(rot) if rot else None, x, xs, t, heads, pos, ps, out, os_, None)


BAD_ROTARIES = [dict(dim=0), dict(dim=24), dict(dim=528), dict(pairs=0), dict(pairs=12), dict(pairs=72), dict(pairs=-8),
                dict(axes=0), dict(axes=5), dict(interleaved=2), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(freq=None), dict(freq=0x1004), dict(axis=0x1002)]


def _append(cache, rot, q=0x2000, qs=512, heads=4, k=0x3000, ks=256, v=0x4000, vs=256, pos=0x5000, ps=3, slots=0x6000,
            t=3, out=0x7000, os_=512):
    return L.lib().moe_nvfp4_kv_append_rotary(ctypes.byref(cache) if cache else None, ctypes.byref(rot) if rot else None,
                                              q, qs, heads, k, ks, v, vs, pos, ps, slots, t, out, os_, None)


def _cache(p=4, page=64, h=2, d=128, k=1.0, v=1.0, pages=0x10000):
    return L.KvCache(p, page, h, d, k, v, pages)


@pytest.mark.parametrize("bad", BAD_ROTARIES)
def test_a_bad_rotary_is_refused(bad):
    assert _rotary(_rot(**bad)) == INV
    assert _append(_cache(), _rot(**bad)) == INV


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=0x2008), dict(xs=255), dict(xs=248), dict(xs=260), dict(t=-1),
                                 dict(heads=0), dict(heads=1 << 17), dict(pos=None), dict(pos=0x3002), dict(out=None),
                                 dict(out=0x4008), dict(os_=248), dict(os_=257), dict(out=0x2000, os_=512),
                                 dict(t=1 << 24), dict(t=1 << 23, heads=128, xs=1 << 14, os_=1 << 14)])
def test_rotary_refusals(bad):
    assert _rotary(_rot(), **bad) == INV
    assert _rotary(_rot(), t=0, **{k: v for k, v in bad.items() if k in ("x", "pos", "out")}) == L.MOE_OK


def test_positions_of_several_axes_must_not_overlap():
    assert _rotary(_rot(axes=3, axis=0x9000), ps=2) == INV
    assert _append(_cache(), _rot(axes=3, axis=0x9000), ps=2) == INV


@pytest.mark.parametrize("bad", [dict(q=None), dict(q=0x2008), dict(qs=504), dict(heads=0), dict(k=None), dict(k=0x3008),
                                 dict(ks=248), dict(v=None), dict(v=0x4004), dict(vs=260), dict(pos=None),
                                 dict(slots=None), dict(slots=0x6002), dict(t=-1), dict(out=None), dict(out=0x7008),
                                 dict(os_=504), dict(out=0x2000, os_=1024), dict(t=1 << 24)])
def test_append_rotary_refusals(bad):
    assert _append(_cache(), _rot(), **bad) == INV


def test_append_rotary_refuses_a_bad_cache_and_another_head_dim():
    for bad in (dict(p=0), dict(page=40), dict(h=0), dict(d=96), dict(k=0.0), dict(pages=None)):
        assert _append(_cache(**bad), _rot()) == INV
    assert _append(None, _rot()) == _append(_cache(), None) == INV
    assert _append(_cache(d=64), _rot()) == INV
    assert _append(_cache(), _rot(), t=0) == L.MOE_OK


def test_wrappers_refuse_cpu_tensors_and_wrong_types():
    f = torch.ones(64, dtype=torch.float64)
    with pytest.raises(ValueError):
        moe.Rotary(f, 128)
    with pytest.raises(TypeError):
        moe.Rotary(f.float(), 128)
    with pytest.raises(ValueError):
        moe.Rotary.from_theta(128, rotary_dim=63, device="cpu")
    with pytest.raises(ValueError):
        moe.Rotary.from_theta(128, theta=0.0, device="cpu")
    with pytest.raises(ValueError):
        moe.Rotary.from_theta(128, sections=(16, 24, 23), device="cpu")
    with pytest.raises(ValueError):
        moe.Rotary.from_theta(128, sections=(0, 0, 64), spread=True, device="cpu")
