"""Appends on both sides of the size from which quads of positions are quantized together: the oracle's bytes, for runs
that fill, begin and end inside units and quads, for scattered slots, and for slots outside the cache among them."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_weight_quantized_amd import kv
from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu
QUADS = 1 << 19      # rows * groups


def _slots(rng, runs, page):
    out, at = [], 0
    for first, n in runs:                          # each run has pages of its own
        pages_of = rng.permutation(-(-(first + n) // page)) + at
        at += len(pages_of)
        pos = first + np.arange(n)
        out.append(pages_of[pos // page] * page + pos % page)
    return np.concatenate(out), at


@pytest.mark.parametrize("dim,heads", [(64, 128), (128, 64), (256, 32)])
@pytest.mark.parametrize("kind", ["runs", "one", "scattered", "holes"])
@pytest.mark.parametrize("rows", [511, 515])
def test_append_around_the_size_of_quads(dim, heads, kind, rows):
    rng = np.random.default_rng(dim + rows)
    page = 64
    runs = [(0, rows)] if kind != "runs" else [(3, 40), (64, 33), (31, 1), (0, 200), (90, rows - 274)]
    slots, n_pages = _slots(rng, runs, page)
    if kind == "scattered":
        slots = rng.permutation(n_pages * page)[:rows]
    if kind == "holes":
        slots = slots.copy()
        slots[2::7] = rng.choice([-1, n_pages * page, 2 ** 31 - 1, -2 ** 31], len(slots[2::7]))
    slots = slots.astype(np.int32)
    assert (2 * rows * heads * (dim // 16) >= QUADS) == (rows > 512)
    k, v = kh.bf16(rng, (2, rows, heads, dim))
    pages = rng.integers(0, 256, (n_pages, heads, page // 32, 36 * dim)).astype(np.uint8)
    want = pages.copy()
    okv.append(want, page, k, slots, 0.0625, False)
    okv.append(want, page, v, slots, 0.5, True)
    cache = kv.NvFp4KvCache(torch.from_numpy(pages).to("cuda"), page, 0.0625, 0.5)
    kv.kv_append(cache, kh.to_bf16(k), kh.to_bf16(v), torch.from_numpy(slots).to("cuda"))
    assert np.array_equal(cache.pages.cpu().numpy(), want)
