"""Rows of a padded batch that belong to no request, where the call makes its outputs itself: zeros and -inf, not
what the memory held before."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_weight_quantized_amd import kv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dirty(case):
    """Leaves blocks of NaN of the outputs' sizes with the allocator."""
    n = case.tokens * case.heads
    for _ in range(3):
        held = [torch.full((n * case.dim,), float("nan"), dtype=torch.bfloat16, device=DEV),
                torch.full((n,), float("nan"), dtype=torch.float32, device=DEV)]
        torch.cuda.synchronize()
        del held


@pytest.mark.parametrize("reqs,extra", [
    ([(1, 50), (1, 3)], 1), ([(1, 50), (1, 3)], 900), ([(60, 9), (1, 100), (3, 3)], 1), ([(300, 0)], 40000),
    ([(1, 5)] * 70, 1), ([(0, 10)], 1)])
@pytest.mark.parametrize("dim,pad,shift", [(64, 1, 0), (128, 21, 5), (256, 333, 0), (128, 1200, 40)])
def test_rows_of_no_request_are_zeros(reqs, extra, dim, pad, shift):
    case = kh.Case(60, dim, 2, 3, 32, reqs, pad=pad, width_extra=extra)
    case.offsets += min(shift, pad)
    a, b = int(case.offsets[0]), int(case.offsets[-1])
    cache, q, args = case.cache(), kh.to_bf16(case.q), case.args()
    _dirty(case)
    out, lse = kv.kv_attention(cache, q, *args, return_lse=True)
    for rows in (slice(0, a), slice(b, None)):
        assert (out[rows] == 0).all() and torch.isneginf(lse[rows]).all()
    if b > a:
        kh.check_attention(case, out, lse, rows=slice(a, b))
    # lse alone is the call's
    given = torch.full_like(out, 7.0)
    _dirty(case)
    _, lse = kv.kv_attention(cache, q, *args, return_lse=True, out=given)
    assert torch.equal(given[a:b], out[a:b])
    for rows in (slice(0, a), slice(b, None)):
        assert (given[rows] == 7.0).all() and torch.isneginf(lse[rows]).all()


def test_a_step_without_requests_is_zeros():
    case = kh.Case(61, 64, 1, 2, 32, [(1, 10)], pad=40)
    cache, q = case.cache(), kh.to_bf16(case.q)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    _dirty(case)
    out, lse = kv.kv_attention(cache, q, z, z[:0], torch.zeros(0, 4, dtype=torch.int32, device=DEV), return_lse=True)
    assert (out == 0).all() and torch.isneginf(lse).all()


def test_captured_padding_follows_the_offsets():
    """One captured step, the requests' share of the batch changes between replays."""
    case = kh.Case(62, 128, 2, 4, 32, [(1, 80), (1, 7), (1, 200)], pad=9)
    cache, q, (off, lens, table) = case.cache(), kh.to_bf16(case.q), case.args()
    kv.kv_attention(cache, q, off, lens, table)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = kv.kv_attention(cache, q, off, lens, table, return_lse=True)
    for offsets in ([0, 1, 2, 3], [0, 1, 1, 2], [4, 5, 6, 7], [0, 0, 0, 0], [0, 1, 2, 3]):
        off.copy_(torch.tensor(offsets, dtype=torch.int32))
        out.fill_(float("nan"))
        lse.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, want_lse = kv.kv_attention(cache, q, off, lens, table, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        keep = np.arange(case.tokens)
        idle = torch.from_numpy((keep < offsets[0]) | (keep >= offsets[-1])).to(DEV)
        assert (out[idle] == 0).all() and torch.isneginf(lse[idle]).all() and torch.isfinite(out).all()
