"""Attention steps of many requests, up to the limit: tiles cut at the ends of shares are joined wherever they lie, and
padded batches that launch the kernel of many rows as well."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_weight_quantized_amd import kv

pytestmark = pytest.mark.gpu


def _case(seed, dim, kv_heads, group, reqs, **kw):
    return kh.Case(seed, dim, kv_heads, group, 32, reqs, **kw)


@pytest.mark.parametrize("requests,most_new,most_old,dim,kv_heads,group,pad,extra", [
    (1100, 1, 60, 64, 2, 1, 0, 1),       # more tiles than shares, each share with some whole ones
    (1100, 1, 60, 64, 2, 1, 30, 70),     # padded past 1024 rows
    (600, 1, 20, 64, 1, 16, 2600, 70),    # padded by so many that the kernel of many rows is launched too
    (700, 3, 30, 128, 4, 2, 0, 1),
    (900, 2, 20, 256, 2, 3, 0, 40),
    (4096, 1, 20, 64, 1, 2, 0, 1),
    (520, 1, 60, 64, 2, 17, 0, 1),        # 32-row tiles
])
def test_steps_of_many_requests(requests, most_new, most_old, dim, kv_heads, group, pad, extra):
    rng = np.random.default_rng(requests + dim)
    reqs = [(int(rng.integers(0, most_new + 1)), int(rng.integers(0, most_old + 1))) for _ in range(requests)]
    case = _case(70, dim, kv_heads, group, reqs, pad=pad, width_extra=extra)
    cache, q, args = case.cache(), kh.to_bf16(case.q), case.args()
    out, lse = kv.kv_attention(cache, q, *args, scale=case.scale, return_lse=True)
    kh.check_attention(case, out, lse)
    again, again_lse = kv.kv_attention(cache, q, *args, scale=case.scale, return_lse=True)
    assert torch.equal(again, out) and torch.equal(again_lse, lse)


def test_long_rows_among_many_short_ones():
    """A few rows that span many shares, at the ends and in the middle of hundreds that fill a part of one."""
    reqs = [(1, 3000)] + [(1, 5 + i % 40) for i in range(500)] + [(2, 5000), (1, 0), (1, 2047)] + \
        [(1, i % 33) for i in range(500)] + [(1, 4000)]
    case = _case(71, 64, 2, 2, reqs)
    kh.check_attention(case, *case.run())
