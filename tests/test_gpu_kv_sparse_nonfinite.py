"""Sparse attention with query rows that hold NaN or infinities and whose scores are NaN: such a row is NaN where it sees a
position, zeros and lse = -inf where it sees none, and the rows beside it in a tile keep their bounds."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from test_gpu_kv_sparse import _lists, check_sparse

pytestmark = pytest.mark.gpu


# Tiles of sixteen, four, three and eight tokens (16 or 32 rows), of one token (four and eight waves), of a part of a token,
# and splits joined by a second launch.
@pytest.mark.parametrize("dim,kv_heads,group,page,reqs,top_k", [
    (64, 1, 1, 32, [(520, 300)], 5),
    (128, 2, 4, 64, [(131, 900), (150, 0)], 4),
    (256, 3, 5, 32, [(175, 250)], 5),
    (64, 10, 16, 32, [(260, 60)], 3),
    (64, 4, 4, 32, [(2510, 60)], 3),
    (128, 2, 4, 32, [(9, 400), (1, 700)], 6),
    (64, 8, 2, 32, [(33, 2500)], 64),
    (64, 2, 40, 32, [(5, 200)], 4),
    (128, 1, 4, 64, [(1, 3000), (1, 2000)], 40),
])
def test_rows_that_see_nothing_stay_zeros(dim, kv_heads, group, page, reqs, top_k):
    c = kh.Case(200, dim, kv_heads, group, page, reqs)
    rng = np.random.default_rng(201)
    lists = _lists(rng, c, top_k)
    if c.tokens == 2:
        lists[1] = -1
    else:
        lists[rng.random(c.tokens) < 0.3] = -1                      # no list for any head
        lists[rng.random((c.tokens, kv_heads)) < 0.2] = -1          # or for one
    bad = rng.random((c.tokens, c.heads)) < 0.4
    if c.tokens == 2:
        bad[1] = True
    for i, (t, h) in enumerate(np.argwhere(bad)):
        if i % 3 == 0:
            c.q[t, h, i % dim] = np.nan
        elif i % 3 == 1:
            c.q[t, h] = np.inf                                      # products of both signs
        else:
            c.q[t, h, ::2], c.q[t, h, 1::2] = np.nan, -np.inf
    empty = np.repeat((lists < 0).all(-1), group, 1)
    assert (empty & bad).any()
    with np.errstate(invalid="ignore"):
        out, lse = check_sparse(c, lists)
    out, lse = out.float().cpu().numpy(), lse.cpu().numpy()
    assert (out[empty] == 0).all() and np.isneginf(lse[empty]).all()
    assert np.isnan(out[bad & ~empty]).all() and np.isfinite(out[~bad]).all()


def test_they_are_the_rows_of_one_token_at_a_time():
    """Which rows are NaN and which are zeros does not depend on how many tokens a call holds."""
    c = kh.Case(202, 64, 1, 4, 32, [(530, 100)])
    rng = np.random.default_rng(203)
    lists = _lists(rng, c, 4)
    lists[::5] = -1
    c.q[::10] = np.nan
    off, lens, table = c.args()
    cache, q, chosen = c.cache(), kh.to_bf16(c.q), torch.from_numpy(lists).cuda()
    many, many_lse = moe.kv_sparse_attention(cache, q, off, lens, table, chosen, return_lse=True)
    for t in (0, 5, 10, 20, 525):
        one = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        at = torch.tensor([100 + t + 1], dtype=torch.int32, device="cuda")
        out, lse = moe.kv_sparse_attention(cache, q[t:t + 1], one, at, table, chosen[t:t + 1], return_lse=True)
        assert torch.equal(out.isnan(), many[t:t + 1].isnan()) and torch.equal(lse.isneginf(), many_lse[t:t + 1].isneginf())
        assert torch.equal(out == 0, many[t:t + 1] == 0)
