"""The launches of the sparse attention (tiles of several tokens, of 32 rows, splits joined by a second launch), each at
the sizes that take it, against the float64 oracle within the bounds that tests/kv_helpers.py derives."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from nvfp4_weight_quantized_amd import kv_sparse
from test_gpu_kv_sparse import _i32, _lists, check_sparse

pytestmark = pytest.mark.gpu
DEV = "cuda"


# More than 512 tokens and heads: tiles of several tokens, which go through the union of their lists.
@pytest.mark.parametrize("seed,dim,kv_heads,group,page,reqs,top_k,pad,overlap", [
    (0, 64, 1, 1, 32, [(300, 90), (220, 400)], 5, 0, 0.5),            # sixteen tokens a tile, the last not full
    (1, 64, 1, 1, 32, [(530, 30)], 7, 3, 0.0),                        # lists that share little
    (2, 64, 3, 2, 32, [(180, 200)], 6, 0, 1.0),                       # and all
    (3, 128, 2, 5, 64, [(131, 300), (1, 900), (0, 64), (150, 0)], 4, 2, 0.5),      # three tokens a tile
    (4, 256, 3, 4, 32, [(175, 250)], 5, 0, 0.5),
    (5, 64, 2, 7, 96, [(270, 500)], 3, 0, 0.5),
    (6, 128, 2, 16, 32, [(260, 100)], 4, 0, 0.5),                     # one token a tile after all
    (7, 64, 8, 40, 32, [(66, 100)], 3, 0, 0.5),                       # two tiles per token
    (8, 64, 1, 1, 32, [(1, 10 + i % 90) for i in range(530)], 3, 0, 0.5),
    (9, 64, 1, 1, 32, [(520, 3000)], 100, 0, 0.8),                    # ten tokens' lists fill the entries
])
def test_tiles_of_several_tokens(seed, dim, kv_heads, group, page, reqs, top_k, pad, overlap):
    c = kh.Case(100 + seed, dim, kv_heads, group, page, reqs, pad=pad)
    assert c.tokens * kv_heads > 512
    out, _ = check_sparse(c, _lists(np.random.default_rng(seed), c, top_k, overlap))
    if pad:
        assert (out[-pad:] == 0).all()


def test_tiles_of_32_rows():
    c = kh.Case(120, 64, 8, 16, 32, [(200, 60), (130, 300)])
    assert c.tokens * c.heads >= 40000
    check_sparse(c, _lists(np.random.default_rng(121), c, 4))


def test_a_bad_page_of_a_union():
    """Only the rows whose own list holds the page, and that reach it, are NaN."""
    c = kh.Case(122, 64, 2, 4, 32, [(280, 200)])
    lists = _lists(np.random.default_rng(123), c, 4)
    c.table[0, [2, 14]] = -1, c.pages.shape[0]
    out, _ = check_sparse(c, lists)
    bad = torch.isnan(out).all(-1)
    assert bad.any() and not bad.all(-1).all()


# One token per tile, long lists: splits of the units.
@pytest.mark.parametrize("seed,dim,kv_heads,group,page,reqs,top_k", [
    (0, 128, 1, 4, 64, [(1, 5000)], 40),
    (1, 128, 2, 8, 64, [(1, 3000), (1, 64), (3, 2600), (0, 40), (1, 900)], 30),
    (2, 64, 1, 16, 32, [(1, 9000)], 130),
    (3, 256, 2, 2, 32, [(2, 3000)], 50),
    (4, 128, 1, 33, 32, [(1, 3000)], 64),                             # 32 rows, two tiles
    (5, 64, 1, 1, 32, [(1, 40000)], 1024),
    (6, 128, 3, 3, 256, [(1, 6000), (1, 20)], 9),
])
def test_splits_of_long_lists(seed, dim, kv_heads, group, page, reqs, top_k):
    c = kh.Case(140 + seed, dim, kv_heads, group, page, reqs, pad=1)
    assert moe.kv_sparse_attention_workspace_size(c.tokens, len(reqs), c.heads, kv_heads, dim, page, top_k) > 0
    lists = _lists(np.random.default_rng(seed), c, top_k)
    lists[0, 0, 1:] = -1                                              # most splits of this tile are empty
    out, lse = check_sparse(c, lists)
    assert (out[-1] == 0).all() and torch.isneginf(lse[-1]).all()
    lists[0, 0, :] = -1                                               # and all of them
    check_sparse(c, lists)


def test_a_given_workspace():
    c = kh.Case(150, 128, 2, 4, 64, [(1, 3000), (1, 700)])
    lists = _lists(np.random.default_rng(151), c, 40)
    need = moe.kv_sparse_attention_workspace_size(2, 2, 8, 2, 128, 64, 40)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)           # NaN everywhere
    a, la = check_sparse(c, lists)
    b, lb = check_sparse(c, lists, workspace=ws[:need])
    assert torch.equal(a, b) and torch.equal(la, lb) and (ws[need:] == 0xFF).all()
    args = (c.cache(), kh.to_bf16(c.q), *c.args(), _i32(lists))
    with pytest.raises(moe.MoeError):
        kv_sparse.kv_sparse_attention(*args, workspace=ws[:need - 1])
    with pytest.raises(moe.MoeError):
        kv_sparse.kv_sparse_attention(*args, workspace=ws[8:])
    with pytest.raises(TypeError):
        kv_sparse.kv_sparse_attention(*args, workspace=ws.view(torch.int8))


def test_graphs_that_share_a_workspace_and_calls_at_once():
    """Two captured calls with one workspace, replayed in turn; and two streams with workspaces of their own."""
    cases = [kh.Case(160 + i, 128, 2, 4, 64, [(1, 2000 + 900 * i), (1, 500)]) for i in range(2)]
    lists = [_i32(_lists(np.random.default_rng(i), c, 40)) for i, c in enumerate(cases)]
    inputs = [(c.cache(), kh.to_bf16(c.q), *c.args(), x) for c, x in zip(cases, lists)]
    want = [moe.kv_sparse_attention(*x) for x in inputs]
    ws = torch.empty(moe.kv_sparse_attention_workspace_size(2, 2, 8, 2, 128, 64, 40), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in inputs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(moe.kv_sparse_attention(*x, workspace=ws))
            graphs.append(g)
        for _ in range(3):
            for g in graphs:
                g.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
            ws.fill_(0xFF)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(moe.kv_sparse_attention(*inputs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])
