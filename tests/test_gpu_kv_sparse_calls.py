"""Calls of rotary positions and sparse attention at the edges of what is documented: pages past 4 GiB, lists with repeats and
pages ahead in tiles of several tokens, lists in no order, large pages of odd unit counts, strided rows, repeated calls."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from test_gpu_kv_sparse import Choice, _gpu_index, _i32, _lists, check_sparse, check_update
from oracle import kv_sparse as osp

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_pages_past_four_gib():
    """The step of a small cache on the last pages of a large one: the same bytes, index, lists and rows."""
    dim, kv_heads, heads, page, few, many = 128, 8, 32, 64, 40, 70000
    rng = np.random.default_rng(1)
    small = moe.NvFp4KvCache.allocate(few, page, kv_heads, dim, 0.02, 0.02)
    big = moe.NvFp4KvCache(torch.empty(many, kv_heads, page // 32, 36 * dim, dtype=torch.uint8, device=DEV), page, 0.02, 0.02)
    ahead = (many - few) * kv_heads * (page // 32) * 36 * dim
    assert ahead > 4 << 30
    shift = many - few
    lens = np.array([1500, 800], np.int32)
    table = np.full((2, 24), -1, np.int32)
    perm = rng.permutation(few).astype(np.int32)
    table[0], table[1, :13] = perm[:24], perm[24:37]
    tokens = int(lens.sum())
    offsets = np.array([0, lens[0], tokens], np.int32)
    fused = kh.to_bf16(kh.bf16(rng, (tokens, heads + 2 * kv_heads, dim)))
    at = np.concatenate([np.arange(n) for n in lens])
    pos = _i32(at)
    slots = np.concatenate([table[r, np.arange(n) // page] * page + np.arange(n) % page for r, n in enumerate(lens)])
    rot = moe.Rotary.from_theta(dim)

    def step(cache, shift):
        q = moe.kv_append_rotary(cache, rot, fused[:, :heads], fused[:, heads:heads + kv_heads], fused[:, heads + kv_heads:],
                                 pos, _i32(slots + shift * page))
        args = (_i32(offsets), _i32(lens), _i32(np.where(table >= 0, table + shift, -1)))
        index = moe.NvFp4KvIndex.allocate(cache)
        moe.kv_index_update(cache, index, *args, tokens)
        chosen = moe.kv_select(index, q, *args, 6)
        out, lse = moe.kv_sparse_attention(cache, q, *args, chosen, return_lse=True)
        return index.codes[shift:shift + few], index.scales[shift:shift + few], q, chosen, out, lse, \
            moe.kv_gather(cache, _i32(slots + shift * page))[0]

    for a, b in zip(step(small, 0), step(big, shift)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dim,kv_heads,group,reqs", [
    (64, 1, 1, [(300, 90), (240, 300)]),               # sixteen tokens a tile
    (128, 2, 4, [(131, 300), (150, 20)]),              # four
    (64, 10, 16, [(260, 60)]),                         # two, of 32 rows
])
def test_repeats_and_pages_ahead_in_tiles_of_several_tokens(dim, kv_heads, group, reqs):
    c = kh.Case(400, dim, kv_heads, group, 32, reqs)
    rng = np.random.default_rng(401)
    lists = np.sort(rng.integers(0, c.table.shape[1] + 3, (c.tokens, kv_heads, 7)).astype(np.int32), -1)
    few = rng.random((c.tokens, kv_heads)) < 0.5
    lists[few] = np.sort(rng.integers(0, 3, (int(few.sum()), 7)).astype(np.int32), -1)       # the same few pages, repeated
    lists[rng.random((c.tokens, kv_heads)) < 0.2, 4:] = -1
    lists[rng.random((c.tokens, kv_heads)) < 0.1, -1] = 2 ** 31 - 1
    check_sparse(c, lists)


def test_lists_in_no_order_leave_other_tokens_alone():
    c = kh.Case(410, 64, 2, 2, 32, [(400, 300)])
    rng = np.random.default_rng(411)
    lists = _lists(rng, c, 6)
    want = moe.kv_sparse_attention(c.cache(), kh.to_bf16(c.q), *c.args(), _i32(lists), scale=c.scale)
    broken = lists.copy()
    for t in (100, 101, 255):
        broken[t] = rng.permuted(rng.integers(-5, 40, (2, 6)).astype(np.int32), axis=-1)
        broken[t, 0] = [20, -1, 3, 2 ** 31 - 1, 3, -2 ** 31]
    got = moe.kv_sparse_attention(c.cache(), kh.to_bf16(c.q), *c.args(), _i32(broken), scale=c.scale)
    far = np.ones(400, bool)
    for t in (100, 101, 255):
        far[max(t - 16, 0):t + 17] = False             # a tile holds at most sixteen tokens
    far = torch.from_numpy(far).to(DEV)
    assert torch.equal(got[far], want[far])


@pytest.mark.parametrize("dim,kv_heads,group,page,reqs,top_k", [
    (64, 2, 2, 1056, [(300, 2000), (1, 5000)], 3),     # 33 units a page, several tokens a tile
    (64, 1, 4, 8160, [(3, 30000)], 3),                 # 255 units, splits
    (128, 1, 1, 32768, [(1, 40000)], 2),
    (64, 1, 1, 65536, [(2, 70000)], 2),
])
def test_large_pages(dim, kv_heads, group, page, reqs, top_k):
    c = kh.Case(420, dim, kv_heads, group, page, reqs, spare=1, width_extra=0)
    rng = np.random.default_rng(421)
    check_sparse(c, _lists(rng, c, top_k))
    check_update(c)


@pytest.mark.parametrize("reqs,kv_heads", [([(1, 900), (1, 70)], 4), ([(40, 500), (25, 10)], 4), ([(700, 100), (390, 77)], 8)])
def test_choice_for_rows_of_a_fused_projection(reqs, kv_heads):
    c = Choice(430, 64, kv_heads, 4, 32, reqs)
    t = len(c.q)
    want = c.check(5)
    fused = torch.full((t, kv_heads * 6 + 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    rows = fused[:, 2:2 + 4 * kv_heads]
    rows.copy_(kh.to_bf16(c.q))
    index = _gpu_index(c.codes, c.scales, 32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [moe.kv_select(index, rows, _i32(c.offsets), _i32(c.lens), _i32(c.table), 5) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(np.array_equal(x.cpu().numpy(), want) for x in got)


def test_append_with_positions_of_a_wider_buffer_and_in_place():
    rng = np.random.default_rng(440)
    rot = moe.Rotary.from_theta(128, sections=(16, 24, 24))
    a, b = (moe.NvFp4KvCache.allocate(6, 32, 2, 128, 0.02, 0.02) for _ in range(2))
    x = kh.to_bf16(kh.bf16(rng, (90, 9, 128)))
    wide = torch.full((3, 200), -7, dtype=torch.int32, device=DEV)
    wide[:, 5:95] = _i32(rng.integers(0, 5000, (3, 90)))
    pos, slots = wide[:, 5:95], _i32(rng.permutation(192)[:90])
    want = moe.kv_append_rotary(a, rot, x[:, :5], x[:, 5:7], x[:, 7:], pos.contiguous(), slots)
    got = moe.kv_append_rotary(b, rot, x[:, :5], x[:, 5:7], x[:, 7:], pos, slots, out=x[:, :5])
    assert got.data_ptr() == x.data_ptr() and torch.equal(x[:, :5], want) and torch.equal(a.pages, b.pages)


def test_calls_repeat_themselves():
    """The same bits call after call, in launches with and without splits."""
    for reqs, kv_heads, top_k in (([(1, 5000)], 2, 60), ([(300, 500), (1, 900)], 4, 6)):
        c = kh.Case(450, 128, kv_heads, 4, 64, reqs)
        cache, q, args = c.cache(), kh.to_bf16(c.q), c.args()
        index = moe.NvFp4KvIndex.allocate(cache)
        whole = _i32(np.concatenate([[0], np.cumsum(c.lens)]))
        moe.kv_index_update(cache, index, whole, args[1], args[2], int(c.lens.sum()))
        first = None
        for _ in range(4):
            chosen = moe.kv_select(index, q, *args, top_k)
            res = (chosen, *moe.kv_sparse_attention(cache, q, *args, chosen, return_lse=True))
            assert first is None or all(torch.equal(x, y) for x, y in zip(res, first))
            first = res
        codes, scales = index.codes.cpu().numpy(), index.scales.cpu().numpy()
        assert np.array_equal(first[0].cpu().numpy(), osp.select(c.q, codes, scales, c.page, c.offsets, c.lens, c.table, top_k))
