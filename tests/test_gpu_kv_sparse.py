"""Sparse attention over the cache on the GPU: the index and the choice of pages against the oracle value for value, the
attention over chosen pages against the float64 oracle within the bounds that tests/kv_helpers.py derives."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from oracle import kv_cache as okv
from oracle import kv_sparse as osp
from oracle import nvfp4 as onv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).to(DEV)


# ----------------------------------------------------------------------------- the index

def _random_index(rng, pages, heads, dim):
    codes = rng.integers(-127, 128, (pages, heads, dim)).astype(np.int8)
    return codes, rng.uniform(0.05, 4.0, (pages, heads)).astype(np.float32)


def _gpu_index(codes, scales, page):
    return moe.NvFp4KvIndex(torch.from_numpy(codes.copy()).to(DEV), torch.from_numpy(scales.copy()).to(DEV), page)


def check_update(c, tokens=None):
    rng = np.random.default_rng(9)
    tokens = c.tokens if tokens is None else tokens
    codes, scales = _random_index(rng, c.pages.shape[0], c.kv_heads, c.dim)
    index = _gpu_index(codes, scales, c.page)
    moe.kv_index_update(c.cache(), index, *c.args(), tokens)
    osp.index_update(codes, scales, c.pages, c.page, c.offsets, c.lens, c.table, tokens)
    assert np.array_equal(index.codes.cpu().numpy(), codes)
    assert np.array_equal(index.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("seed,dim,kv_heads,page,reqs,pad", [
    (0, 64, 1, 32, [(1, 0)], 0),
    (1, 128, 8, 64, [(1, 63), (1, 64), (1, 65), (1, 300)], 0),
    (2, 128, 3, 96, [(200, 0), (1, 17), (0, 90), (97, 95)], 5),
    (3, 256, 2, 32, [(33, 31), (0, 0), (5, 400)], 1),
    (4, 64, 5, 256, [(3, 254), (700, 11)], 0),
    (5, 128, 1, 128, [(1, i * 7) for i in range(70)], 3),
])
def test_index_matches_the_oracle(seed, dim, kv_heads, page, reqs, pad):
    check_update(kh.Case(seed, dim, kv_heads, 1, page, reqs, pad=pad))


def test_index_of_fewer_rows_than_tokens_and_of_bad_pages():
    c = kh.Case(11, 64, 2, 1, 32, [(40, 5), (3, 60), (50, 0)])
    for tokens in (0, 1, 39, 41, 60):
        check_update(c, tokens)
    c.table[1, 1], c.table[2, 0] = -1, c.pages.shape[0]
    check_update(c)
    c.table = c.table[:, :1].copy()           # a table that ends before the rows do
    check_update(c)


def test_index_of_zeros_and_of_the_largest_values_in_a_large_page():
    page, dim = 40960, 64
    pages = okv.new_pages(2, page, 1, dim)
    unit = pages.reshape(-1, 36 * dim)
    unit[:, :32 * dim], unit[:, 32 * dim:] = 0x77, 0x7E          # 6 * 448 everywhere
    n = 40009
    table, lens, offsets = np.array([[1, 0]], np.int32), np.array([page + n], np.int32), np.array([0, page + n], np.int32)
    codes, scales = np.zeros((2, 1, dim), np.int8), np.zeros((2, 1), np.float32)
    cache = moe.NvFp4KvCache(torch.from_numpy(pages).to(DEV), page)
    index = _gpu_index(codes, scales, page)
    moe.kv_index_update(cache, index, _i32(offsets), _i32(lens), _i32(table), int(lens[0]))
    assert (index.codes == 127).all()
    assert np.array_equal(index.scales.cpu().numpy(), np.full((2, 1), np.float32(2688 / 127)))
    zero = moe.NvFp4KvCache.allocate(2, page, 1, dim)
    moe.kv_index_update(zero, index, _i32(offsets), _i32(lens), _i32(table), int(lens[0]))
    assert (index.codes == 0).all() and (index.scales == 0).all()


def test_index_grows_with_its_page():
    """Token by token, an index equals the one built at once from whole lengths."""
    c = kh.Case(12, 128, 2, 1, 32, [(0, 75), (0, 40)])
    cache, table = c.cache(), _i32(c.table)
    total = c.pages.shape[0]
    a = moe.NvFp4KvIndex.allocate(cache)
    for i in range(75):
        lens = np.minimum(c.lens, i + 1)
        new = np.array([1, 1 if i < 40 else 0])
        moe.kv_index_update(cache, a, _i32(np.concatenate([[0], np.cumsum(new)])), _i32(lens), table, 2)
    b = moe.NvFp4KvIndex.allocate(cache)
    moe.kv_index_update(cache, b, _i32(np.concatenate([[0], np.cumsum(c.lens)])), _i32(c.lens), table, int(c.lens.sum()))
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    assert a.codes.shape == (total, 2, 128) and (a.codes != 0).any()


# ----------------------------------------------------------------------------- the choice

class Choice:
    def __init__(self, seed, dim, kv_heads, group, page, reqs, pad=0, spare=3, width_extra=2, sigma=1.0):
        rng = np.random.default_rng(seed)
        new = [n for n, _ in reqs]
        self.rng, self.page = rng, page
        self.lens = np.array([n + o for n, o in reqs], np.int32)
        self.offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        need = [-(-int(n) // page) for n in self.lens]
        total = sum(need) + spare
        perm = rng.permutation(total)
        self.table = np.full((len(reqs), max(need + [0]) + width_extra), -3, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = perm[at:at + n]
            at += n
        self.codes, self.scales = _random_index(rng, total, kv_heads, dim)
        self.q = kh.bf16(rng, (int(self.offsets[-1]) + pad, kv_heads * group, dim), sigma)

    def check(self, top_k, first=1, last=1):
        index = _gpu_index(self.codes, self.scales, self.page)
        got = moe.kv_select(index, kh.to_bf16(self.q), _i32(self.offsets), _i32(self.lens), _i32(self.table), top_k, first,
                            last).cpu().numpy()
        want = osp.select(self.q, self.codes, self.scales, self.page, self.offsets, self.lens, self.table, top_k, first,
                          last)
        assert np.array_equal(got, want)
        return got


@pytest.mark.parametrize("seed,dim,kv_heads,group,page,reqs,pad,top_k,first,last", [
    (0, 64, 1, 1, 32, [(1, 0)], 0, 2, 1, 1),
    (1, 128, 8, 4, 64, [(1, 5000)], 0, 16, 1, 1),
    (2, 128, 2, 8, 64, [(1, 63), (1, 64), (3, 700), (0, 90), (1, 9000)], 4, 9, 1, 2),
    (3, 256, 3, 5, 32, [(5, 1000), (2, 30)], 0, 12, 0, 1),
    (4, 64, 2, 16, 96, [(7, 3000)], 2, 5, 2, 3),
    (5, 128, 1, 3, 32, [(70, 900)], 0, 8, 1, 1),
    (6, 64, 1, 64, 32, [(2, 4000), (1, 10)], 0, 64, 3, 4),
    (7, 256, 1, 33, 128, [(1, 20000)], 0, 7, 0, 7),
    (8, 64, 4, 2, 32, [(40, 0), (33, 31), (1, 0)], 0, 3, 1, 1),
    (9, 128, 2, 6, 32, [(1, 70 * i) for i in range(9)], 0, 1, 0, 1),
    (10, 64, 1, 1, 32, [(17, 2000)], 0, 100, 0, 1),              # more than there are
    (11, 64, 1, 1, 32, [(2, 32 * 5000)], 0, 1024, 1, 1),
    (12, 64, 1, 4, 32, [(9, 32 * 3000), (1, 40)], 0, 48, 1, 1),      # keys over all waves, several tokens
    (13, 128, 1, 2, 32, [(10, 32 * 2100)], 0, 1000, 2, 2),
    (14, 256, 1, 1, 64, [(3, 64 * 2500)], 0, 5, 1, 1),
    (15, 256, 1, 48, 32, [(1, 32 * 1900)], 0, 200, 1, 1),
    (16, 128, 2, 4, 32, [(20, 32 * 1000)], 0, 24, 1, 1),             # a list of candidates
    (17, 128, 2, 1, 32, [(1, 32 * 2040), (1, 32 * 700)], 0, 63, 0, 1),
])
def test_choice_matches_the_oracle(seed, dim, kv_heads, group, page, reqs, pad, top_k, first, last):
    Choice(seed, dim, kv_heads, group, page, reqs, pad=pad).check(top_k, first, last)


def test_choice_of_equal_scores_takes_the_lowest_pages():
    c = Choice(20, 64, 2, 2, 32, [(3, 3200)])
    c.codes[:] = c.codes[0]
    c.scales[:] = 0.5
    got = c.check(10)
    assert np.array_equal(got[0, 0], list(range(9)) + [100])
    c.scales[:, 1] = np.where(np.arange(len(c.scales)) % 3 == 0, 0.5, 0.25)      # two values, many ties each
    c.check(60)
    c.codes[:] = 0
    c.check(33, 2, 2)
    for width in (1500, 5000):                                        # many equal keys, one wave and all of them
        c = Choice(25, 64, 1, 4, 32, [(5, 32 * width)])
        c.codes[:] = c.codes[0]
        c.scales[:] = np.where(np.arange(len(c.scales)) % 7 == 0, 2.0, 1.0)[:, None].astype(np.float32)
        c.check(100, 1, 3)
        c.check(1000)
        c.scales[:] = np.float32(0.25)
        c.check(70)


def test_choice_of_rows_without_a_usable_value():
    """Zeros, magnitudes outside 2^-100 .. 2^100, infinities and NaN count as zeros, head by head."""
    c = Choice(21, 128, 1, 4, 32, [(8, 2000)])
    c.q[0] = 0.0
    c.q[1, 2, 5], c.q[2, :, 9] = np.inf, np.nan
    c.q[3], c.q[4, 1] = c.q[3] * 2.0 ** -110, c.q[4, 1] * 2.0 ** 110
    c.q[5] = np.where(np.arange(128) == 3, 2.0 ** 100, 0.0)
    c.q[6, 0] = np.where(np.arange(128) == 3, 2.0 ** -100, 0.0)
    index = _gpu_index(c.codes, c.scales, c.page)
    q = torch.from_numpy(c.q).to(torch.bfloat16).to(DEV)
    got = moe.kv_select(index, q, _i32(c.offsets), _i32(c.lens), _i32(c.table), 12).cpu().numpy()
    want = osp.select(c.q, c.codes, c.scales, c.page, c.offsets, c.lens, c.table, 12)
    assert np.array_equal(got, want)


def test_choice_with_bad_pages_and_lengths_behind_the_table():
    c = Choice(22, 64, 2, 3, 32, [(4, 1500), (2, 700), (1, 300), (2, 31)])
    c.table[0, 3:9], c.table[0, 47], c.table[1, 0] = -1, 10 ** 6, -1
    c.check(11, 1, 2)
    c.check(40, 1, 1)
    c.table = np.ascontiguousarray(c.table[:, :12])              # own pages behind it are listed all the same
    got = c.check(9, 1, 3)
    assert list(got[3, 0, -3:]) == [44, 45, 46]
    c.table = np.ascontiguousarray(c.table[:, :0])
    c.check(5, 1, 2)


def test_choice_of_padded_rows_and_of_more_tokens_than_rows():
    c = Choice(23, 64, 1, 2, 32, [(5, 600), (3, 900)], pad=6)
    c.check(7)
    c.offsets += 2                                               # rows before the first request
    c.check(7)
    c.q = c.q[:6]                                                # tokens past the last row have none
    c.check(7)
    c.lens[:] = [3, -4]                                          # rows before the first position
    got = c.check(7)
    assert (got[:2] == -1).all()


def test_choice_without_requests_and_without_rows():
    c = Choice(24, 64, 2, 2, 32, [(1, 50)])
    index, q = _gpu_index(c.codes, c.scales, 32), kh.to_bf16(c.q)
    empty, table = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(0, 5, dtype=torch.int32, device=DEV)
    assert (moe.kv_select(index, q, empty, empty[:0], table, 3) == -1).all()
    assert moe.kv_select(index, q[:0], _i32(c.offsets), _i32(c.lens), _i32(c.table), 3).shape == (0, 2, 3)


# ----------------------------------------------------------------------------- the attention

def _lists(rng, c, top_k, overlap=0.5):
    """Ascending lists with -1 behind: neighbours share part of theirs, some rows list little or nothing."""
    width = c.table.shape[1]
    out = np.full((c.tokens, c.kv_heads, top_k), -1, np.int32)
    for r in range(len(c.lens)):
        a, b = int(c.offsets[r]), int(c.offsets[r + 1])
        common = rng.random((c.kv_heads, width))
        for t in range(a, b):
            own = (int(c.lens[r]) - (b - a) + t - a) // c.page
            for h in range(c.kv_heads):
                n = min(own + 1, int(rng.integers(0, top_k + 1)) if rng.random() < 0.3 else top_k)
                score = overlap * common[h] + (1 - overlap) * rng.random(width)
                pick = np.sort(np.argsort(score[:own + 1])[:n])
                out[t, h, :n] = pick
    return out


def check_sparse(c, lists, **kw):
    out, lse = moe.kv_sparse_attention(c.cache(), kh.to_bf16(c.q), *c.args(), _i32(lists), scale=c.scale, return_lse=True,
                                       **kw)
    ref, ref_lse, mags = osp.attention(c.q, c.pages, c.page, c.d_k, c.d_v, c.offsets, c.lens, c.table, lists, c.scale)
    inside = np.zeros(c.tokens, bool)
    inside[int(c.offsets[0]):int(c.offsets[-1])] = True
    got, got_lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bad = np.isnan(ref).any(-1) & inside[:, None]
    assert np.array_equal(np.isnan(got).all(-1)[inside], bad[inside]) and np.isnan(got_lse[bad]).all()
    sel = inside[:, None] & ~bad
    most = lists.shape[2] * c.page
    tol, tol_lse = kh.bounds(ref, ref_lse, mags, sel, min(most, int(c.lens.max())), c.dim)
    empty = np.isneginf(ref_lse[sel])
    assert np.array_equal(np.isneginf(got_lse[sel]), empty) and np.all(got[sel][empty] == 0)
    over = np.abs(got[sel] - ref[sel]) / tol
    assert np.all(over <= 1), f"out: {np.nanmax(over)} times the bound"
    over = np.abs(got_lse[sel][~empty] - ref_lse[sel][~empty]) / tol_lse[~empty]
    assert np.all(over <= 1), f"lse: {over.max()} times the bound"
    return out, lse


@pytest.mark.parametrize("seed,dim,kv_heads,group,page,reqs,top_k,pad", [
    (0, 64, 1, 1, 32, [(1, 0)], 1, 0),
    (1, 128, 4, 8, 64, [(1, 1500)], 9, 0),
    (2, 128, 2, 4, 64, [(1, 63), (1, 64), (0, 30), (5, 500), (1, 1200)], 6, 3),
    (3, 256, 2, 8, 32, [(3, 400), (1, 31)], 7, 0),
    (4, 64, 3, 6, 32, [(5, 700), (2, 20), (4, 100)], 12, 0),
    (5, 128, 1, 16, 96, [(4, 900)], 4, 1),
    (6, 64, 2, 1, 32, [(37, 300), (16, 0)], 5, 0),               # sixteen tokens a tile
    (7, 64, 1, 5, 256, [(20, 1100)], 3, 0),                      # three tokens a tile
    (8, 128, 1, 17, 32, [(3, 300)], 6, 0),                       # blocks of 32 rows
    (9, 64, 1, 64, 64, [(2, 500), (1, 3)], 5, 0),                # two tiles per token
    (10, 256, 1, 33, 32, [(2, 200)], 4, 2),
    (11, 64, 1, 2, 32, [(9, 3000)], 90, 0),
    (12, 128, 2, 2, 32, [(70, 0), (33, 31)], 3, 0),
])
def test_sparse_attention_matches_the_oracle(seed, dim, kv_heads, group, page, reqs, top_k, pad):
    c = kh.Case(seed, dim, kv_heads, group, page, reqs, pad=pad)
    lists = _lists(np.random.default_rng(seed), c, top_k)
    out, lse = check_sparse(c, lists)
    if pad:
        assert (out[-pad:] == 0).all() and torch.isneginf(lse[-pad:]).all()
        given = torch.full_like(out, 3.0)
        again, lse2 = check_sparse(c, lists, out=given)
        assert again is given and (given[-pad:] == 3).all() and torch.isneginf(lse2[-pad:]).all()
        assert torch.equal(given[:-pad], out[:-pad])


@pytest.mark.parametrize("overlap", [0.0, 1.0])
@pytest.mark.parametrize("group,dim", [(1, 64), (4, 128), (8, 256)])
def test_lists_that_share_all_or_nothing(group, dim, overlap):
    c = kh.Case(30, dim, 2, group, 32, [(33, 900)])
    check_sparse(c, _lists(np.random.default_rng(31), c, 10, overlap))


def test_every_page_listed_is_the_attention():
    c = kh.Case(32, 128, 2, 4, 32, [(9, 200), (1, 330), (40, 0)])
    every = np.broadcast_to(np.arange(c.table.shape[1], dtype=np.int32), (c.tokens, 2, c.table.shape[1]))
    out, lse = check_sparse(c, every)
    ref, ref_lse = c.run()
    # both lie within the same bound of the exact rows
    assert torch.allclose(out.float(), ref.float(), rtol=2.0 ** -7, atol=1e-4) and torch.allclose(lse, ref_lse, atol=1e-4)


def test_lists_with_repeats_pages_ahead_and_nothing():
    c = kh.Case(33, 64, 2, 4, 32, [(6, 200), (1, 5)])
    lists = np.full((c.tokens, 2, 8), -1, np.int32)
    lists[0, 0, :5] = [1, 1, 2, 2, 2]
    lists[0, 1, :3] = [0, 50, 2 ** 31 - 1]                        # the last two lie ahead: behind the table, unseen
    lists[1, :, :4] = [2, 6, 7, 7]
    lists[2, :, :3] = [6, 6, 6]
    lists[4, 1, :1] = 3
    lists[6, 0, :2] = [0, 0]
    check_sparse(c, lists)


def test_a_bad_page_makes_only_the_rows_that_see_it_nan():
    c = kh.Case(34, 64, 1, 2, 32, [(16, 300), (3, 100)])
    lists = _lists(np.random.default_rng(35), c, 4)
    c.table[0, lists[3, 0, 1]] = c.pages.shape[0] + 5
    c.table[1, 0] = -1
    out, _ = check_sparse(c, lists)
    assert torch.isnan(out).any() and not torch.isnan(out).all()
    c.table = np.ascontiguousarray(c.table[:, :5])               # some lists reach behind the table
    check_sparse(c, lists)


def test_more_tokens_than_rows_and_rows_before_the_first_request():
    c = kh.Case(36, 64, 2, 4, 32, [(6, 200), (5, 50)], pad=4)
    lists = _lists(np.random.default_rng(37), c, 4)
    c.offsets = c.offsets + 2
    lists[2:] = lists[:-2].copy()
    check_sparse(c, lists)
    c.tokens, c.q, lists = 9, c.q[:9], lists[:9]
    check_sparse(c, lists)


@pytest.mark.parametrize("sigma", [1e-30, 0.1, 30.0])
def test_scores_of_any_size(sigma):
    c = kh.Case(38, 64, 1, 4, 32, [(7, 500)], sigma_q=sigma)
    check_sparse(c, _lists(np.random.default_rng(39), c, 6))


def test_many_requests_of_one_token():
    c = kh.Case(40, 64, 1, 2, 32, [(1, (i * 37) % 150) for i in range(700)])
    check_sparse(c, _lists(np.random.default_rng(41), c, 3))
    check_update(c)


def test_strided_queries_other_stream_and_refusals():
    c = kh.Case(42, 128, 2, 4, 32, [(9, 200)])
    lists = _i32(_lists(np.random.default_rng(43), c, 4))
    cache, args = c.cache(), c.args()
    q = kh.to_bf16(c.q)
    want = moe.kv_sparse_attention(cache, q, *args, lists)
    fused = torch.zeros(9, 12, 128, dtype=torch.bfloat16, device=DEV)
    fused[:, 2:10] = q
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = moe.kv_sparse_attention(cache, fused[:, 2:10], *args, lists)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    for bad in (lists[:8], lists[:, :1], lists[:, :, :0], lists.long(), lists.cpu(), lists.transpose(0, 2)):
        with pytest.raises((TypeError, ValueError)):
            moe.kv_sparse_attention(cache, q, *args, bad)
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(out=q[:, :4]), dict(out=q.float())):
        with pytest.raises((TypeError, ValueError)):
            moe.kv_sparse_attention(cache, q, *args, lists, **kw)
    index = moe.NvFp4KvIndex.allocate(cache)
    for kw in (dict(top_k=1), dict(top_k=0), dict(top_k=2000), dict(top_k=4, first=-1), dict(top_k=4, last=0),
               dict(top_k=4, first=3, last=2)):
        with pytest.raises(ValueError):
            moe.kv_select(index, q, *args, **kw)
    with pytest.raises(ValueError):
        moe.kv_select(index, q, args[0], args[1], torch.zeros(1, 16385, dtype=torch.int32, device=DEV), 4)
    other = moe.NvFp4KvIndex(index.codes, index.scales, 64)
    with pytest.raises(ValueError):
        moe.kv_index_update(cache, other, *args, 9)
    with pytest.raises(ValueError):
        moe.NvFp4KvIndex(index.codes.view(-1)[1:2 * 128 + 1].view(1, 2, 128), index.scales[:1].contiguous(), 32)
