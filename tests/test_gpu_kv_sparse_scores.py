"""Sparse attention at scores far beyond those of a trained model (products with log2(e) of 2^20 and more), in every launch:
tiles of several tokens whose lists differ, of 32 rows, of eight waves, and splits."""

import numpy as np
import pytest

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from oracle import kv_cache as okv
from oracle import kv_sparse as osp
from test_gpu_kv_sparse import _i32, _lists

pytestmark = pytest.mark.gpu

# dim, kv_heads, group, requests, top_k
SHAPES = [
    (64, 1, 1, [(300, 90), (220, 200)], 4),            # sixteen tokens a tile
    (128, 2, 4, [(131, 300), (1, 500), (130, 0)], 4),  # four
    (256, 3, 5, [(175, 150)], 3),                      # three
    (64, 10, 16, [(260, 60)], 3),                      # 32 rows of two tokens
    (64, 4, 4, [(2510, 60)], 2),                        # and of eight
    (128, 2, 4, [(9, 400), (1, 700)], 6),              # one token, eight waves
    (64, 8, 2, [(33, 2500)], 64),
    (64, 2, 40, [(5, 200)], 4),                        # 32 rows, two tiles per token
    (128, 1, 4, [(1, 3000), (1, 2000)], 90),           # splits
    (256, 1, 2, [(2, 3000)], 60),
]


def _case(dim, kv_heads, group, reqs, exponent, seed=60):
    return kh.Case(seed, dim, kv_heads, group, 32, reqs, d_k=0.0371 * 2.0 ** exponent, sigma_k=2.0 ** exponent)


def _run(c, lists):
    out, lse = moe.kv_sparse_attention(c.cache(), kh.to_bf16(c.q), *c.args(), _i32(lists), scale=c.scale, return_lse=True)
    return out.double().cpu().numpy(), lse.double().cpu().numpy()


def _leads(c, lists, mag):
    """Rows whose largest score leads the next by 40 and twice the rounding of one."""
    lead = np.zeros(mag.shape, bool)
    g = c.heads // c.kv_heads
    for r in range(len(c.lens)):
        slots = okv.slots_of(c.table[r], c.page, 0, int(c.lens[r]))
        k = okv.decode(c.pages, c.page, slots, c.d_k, False)
        a, b = int(c.offsets[r]), int(c.offsets[r + 1])
        for t in range(a, b):
            pos = int(c.lens[r]) - (b - a) + t - a
            for h in range(c.kv_heads):
                at = np.concatenate([np.arange(p * c.page, min((p + 1) * c.page, pos + 1)) for p in lists[t, h] if p >= 0] +
                                    [np.zeros(0, int)]).astype(int)
                if not len(at):
                    continue
                s = np.sort(c.scale * (c.q[t, h * g:(h + 1) * g] @ k[at, h].T), -1)
                ds = (c.dim + 12) * 2.0 ** -24 * mag[t, h * g:(h + 1) * g]
                lead[t, h * g:(h + 1) * g] = True if s.shape[1] == 1 else s[:, -1] - s[:, -2] > 2 * ds + 40
    return lead


def _check_largest(c, lists, out, lse, least):
    """The arithmetic of test_gpu_kv_scores: a row whose largest score leads gives that position's value times p / p, the
    upper p rounded to fp16 (2^-11), in fp32 (at most 16 roundings of 2^-24), rounded to bf16 (2^-8, half a step); the other
    positions, each below 2^-57, add at most 2^-57 sum|v| / sum p to out and to the reference each.  lse is the score: ds, 8
    roundings of it, and the logarithm of the sum."""
    ref, ref_lse, (_, plain, mag) = osp.attention(c.q, c.pages, c.page, c.d_k, c.d_v, c.offsets, c.lens, c.table, lists,
                                                  c.scale)
    empty = np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), empty) and (out[empty] == 0).all()
    assert np.isfinite(out).all() and np.isfinite(lse[~empty]).all()
    ds = (c.dim + 12) * 2.0 ** -24 * mag
    tol = ds + 8 * 2.0 ** -24 * np.abs(np.where(empty, 0, ref_lse)) + 1e-3
    assert np.all(np.abs(lse[~empty] - ref_lse[~empty]) <= tol[~empty])
    lead = _leads(c, lists, mag)
    assert lead[~empty].mean() >= least
    tol = np.abs(ref) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) + 2 * 2.0 ** -57 * plain
    assert np.all(np.abs(out - ref)[lead] <= tol[lead])


@pytest.mark.parametrize("exponent", [20, 30, 50])
@pytest.mark.parametrize("dim,kv_heads,group,reqs,top_k", SHAPES)
def test_large_scores_take_the_largest(dim, kv_heads, group, reqs, top_k, exponent):
    c = _case(dim, kv_heads, group, reqs, exponent)
    lists = _lists(np.random.default_rng(61), c, top_k)
    _check_largest(c, lists, *_run(c, lists), 0.7)


@pytest.mark.parametrize("dim,kv_heads,group,reqs,top_k", SHAPES)
def test_rows_of_ordinary_scores_beside_large_ones_keep_their_bounds(dim, kv_heads, group, reqs, top_k):
    """Rows of one tile whose scores differ by 2^30."""
    c = kh.Case(62, dim, kv_heads, group, 32, reqs)
    lists = _lists(np.random.default_rng(63), c, top_k)
    big = np.zeros(c.q.shape[:2], bool)
    big[::3, ::2] = big[1::3, 1::2] = True
    c.q[big] *= 2.0 ** 30
    out, lse = _run(c, lists)
    _check_largest(c, lists, out, lse, 0.0)
    ref, ref_lse, mags = osp.attention(c.q, c.pages, c.page, c.d_k, c.d_v, c.offsets, c.lens, c.table, lists, c.scale)
    sel = ~big & ~np.isneginf(ref_lse)
    tol, tol_lse = kh.bounds(ref, ref_lse, mags, sel, min(top_k * 32, int(c.lens.max())), dim)
    assert np.all(np.abs(out[sel] - ref[sel]) <= tol) and np.all(np.abs(lse[sel] - ref_lse[sel]) <= tol_lse)


@pytest.mark.parametrize("exponent", [16, 30])
@pytest.mark.parametrize("dim,kv_heads,group,reqs,top_k", SHAPES)
def test_equal_large_scores_share(dim, kv_heads, group, reqs, top_k, exponent):
    """All keys alike: equal scores, whatever their size; out is the mean of the values listed."""
    c = _case(dim, kv_heads, group, reqs, exponent, seed=64)
    rng = np.random.default_rng(64)
    lists = _lists(rng, c, top_k)
    one = kh.bf16(rng, (1, kv_heads, dim), 2.0 ** exponent)
    for r in range(len(reqs)):
        slots = okv.slots_of(c.table[r], 32, 0, int(c.lens[r]))
        okv.append(c.pages, 32, np.repeat(one, len(slots), 0), slots, c.d_k, False)
    out, lse = _run(c, lists)
    _, ref_lse, (_, _, mag) = osp.attention(c.q, c.pages, c.page, c.d_k, c.d_v, c.offsets, c.lens, c.table, lists, c.scale)
    ref, _, (terms, _, _) = osp.attention(np.zeros_like(c.q), c.pages, c.page, c.d_k, c.d_v, c.offsets, c.lens, c.table,
                                          lists, c.scale)
    # p is the same number for every position (2^-11 once rounded); fp32 sums of n terms and the rounding to bf16
    n = min(top_k * 32, int(c.lens.max()))
    tol = np.abs(ref) * 2.0 ** -8 + terms * (1 + 2.0 ** -8) * (2.0 ** -11 + 2 * (n + 64) * 2.0 ** -24)
    assert np.all(np.abs(out - ref) <= tol)
    seen = ~np.isneginf(ref_lse)
    assert np.array_equal(np.isneginf(lse), ~seen)
    ds = (dim + 12) * 2.0 ** -24 * mag
    got, want = lse[seen], ref_lse[seen]
    assert np.all(np.abs(got - want) <= ds[seen] + 8 * 2.0 ** -24 * np.abs(want) + 1e-3)
