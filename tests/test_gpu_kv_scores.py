"""Attention over the cache at scores far beyond those of a trained model: products with log2(e) of 2^20 and
more, where one unit in the last place of a score is many powers of two in its exponential."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu

# few rows per request, cut and whole; many rows, wide and narrow waves; a wide table cuts positions
SHAPES = [
    (64, 3, [(1, 0), (1, 40), (3, 200)], 1),
    (128, 2, [(2, 300), (1, 0)], 1200),
    (128, 20, [(1, 90), (2, 31)], 1),
    (256, 1, [(1, 130), (1, 0)], 500),
    (64, 4, [(90, 0), (70, 50)], 1),
    (128, 4, [(140, 20)], 40000),
    (256, 2, [(70, 9), (1, 300)], 1),
]


def _case(dim, group, reqs, extra, exponent, seed=50, sign=0):
    """Scores of about 2^exponent: unit queries, keys of 2^exponent; sign: all scores of that sign."""
    case = kh.Case(seed, dim, 2, group, 32, reqs, width_extra=extra, d_k=0.0371 * 2.0 ** exponent,
                   sigma_k=2.0 ** exponent)
    if sign:
        case.q = np.abs(case.q)
        rng = np.random.default_rng(seed)
        for r in range(len(reqs)):
            slots = okv.slots_of(case.table[r], 32, 0, int(case.lens[r]))
            k = sign * np.abs(kh.bf16(rng, (len(slots), 2, dim), 2.0 ** exponent))
            okv.append(case.pages, 32, k, slots, case.d_k, False)
    return case


def _check_largest(case, out, lse, least=0.7):
    """Rows whose largest score leads the next by more than every rounding of both: out is that position's
    value.  A score's rounding is at most (dim + 12) 2^-24 of its terms (kv_helpers.bounds), twice for a
    difference; 40 more leave the rest of the row below 2^-57 of the largest.  out is the largest's value times
    p / p, the upper p rounded to fp16 (2^-11), in fp32 (at most 16 roundings of 2^-24), rounded to bf16 (2^-8).
    The other positions, each below 2^-57, give out and the reference at most 2^-57 sum|v| / sum p each: all there is
    where the largest's value is 0.  lse is the score: 8 roundings of it beside ds, and the logarithm of the sum."""
    ref, ref_lse, (_, plain, mag) = case.reference()
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    ds = (case.dim + 12) * 2.0 ** -24 * mag
    assert np.all(np.abs(lse - ref_lse) <= ds + 8 * 2.0 ** -24 * np.abs(ref_lse) + 1e-3)
    sure = np.zeros(ref_lse.shape, bool)
    g = case.heads // case.pages.shape[1]
    for r in range(len(case.lens)):
        slots = okv.slots_of(case.table[r], case.page, 0, int(case.lens[r]))
        k = okv.decode(case.pages, case.page, slots, case.d_k, False)
        a, b = int(case.offsets[r]), int(case.offsets[r + 1])
        for t in range(a, b):
            pos = int(case.lens[r]) - (b - a) + t - a
            for h in range(case.heads):
                s = np.sort(case.scale * (k[:pos + 1, h // g] @ case.q[t, h]))
                sure[t, h] = len(s) == 1 or s[-1] - s[-2] > 2 * ds[t, h] + 40
    assert sure.mean() >= least
    # 2^-18: the 16 roundings and the products of the terms
    tol = np.abs(ref) * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) + 2 * 2.0 ** -57 * plain
    assert np.all(np.abs(out - ref)[sure] <= tol[sure])


@pytest.mark.parametrize("exponent", [18, 24, 27, 30, 34, 50])
@pytest.mark.parametrize("dim,group,reqs,extra", SHAPES)
def test_large_scores_take_the_largest(dim, group, reqs, extra, exponent):
    case = _case(dim, group, reqs, extra, exponent)
    _check_largest(case, *case.run())


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("exponent", [20, 31])
@pytest.mark.parametrize("dim,group,reqs,extra", SHAPES)
def test_large_scores_of_one_sign(dim, group, reqs, extra, exponent, sign):
    case = _case(dim, group, reqs, extra, exponent, sign=sign)
    _check_largest(case, *case.run())


@pytest.mark.parametrize("dim,group,reqs,extra", SHAPES)
def test_scores_near_the_end_of_fp32(dim, group, reqs, extra):
    """Scores of about 2^120, from large keys and large queries."""
    case = _case(dim, group, reqs, extra, 62, seed=54)
    case.q *= 2.0 ** 58
    _check_largest(case, *case.run())


@pytest.mark.parametrize("exponent", [16, 30, 40])
@pytest.mark.parametrize("dim,group,reqs,extra", SHAPES)
def test_equal_large_scores_share(dim, group, reqs, extra, exponent):
    """All keys alike: equal scores, whatever their size; out is the mean of the values seen."""
    case = _case(dim, group, reqs, extra, exponent, seed=51)
    rng = np.random.default_rng(51)
    one = kh.bf16(rng, (1, 2, dim), 2.0 ** exponent)
    for r in range(len(reqs)):
        slots = okv.slots_of(case.table[r], 32, 0, int(case.lens[r]))
        okv.append(case.pages, 32, np.repeat(one, len(slots), 0), slots, case.d_k, False)
    _, ref_lse, (_, _, mag) = case.reference()
    out, lse = case.run()
    case.q = np.zeros_like(case.q)
    ref, _, (terms, _, _) = case.reference()
    got = out.double().cpu().numpy()
    # p is the same number for every position: fp32 sums of n terms and the rounding to bf16
    n = int(case.lens.max())
    tol = np.abs(ref) * 2.0 ** -8 + terms * (2.0 ** -11 + 2 * (n + 64) * 2.0 ** -24)
    assert np.all(np.abs(got - ref) <= tol)
    ds = (dim + 12) * 2.0 ** -24 * mag
    assert np.all(np.abs(lse.double().cpu().numpy() - ref_lse) <= ds + 8 * 2.0 ** -24 * np.abs(ref_lse) + 1e-3)


@pytest.mark.parametrize("dim,group,reqs,extra", SHAPES)
def test_rows_of_ordinary_scores_beside_large_ones_keep_their_bounds(dim, group, reqs, extra):
    """Rows of one wave whose scores differ by 2^30: the ordinary ones keep the bounds of ordinary scores."""
    case = kh.Case(52, dim, 2, group, 32, reqs, width_extra=extra)
    big = np.zeros(case.q.shape[:2], bool)
    big[::3, 1::2] = True
    case.q[big] *= 2.0 ** 30
    out, lse = case.run()
    kh.check_attention(case, out, lse, rows=~big)
    _check_largest(case, out, lse, least=0.0)


def test_zero_scores_of_large_rows_are_zero():
    """Queries and scales whose factor alone leaves the fp32 range, keys of zeros: every score is 0, not 0 * inf."""
    for reqs in ([(1, 40), (2, 3)], [(90, 10)]):
        case = kh.Case(53, 64, 2, 4, 32, reqs, d_k=2.0 ** 60)
        for r in range(len(reqs)):
            slots = okv.slots_of(case.table[r], 32, 0, int(case.lens[r]))
            okv.append(case.pages, 32, np.zeros((len(slots), 2, 64)), slots, case.d_k, False)
        case.q = kh.bf16(np.random.default_rng(2), case.q.shape, 2.0 ** 110)
        out, lse = case.run()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        kh.check_attention(case, out, lse)
