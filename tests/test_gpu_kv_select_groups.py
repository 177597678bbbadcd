"""The launches of the choice of pages that share what a workgroup reads among several groups of tokens, and the widest
block tables, each against the oracle value for value."""

import numpy as np
import pytest

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from test_gpu_kv_sparse import Choice, _gpu_index, _i32

pytestmark = pytest.mark.gpu


def groups_of(tokens, requests, kv_heads, group, dim, width):
    """Groups of tokens of a workgroup, by the rule of csrc/kv_index.hip (0: a workgroup takes one token)."""
    if tokens <= requests:
        return 0
    per = 16 // (group if group <= 2 else 4)
    blocks, stride = (group + 3) // 4, (width + 63) // 64 * 64 + 16
    for groups in (4, 2, 1):
        lds = groups * per * stride * 4 + 16 * blocks * groups * (4 + dim) + 8 * 16 * dim
        if lds <= (52 if groups > 1 else 150) << 10 and (groups == 1 or tokens // (groups * per) * kv_heads >= 512):
            return groups
    return 0


# Requests that end inside a group and inside a workgroup's tokens, one of a single row, padded rows.
@pytest.mark.parametrize("seed,dim,kv_heads,group,page,reqs,pad,top_k,first,last,width_extra,groups", [
    (0, 64, 16, 1, 256, [(1311, 700), (1, 2000), (739, 40)], 5, 4, 1, 1, 2, 4),
    (1, 64, 16, 2, 128, [(700, 333), (331, 900), (1, 1)], 0, 5, 1, 2, 2, 4),
    (2, 64, 8, 4, 64, [(641, 500), (390, 77)], 3, 6, 1, 1, 2, 4),
    (3, 64, 16, 5, 128, [(333, 600), (1, 500), (190, 0)], 0, 4, 0, 1, 2, 4),
    (4, 128, 8, 4, 64, [(700, 300), (333, 900)], 0, 7, 1, 1, 250, 4),
    (5, 64, 16, 1, 256, [(801, 700), (223, 40), (2, 999)], 1, 4, 1, 1, 2, 2),
    (6, 128, 16, 2, 128, [(333, 500), (219, 900)], 0, 5, 2, 1, 2, 2),
    (7, 256, 8, 4, 64, [(300, 500), (1, 700), (222, 60)], 2, 6, 1, 1, 2, 2),
    (8, 128, 8, 5, 64, [(301, 400), (219, 0)], 0, 5, 1, 1, 2, 2),
    (9, 128, 8, 4, 64, [(701, 300), (333, 900)], 0, 7, 1, 1, 880, 2),          # four groups do not fit
    (10, 64, 4, 2, 32, [(1100, 400), (960, 2000)], 0, 40, 1, 1, 2, 2),
    (11, 128, 8, 4, 64, [(701, 300), (333, 900)], 0, 7, 1, 1, 1200, 1),        # nor two
])
def test_groups_of_tokens(seed, dim, kv_heads, group, page, reqs, pad, top_k, first, last, width_extra, groups):
    c = Choice(300 + seed, dim, kv_heads, group, page, reqs, pad=pad, width_extra=width_extra)
    assert groups_of(len(c.q), len(reqs), kv_heads, group, dim, c.table.shape[1]) == groups
    got = c.check(top_k, first, last)
    assert (got[len(got) - pad:] == -1).all()


def test_bad_pages_and_short_tables_of_groups():
    c = Choice(320, 64, 8, 4, 64, [(641, 500), (390, 77)])
    c.table[0, 3:7], c.table[1, 0] = -1, 10 ** 6
    c.check(6, 1, 2)
    c.table = np.ascontiguousarray(c.table[:, :9])                    # own pages behind the table
    c.check(6, 1, 2)


@pytest.mark.parametrize("dim,kv_heads,group,new,top_k,groups", [
    (256, 1, 64, 1, 64, 0),          # the most LDS: 147776 bytes
    (256, 1, 64, 3, 33, 0),          # several tokens do not fit either
    (64, 1, 4, 1, 1024, 0),
    (64, 2, 2, 5, 1000, 0),
])
def test_the_widest_table(dim, kv_heads, group, new, top_k, groups):
    width = 16384
    c = Choice(330, dim, kv_heads, group, 32, [(new, 32 * width - 7 - new)], width_extra=0)
    assert c.table.shape[1] == width and groups_of(new, 1, kv_heads, group, dim, width) == groups
    c.check(top_k, 2, 3)


@pytest.mark.parametrize("dim,group,pages,top_k,width", [
    (64, 4, 1500, 1024, 1502),       # more than a row's candidates
    (128, 4, 4000, 48, 4002),        # one workgroup per compute unit
    (64, 1, 1200, 300, 1202),
    (64, 4, 300, 24, 8000),          # a table much wider than the request
    (128, 4, 300, 24, 16384),
])
def test_wide_tables_and_several_tokens(dim, group, pages, top_k, width):
    c = Choice(340, dim, 2, group, 32, [(21, 32 * pages - 40), (3, 900)], width_extra=2)
    wide = np.full((2, width), -3, np.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    c.check(top_k, 1, 2)


def test_the_choice_does_not_depend_on_the_tables_width():
    c = Choice(350, 128, 8, 4, 64, [(300, 6000), (251, 3000)])
    want = c.check(32)
    for width in (960, 1030, 2048, 5000, 16384):
        table = np.full((2, width), -3, np.int32)
        table[:, :c.table.shape[1]] = c.table
        got = moe.kv_select(_gpu_index(c.codes, c.scales, c.page), kh.to_bf16(c.q), _i32(c.offsets), _i32(c.lens),
                            _i32(table), 32).cpu().numpy()
        assert np.array_equal(got, want), width
