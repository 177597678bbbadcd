"""GPU parity of the attention over the paged NVFP4 cache against the float64 oracle, within bounds
derived from the arithmetic (kv_helpers.bounds), over head layouts, lengths, windows, paddings and
masks that leave rows empty; and its behaviour in graphs, on streams and with bad pages."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
from nvfp4_weight_quantized_amd import kv
from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu
DEV = "cuda"

# (new, old) per request
DECODE = [(1, 0), (1, 30), (1, 31), (1, 32), (1, 63), (1, 64), (1, 200), (1, 511)]
MIXED = [(5, 0), (0, 40), (1, 100), (33, 20), (2, 0), (0, 0), (70, 5), (1, 0)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv_heads,group,page", [(1, 1, 32), (2, 5, 64), (3, 8, 96), (1, 16, 32), (2, 17, 128), (1, 64, 64)])
def test_decode_rows(dim, kv_heads, group, page):
    case = kh.Case(dim + group, dim, kv_heads, group, page, DECODE)
    kh.check_attention(case, *case.run())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,window", [(1, 0), (3, 0), (4, 1), (8, 33), (16, 64), (2, 100000)])
def test_mixed_rows_and_windows(dim, group, window):
    case = kh.Case(dim + window, dim, 2, group, 32, MIXED, window=window, pad=3)
    kh.check_attention(case, *case.run())


@pytest.mark.parametrize("dim,group,reqs,window", [
    (128, 8, [(1, 5000)], 0),                       # one request: the keys are split
    (64, 6, [(3, 3000), (1, 10), (2, 4000)], 0),
    (256, 4, [(1, 2500), (4, 1000)], 700),
    (128, 2, [(300, 0)], 0),                        # a prompt
    (64, 4, [(129, 400), (200, 0), (1, 900)], 0),   # chunks beside a single token
    (128, 1, [(257, 31)], 40),
    (256, 2, [(65, 130), (64, 0)], 0),
])
def test_longer_rows(dim, group, reqs, window):
    case = kh.Case(dim + len(reqs), dim, 2, group, 64, reqs, window=window)
    kh.check_attention(case, *case.run())


@pytest.mark.parametrize("sigma_q,sigma_k", [(30.0, 8.0), (1e-3, 1.0), (2.0 ** 60, 2.0 ** -60), (2.0 ** -60, 1.0)])
def test_score_magnitudes(sigma_q, sigma_k):
    """Sharp and flat softmax, rows far from 1 (each row is scaled by its own power of two)."""
    d_k = 0.0371 if sigma_k > 1e-9 else 2.0 ** -60
    case = kh.Case(11, 128, 2, 4, 32, [(9, 100), (1, 300), (40, 0)], sigma_q=sigma_q, sigma_k=sigma_k, d_k=d_k)
    kh.check_attention(case, *case.run())


def test_rows_with_elements_of_many_magnitudes():
    """Elements far below their row's largest, down to the range of the fp16 re-encoding."""
    case = kh.Case(12, 64, 1, 4, 32, [(3, 60), (1, 7)])
    rng = np.random.default_rng(3)
    case.q = kh.omoe.bf16_to_float(kh.oa4.float_to_bf16_bits(case.q * np.exp2(rng.integers(-25, 1, case.q.shape))))
    kh.check_attention(case, *case.run())


def test_zero_rows_and_equal_scores():
    case = kh.Case(13, 128, 1, 4, 32, [(4, 60)])
    case.q[:] = 0.0                                  # every score 0: the mean of the values
    out, lse = case.run()
    kh.check_attention(case, out, lse)
    assert np.allclose(lse.cpu().numpy()[:, 0], np.log(np.arange(61, 65)), rtol=1e-6)


def test_rows_before_the_first_position_are_empty():
    """seq_lens smaller than the request's rows: the first rows see nothing, zeros and -inf."""
    case = kh.Case(14, 64, 2, 3, 32, [(6, 0), (4, 40), (3, 0)])
    case.lens = np.array([2, 44, 0], np.int32)
    out, lse = case.run()
    kh.check_attention(case, out, lse)
    assert torch.isneginf(lse[:4]).all() and (out[:4] == 0).all() and torch.isneginf(lse[10:]).all()


@pytest.mark.parametrize("reqs", [[(1, 50), (1, 3)], [(60, 9), (1, 100), (3, 3)]])
def test_rows_outside_every_request_stay(reqs):
    case = kh.Case(15, 128, 1, 4, 32, reqs, pad=21)
    out = torch.full((case.tokens, case.heads, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got, lse = case.run(out=out)
    assert got is out and (out[int(case.offsets[-1]):] == 7.0).all()
    kh.check_attention(case, out, lse)
    # and before the first request
    case.offsets += 5
    out.fill_(7.0)
    _, lse = case.run(out=out)
    assert (out[:5] == 7.0).all() and (out[int(case.offsets[-1]):] == 7.0).all()
    ref, ref_lse, mags = case.reference()
    sel = slice(5, int(case.offsets[-1]))
    tol, _ = kh.bounds(ref, ref_lse, mags, sel, int(case.lens.max()), 128)
    assert np.all(np.abs(out.double().cpu().numpy()[sel] - ref[sel]) <= tol)


@pytest.mark.parametrize("reqs", [[(1, 130), (1, 70)], [(40, 90), (50, 20)]])
def test_a_bad_page_makes_the_rows_that_see_it_nan(reqs):
    case = kh.Case(16, 64, 2, 4, 32, reqs, window=35)
    good, good_lse = case.run()
    for entry in (-1, case.pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = case.table.copy()
        bad[0, 2] = entry                            # positions 64..95 of request 0
        save, case.table = case.table, bad
        out, lse = case.run()
        case.table = save
        n0 = reqs[0][0]
        pos = case.lens[0] - n0 + np.arange(n0)
        hit = np.zeros(case.tokens, bool)
        hit[:n0] = (pos >= 64) & (pos - 35 < 95)
        h = torch.from_numpy(hit).to(DEV)
        assert torch.isnan(out[h]).all() and torch.isnan(lse[h]).all()
        assert torch.equal(out[~h], good[~h]) and torch.equal(lse[~h], good_lse[~h])
    # a length past the table: the rows that see positions behind it are NaN
    case.lens = case.lens.copy()
    case.lens[1] = case.table.shape[1] * 32 + 3
    out, lse = case.run()
    assert torch.isnan(out[int(case.offsets[2]) - 1]).all()
    assert torch.equal(out[:reqs[0][0]], good[:reqs[0][0]])


def test_nonfinite_query_rows_do_not_spread():
    case = kh.Case(17, 128, 1, 4, 32, [(20, 40), (1, 9)])
    q = kh.to_bf16(case.q)
    good, _ = case.run()
    q[3, 1, 5], q[7, 0, 0] = float("nan"), float("inf")
    out, lse = kv.kv_attention(case.cache(), q, *case.args(), scale=case.scale, return_lse=True)
    assert torch.isnan(out[3, 1]).all() and torch.isnan(lse[3, 1])
    assert not torch.isfinite(lse[7, 0])
    mask = torch.ones(out.shape[:2], dtype=torch.bool, device=DEV)
    mask[3, 1] = mask[7, 0] = False
    assert torch.equal(out[mask], good[mask])


def test_query_slices_default_scale_and_no_lse():
    case = kh.Case(18, 64, 2, 3, 64, MIXED)
    wide = torch.randn(case.tokens, 8 + 6 * 64 + 40, device=DEV).to(torch.bfloat16)
    q = wide[:, 8:8 + 6 * 64].unflatten(1, (6, 64))
    q.copy_(kh.to_bf16(case.q))
    out = kv.kv_attention(case.cache(), q, *case.args())
    ref, _ = case.run()
    assert torch.equal(out, ref)


def test_repeated_calls_are_bitwise_equal_and_need_no_clean_workspace():
    case = kh.Case(19, 128, 2, 8, 64, [(1, 3000), (1, 40), (7, 900), (1, 0)])
    cache, args, q = case.cache(), case.args(), kh.to_bf16(case.q)
    need = kv.kv_attention_workspace_size(case.tokens, 4, case.heads, 2, 128)
    first = None
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((max(need, 16),), fill, dtype=torch.uint8, device=DEV)
        got = kv.kv_attention(cache, q, *args, scale=case.scale, return_lse=True, workspace=ws)
        if first is None:
            first = got
            kh.check_attention(case, *got)
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


@pytest.mark.parametrize("reqs", [[(1, 700), (1, 20)], [(90, 30), (1, 400)]])
def test_graph_replays_on_changing_contents(reqs):
    """Captured once; lengths, tables, queries and cache bytes change between the replays, eager work
    and synchronizations in between; every replay equals the eager call."""
    cases = [kh.Case(20 + i, 128, 2, 4, 64, [(n, max(0, o - 9 * i)) for n, o in reqs], spare=40 + i) for i in range(3)]
    p_max = max(c.pages.shape[0] for c in cases)
    w_max = max(c.table.shape[1] for c in cases)
    for c in cases:
        c.pages = np.concatenate([c.pages, np.zeros((p_max - c.pages.shape[0], *c.pages.shape[1:]), np.uint8)])
        c.table = np.pad(c.table, ((0, 0), (0, w_max - c.table.shape[1])), constant_values=-1)
    s = cases[0]
    pages = torch.from_numpy(s.pages).to(DEV)
    cache = kv.NvFp4KvCache(pages, 64, s.d_k, s.d_v)
    off, lens, table = s.args()
    q = kh.to_bf16(s.q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.kv_attention(cache, q, off, lens, table, return_lse=True)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = kv.kv_attention(cache, q, off, lens, table, return_lse=True)
    for i in (0, 1, 2, 0, 1):
        c = cases[i]
        pages.copy_(torch.from_numpy(c.pages))
        q.copy_(kh.to_bf16(c.q))
        off.copy_(torch.from_numpy(c.offsets))
        lens.copy_(torch.from_numpy(c.lens))
        table.copy_(torch.from_numpy(c.table))
        graph.replay()
        torch.cuda.synchronize()
        eager = kv.kv_attention(cache, q, off, lens, table, return_lse=True)
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        kh.check_attention(c, out, lse)


def test_two_streams_at_once():
    a = kh.Case(30, 128, 2, 8, 64, [(1, 2000), (1, 300)])
    b = kh.Case(31, 64, 2, 4, 32, [(80, 100), (1, 700)])
    streams = [torch.cuda.Stream() for _ in range(2)]
    sets = [(c.cache(), kh.to_bf16(c.q), c.args(), c) for c in (a, b)]
    torch.cuda.synchronize()
    res = [[], []]
    for _ in range(6):
        for i, (cache, q, args, c) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                res[i].append(kv.kv_attention(cache, q, *args, scale=c.scale, return_lse=True))
    torch.cuda.synchronize()
    for i, (_, _, _, c) in enumerate(sets):
        kh.check_attention(c, *res[i][0])
        for out, lse in res[i][1:]:
            assert torch.equal(out, res[i][0][0]) and torch.equal(lse, res[i][0][1])


def test_attention_wrappers_refuse_before_any_launch():
    case = kh.Case(32, 64, 2, 3, 32, [(2, 10), (1, 5)])
    cache, (off, lens, table), q = case.cache(), case.args(), kh.to_bf16(case.q)
    ok = dict(q=q, query_offsets=off, seq_lens=lens, block_table=table)
    for bad in (dict(q=q[:, :5]), dict(q=q[..., :32]), dict(q=q.transpose(0, 1)), dict(query_offsets=off[:2]),
                dict(block_table=table[:1]), dict(scale=0.0), dict(scale=float("nan")), dict(window=-1),
                dict(window=2 ** 32 + 5),
                dict(out=torch.empty_like(q[:1])), dict(seq_lens=lens.cpu()),
                dict(block_table=table.t().contiguous().t())):
        with pytest.raises(ValueError):
            kv.kv_attention(cache, **{**ok, **bad})
    for bad in (dict(q=q.float()), dict(seq_lens=lens.long()), dict(block_table=table.long()),
                dict(out=torch.empty_like(q).float())):
        with pytest.raises(TypeError):
            kv.kv_attention(cache, **{**ok, **bad})


def test_no_rows_and_no_requests():
    case = kh.Case(33, 64, 1, 2, 32, [(0, 10)])
    out, lse = case.run()
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    z = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 3.0)
    kv.kv_attention(case.cache(), q, z, z[:0], torch.zeros(0, 4, dtype=torch.int32, device=DEV), out=out)
    assert (out == 3.0).all()


# The host knows the width of the block table only: a narrow one lets tiles be taken whole, and few rows by the
# kernel for many; a wider one makes the call cut positions into shares and splits, and a very wide one take
# 32-row waves.
WIDE = 40000


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,reqs,window,pad", [
    (8, DECODE, 0, 0),
    (17, DECODE, 40, 3),
    (64, [(1, 3), (2, 700), (1, 0)], 0, 0),
    (4, MIXED, 0, 5),
    (16, MIXED, 64, 0),
    (1, [(300, 0)], 0, 2),
    (1, [(270, 1500)], 333, 0),                      # every tile's window is cut
    (4, [(333, 0), (1, 1800), (65, 1)], 0, 0),       # the first tiles see little: splits of theirs are empty
    (3, [(100, 2000), (96, 0), (0, 50), (2, 31)], 70, 7),
])
@pytest.mark.parametrize("extra", [400, WIDE])
def test_wide_block_tables(extra, dim, group, reqs, window, pad):
    case = kh.Case(dim + group, dim, 2, group, 32, reqs, window=window, pad=pad, width_extra=extra)
    kh.check_attention(case, *case.run())


@pytest.mark.parametrize("reqs", [[(1, 130), (1, 70)], [(40, 90), (50, 20)]])
def test_a_bad_page_of_a_wide_table(reqs):
    case = kh.Case(40, 128, 2, 4, 32, reqs, window=35, width_extra=WIDE)
    good, good_lse = case.run()
    for entry in (-1, case.pages.shape[0]):
        save = case.table[0, 2]
        case.table[0, 2] = entry                     # positions 64..95 of request 0
        out, lse = case.run()
        case.table[0, 2] = save
        n0 = reqs[0][0]
        pos = case.lens[0] - n0 + np.arange(n0)
        hit = np.zeros(case.tokens, bool)
        hit[:n0] = (pos >= 64) & (pos - 35 < 95)
        h = torch.from_numpy(hit).to(DEV)
        assert torch.isnan(out[h]).all() and torch.isnan(lse[h]).all()
        assert torch.equal(out[~h], good[~h]) and torch.equal(lse[~h], good_lse[~h])


@pytest.mark.parametrize("extra", [1, WIDE])
def test_rows_before_the_first_position_beside_many_rows(extra):
    case = kh.Case(41, 64, 2, 3, 32, [(90, 0), (4, 40), (70, 0)], width_extra=extra)
    case.lens = np.array([31, 44, 0], np.int32)
    out, lse = case.run()
    kh.check_attention(case, out, lse)
    assert torch.isneginf(lse[:59]).all() and (out[:59] == 0).all() and torch.isneginf(lse[94:]).all()


@pytest.mark.parametrize("requests,most_new,most_old,extra", [
    (65, 1, 90, 1), (130, 1, 300, 1), (600, 1, 3, 1), (600, 2, 3, 1), (70, 130, 40, 1), (70, 130, 40, 200), (200, 1, 0, 1)])
def test_many_requests(requests, most_new, most_old, extra):
    """More requests than lanes; shares that hold many short tiles; idle requests among them."""
    rng = np.random.default_rng(requests + most_new)
    reqs = [(int(rng.integers(0, most_new + 1)), int(rng.integers(0, most_old + 1))) for _ in range(requests)]
    case = kh.Case(42, 64, 4, 2, 32, reqs, width_extra=extra)
    kh.check_attention(case, *case.run())


@pytest.mark.parametrize("reqs", [[(3, 60), (5, 20), (4, 9)], [(40, 60), (50, 20), (90, 3)]])
@pytest.mark.parametrize("tokens", [1, 2, 6, 8, 60, 97])
def test_fewer_rows_than_tokens(reqs, tokens):
    """Tokens past the last row have no row; the others keep their positions."""
    case = kh.Case(43, 64, 2, 4, 32, reqs)
    tokens = min(tokens, case.tokens)
    full, full_lse = case.run()
    case.q = case.q[:tokens]
    out, lse = case.run()
    kh.check_attention(case, out, lse, rows=slice(0, tokens))
    # the same rows of the whole step, within the bounds of both
    ref, ref_lse, mags = case.reference()
    tol, _ = kh.bounds(ref, ref_lse, mags, slice(0, tokens), int(case.lens.max()), 64)
    assert np.all(np.abs((full[:tokens].double() - out.double()).cpu().numpy()) <= 2 * tol)


@pytest.mark.parametrize("scale,d_k", [(2.0 ** -62, 2.0 ** -64), (2.0 ** -60, 2.0 ** -60), (2.0 ** 36, 2.0 ** 64)])
@pytest.mark.parametrize("n", [2, 80])
def test_zero_rows_at_the_ends_of_the_scales(scale, d_k, n):
    """The factor of the scores at both ends of its range, rows of zeros and (below) of small elements
    beside masked positions: no 0 * inf."""
    case = kh.Case(44, 64, 1, 2, 32, [(n, 45), (1, 0)], d_k=d_k, sigma_k=d_k)
    case.scale = scale
    case.q[:] = 0.0
    if scale < 1:
        case.q[::2] = kh.bf16(np.random.default_rng(1), case.q[::2].shape, 2.0 ** -100)
    out, lse = case.run()
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    kh.check_attention(case, out, lse)


def test_two_graphs_replayed_on_two_streams():
    """Two captured calls have workspaces of their own: replayed at once, each gives the eager result."""
    cases = [kh.Case(45, 128, 2, 8, 64, [(1, 2500), (1, 300)], width_extra=300), kh.Case(46, 128, 2, 4, 32, [(80, 900)])]
    sets = [(c.cache(), kh.to_bf16(c.q), c.args()) for c in cases]
    eager = [kv.kv_attention(c, q, *a, return_lse=True) for c, q, a in sets]
    graphs, outs = [], []
    for c, q, a in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(kv.kv_attention(c, q, *a, return_lse=True))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for out in outs:
            out[0].zero_()
            out[1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, eager):
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for c, got in zip(cases, eager):
        kh.check_attention(c, *got)


@pytest.mark.parametrize("group,n", [(1, 3), (1, 200), (4, 90), (8, 5), (8, 150)])
@pytest.mark.parametrize("window", [0, 1, 40, 10 ** 6])
def test_rows_behind_the_table_are_nan(group, n, window):
    """A table of 64 positions: rows before its end are right, the others NaN, however far they lie behind
    it and whatever their windows reach."""
    case = kh.Case(47, 64, 2, group, 32, [(n, 20), (2, 5)], window=window)
    full, case.table = case.table, np.ascontiguousarray(case.table[:, :2])
    out, lse = case.run()
    tail = slice(max(0, 64 - 20), n)
    assert torch.isnan(out[tail]).all() and torch.isnan(lse[tail]).all()
    case.table = full
    keep = np.array([t for t in range(case.tokens) if t >= n or t < 64 - 20])
    kh.check_attention(case, out, lse, rows=keep)
    case.table = np.ascontiguousarray(full[:, :2])
    for far in (70000, 2 ** 31 - 1):
        case.lens[0] = far
        again, again_lse = case.run()
        assert torch.isnan(again[:n]).all() and torch.isnan(again_lse[:n]).all()
        kh.check_attention(_second(case), again[n:], again_lse[n:])


def _second(case):
    """The second request of a case, as a case of its own."""
    import copy
    c = copy.copy(case)
    n = int(case.offsets[1])
    c.q, c.offsets, c.lens, c.table = case.q[n:], case.offsets[1:] - n, case.lens[1:], case.table[1:]
    return c
