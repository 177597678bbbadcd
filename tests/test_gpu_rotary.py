"""Rotary positions on the GPU: rows against the float64 oracle within derived bounds, and the rotating append against
its parts, bit for bit."""

import numpy as np
import pytest
import torch

import kv_helpers as kh
import nvfp4_weight_quantized_amd as moe
from oracle import rotary as orot

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _i32(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).to(DEV)


def _make(rng, tokens, heads, dim, pairs, axes, interleaved, scale=1.0, far=200000):
    freq = 500000.0 ** (-np.arange(pairs) / pairs)
    axis = rng.integers(0, axes, pairs).astype(np.int32) if axes > 1 else None
    pos = rng.integers(0, far, (axes, tokens)).astype(np.int32)
    rot = moe.Rotary(torch.from_numpy(freq).to(DEV), dim, _i32(axis) if axes > 1 else None, axes, interleaved, scale)
    x = kh.bf16(rng, (tokens, heads, dim))
    return rot, freq, axis, pos, x


def check(got, x, pos, freq, axis, interleaved, scale=1.0):
    """Cosine and sine are off by half a step of fp32 (2^-24 relative; the angle, in 64 bits, by less than 2^-34 for
    these positions), each product and the sum by another: 3 * 2^-24 of |x1 c| + |x2 s|, and the result is rounded to bf16
    once, half a step (2^-8 relative)."""
    ref, mag = orot.rotate(x, pos, freq, axis, interleaved, scale)
    err = np.abs(got.double().cpu().numpy() - ref)
    fp32 = (3.1 * 2.0 ** -24 + 2.0 ** -33) * mag
    tol = np.abs(ref) * 2.0 ** -8 + (1 + 2.0 ** -8) * fp32 + 2.0 ** -126
    tol[mag == 0] = 0.0
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("seed,tokens,heads,dim,pairs,axes,interleaved,scale", [
    (0, 1, 1, 64, 32, 1, False, 1.0),
    (1, 1, 40, 128, 64, 1, False, 1.0),
    (2, 5, 3, 128, 64, 3, False, 1.0),
    (3, 7, 2, 256, 32, 1, True, 1.0),
    (4, 33, 5, 128, 24, 2, False, 0.7),         # pairs end inside a group of 16
    (5, 33, 5, 128, 40, 2, True, 1.25),
    (6, 300, 4, 64, 8, 4, False, 1.0),
    (7, 2100, 3, 64, 32, 3, True, 1.0),         # two tokens per block, an odd last one
    (8, 9001, 1, 256, 128, 1, False, 1.0),
    (9, 3, 7, 512, 256, 2, False, 1.0),         # no cache has this head dimension
    (10, 2, 9, 16, 8, 1, False, 1.0),
    (11, 4099, 2, 48, 16, 1, False, 1.0),
])
def test_rows_match_the_oracle(seed, tokens, heads, dim, pairs, axes, interleaved, scale):
    rng = np.random.default_rng(seed)
    rot, freq, axis, pos, x = _make(rng, tokens, heads, dim, pairs, axes, interleaved, scale)
    got = moe.rotary(rot, kh.to_bf16(x), _i32(pos if axes > 1 else pos[0]))
    check(got, x, pos, freq, axis, interleaved, scale)


def test_angles_of_far_and_negative_positions():
    """Positions up to 2^31 - 1: the angle's 64 bits leave an error of at most 2^31 * 2^-53 of a turn's radians."""
    rng = np.random.default_rng(20)
    pos = np.array([0, 1, -1, 2 ** 20 + 1, -2 ** 20, 2 ** 31 - 1, -2 ** 31, 12345678], np.int32)
    freq = np.concatenate([2.0 ** -np.arange(0, 12), [0.0, 1.7, 256.0, -0.3]])
    x = kh.bf16(rng, (len(pos), 2, 32))
    rot = moe.Rotary(torch.from_numpy(freq).to(DEV), 32)
    got = moe.rotary(rot, kh.to_bf16(x), _i32(pos))
    ref, mag = orot.rotate(x, pos, freq)
    angle = np.abs(np.outer(pos.astype(np.float64), freq)).max()
    tol = np.abs(ref) * 2.0 ** -8 + 1.01 * (3.1 * 2.0 ** -24 * mag + angle * 2.0 ** -52 * 4)
    assert np.all(np.abs(got.double().cpu().numpy() - ref) <= tol)


def test_in_place_strided_and_into_a_slice():
    rng = np.random.default_rng(21)
    rot, freq, axis, pos, x = _make(rng, 77, 4, 128, 32, 3, False)
    want = moe.rotary(rot, kh.to_bf16(x), _i32(pos))
    fused = torch.full((77, 10, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    part = fused[:, 3:7]
    part.copy_(kh.to_bf16(x))
    other = torch.full((77, 6, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got = moe.rotary(rot, part, _i32(pos), out=other[:, 1:5])
    assert got.data_ptr() == other[:, 1:5].data_ptr() and torch.equal(other[:, 1:5], want)
    assert (other[:, 0] == 7).all() and (other[:, 5] == 7).all()
    assert moe.rotary(rot, part, _i32(pos), out=part).data_ptr() == part.data_ptr()
    assert torch.equal(part, want) and (fused[:, :3] == 7).all() and (fused[:, 7:] == 7).all()
    wide = torch.zeros(3, 200, dtype=torch.int32, device=DEV)      # rows of a wider buffer
    wide[:, :77] = _i32(pos)
    assert torch.equal(moe.rotary(rot, kh.to_bf16(x), wide[:, :77]), want)


def test_refusals_and_empty_steps():
    rot = moe.Rotary.from_theta(128, sections=(16, 24, 24))
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16, device=DEV)
    pos = torch.zeros(3, 4, dtype=torch.int32, device=DEV)
    for bad in (pos[0], pos[:2], pos[:, :3], pos.long(), pos.cpu(), pos.t().contiguous().t(), pos[:1].expand(3, 4)):
        with pytest.raises((TypeError, ValueError)):
            moe.rotary(rot, x, bad)
    for bad in (x.float(), x[:, :, :64], x.cpu(), x.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises((TypeError, ValueError)):
            moe.rotary(rot, bad, pos)
    for bad in (x[:3], x[:, :1], torch.zeros(8, 2, 128, dtype=torch.bfloat16, device=DEV)[::2][:, :1]):
        with pytest.raises(ValueError):
            moe.rotary(rot, x, pos, out=bad)
    assert moe.rotary(rot, x[:0], pos[:, :0]).shape == (0, 2, 128)
    assert moe.rotary(rot, x[:, :0], pos).shape == (4, 0, 128)


def test_sections_in_order_and_in_turn():
    assert moe.Rotary.from_theta(32, sections=(4, 6, 6)).axes.tolist() == [0] * 4 + [1] * 6 + [2] * 6
    spread = moe.Rotary.from_theta(32, sections=(6, 5, 5), spread=True).axes.tolist()
    assert spread == [0, 1, 2] * 5 + [0]
    rot = moe.Rotary.from_theta(64, 500.0, rotary_dim=32)
    assert rot.pairs == 16 and rot.axes is None
    assert np.allclose(rot.inv_freq.cpu().numpy(), 500.0 ** (-np.arange(16) / 16), rtol=1e-15)


def test_an_axis_outside_counts_as_the_nearest_one():
    rng = np.random.default_rng(22)
    rot, freq, _, pos, x = _make(rng, 9, 2, 64, 32, 2, False)
    axis = np.array([-5, 0, 1, 99] * 8, np.int32)
    rot = moe.Rotary(torch.from_numpy(freq).to(DEV), 64, _i32(axis), 2)
    check(moe.rotary(rot, kh.to_bf16(x), _i32(pos)), x, pos, freq, np.clip(axis, 0, 1), False)


# ----------------------------------------------------------------------------- on the way into the cache

def _cache(rng, pages, page, kv_heads, dim):
    init = torch.from_numpy(rng.integers(0, 255, (pages, kv_heads, page // 32, 36 * dim)).astype(np.uint8))
    return [moe.NvFp4KvCache(init.to(DEV).clone(), page, 0.0371, 0.0113) for _ in range(2)]


@pytest.mark.parametrize("seed,tokens,heads,kv_heads,dim,pairs,axes,interleaved,page,order", [
    (0, 1, 1, 1, 64, 32, 1, False, 32, "run"),
    (1, 1, 32, 8, 128, 64, 1, False, 64, "run"),
    (2, 45, 24, 3, 256, 32, 1, True, 64, "scattered"),
    (3, 70, 6, 2, 128, 24, 3, False, 96, "run"),
    (4, 70, 5, 1, 128, 40, 2, True, 32, "padded"),
    (5, 2100, 8, 8, 64, 32, 3, False, 128, "run"),
    (6, 5001, 4, 8, 128, 64, 3, False, 64, "run"),          # values in quads
    (7, 5001, 4, 8, 128, 64, 1, False, 64, "scattered"),
    (8, 3001, 7, 7, 256, 128, 4, True, 32, "padded"),
    (9, 17, 3, 3, 64, 8, 1, False, 32, "outside"),
])
def test_append_rotary_is_its_parts(seed, tokens, heads, kv_heads, dim, pairs, axes, interleaved, page, order):
    rng = np.random.default_rng(100 + seed)
    rot, _, _, pos, _ = _make(rng, tokens, 1, dim, pairs, axes, interleaved)
    pages = -(-(tokens + 7) // page) + 2
    a, b = _cache(rng, pages, page, kv_heads, dim)
    perm = rng.permutation(pages)
    at = np.arange(tokens) + 5
    slots = perm[at // page] * page + at % page
    if order == "scattered":
        slots = rng.permutation(pages * page)[:tokens]
    elif order == "padded":
        slots[-9:] = -1
        slots[3] = -1
    elif order == "outside":
        slots[[1, 5]] = pages * page, 2 ** 31 - 1
    fused = kh.to_bf16(kh.bf16(rng, (tokens, heads + 2 * kv_heads, dim)))
    q, k, v = fused[:, :heads], fused[:, heads:heads + kv_heads], fused[:, heads + kv_heads:]
    p = _i32(pos if axes > 1 else pos[0])
    got = moe.kv_append_rotary(a, rot, q, k, v, p, _i32(slots))
    assert torch.equal(got, moe.rotary(rot, q, p))
    moe.kv_append(b, moe.rotary(rot, k, p), v, _i32(slots))
    assert torch.equal(a.pages, b.pages)
    # the same into q itself
    assert torch.equal(moe.kv_append_rotary(a, rot, q, k, v, p, _i32(slots), out=q), got) and torch.equal(q, got)
    assert torch.equal(a.pages, b.pages)


def test_append_rotary_of_extreme_rows():
    """Zeros, subnormals, the largest values, infinities and NaN: q carries them on, the cache holds finite values."""
    rng = np.random.default_rng(30)
    rot, _, _, pos, _ = _make(rng, 16, 1, 64, 16, 1, False)
    a, b = _cache(rng, 3, 32, 1, 64)
    x = kh.to_bf16(kh.bf16(rng, (16, 4, 64)))
    x[0], x[1], x[2] = 0.0, -0.0, 1e-39
    x[3, :, ::5], x[4, :, 3], x[5, :, 20], x[6] = 3e38, float("inf"), float("nan"), -3e38
    p, slots = _i32(pos[0]), _i32(np.arange(16) + 9)
    got = moe.kv_append_rotary(a, rot, x[:, :2], x[:, 2:3], x[:, 3:], p, slots)
    moe.kv_append(b, moe.rotary(rot, x[:, 2:3], p), x[:, 3:], slots)
    assert torch.equal(a.pages, b.pages)
    assert torch.equal(got.nan_to_num(9.0), moe.rotary(rot, x[:, :2], p).nan_to_num(9.0))
    k, v = moe.kv_gather(a, slots)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_append_rotary_refusals():
    rot = moe.Rotary.from_theta(64)
    cache = moe.NvFp4KvCache.allocate(4, 32, 2, 64)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos, slots = torch.zeros(3, dtype=torch.int32, device=DEV), torch.arange(3, dtype=torch.int32, device=DEV)
    for args in ((cache, moe.Rotary.from_theta(128), q, k, k, pos, slots), (cache, rot, q[:2], k, k, pos, slots),
                 (cache, rot, q[:, :0], k, k, pos, slots), (cache, rot, q, k[:, :1], k, pos, slots),
                 (cache, rot, q, k, k, pos[:2], slots), (cache, rot, q, k, k, pos, slots[:2]),
                 (cache, rot, q, k, k, pos, slots.cpu())):
        with pytest.raises(ValueError):
            moe.kv_append_rotary(*args)
    assert moe.kv_append_rotary(cache, rot, q[:0], k[:0], k[:0], pos[:0], slots[:0]).shape == (0, 4, 64)


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(31)
    rot, _, _, pos, _ = _make(rng, 40, 1, 128, 64, 3, False)
    a, b = _cache(rng, 4, 32, 2, 128)
    x = kh.to_bf16(kh.bf16(rng, (40, 8, 128)))
    p, slots = _i32(pos), _i32(np.arange(40) + 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        moe.kv_append_rotary(a, rot, x[:, :4], x[:, 4:6], x[:, 6:], p, slots)
        with torch.cuda.graph(graph, stream=side):
            got = moe.kv_append_rotary(a, rot, x[:, :4], x[:, 4:6], x[:, 6:], p, slots)
    torch.cuda.current_stream().wait_stream(side)
    for i in range(3):
        x.copy_(kh.to_bf16(kh.bf16(rng, (40, 8, 128))))
        p.add_(1000 * i)
        graph.replay()
        torch.cuda.synchronize()
        want = moe.kv_append_rotary(b, rot, x[:, :4], x[:, 4:6], x[:, 6:], p, slots)
        assert torch.equal(got, want) and torch.equal(a.pages.view(-1), b.pages.view(-1)), i
