"""The rotating append of long steps, in which a thread takes half a key row: every head dimension, both pairings, heads
rotated in whole and in part, against rotation and append on their own, bit for bit."""

import pytest

import test_gpu_rotary as base

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed,tokens,heads,kv_heads,dim,pairs,axes,interleaved,page,order", [
    (20, 8201, 2, 8, 64, 32, 1, False, 64, "run"),
    (21, 8201, 2, 8, 64, 32, 3, False, 32, "scattered"),
    (22, 8193, 3, 8, 64, 24, 2, False, 128, "run"),
    (23, 8193, 1, 8, 64, 8, 1, False, 64, "padded"),
    (24, 8193, 2, 8, 64, 32, 1, True, 64, "scattered"),
    (25, 16387, 1, 4, 64, 16, 4, True, 96, "run"),
    (26, 4099, 2, 4, 256, 128, 1, False, 64, "run"),
    (27, 4099, 3, 4, 256, 128, 3, False, 32, "scattered"),
    (28, 4097, 1, 4, 256, 40, 2, False, 64, "run"),
    (29, 4097, 2, 4, 256, 120, 1, True, 128, "padded"),
    (30, 8193, 1, 4, 128, 24, 1, False, 64, "scattered"),
    (31, 8193, 1, 4, 128, 64, 2, True, 64, "outside"),
    (32, 1025, 1, 64, 64, 32, 1, False, 32, "run"),               # more half rows of a token than threads
])
def test_long_steps_are_their_parts(seed, tokens, heads, kv_heads, dim, pairs, axes, interleaved, page, order):
    assert 2 * tokens * kv_heads * (dim // 16) >= 1 << 19          # by the rule of csrc/rotary_launch.h
    base.test_append_rotary_is_its_parts(seed, tokens, heads, kv_heads, dim, pairs, axes, interleaved, page, order)
