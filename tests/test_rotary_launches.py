"""The launches of the rotary kernels, planned on the host (csrc/rotary_launch.h, compiled here without HIP): they hold every
row, and fewer than 2^32 work-items for every call within the limits of the arguments."""

import json
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROWS, APPEND, TOKENS = 1 << 36, 1 << 35, (1 << 24) - 1      # include/moe_nvfp4.h


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("launches") / "rotary_launches")
    subprocess.run(["g++", "-O1", "-std=c++17", os.path.join(HERE, "rotary_launches.cpp"), "-o", exe], check=True)

    def plan(calls):
        text = "".join("%d %d %d %d %d %d\n" % c for c in calls)
        res = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        return [json.loads(line) for line in res.stdout.splitlines()]

    return plan


def _calls(n, seed):
    """Steps of every size, half of them as long as the limits allow."""
    rng = random.Random(seed)
    for _ in range(n):
        dim = rng.choice([64, 128, 256])
        heads, hkv = int(2 ** rng.uniform(0, 16)), int(2 ** rng.uniform(0, 10))
        most = min(TOKENS, APPEND // (heads * dim), APPEND // (hkv * dim))
        t = most if rng.random() < 0.5 else int(2 ** rng.uniform(0, 24))
        yield min(t, most), heads, hkv, dim, 8 * rng.randrange(1, dim // 16 + 1), rng.randrange(2)


def _hold(x, t, heads, pairs):
    """Rows: every token has a workgroup, its angles fit, and the divisions by multiplication are exact (i * d < 2^32)."""
    assert (x["blocks"] - 1) * x["per_block"] < t <= x["blocks"] * x["per_block"]
    assert 1 <= x["per_block"] * pairs <= x["entries"]
    items = x["per_block"] * heads * x["pieces"]
    assert items * x["pieces"] < 1 << 32 and x["per_block"] * heads * heads <= 1 << 32 and items + 1024 < 1 << 31


def test_every_row_is_held_and_every_launch_fits(launches):
    corners = [(TOKENS, 1, 1, 64, 32, 0), (TOKENS, 8, 8, 256, 128, 1), (8259552, 65, 65, 64, 24, 1), (1, 65536, 1024, 256, 8, 1),
               (1 << 11, 65536, 1024, 256, 128, 0), (1 << 22, 128, 128, 64, 32, 0), (1, 1, 1, 64, 8, 0)]
    calls = corners + list(_calls(20000, 1))
    most = 0
    for call, x in zip(calls, launches(calls)):
        t, heads, hkv, dim, pairs, _ = call
        _hold(x, t, heads, pairs)
        assert x["fits"] and x["append_fits"], call
        most = max(most, x["append_blocks"] * x["threads"])
        assert 8 * x["q"] >= x["blocks"] and 8 * x["k"] * x["k_tokens"] >= t and x["k_tokens"] * pairs <= x["entries"]
        rows = -(-t // 4) if x["quads"] else t
        assert 8 * x["v"] * x["threads"] >= rows * hkv * (dim // 16)
        assert x["k_tokens"] * x["k_per"] ** 2 < 1 << 32
        assert x["append_blocks"] == 8 * (x["q"] + x["k"] + x["v"])
    assert most > 3 << 30      # the longest calls are among them


def test_rows_alone_fit_up_to_their_limits(launches):
    rng = random.Random(2)
    calls = []
    for _ in range(5000):
        dim = 16 * rng.randrange(1, 33)
        heads = int(2 ** rng.uniform(0, 16))
        calls.append((min(TOKENS, ROWS // (heads * dim)), heads, 1, dim, 8 * rng.randrange(1, dim // 16 + 1),
                      rng.randrange(2)))
    for call, x in zip(calls, launches(calls)):
        _hold(x, call[0], call[1], call[4])
        assert x["fits"], call


def test_a_launch_of_more_work_items_does_not_fit(launches):
    """Past the limits of the arguments, so that the check is seen to count."""
    x, y = launches([(1 << 24, 1, 1, 256, 128, 0), (1 << 28, 64, 64, 64, 24, 0)])
    assert x["fits"] and not y["fits"] and not y["append_fits"]
