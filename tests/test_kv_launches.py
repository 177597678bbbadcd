"""The launches of an attention call, planned on the host (csrc/kv_launch.h, compiled here without HIP): grids hold
every tile and share that a step can have, and no more than its rows make."""

import json
import os
import random
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def launches(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("launches") / "kv_launches")
    subprocess.run(["g++", "-O1", "-std=c++17", os.path.join(HERE, "kv_launches.cpp"), "-o", exe], check=True)

    def plan(calls):
        text = "".join("%d %d %d %d %d %d\n" % c for c in calls)
        res = subprocess.run([exe], input=text, capture_output=True, text=True, check=True)
        return [json.loads(f"[{line}]") for line in res.stdout.splitlines()]

    return plan


def _calls(n, seed):
    rng = random.Random(seed)
    out = []
    for _ in range(n):
        g = rng.choice([1, 2, 4, 5, 8, 16, 64])
        hkv = rng.choice([1, 2, 3, 8, 16, 128])
        r = int(2 ** rng.uniform(0, 12))
        t = int(2 ** rng.uniform(0, 15))
        out.append((t, r, g, hkv, rng.choice([64, 128, 256]), int(2 ** rng.uniform(0, 17))))
    return out


def _steps(rng, call):
    """Token counts of requests that a call of these sizes may hold: even, one long, threshold-sized, some idle."""
    t, r, g = call[:3]
    yield [t // r + (i < t % r) for i in range(r)]
    yield [t - min(r - 1, t - 1)] + [1] * min(r - 1, t - 1)
    for rows in (64, 65, 16, 17, 128, 129):
        n = -(-rows // g)
        k = min(r, t // n) if n <= t else 0
        yield [n] * k
    left, some = t, []
    while left and len(some) < r:
        some.append(min(left, int(2 ** rng.uniform(0, 9))))
        left -= some[-1]
    yield some


def test_grids_hold_every_tile(launches):
    """Every request belongs to one launch, and the row tiles of any step fit its grid."""
    rng = random.Random(3)
    calls = _calls(400, 1)
    for call, plan in zip(calls, launches(calls)):
        t, r, g, hkv, dim, units = call
        for new in _steps(rng, call):
            assert sum(new) <= t and len(new) <= r
            mine = [0] * len(plan)
            for n in new:
                if n:
                    hits = [i for i, p in enumerate(plan) if p["min_rows"] < n * g <= p["max_rows"]]
                    assert len(hits) == 1, (call, n)
                    mine[hits[0]] += -(-n * g // plan[hits[0]]["bm"]) * hkv
            for tiles, p in zip(mine, plan):
                assert tiles <= p["tiles"], (call, new)
                if p["whole"]:
                    assert tiles <= p["grid"]
                elif not p["shares"]:      # cut tiles: at most `target` items more per head
                    assert tiles + p["target"] * hkv <= p["grid"]


def test_launches_are_of_the_steps_size(launches):
    """Tiles that a grid allows for: at most those that T rows make, not one for each request whatever its rows."""
    calls = _calls(400, 2) + [(1024, 1000, 4, 8, 128, 400), (4200, 4096, 4, 8, 128, 4096), (1100, 1024, 1, 8, 64, 64)]
    for call, plan in zip(calls, launches(calls)):
        t, r, g, hkv, dim, units = call
        for p in plan:
            most = t * g // (p["min_rows"] + 1)
            assert p["tiles"] <= hkv * (min(r, t, most) + t * g // p["bm"]), call


def test_the_joining_launch_is_of_the_size_of_what_is_cut(launches):
    """Partial sums number at most two per share or item aimed at, and the tiles to join half of that, however many
    requests or rows a step has."""
    calls = _calls(400, 4) + [(r, r, 4, 8, 128, 40) for r in (64, 1024, 4096)] + [(1 << 18, 4096, 4, 8, 128, 4096)]
    for call, plan in zip(calls, launches(calls)):
        hkv, dim = call[3], call[4]
        for p in plan:
            slots = p["bytes"] // (p["bm"] * (dim + 2) * 4)
            assert p["join"] <= slots / 2
            if p["whole"]:
                assert p["join"] == slots == 0
            elif p["shares"]:
                assert p["join"] == min(p["tiles"], p["grid"] - 1)      # a boundary between shares each
            else:
                assert p["join"] <= p["target"] * hkv


def test_padding_does_not_bring_the_kernel_of_many_rows(launches):
    """Batches of single tokens and short drafts past 1024 rows take one kernel; a prompt among them takes both."""
    for r, t in ((1000, 1024), (1023, 1030), (4000, 4096), (600, 1200)):
        (plan,) = launches([(t, r, 4, 8, 128, 400)])
        assert [p["shares"] for p in plan] == [1], (r, t)
    (plan,) = launches([(3400, 400, 4, 8, 128, 400)])
    assert [p["shares"] for p in plan] == [0, 1]
