"""The package imports, and its host-side parts work, on a torch without a GPU runtime."""

import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CPU_TORCH = """
import torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):      # a CPU build of torch has neither
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import nvfp4_weight_quantized_amd as moe
assert moe.synth.WORKLOADS["tiny"].T > 0
z = torch.zeros(4, dtype=torch.int32)
try:
    moe.kv_plan(z, z, torch.zeros(4, 2, dtype=torch.int32), z, 64, 8, 4)
except ValueError as e:
    print("refused:", e)
"""


def test_imports_without_the_private_stream_names():
    res = subprocess.run([sys.executable, "-c", CPU_TORCH], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stderr
    assert res.stdout.startswith("refused: kv_lens")


def test_public_names_serve_the_launches(monkeypatch):
    """The names taken instead: the current stream's handle and the current device."""
    import torch

    from nvfp4_weight_quantized_amd import kv

    class Stream:
        cuda_stream = 0x1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: Stream() if index == 3 else None)
    assert kv._public_stream(3) == 0x1234
    monkeypatch.setattr(kv, "_current_device", lambda: 3)
    assert kv._on(3) is kv._NOTHING


@pytest.mark.gpu
def test_public_names_give_the_same_streams(monkeypatch):
    import torch

    from nvfp4_weight_quantized_amd import kv

    def plan():
        z = torch.zeros(4, dtype=torch.int32, device="cuda")
        return kv.kv_plan(z, z + 1, torch.full((4, 2), -1, dtype=torch.int32, device="cuda"),
                          torch.arange(4, dtype=torch.int32, device="cuda"), 64, 4, 4)

    want = plan()
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert kv._public_stream(0) == kv._raw_stream(0) == stream.cuda_stream
    monkeypatch.setattr(kv, "_raw_stream", kv._public_stream)
    monkeypatch.setattr(kv, "_current_device", torch.cuda.current_device)
    with torch.cuda.stream(side):
        got = plan()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
