"""The package imports, and what needs no GPU works, on a build of torch without CUDA."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = """
import torch
for name in dir(torch._C):  # as in a CPU build
    if name.startswith("_cuda_"):
        delattr(torch._C, name)
import hybrid_linear_attention_chunk_gb300 as kda
x = torch.zeros(4, 1, 8)
kda.chunk_desc(torch.zeros(64, 1, 64), torch.zeros(64, 1, 64))
try:
    kda._lib._elsewhere(x.get_device(), None)
except ValueError as e:
    print("refused:", e)
"""


def test_import_without_cuda():
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert "refused: tensors must be on a CUDA device" in r.stdout


@pytest.mark.gpu
def test_public_ways_to_device_and_stream(kda, monkeypatch):
    """What stands in for torch's own short cuts gives the same device and stream, on a side stream too."""
    x = torch.randn(50, 2, 16, device="cuda:0")
    want, _ = kda.kda_scan_fwd(x, -x.abs())
    torch.cuda.synchronize()
    assert kda._lib._current_device() == torch.cuda.current_device()
    for s in (torch.cuda.current_stream(), torch.cuda.Stream()):
        with torch.cuda.stream(s):
            assert kda._lib._current_stream(0) == kda._lib._stream_of(0) == s.cuda_stream
            with monkeypatch.context() as m:
                m.setattr(kda._lib, "_current_stream", kda._lib._stream_of)
                m.setattr(kda._lib, "_current_device", torch.cuda.current_device)
                out, _ = kda.kda_scan_fwd(x, -x.abs())
        s.synchronize()
        assert torch.equal(out, want)
