"""The binding of include/ss_block.h: import, current stream and device, arguments."""
import os
import subprocess
import sys

import pytest
import torch

import sampled_softmax_output_gb300 as ss
from sampled_softmax_output_gb300 import block


def _without(names):
    """Runs the package's import and a refusal in a process whose torch lacks `names`."""
    code = f"""
import torch
for n in {names!r}:
    if hasattr(torch._C, n):
        delattr(torch._C, n)
import sampled_softmax_output_gb300 as ss
try:
    ss.dropout(torch.zeros(4), 0.1, 0)
except ValueError:
    print("imported")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    return subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                          timeout=300)


def test_import_without_torchs_private_names():
    r = _without(["_cuda_getCurrentRawStream", "_cuda_getDevice"])
    assert r.returncode == 0 and "imported" in r.stdout, r.stderr[-2000:]


@pytest.mark.gpu
def test_current_stream_by_the_public_calls(monkeypatch):
    """As where torch lacks the private names; on a stream of its own."""
    x = torch.randn(5003, device="cuda")
    want = ss.dropout(x, 0.1, 3)
    monkeypatch.setattr(block, "_raw_stream", block._public_stream)
    monkeypatch.setattr(block, "_current_device", torch.cuda.current_device)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert block._raw_stream(0) == side.cuda_stream
        y = ss.dropout(x, 0.1, 3)
    side.synchronize()
    assert torch.equal(y, want)
