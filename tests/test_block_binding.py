"""The binding of include/ss_block.h: import, current stream and device, arguments."""
import os
import subprocess
import sys

import numpy as np
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


def _spec(seed, offset=0):
    s = block._dropout_spec(0.1, seed, offset, None)
    return s.seed, s.offset


def test_seeds_and_offsets():
    """Whole numbers of any kind, taken modulo 2^64 (seed) or as they are (offset);
    nothing is cut off in silence."""
    for one in (1, True, np.int32(1), np.uint64(1)):
        assert _spec(one, 5) == (1, 5)
    assert _spec(-1)[0] == 2 ** 64 - 1 and _spec(2 ** 64 + 3)[0] == 3
    assert _spec(0, 2 ** 64 - 1)[1] == 2 ** 64 - 1
    for seed in (0.5, 1.0, "1", None, np.float64(2)):
        with pytest.raises(TypeError):
            _spec(seed)
    for offset in (-1, 2 ** 64, 2 ** 64 + 5):
        with pytest.raises(ValueError):
            _spec(0, offset)
    with pytest.raises(TypeError):
        _spec(0, 3.0)
