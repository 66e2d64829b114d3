"""Host-side checks of include/ss_block.h: exported symbols, workspace sizes, and
arguments refused before the device is touched (the fake device addresses are
never dereferenced). Also the mask's definition against SplitMix64's vectors."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

import sampled_softmax_output_gb300 as ss
from block_util import keep_mask

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
FAKE = 0x7F0000000000
p = ctypes.c_void_p


def test_exports_every_declared_symbol():
    names = ss.header_symbols(ss.HEADER_BLOCK)
    assert set(names) == {"ss_dropout", "ss_dropout_backward", "ss_ffn_workspace_size",
                          "ss_ffn_low_bits_pitch", "ss_ffn_forward", "ss_ffn_backward"}
    for n in names:
        assert hasattr(ss.lib(), n), n


def test_mask_is_halves_of_splitmix64_outputs():
    path = os.path.join(os.path.dirname(__file__), "golden", "splitmix64_vectors.txt")
    by_seed = {}
    for line in open(path):
        if line.strip() and not line.startswith("#"):
            seed, k, out = line.split()[:3]
            by_seed[int(seed, 0), int(k, 0)] = int(out, 0)
    assert by_seed
    for (seed, k), z in by_seed.items():
        for half, e in ((z & 0xFFFFFFFF, 2 * k), (z >> 32, 2 * k + 1)):
            # p on either side of the element's bits decides it
            assert keep_mask(1, half / 2 ** 32, seed, e)[0]
            assert not keep_mask(1, (half + 1) / 2 ** 32, seed, e)[0]


def _drop(fn="ss_dropout", **kw):
    a = dict(x=FAKE, residual=FAKE, n=16, dtype=0, spec=ss.DropoutSpec(0.1, 1, None, 0), y=FAKE)
    a.update(kw)
    spec = None if a["spec"] is None else ctypes.byref(a["spec"])
    if fn == "ss_dropout":
        return ss.lib().ss_dropout(p(a["x"]), p(a["residual"]), a["n"], a["dtype"], spec,
                                   p(a["y"]), None)
    return ss.lib().ss_dropout_backward(p(a["x"]), a["n"], a["dtype"], spec, p(a["y"]), None)


@pytest.mark.parametrize("fn", ["ss_dropout", "ss_dropout_backward"])
def test_dropout_argument_errors(fn):
    assert _drop(fn, n=0) == OK and _drop(fn, n=0, spec=None, x=0, y=0) == OK
    assert _drop(fn, n=-1) == INVALID and _drop(fn, n=1 << 62) == UNSUPPORTED
    assert _drop(fn, dtype=2) == INVALID and _drop(fn, dtype=-1) == INVALID
    for bad in (-0.1, 1.0000001, math.nan, math.inf):
        assert _drop(fn, spec=ss.DropoutSpec(bad, 0, None, 0)) == INVALID, bad
    assert _drop(fn, spec=ss.DropoutSpec(0.5, 0, FAKE + 4, 0)) == INVALID  # seed_dev alignment
    assert _drop(fn, x=0) == INVALID and _drop(fn, y=0) == INVALID
    assert _drop(fn, x=FAKE + 1) == INVALID and _drop(fn, y=FAKE + 2, dtype=1) == INVALID
    if fn == "ss_dropout":
        assert _drop(fn, residual=FAKE + 1) == INVALID


def test_low_bits_pitch():
    f = ss.lib().ss_ffn_low_bits_pitch
    assert [f(n) for n in (-8, 0, 8, 64, 72, 2048)] == [0, 0, 64, 64, 128, 2048]


def test_ffn_workspace_size():
    f = ss.lib().ss_ffn_workspace_size
    n = f(1000, 768, 2048)
    assert n >= 1024 + 2 * 1000 * 2048 * 2 + 1000 * 768 * 2 and n % 1024 == 0
    assert f(0, 768, 2048) > 0 and f(999, 768, 2048) <= n
    for bad in ((-1, 768, 2048), (1, 0, 2048), (1, 768, 0), (1, 100, 2048), (1, 768, 2044),
                (1, 16392, 64), (1, 64, 65544), (1 << 31, 64, 64), (1 << 30, 64, 65536)):
        assert f(*bad) == 0, bad
    with pytest.raises(ss.SSError):
        ss.ffn_workspace_size(1, 100, 64)


FWD = ("X", "Wg", "Wu", "Wd", "residual", "T", "D", "F", "act", "spec", "Y", "G", "U", "A", "R",
       "ws", "wsb")
BWD = ("dY", "X", "Wg", "Wu", "Wd", "G", "U", "A", "R", "T", "D", "F", "act", "spec", "dw", "acc",
       "dX", "dWg", "dWu", "dWd", "ws", "wsb")


def _ffn(fn, names, **kw):
    a = {n: FAKE for n in names}
    a.update(T=64, D=768, F=2048, act=0, spec=None, dw=1, acc=0, wsb=1 << 40)
    a.update(kw)
    plain = ("T", "D", "F", "act", "dw", "acc", "wsb")
    args = [a[n] if n in plain else (None if a[n] is None else ctypes.byref(a[n]))
            if n == "spec" else p(a[n]) for n in names]
    return getattr(ss.lib(), fn)(*args, None)


def _fwd(**kw):
    return _ffn("ss_ffn_forward", FWD, **kw)


def _bwd(**kw):
    return _ffn("ss_ffn_backward", BWD, **kw)


@pytest.mark.parametrize("fn", [_fwd, _bwd])
def test_ffn_argument_errors(fn):
    assert fn(T=-1) == INVALID and fn(D=0) == INVALID and fn(F=-8) == INVALID
    assert fn(T=1 << 31) == UNSUPPORTED and fn(D=772) == UNSUPPORTED and fn(F=2050) == UNSUPPORTED
    assert fn(D=16392) == UNSUPPORTED and fn(F=65544) == UNSUPPORTED
    assert fn(act=-1) == INVALID and fn(act=4) == INVALID
    assert fn(spec=ss.DropoutSpec(1.5, 0, None, 0)) == INVALID
    assert fn(spec=ss.DropoutSpec(0.5, 0, FAKE + 1, 0)) == INVALID
    need = ss.lib().ss_ffn_workspace_size(64, 768, 2048)
    assert fn(wsb=need - 1) == WORKSPACE
    for k in ("X", "Wg", "Wu", "Wd", "ws"):
        assert fn(**{k: 0}) == INVALID and fn(**{k: FAKE + 8}) == INVALID, k


def test_ffn_forward_argument_errors():
    assert _fwd(Y=0) == INVALID and _fwd(Y=FAKE + 2) == INVALID and _fwd(residual=FAKE + 8) == INVALID
    for k in ("G", "U", "A"):  # all three or none
        assert _fwd(**{k: 0}) == INVALID, k
        assert _fwd(**{k: FAKE + 8}) == INVALID, k
    assert _fwd(R=FAKE + 16) == INVALID            # 32-byte alignment
    assert _fwd(G=0, U=0, A=0) == INVALID          # low bits of nothing
    assert _fwd(T=0, X=0, Y=0, G=0, U=0, A=0, R=0) == OK


def test_ffn_backward_argument_errors():
    for k in ("dY", "G", "U", "A", "dX", "dWg", "dWu", "dWd"):
        assert _bwd(**{k: 0}) == INVALID and _bwd(**{k: FAKE + 8}) == INVALID, k
    assert _bwd(dw=2) == INVALID and _bwd(acc=2) == INVALID
    assert _bwd(R=FAKE + 16) == INVALID
    assert _bwd(T=0, dY=0, X=0, G=0, U=0, A=0, R=0, dX=0, acc=1) == OK


def test_python_refusals_on_host_tensors():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ss.dropout(x, 0.1, 0)  # not a CUDA tensor
    with pytest.raises(TypeError):
        ss.dropout(x.to(torch.float16), 0.1, 0)
    with pytest.raises(TypeError):
        ss.dropout_backward(np.zeros(4), 0.1, 0)
    w = torch.zeros(16, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ss.ffn_forward(x, w, w, w, torch.zeros(1024, dtype=torch.uint8))
    with pytest.raises(TypeError):
        ss.ffn_forward(x.float(), w, w, w, torch.zeros(1024, dtype=torch.uint8))
