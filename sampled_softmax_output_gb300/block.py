"""Python binding of include/ss_block.h: dropout from a counter-based generator
and the gated feed-forward block in front of the output head.

    ws = ss.ffn_workspace(T, D, F)
    H, saved = ss.ffn_forward(X, Wg, Wu, Wd, ws, residual=R, p=0.1, seed=s, save=True)
    out = ss.step(H, W, targets, C, seed, head_ws, scale=1.0 / T)
    g = ss.ffn_backward(out["dH"], X, Wg, Wu, Wd, saved, ws, p=0.1, seed=s)

As in the package's other calls: argument marshalling only, contiguous CUDA
tensors, results on the current stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

from . import WORKSPACE_HEADER_BYTES, SSError, _check, _lib, _need, _ptr, _stream

HEADER_BLOCK = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "include", "ss_block.h")
MAX_F = 65536
ACTS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


class DropoutSpec(ctypes.Structure):
    """ss_dropout_spec: p, seed (+ the word at seed_dev, if any), offset."""
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("seed_dev", ctypes.c_void_p),
                ("offset", ctypes.c_uint64)]


def _declare(L):
    p, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    dp = ctypes.POINTER(DropoutSpec)
    L.ss_dropout.restype = i32
    L.ss_dropout.argtypes = [p, p, i64, i32, dp, p, p]
    L.ss_dropout_backward.restype = i32
    L.ss_dropout_backward.argtypes = [p, i64, i32, dp, p, p]
    L.ss_ffn_workspace_size.restype = sz
    L.ss_ffn_workspace_size.argtypes = [i64, i64, i64]
    L.ss_ffn_forward.restype = i32
    L.ss_ffn_forward.argtypes = [p] * 5 + [i64, i64, i64, i32, dp] + [p] * 4 + [p, sz, p]
    L.ss_ffn_backward.restype = i32
    L.ss_ffn_backward.argtypes = ([p] * 8 + [i64, i64, i64, i32, dp, i32, i32] + [p] * 4
                                  + [p, sz, p])


_declare(_lib)


def _on(device):
    """The library launches on the current device: make it the tensors'."""
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _dropout_spec(p, seed, offset, device):
    if isinstance(seed, torch.Tensor):
        _need(seed, "seed", torch.int64, device)
        if seed.numel() != 1:
            raise ValueError(f"seed must hold one value, got {seed.numel()}")
        return DropoutSpec(float(p), 0, seed.data_ptr(), offset)
    return DropoutSpec(float(p), seed & (2**64 - 1), None, offset)


def _float_tensor(t, name, device=None, shape=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    _need(t, name, dtype if dtype is not None else t.dtype, device, shape)


def dropout(x: torch.Tensor, p: float, seed, residual: torch.Tensor | None = None,
            offset: int = 0, out: torch.Tensor | None = None):
    """residual + dropout(x) (ss_dropout): x of any shape, bf16 or fp32; no mask
    is stored. seed: an int, or an int64 CUDA tensor of one value that the
    kernel reads when it runs (a captured graph then draws a new mask whenever
    the tensor has changed). offset: the position of x's first element in the
    stream of random numbers. out may be x or residual."""
    _float_tensor(x, "x")
    dev = x.device
    if residual is not None:
        _need(residual, "residual", x.dtype, dev, x.shape)
    if offset < 0:
        raise ValueError(f"offset must not be negative, got {offset}")
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", x.dtype, dev, x.shape)
    spec = _dropout_spec(p, seed, offset, dev)
    with _on(dev):
        code = _lib.ss_dropout(_ptr(x), _ptr(residual), x.numel(), _DTYPES[x.dtype], spec,
                               _ptr(out), _stream(dev))
    _check(code, "ss_dropout")
    return out


def dropout_backward(dy: torch.Tensor, p: float, seed, offset: int = 0,
                     out: torch.Tensor | None = None):
    """The gradient of dropout(x, p, seed, offset=offset) with respect to x
    (ss_dropout_backward); that of its residual is dy itself. out may be dy."""
    _float_tensor(dy, "dy")
    dev = dy.device
    if offset < 0:
        raise ValueError(f"offset must not be negative, got {offset}")
    if out is None:
        out = torch.empty_like(dy)
    else:
        _need(out, "out", dy.dtype, dev, dy.shape)
    spec = _dropout_spec(p, seed, offset, dev)
    with _on(dev):
        code = _lib.ss_dropout_backward(_ptr(dy), dy.numel(), _DTYPES[dy.dtype], spec, _ptr(out),
                                        _stream(dev))
    _check(code, "ss_dropout_backward")
    return out


def ffn_workspace_size(T: int, D: int, F: int) -> int:
    n = _lib.ss_ffn_workspace_size(T, D, F)
    if n == 0:
        raise SSError(1, "ss_ffn_workspace_size")
    return int(n)


def ffn_workspace(T: int, D: int, F: int, device=None) -> torch.Tensor:
    """A device byte buffer for the forward and the backward of one block of up
    to T tokens, its header zeroed as include/ss_block.h requires."""
    ws = torch.empty(ffn_workspace_size(T, D, F), dtype=torch.uint8,
                     device=device if device is not None else "cuda")
    ws[:WORKSPACE_HEADER_BYTES].zero_()
    return ws


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return ACTS[act]


def _block_args(X, Wg, Wu, Wd, ws):
    bf16 = torch.bfloat16
    _need(X, "X", bf16)
    if X.dim() != 2:
        raise ValueError(f"X must be [T, D], got {tuple(X.shape)}")
    dev = X.device
    T, D = X.shape
    _need(Wg, "Wg", bf16, dev)
    F = Wg.shape[0]
    _need(Wg, "Wg", bf16, dev, (F, D))
    _need(Wu, "Wu", bf16, dev, (F, D))
    _need(Wd, "Wd", bf16, dev, (D, F))
    _need(ws, "workspace", torch.uint8, dev)
    return dev, T, D, F


def ffn_forward(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
                ws: torch.Tensor, act: str = "silu", residual: torch.Tensor | None = None,
                p: float = 0.0, seed=0, offset: int = 0, save: bool = False,
                out: torch.Tensor | None = None):
    """The gated feed-forward block (ss_ffn_forward):
        Y = residual + dropout((act(X Wg^T) * (X Wu^T)) Wd^T)
    X [T, D], Wg, Wu [F, D], Wd [D, F], all bf16. Returns Y, or with save=True
    (Y, (G, U, A)), what ffn_backward needs. out may be residual. p, seed and
    offset as for dropout()."""
    dev, T, D, F = _block_args(X, Wg, Wu, Wd, ws)
    bf16 = torch.bfloat16
    if residual is not None:
        _need(residual, "residual", bf16, dev, (T, D))
    if offset < 0:
        raise ValueError(f"offset must not be negative, got {offset}")
    if out is None:
        out = torch.empty(T, D, dtype=bf16, device=dev)
    else:
        _need(out, "out", bf16, dev, (T, D))
    saved = (tuple(torch.empty(T, F, dtype=bf16, device=dev) for _ in range(3)) if save
             else (None, None, None))
    spec = _dropout_spec(p, seed, offset, dev)
    with _on(dev):
        code = _lib.ss_ffn_forward(_ptr(X), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(residual), T, D, F,
                                   _act(act), spec, _ptr(out), *(_ptr(t) for t in saved),
                                   _ptr(ws), ws.numel(), _stream(dev))
    _check(code, "ss_ffn_forward")
    return (out, saved) if save else out


def ffn_backward(dY: torch.Tensor, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                 Wd: torch.Tensor, saved, ws: torch.Tensor, act: str = "silu", p: float = 0.0,
                 seed=0, offset: int = 0, dw_dtype=torch.float32, accumulate: bool = False,
                 dX: torch.Tensor | None = None, dWg: torch.Tensor | None = None,
                 dWu: torch.Tensor | None = None, dWd: torch.Tensor | None = None):
    """The gradients of ffn_forward (ss_ffn_backward) from dY [T, D] and the
    `saved` tensors: {"dX", "dWg", "dWu", "dWd"}, dX bf16 and the weight
    gradients of dw_dtype (fp32 or bf16), zero-filled when accumulate=True and
    none is given. The gradient of the residual is dY itself."""
    dev, T, D, F = _block_args(X, Wg, Wu, Wd, ws)
    bf16 = torch.bfloat16
    if dw_dtype not in _DTYPES:
        raise TypeError(f"dw_dtype must be torch.bfloat16 or torch.float32, got {dw_dtype}")
    if offset < 0:
        raise ValueError(f"offset must not be negative, got {offset}")
    _need(dY, "dY", bf16, dev, (T, D))
    G, U, A = saved
    for t, name in ((G, "G"), (U, "U"), (A, "A")):
        _need(t, name, bf16, dev, (T, F))
    if dX is None:
        dX = torch.empty(T, D, dtype=bf16, device=dev)
    else:
        _need(dX, "dX", bf16, dev, (T, D))
    new = torch.zeros if accumulate else torch.empty
    grads = []
    for t, name, shape in ((dWg, "dWg", (F, D)), (dWu, "dWu", (F, D)), (dWd, "dWd", (D, F))):
        if t is None:
            t = new(shape, dtype=dw_dtype, device=dev)
        else:
            _need(t, name, dw_dtype, dev, shape)
        grads.append(t)
    spec = _dropout_spec(p, seed, offset, dev)
    with _on(dev):
        code = _lib.ss_ffn_backward(_ptr(dY), _ptr(X), _ptr(Wg), _ptr(Wu), _ptr(Wd), _ptr(G),
                                    _ptr(U), _ptr(A), T, D, F, _act(act), spec,
                                    _DTYPES[dw_dtype], 1 if accumulate else 0, _ptr(dX),
                                    *(_ptr(t) for t in grads), _ptr(ws), ws.numel(), _stream(dev))
    _check(code, "ss_ffn_backward")
    return {"dX": dX, "dWg": grads[0], "dWu": grads[1], "dWd": grads[2]}
