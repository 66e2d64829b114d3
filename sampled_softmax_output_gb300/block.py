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

import ctypes
import operator
import os

import torch

from . import WORKSPACE_HEADER_BYTES, SSError, _lib, _need

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
    L.ss_ffn_low_bits_pitch.restype = i64
    L.ss_ffn_low_bits_pitch.argtypes = [i64]
    L.ss_ffn_forward.restype = i32
    L.ss_ffn_forward.argtypes = [p] * 5 + [i64, i64, i64, i32, dp] + [p] * 5 + [p, sz, p]
    L.ss_ffn_backward.restype = i32
    L.ss_ffn_backward.argtypes = ([p] * 9 + [i64, i64, i64, i32, dp, i32, i32] + [p] * 4
                                  + [p, sz, p])


_declare(_lib)


def _public_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle by device index, and the current device's index: by
# torch's own short cuts (a call of 4.6 us instead of 6.1), which builds of torch without
# CUDA lack and a release may rename, else by the public calls.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or _public_stream
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# The checks below run in front of launches of a few microseconds, so each call
# asks the cheap questions first and goes through _need, which says what is
# wrong, only where one of them fails.

_BF16, _U8 = torch.bfloat16, torch.uint8
_U64 = 0xFFFFFFFFFFFFFFFF


def _fits(t, dtype, index, shape) -> bool:
    try:
        return (t.dtype is dtype and t.get_device() == index and t.shape == shape
                and t.is_contiguous())
    except AttributeError:  # no tensor: _need says so
        return False


def _call(fn, index, *args):
    """fn(*args, stream) with device `index` current: the library launches on
    the current device. The C entry point's name is the function's."""
    if index == _current_device():
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        raise SSError(code, fn.__name__)


def _dropout_spec(p, seed, offset, device):
    if not 0 <= offset <= _U64:
        raise ValueError(f"offset must be in [0, 2^64), got {offset}")
    if seed.__class__ is int:
        return DropoutSpec(p, seed & _U64, None, offset)
    if isinstance(seed, torch.Tensor):
        _need(seed, "seed", torch.int64, device)
        if seed.numel() != 1:
            raise ValueError(f"seed must hold one value, got {seed.numel()}")
        return DropoutSpec(p, 0, seed.data_ptr(), offset)
    try:
        seed = operator.index(seed)
    except TypeError:
        raise TypeError(f"seed must be an int or an int64 CUDA tensor, got {seed!r}") from None
    return DropoutSpec(p, seed & _U64, None, offset)


def _dropout_args(x, name, out, p, seed, offset):
    """Checked (dtype code, device index, out, spec) of an elementwise call."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {x.dtype}")
    index = x.get_device()
    if index < 0 or not x.is_contiguous():
        _need(x, name, x.dtype)
    if out is None:
        out = torch.empty_like(x)
    elif not _fits(out, x.dtype, index, x.shape):
        _need(out, "out", x.dtype, x.device, x.shape)
    return code, index, out, _dropout_spec(p, seed, offset, x.device)


def dropout(x: torch.Tensor, p: float, seed, residual: torch.Tensor | None = None,
            offset: int = 0, out: torch.Tensor | None = None):
    """residual + dropout(x) (ss_dropout): x of any shape, bf16 or fp32; no mask
    is stored. seed: an int, or an int64 CUDA tensor of one value that the
    kernel reads when it runs (a captured graph then draws a new mask whenever
    the tensor has changed). offset: the position of x's first element in the
    stream of random numbers. out may be x or residual."""
    code, index, out, spec = _dropout_args(x, "x", out, p, seed, offset)
    if residual is not None and not _fits(residual, x.dtype, index, x.shape):
        _need(residual, "residual", x.dtype, x.device, x.shape)
    _call(_lib.ss_dropout, index, x.data_ptr(), None if residual is None else residual.data_ptr(),
          x.numel(), code, spec, out.data_ptr())
    return out


def dropout_backward(dy: torch.Tensor, p: float, seed, offset: int = 0,
                     out: torch.Tensor | None = None):
    """The gradient of dropout(x, p, seed, offset=offset) with respect to x
    (ss_dropout_backward); that of its residual is dy itself. out may be dy."""
    code, index, out, spec = _dropout_args(dy, "dy", out, p, seed, offset)
    _call(_lib.ss_dropout_backward, index, dy.data_ptr(), dy.numel(), code, spec, out.data_ptr())
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


class FfnSaved:
    """What ffn_forward(save=True) keeps for ffn_backward: G, U and A ([T, F]
    bf16, also saved[0], saved[1], saved[2]) and the low bits of G and U (R of
    include/ss_block.h), in one buffer. They belong together: to change one of
    them, pass three tensors of your own."""

    __slots__ = ("buffer", "T", "F")

    def __init__(self, T: int, F: int, device):
        self.T, self.F = T, F
        self.buffer = torch.empty((self._low_offset() + T * _low_pitch(F)) // 2, dtype=_BF16,
                                  device=device)

    def _low_offset(self) -> int:
        return (6 * self.T * self.F + 31) // 32 * 32

    def pointers(self):
        """Device addresses of G, U, A and R."""
        g, n = self.buffer.data_ptr(), 2 * self.T * self.F
        return g, g + n, g + 2 * n, g + self._low_offset()

    def __len__(self):
        return 3

    def __getitem__(self, i: int) -> torch.Tensor:
        if not 0 <= i < 3:
            raise IndexError(i)
        n = self.T * self.F
        return self.buffer[i * n:(i + 1) * n].view(self.T, self.F)

    def low_bits(self) -> torch.Tensor:
        """R [T, F]: uint8, G's half byte low, U's high."""
        pitch = _low_pitch(self.F)
        raw = self.buffer.view(torch.uint8)[self._low_offset():]
        return raw[:self.T * pitch].view(self.T, pitch)[:, :self.F]


def _low_pitch(F: int) -> int:
    return (F + 63) // 64 * 64


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}, got {act!r}")
    return code


def _block_args(X, Wg, Wu, Wd, ws):
    """Checked (device index, T, D, F)."""
    try:
        index = X.get_device()
        T, D = X.shape
        up = Wg.shape
        F = up[0]
        if (index >= 0 and X.dtype is Wg.dtype is Wu.dtype is Wd.dtype is _BF16
                and ws.dtype is _U8 and up[1] == D and Wu.shape == up and Wd.shape == (D, F)
                and Wg.get_device() == Wu.get_device() == Wd.get_device() == ws.get_device()
                == index and X.is_contiguous() and Wg.is_contiguous() and Wu.is_contiguous()
                and Wd.is_contiguous() and ws.is_contiguous()):
            return index, T, D, F
    except (AttributeError, IndexError, ValueError):
        pass
    _need(X, "X", _BF16)
    if X.dim() != 2:
        raise ValueError(f"X must be [T, D], got {tuple(X.shape)}")
    T, D = X.shape
    _need(Wg, "Wg", _BF16, X.device)
    F = Wg.shape[0] if Wg.dim() else 0
    for t, name, shape in ((Wg, "Wg", (F, D)), (Wu, "Wu", (F, D)), (Wd, "Wd", (D, F))):
        _need(t, name, _BF16, X.device, shape)
    _need(ws, "workspace", _U8, X.device)
    raise AssertionError("unreachable: one of the checks above fails")


def ffn_forward(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, Wd: torch.Tensor,
                ws: torch.Tensor, act: str = "silu", residual: torch.Tensor | None = None,
                p: float = 0.0, seed=0, offset: int = 0, save: bool = False,
                out: torch.Tensor | None = None):
    """The gated feed-forward block (ss_ffn_forward):
        Y = residual + dropout((act(X Wg^T) * (X Wu^T)) Wd^T)
    X [T, D], Wg, Wu [F, D], Wd [D, F], all bf16. Returns Y, or with save=True
    (Y, saved), an FfnSaved for ffn_backward. out may be residual. p, seed and
    offset as for dropout()."""
    index, T, D, F = _block_args(X, Wg, Wu, Wd, ws)
    if residual is not None and not _fits(residual, _BF16, index, X.shape):
        _need(residual, "residual", _BF16, X.device, X.shape)
    if out is None:
        out = torch.empty_like(X)
    elif not _fits(out, _BF16, index, X.shape):
        _need(out, "out", _BF16, X.device, X.shape)
    saved, g, u, a, r = None, None, None, None, None
    if save:
        saved = FfnSaved(T, F, X.device)
        g, u, a, r = saved.pointers()
    _call(_lib.ss_ffn_forward, index, X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(),
          None if residual is None else residual.data_ptr(), T, D, F, _act(act),
          _dropout_spec(p, seed, offset, X.device), out.data_ptr(), g, u, a, r, ws.data_ptr(),
          ws.numel())
    return (out, saved) if save else out


def ffn_backward(dY: torch.Tensor, X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor,
                 Wd: torch.Tensor, saved, ws: torch.Tensor, act: str = "silu", p: float = 0.0,
                 seed=0, offset: int = 0, dw_dtype=torch.float32, accumulate: bool = False,
                 dX: torch.Tensor | None = None, dWg: torch.Tensor | None = None,
                 dWu: torch.Tensor | None = None, dWd: torch.Tensor | None = None):
    """The gradients of ffn_forward (ss_ffn_backward) from dY [T, D] and `saved`
    (that of ffn_forward, or three [T, F] tensors G, U, A): {"dX", "dWg",
    "dWu", "dWd"}, dX bf16 and the weight gradients of dw_dtype (fp32 or bf16),
    zero-filled when accumulate=True and none is given. Outputs that are given must
    not overlap the inputs or one another. The gradient of the residual is dY
    itself."""
    index, T, D, F = _block_args(X, Wg, Wu, Wd, ws)
    dev = X.device
    dw = _DTYPES.get(dw_dtype)
    if dw is None:
        raise TypeError(f"dw_dtype must be torch.bfloat16 or torch.float32, got {dw_dtype}")
    if not _fits(dY, _BF16, index, X.shape):
        _need(dY, "dY", _BF16, dev, X.shape)
    if isinstance(saved, FfnSaved):
        if (saved.T, saved.F) != (T, F) or saved.buffer.get_device() != index:
            raise ValueError(f"saved is of [{saved.T}, {saved.F}] on {saved.buffer.device}, "
                             f"expected [{T}, {F}] on {dev}")
        g, u, a, r = saved.pointers()
    else:
        G, U, A = saved
        for t, name in ((G, "G"), (U, "U"), (A, "A")):
            if not _fits(t, _BF16, index, (T, F)):
                _need(t, name, _BF16, dev, (T, F))
        g, u, a, r = G.data_ptr(), U.data_ptr(), A.data_ptr(), None
    if dX is None:
        dX = torch.empty_like(X)
    elif not _fits(dX, _BF16, index, X.shape):
        _need(dX, "dX", _BF16, dev, X.shape)
    new = torch.zeros if accumulate else torch.empty
    up, down = (F, D), (D, F)
    if dWg is None:
        dWg = new(up, dtype=dw_dtype, device=dev)
    elif not _fits(dWg, dw_dtype, index, up):
        _need(dWg, "dWg", dw_dtype, dev, up)
    if dWu is None:
        dWu = new(up, dtype=dw_dtype, device=dev)
    elif not _fits(dWu, dw_dtype, index, up):
        _need(dWu, "dWu", dw_dtype, dev, up)
    if dWd is None:
        dWd = new(down, dtype=dw_dtype, device=dev)
    elif not _fits(dWd, dw_dtype, index, down):
        _need(dWd, "dWd", dw_dtype, dev, down)
    _call(_lib.ss_ffn_backward, index, dY.data_ptr(), X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
          Wd.data_ptr(), g, u, a, r, T, D, F, _act(act), _dropout_spec(p, seed, offset, dev), dw,
          1 if accumulate else 0, dX.data_ptr(), dWg.data_ptr(), dWu.data_ptr(), dWd.data_ptr(),
          ws.data_ptr(), ws.numel())
    return {"dX": dX, "dWg": dWg, "dWu": dWu, "dWd": dWd}
