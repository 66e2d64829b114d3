"""Python binding of include/ss_logprob.h: the log-probabilities of chosen ids over
the whole vocabulary, forward and backward, and the losses made of them.

    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)                       # ids [T] or [T, K]
    out = ss.policy_loss(logp, old_logp, advantage, ref_logp=ref, weight=m, kl=0.05)
    dH, dW = ss.logprobs_backward(out["dlogp"], H, W, ids, logp, lse, ws)

As in the package's other calls: argument marshalling only, contiguous CUDA
tensors, results on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import Head, SSError, WORKSPACE_HEADER_BYTES, _lib, _need
from .block import _BF16, _DTYPES, _U8, _call, _fits

HEADER_LOGPROB = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                              "include", "ss_logprob.h")
MAX_IDS = 128
PREFERENCES = {"sigmoid": 0, "hinge": 1, "ipo": 2}
_F32, _I32 = torch.float32, torch.int32


def _declare(L):
    p, i64, i32, f, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float,
                          ctypes.c_size_t)
    hp = ctypes.POINTER(Head)
    L.ss_logprob_workspace_size.restype = sz
    L.ss_logprob_workspace_size.argtypes = [i64, i64, i64, i32]
    L.ss_logprob_forward.restype = i32
    L.ss_logprob_forward.argtypes = [p, p, p, i64, i64, i64, i64, hp, p, p, p, sz, p]
    L.ss_logprob_backward.restype = i32
    L.ss_logprob_backward.argtypes = [p] * 6 + [i64, i64, i64, i64, hp, i32, i32, p, p, p, sz, p]
    L.ss_policy_loss.restype = i32
    L.ss_policy_loss.argtypes = [p] * 5 + [i64, f, f, f, f, p, p, p, p]
    L.ss_preference_loss.restype = i32
    L.ss_preference_loss.argtypes = [p] * 4 + [i64, i64, i32, f, f, i32, f, p, p, p, p, sz, p]
    L.ss_distill_loss.restype = i32
    L.ss_distill_loss.argtypes = [p, p, i32, p, p, i64, i64, i32, f, p, p, p]


_declare(_lib)


def _at(t):
    return None if t is None else t.data_ptr()


def _head_of(cap, tau):
    return None if cap == 0 else Head(cap, tau, 0)


# As in block.py, the checks run in front of launches of a few microseconds: the cheap
# questions first, _need, which says what is wrong, only where one of them fails.

def _expect(t, name, dtype, index, shape, device):
    if not _fits(t, dtype, index, shape):
        _need(t, name, dtype, device, shape)


def _out(t, name, dtype, like_shape, index, device):
    if t is None:
        return torch.empty(like_shape, dtype=dtype, device=device)
    _expect(t, name, dtype, index, like_shape, device)
    return t


def _rows_like(logp, **others):
    """The device index of logp, an fp32 tensor, which `others` (None: not given) are
    like."""
    try:
        index, shape = logp.get_device(), logp.shape
        if index >= 0 and logp.dtype is _F32 and logp.is_contiguous():
            for t in others.values():
                if t is not None and not (t.dtype is _F32 and t.shape == shape
                                          and t.get_device() == index and t.is_contiguous()):
                    break
            else:
                return index
    except AttributeError:  # no tensor
        pass
    _need(logp, "logp", _F32)
    for name, t in others.items():
        if t is not None:
            _need(t, name, _F32, logp.device, logp.shape)
    raise AssertionError("unreachable: one of the checks above fails")


def logprob_workspace_size(T: int, V: int, D: int, backward: bool = True) -> int:
    n = _lib.ss_logprob_workspace_size(T, V, D, 1 if backward else 0)
    if n == 0:
        raise SSError(1, "ss_logprob_workspace_size")
    return int(n)


def logprob_workspace(T: int, V: int, D: int, backward: bool = True, device=None) -> torch.Tensor:
    """A device byte buffer for the log-probabilities of up to T tokens (with
    backward=False without their backward pass), its header zeroed as
    include/ss_logprob.h requires."""
    ws = torch.empty(logprob_workspace_size(T, V, D, backward), dtype=_U8,
                     device=device if device is not None else "cuda")
    ws[:WORKSPACE_HEADER_BYTES].zero_()
    return ws


def _logprob_args(H, W, ids, ws):
    """Checked (device index, T, V, D, K)."""
    try:
        index = H.get_device()
        T, D = H.shape
        V = W.shape[0]
        n = ids.shape
        if (index >= 0 and H.dtype is W.dtype is _BF16 and ids.dtype is _I32 and ws.dtype is _U8
                and W.shape == (V, D) and 1 <= len(n) <= 2 and n[0] == T
                and W.get_device() == ids.get_device() == ws.get_device() == index
                and H.is_contiguous() and W.is_contiguous() and ids.is_contiguous()
                and ws.is_contiguous()):
            return index, T, V, D, n[1] if len(n) == 2 else 1
    except (AttributeError, IndexError, ValueError):
        pass
    _need(H, "H", _BF16)
    if H.dim() != 2:
        raise ValueError(f"H must be [T, D], got {tuple(H.shape)}")
    T, D = H.shape
    dev = H.device
    _need(W, "W", _BF16, dev)
    _need(W, "W", _BF16, dev, (W.shape[0] if W.dim() else 0, D))
    _need(ids, "ids", _I32, dev)
    if ids.dim() not in (1, 2) or ids.shape[0] != T:
        raise ValueError(f"ids must be [{T}] or [{T}, K], got {tuple(ids.shape)}")
    _need(ws, "workspace", _U8, dev)
    raise AssertionError("unreachable: one of the checks above fails")


def logprobs(H: torch.Tensor, W: torch.Tensor, ids: torch.Tensor, ws: torch.Tensor,
             cap: float = 0.0, tau: float = 1.0, logp: torch.Tensor | None = None,
             lse: torch.Tensor | None = None):
    """Log-probabilities of ids over the whole vocabulary (ss_logprob_forward): H
    [T, D], W [V, D] bf16, ids [T] or [T, K] int32 (-1: absent, 0 there). Returns
    (logp like ids, lse [T]), fp32. cap and tau as for forward()."""
    index, T, V, D, K = _logprob_args(H, W, ids, ws)
    dev = H.device
    logp = _out(logp, "logp", _F32, ids.shape, index, dev)
    lse = _out(lse, "lse", _F32, (T,), index, dev)
    _call(_lib.ss_logprob_forward, index, H.data_ptr(), W.data_ptr(), ids.data_ptr(), K, T, V, D,
          _head_of(cap, tau), logp.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel())
    return logp, lse


def logprobs_backward(dlogp: torch.Tensor, H: torch.Tensor, W: torch.Tensor, ids: torch.Tensor,
                      logp: torch.Tensor, lse: torch.Tensor, ws: torch.Tensor, cap: float = 0.0,
                      tau: float = 1.0, dw_dtype=torch.float32, accumulate: bool = False,
                      dH: torch.Tensor | None = None, dW: torch.Tensor | None = None):
    """(dH [T, D] bf16, dW [V, D] of dw_dtype, fp32 or bf16) of sum(dlogp * logp)
    (ss_logprob_backward), logp and lse those of logprobs() on the same H, W and
    ids. A dW that is not given is zero-filled when accumulate=True."""
    index, T, V, D, K = _logprob_args(H, W, ids, ws)
    dev = H.device
    dw = _DTYPES.get(dw_dtype)
    if dw is None:
        raise TypeError(f"dw_dtype must be torch.bfloat16 or torch.float32, got {dw_dtype}")
    _expect(dlogp, "dlogp", _F32, index, ids.shape, dev)
    _expect(logp, "logp", _F32, index, ids.shape, dev)
    _expect(lse, "lse", _F32, index, (T,), dev)
    dH = _out(dH, "dH", _BF16, (T, D), index, dev)
    if dW is None:
        dW = (torch.zeros if accumulate else torch.empty)((V, D), dtype=dw_dtype, device=dev)
    else:
        _expect(dW, "dW", dw_dtype, index, (V, D), dev)
    _call(_lib.ss_logprob_backward, index, dlogp.data_ptr(), H.data_ptr(), W.data_ptr(),
          ids.data_ptr(), logp.data_ptr(), lse.data_ptr(), K, T, V, D, _head_of(cap, tau), dw,
          1 if accumulate else 0, dH.data_ptr(), dW.data_ptr(), ws.data_ptr(), ws.numel())
    return dH, dW


def policy_loss(logp: torch.Tensor, old_logp: torch.Tensor, advantage: torch.Tensor,
                ref_logp: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                clip=0.2, kl: float = 0.0, scale: float = 1.0):
    """The clipped policy loss with a KL term (ss_policy_loss), fp32 tensors of one
    shape, a value per token:
        weight * (-min(r A, clip(r, 1 - low, 1 + high) A) + kl * (exp(d) - d - 1))
    with r = exp(logp - old_logp), d = ref_logp - logp; clip is (low, high), or one
    number for both. Returns {"loss", "dlogp"} and with ref_logp "kl", each like
    logp; dlogp = scale * d loss / d logp. Tokens of weight 0 give 0."""
    if old_logp is None or advantage is None:
        raise TypeError("old_logp and advantage must be torch.Tensors")
    index = _rows_like(logp, old_logp=old_logp, advantage=advantage, ref_logp=ref_logp,
                       weight=weight)
    low, high = clip if isinstance(clip, (tuple, list)) else (clip, clip)
    loss, dlogp = torch.empty_like(logp), torch.empty_like(logp)
    out = {"loss": loss, "dlogp": dlogp}
    k = None
    if ref_logp is not None:
        out["kl"] = k = torch.empty_like(logp)
    _call(_lib.ss_policy_loss, index, logp.data_ptr(), old_logp.data_ptr(), advantage.data_ptr(),
          _at(ref_logp), _at(weight), logp.numel(), low, high, kl, scale, loss.data_ptr(), _at(k),
          dlogp.data_ptr())
    return out


def preference_loss(logp: torch.Tensor, offsets: torch.Tensor, ws: torch.Tensor,
                    ref_logp: torch.Tensor | None = None, weight: torch.Tensor | None = None,
                    beta: float = 0.1, kind: str = "sigmoid", smoothing: float = 0.0,
                    average: bool = False, scale: float = 1.0):
    """Losses of preference pairs in a packed batch (ss_preference_loss): logp,
    ref_logp, weight [n] fp32; offsets [2 P + 1] int32, sequence s is the tokens
    [offsets[s], offsets[s + 1]) and pair i the sequences 2 i (chosen) and 2 i + 1
    (rejected). kind: "sigmoid" (with label smoothing), "hinge" or "ipo". Any
    workspace of the package records a bad offset. Returns {"loss" [P], "reward"
    [P, 2], "dlogp" [n]}; dlogp = scale * d loss / d logp, 0 outside the sequences."""
    index, dev = _rows_like(logp, ref_logp=ref_logp, weight=weight), logp.device
    if logp.dim() != 1:
        raise ValueError(f"logp must be [n], got {tuple(logp.shape)}")
    if not _fits(offsets, _I32, index, getattr(offsets, "shape", None)):
        _need(offsets, "offsets", _I32, dev)
    if offsets.dim() != 1 or offsets.numel() % 2 != 1:
        raise ValueError(f"offsets must be [2 P + 1], got {tuple(offsets.shape)}")
    if not _fits(ws, _U8, index, getattr(ws, "shape", None)):
        _need(ws, "workspace", _U8, dev)
    code = PREFERENCES.get(kind)
    if code is None:
        raise ValueError(f"kind must be one of {sorted(PREFERENCES)}, got {kind!r}")
    pairs = offsets.numel() // 2
    loss = torch.empty(pairs, dtype=_F32, device=dev)
    reward = torch.empty((pairs, 2), dtype=_F32, device=dev)
    dlogp = torch.empty_like(logp)
    _call(_lib.ss_preference_loss, index, logp.data_ptr(), _at(ref_logp), _at(weight),
          offsets.data_ptr(), pairs, logp.numel(), code, beta, smoothing, 1 if average else 0,
          scale, loss.data_ptr(), reward.data_ptr(), dlogp.data_ptr(), ws.data_ptr(), ws.numel())
    return {"loss": loss, "reward": reward, "dlogp": dlogp}


def distill_loss(logp: torch.Tensor, teacher: torch.Tensor, ids: torch.Tensor | None = None,
                 weight: torch.Tensor | None = None, tail: bool = False, scale: float = 1.0):
    """KL(teacher || student) over the teacher's top ids (ss_distill_loss): logp
    [T, K] fp32 of the student at those ids, teacher [T, K] fp32 or bf16 its values
    there: logits or log-probabilities, renormalised over the K, or with tail=True
    log-probabilities, what they leave of 1 being one more class. ids [T, K]: an
    entry of -1 is absent. weight [T]. Returns {"loss" [T], "dlogp" [T, K]}; dlogp =
    scale * d loss / d logp."""
    index, dev = _rows_like(logp), logp.device
    if logp.dim() != 2:
        raise ValueError(f"logp must be [T, K], got {tuple(logp.shape)}")
    T, K = logp.shape
    if not isinstance(teacher, torch.Tensor):
        raise TypeError("teacher must be a torch.Tensor")
    code = _DTYPES.get(teacher.dtype)
    if code is None:
        raise TypeError(f"teacher must be torch.bfloat16 or torch.float32, got {teacher.dtype}")
    _expect(teacher, "teacher", teacher.dtype, index, logp.shape, dev)
    if ids is not None:
        _expect(ids, "ids", _I32, index, logp.shape, dev)
    if weight is not None:
        _expect(weight, "weight", _F32, index, (T,), dev)
    loss = torch.empty(T, dtype=_F32, device=dev)
    dlogp = torch.empty_like(logp)
    _call(_lib.ss_distill_loss, index, logp.data_ptr(), teacher.data_ptr(), code, _at(ids),
          _at(weight), T, K, 1 if tail else 0, scale, loss.data_ptr(), dlogp.data_ptr())
    return {"loss": loss, "dlogp": dlogp}
