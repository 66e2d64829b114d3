"""The operators of include/ss_block.h in 64 bits, with bounds on how far a
result may be from them, counted from the roundings that the interface states.

Each bf16 rounding is off by at most half a step: BF = finfo(bf16).eps / 2 of
the value. A sum of n products in fp32 is off by at most SUM(n) times the sum of
the products' magnitudes (n additions of half a step each, and a tensor core may
truncate where an adder rounds: one whole step). The activations use the
hardware's exponential and reciprocal: ACT relative.
"""
from __future__ import annotations

import math

import numpy as np
import torch

F64 = torch.float64
BF = torch.finfo(torch.bfloat16).eps / 2
F32 = torch.finfo(torch.float32).eps / 2
ACT = 2.0 ** -18


def SUM(n):
    return (n + 8) * 2 * F32


def keep_mask(n: int, p: float, seed: int, offset: int = 0) -> np.ndarray:
    """Which of the elements offset .. offset + n - 1 of the stream stay."""
    e = np.arange(n, dtype=np.uint64) + np.uint64(offset)
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + ((e >> np.uint64(1)) + np.uint64(1)) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    bits = np.where(e & np.uint64(1), z >> np.uint64(32), z & np.uint64(0xFFFFFFFF))
    return bits >= np.uint64(int(p * 2 ** 32))


def keep_factor(shape, p, seed, offset=0, device="cuda"):
    """1 / (1 - p) where an element stays, else 0."""
    if p == 0.0:
        return torch.ones(shape, dtype=F64, device=device)
    if p == 1.0:
        return torch.zeros(shape, dtype=F64, device=device)
    m = keep_mask(math.prod(shape), p, seed, offset).reshape(shape)
    return torch.from_numpy(m).to(device).to(F64) / (1.0 - p)


def act64(g, act):
    """act(g) and act'(g)."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-g * math.sqrt(0.5))
        return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (g + 0.044715 * g ** 3))  # (1 + tanh(v)) / 2 is sigmoid(2 v)
        return g * s, s + g * s * (1 - s) * c * (1 + 0.134145 * g * g)
    on = (g > 0).to(F64)
    return g * on, on


def forward64(X, Wg, Wu, Wd, act, residual=None, factor=None):
    """{name: (value, bound on the error of the library's result)}."""
    X, Wg, Wu, Wd = (t.to(F64) for t in (X, Wg, Wu, Wd))
    D, F = X.shape[1], Wg.shape[0]
    G, U = X @ Wg.T, X @ Wu.T
    dg, du = SUM(D) * (X.abs() @ Wg.abs().T), SUM(D) * (X.abs() @ Wu.abs().T)
    a, _ = act64(G, act)
    A = a * U
    # |act'| <= 1.13 everywhere; act itself is ACT (1 + |g|) off
    eA = (1.13 * dg + ACT * (a.abs() + dg)) * U.abs() + (a.abs() + 1.13 * dg) * du
    eA_bf = eA + BF * (A.abs() + eA)
    Z = A @ Wd.T
    eZ = eA_bf @ Wd.abs().T + SUM(F) * ((A.abs() + eA_bf) @ Wd.abs().T)
    f = torch.ones_like(Z) if factor is None else factor
    Y = Z * f + (0 if residual is None else residual.to(F64))
    eY = eZ * f + 4 * F32 * (Z.abs() * f + Y.abs())
    return {"Y": (Y, eY + BF * (Y.abs() + eY)), "G": (G, dg + BF * (G.abs() + dg)),
            "U": (U, du + BF * (U.abs() + du)), "A": (A, eA_bf)}


def refined(saved, low=None):
    """G, U (with their low bits: 8 plus 16ths of a bf16 step of their bit patterns,
    a 256th more each) and A of an FfnSaved, or of some rows of one and of its low
    bits, as fp32 tensors."""
    low = (saved.low_bits() if low is None else low).to(torch.int32)

    def add(t, nibble):
        bits = (t.contiguous().view(torch.int16).to(torch.int32) << 16) + (nibble - 8) * 0x1010
        return bits.view(torch.float32)

    return add(saved[0], low & 15), add(saved[1], low >> 4), saved[2]


def backward64(dY, X, Wg, Wu, Wd, saved, act, factor=None, fp32_dw=True):
    """From the saved tensors as they are: {name: (value, bound)}."""
    dY, X, Wg, Wu, Wd = (t.to(F64) for t in (dY, X, Wg, Wu, Wd))
    G, U, A = (t.to(F64) for t in saved)
    T, D = X.shape
    F = Wg.shape[0]
    dZ = dY if factor is None else dY * factor
    dA = dZ @ Wd
    eA = (SUM(D) + 4 * F32) * (dZ.abs() @ Wd.abs())
    a, d = act64(G, act)
    dG, dU = dA * U * d, dA * a
    # the slope is a sum of two terms of at most 1 + |g|, each ACT off
    e_d, e_a = ACT * 2 * (1 + G.abs()), ACT * (a.abs() + 1e-30)
    eG = eA * (U * d).abs() + (dA.abs() + eA) * U.abs() * e_d
    eU = eA * a.abs() + (dA.abs() + eA) * e_a
    eG, eU = eG + BF * (dG.abs() + eG), eU + BF * (dU.abs() + eU)

    def product(l, el, r, n):
        return l @ r, el @ r.abs() + SUM(n) * ((l.abs() + el) @ r.abs())

    x1, ex1 = product(dG, eG, Wg, 2 * F)
    x2, ex2 = product(dU, eU, Wu, 2 * F)
    wg, ewg = product(dG.T, eG.T, X, T)
    wu, ewu = product(dU.T, eU.T, X, T)
    wd, ewd = product(dZ.T, 4 * F32 * dZ.abs().T, A, T)
    out = {"dX": (x1 + x2, ex1 + ex2), "dWg": (wg, ewg), "dWu": (wu, ewu), "dWd": (wd, ewd)}
    for k, (v, e) in out.items():
        step = F32 if fp32_dw and k != "dX" else BF
        out[k] = (v, e + step * (v.abs() + e))
    return out


def assert_within(got: torch.Tensor, ref, name=""):
    value, bound = ref
    off = (got.to(F64) - value).abs()
    bad = ~(off <= bound + 1e-37)
    assert not bad.any(), (
        f"{name}: {int(bad.sum())} of {bad.numel()} values off; worst ratio to the bound "
        f"{float((off / (bound + 1e-37)).nan_to_num(nan=math.inf).max()):.3g} "
        f"at {bad.nonzero()[0].tolist()}")
