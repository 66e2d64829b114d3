"""The operators of include/ss_logprob.h in 64 bits, with bounds on how far a result
may be from them, counted from the roundings that the interface and the kernels'
comments state (BF, F32 and SUM as in block_util).

Logits. A product of two bf16 values is exact in fp32; a sum of D of them is off by
at most SUM(D) times the sum of their magnitudes. With a cap, z is a sum's error times
the largest slope cap / (4 tau), plus the hardware's exponential and reciprocal: ACT
of cap.

Log-sum-exp. Its error is the logits' error averaged over the softmax, plus that of
the sum of exponentials: the exponent's argument is (z - m) log2 e with m log2 e and
the difference rounded, 4 |m| half steps, the exponential itself 2^-21, and the sum
about 64 additions in a tile, bins / 32 + 8 to join them, then the logarithm's own
2 |lse| half steps.
"""
from __future__ import annotations

import math

import torch

from block_util import ACT, BF, F32, F64, SUM, assert_within  # noqa: F401


def logits64(H, W, cap=0.0, tau=1.0):
    """z, dz/ds and the bound on z's error."""
    H, W = H.to(F64), W.to(F64)
    s = H @ W.T
    e = SUM(H.shape[1]) * (H.abs() @ W.abs().T)
    if not cap:
        return s, None, e
    w = torch.special.expit(s / tau)
    slope = cap / tau * w * torch.special.expit(-s / tau)
    return cap * w, slope, e * cap / (4 * tau) + ACT * cap


def logprobs64(H, W, ids, cap=0.0, tau=1.0):
    """{"logp": (value, bound), "lse": (value, bound)}; ids [T, K]."""
    z, _, e = logits64(H, W, cap, tau)
    lse = torch.logsumexp(z, 1)
    P = torch.exp(z - lse[:, None])
    m = z.abs().amax(1)
    bins = 2 * ((W.shape[0] + 255) // 256)
    e_lse = ((P * e).sum(1) * 1.01 + (4 * m + 64 + bins / 32 + 8 + 2 * lse.abs()) * 2 * F32
             + 2.0 ** -21)
    at = ids.clamp(min=0).long()
    logp = z.gather(1, at) - lse[:, None]
    e_logp = e.gather(1, at) + e_lse[:, None] + 2 * F32 * logp.abs()
    gone = ids < 0
    return {"logp": (logp.masked_fill(gone, 0.0), e_logp.masked_fill(gone, 0.0)),
            "lse": (lse, e_lse)}


def grads64(dlogp, H, W, ids, logp, lse, cap=0.0, tau=1.0, fp32_dw=True):
    """From logp and lse as they are: {"dH": (value, bound), "dW": (value, bound)}."""
    T, K = ids.shape
    z, slope, e = logits64(H, W, cap, tau)
    H, W = H.to(F64), W.to(F64)
    w = torch.where(ids >= 0, dlogp, 0.0).to(F64)
    live = (w != 0).any(1)
    a, size = -w.sum(1, keepdim=True), w.abs().sum(1, keepdim=True)
    lse, logp = lse.to(F64)[:, None], logp.to(F64)
    P = torch.exp(torch.where(live[:, None], z - lse, -math.inf))
    G = a * P
    # the exponential's argument: z and lse in half steps, the hardware's 2^-20
    eG = (a.abs() + K * F32 * size) * P * (e + 4 * F32 * (lse.abs() + z.abs()) + 2.0 ** -20)
    eG += K * F32 * size * P
    at = ids.clamp(min=0).long()
    here = (ids >= 0) & live[:, None]
    # at the ids: a exp(logp) + w, from logp
    q = torch.where(here, torch.exp(logp), 0.0)
    onto = torch.zeros_like(G).scatter_add_(1, at, w)
    touched = torch.zeros_like(G).scatter_(1, at, here.to(F64)) > 0
    q_at = torch.zeros_like(G).scatter_(1, at, q)
    # (a row of several absent ids may have written over vocabulary row 0)
    for k in range(K):
        q_at[torch.arange(T, device=G.device)[here[:, k]], at[here[:, k], k]] = q[here[:, k], k]
        touched[torch.arange(T, device=G.device)[here[:, k]], at[here[:, k], k]] = True
    G = torch.where(touched, a * q_at, G) + onto
    eG = torch.where(touched, (K + 8) * F32 * 2 * (size * q_at + size), eG)
    if slope is not None:
        # at the ids z comes back as logp + lse: the rounding of the difference that made
        # logp and that of the sum, and |d slope / dz| = |cap - 2 z| / (cap tau) <= 1 / tau
        e_slope = (cap / (4 * tau)) * (8 * ACT + 4 * e / tau) + 1e-30
        l_at = torch.where(touched, z - lse, 0.0)
        e_slope = e_slope + 2 * F32 * (l_at.abs() + z.abs()) * touched / tau
        eG = eG * slope + (G.abs() + eG) * e_slope
        G = G * slope
    eG = eG + (BF + 8 * F32) * (G.abs() + eG)
    live_H = torch.where(live[:, None], H, 0.0)
    dH, eH = G @ W, eG @ W.abs() + SUM(W.shape[0]) * ((G.abs() + eG) @ W.abs())
    dW = G.T @ live_H
    # one id per token: H may be scaled and rounded too
    more = BF + 8 * F32 if K == 1 else 0.0
    eW = eG.T @ live_H.abs() + (SUM(T) + more) * ((G.abs() + eG).T @ live_H.abs())
    step = F32 if fp32_dw else BF
    return {"dH": (dH, eH + BF * (dH.abs() + eH)), "dW": (dW, eW + step * (dW.abs() + eW))}


# ---------------------------------------------------------------- the losses

# exp, expm1, log, log1p in fp32 are within a few half steps of the result: EXP
EXP = 4 * F32


def policy64(logp, old, A, ref=None, m=None, clip=(0.2, 0.2), kl=0.0, scale=1.0):
    """{name: (value, bound)}; the caller keeps ratios off the clip's ends."""
    x, old, A = logp.to(F64), old.to(F64), A.to(F64)
    m = torch.ones_like(x) if m is None else m.to(F64)
    used = m != 0
    r = torch.exp(x - old)
    # the difference of two fp32 numbers rounds by half a step of it
    e_r = r * (2 * F32 * (x - old).abs() + EXP)
    held = ((A > 0) & (r > 1 + clip[1])) | ((A < 0) & (r < 1 - clip[0]))
    free = torch.where(A == 0, 0.0, r * A)
    gain = torch.where(held, r.clamp(1 - clip[0], 1 + clip[1]) * A, free)
    slope = torch.where(held, 0.0, free)
    e_gain = torch.where(held, 4 * F32 * gain.abs(), e_r * A.abs() + 2 * F32 * free.abs())
    loss, d, e_loss, e_d = -gain, -slope, e_gain, torch.where(held, 0.0, e_gain)
    out = {}
    if ref is not None:
        g = ref.to(F64) - x
        e_g = F32 * g.abs()
        k = torch.expm1(g) - g
        e_k = (torch.expm1(g).abs() * EXP + torch.exp(g) * e_g + e_g + 2 * F32 * k.abs()) * 1.01
        out["kl"] = (torch.where(used, k, 0.0), torch.where(used, e_k, 0.0))
        loss, e_loss = loss + kl * k, e_loss + kl * (e_k + 4 * F32 * k.abs()) + 4 * F32 * loss.abs()
        dk = torch.expm1(g)
        e_dk = dk.abs() * (EXP + 4 * F32) + torch.exp(g) * e_g
        d, e_d = d - kl * dk, e_d + kl * e_dk + 4 * F32 * d.abs()
    for name, v, e, f in (("loss", loss, e_loss, 1.0), ("dlogp", d, e_d, scale)):
        v, e = m * v * f, m.abs() * abs(f) * e
        v, e = torch.where(used, v, 0.0), torch.where(used, e + 6 * F32 * v.abs(), 0.0)
        out[name] = (v, e + 1e-37)
    return out


def preference64(logp, offsets, ref=None, m=None, beta=0.1, kind="sigmoid", smoothing=0.0,
                 average=False, scale=1.0):
    x = logp.to(F64)
    n = x.numel()
    m = torch.ones_like(x) if m is None else m.to(F64)
    ref = torch.zeros_like(x) if ref is None else ref.to(F64)
    gap = torch.where(m != 0, m * (x - ref), 0.0)
    # the difference and the product round once each, the sums are in 64 bits
    e_gap = 2 * F32 * gap.abs() * 1.01
    at = offsets.tolist()
    pairs = len(at) // 2
    R, eR, per = [], [], []
    for s in range(2 * pairs):
        part = slice(at[s], at[s + 1])
        mass = float(m[part].sum())
        p = (1 / mass if mass != 0 else 0.0) if average else 1.0
        R.append(float(gap[part].sum()) * p)
        eR.append(float(e_gap[part].sum()) * abs(p))
        per.append(p)
    loss, e_loss, reward, e_reward = [], [], [], []
    d, e_d = torch.zeros_like(x), torch.zeros_like(x)
    for i in range(pairs):
        X, eX = R[2 * i] - R[2 * i + 1], eR[2 * i] + eR[2 * i + 1] + 1e-12
        h, eh = beta * X, beta * eX + 2 * F32 * abs(beta * X)
        if kind == "sigmoid":
            def sp(v):  # log(1 + exp(v))
                return max(v, 0.0) + math.log1p(math.exp(-abs(v)))
            value = (1 - smoothing) * sp(-h) + smoothing * sp(h)
            e_v = eh + 16 * F32 * (value + 1e-30)
            s_neg = math.exp(-sp(h))
            slope = beta * (smoothing - s_neg)
            e_s = beta * (eh * s_neg + 16 * F32 * (s_neg + smoothing))
        elif kind == "hinge":
            value, e_v = max(0.0, 1 - h), eh + 2 * F32
            slope, e_s = (-beta if h < 1 else 0.0), 2 * F32 * beta
        else:
            u = X - 0.5 / beta
            value, slope = u * u, 2 * u
            # 0.5 / beta with beta in fp32
            eu = eX + 2 * F32 * 0.5 / beta
            e_v, e_s = 2 * abs(u) * eu + eu * eu + 2 * F32 * value, 2 * eu + 4 * F32 * abs(slope)
        loss.append(value)
        e_loss.append(e_v)
        for k, sign in ((0, 1.0), (1, -1.0)):
            s = 2 * i + k
            reward.append(beta * R[s])
            e_reward.append(beta * eR[s] + 4 * F32 * abs(beta * R[s]))
            part = slice(at[s], at[s + 1])
            c, e_c = sign * scale * slope * per[s], abs(scale * per[s]) * e_s
            d[part] = m[part] * c
            e_d[part] = m[part].abs() * (e_c + 6 * F32 * abs(c))
    dev = x.device

    def t(v):
        return torch.tensor(v, dtype=F64, device=dev)

    return {"loss": (t(loss), t(e_loss) + 1e-37),
            "reward": (t(reward).view(-1, 2), t(e_reward).view(-1, 2) + 1e-37),
            "dlogp": (d, e_d + 1e-37)} if n or pairs else {}


FLOOR = 2.0 ** -12


def distill64(logp, teacher, ids=None, m=None, tail=False, scale=1.0):
    """The caller keeps the tail off its floor."""
    T, K = logp.shape
    l, x = logp.to(F64), teacher.to(F64)
    here = torch.ones_like(l, dtype=torch.bool) if ids is None else ids >= 0
    m = torch.ones(T, dtype=F64, device=l.device) if m is None else m.to(F64)
    used = ((m != 0) & here.any(1))[:, None]
    x = torch.where(here, x, -math.inf)
    here = here & used
    if tail:
        p = torch.exp(x)
        q = torch.where(here, torch.exp(l), 0.0)
        p1 = (1 - p.sum(1)).clamp(min=0.0)
        rest = 1 - q.sum(1)
        q1 = rest.clamp(min=FLOOR)
        # the exponentials and their sums are pairs; what they leave of 1, (1 - hi) - lo,
        # is an fp32 number: two roundings of at most F32 of it
        e_p1 = 2.0 ** -27 + 2 * F32 * p1
        e_q1 = 2.0 ** -27 + 2 * F32 * q1
        ratio = torch.where(rest > FLOOR, p1 / q1, 0.0)
        e_ratio = (e_p1 + ratio * e_q1) / q1 * 1.01 + 4 * F32 * ratio
        loss = torch.special.xlogy(p1, p1) - p1 * q1.log()
        e_loss = (e_p1 * ((p1 + 1e-30).log() - q1.log()).abs() + e_p1 + p1 * e_q1 / q1
                  + 8 * F32 * (p1 * (p1 + 1e-30).log()).abs() + 8 * F32 * p1 * q1.log().abs())
        logt = torch.where(p > 0, x, 0.0)
        e_logt = torch.zeros_like(p)
        slope = ratio[:, None] * q - p
        e_slope = e_ratio[:, None] * q + (ratio[:, None] * q + p) * (EXP + 2 * F32)
    else:
        lse = torch.logsumexp(x, 1, keepdim=True)
        logt = torch.where(x > -math.inf, x - lse, 0.0)
        p = torch.where(x > -math.inf, torch.exp(logt), 0.0)
        # the differences from the row's largest value, and log of a sum of up to K
        e_logt = 2 * F32 * (x.abs().nan_to_num(posinf=0.0) + lse.abs() + 12)
        e_logt = torch.where(p > 0, e_logt, 0.0)
        loss, e_loss = torch.zeros_like(m), torch.zeros_like(m)
        slope, e_slope = -p, p * (e_logt + 4 * EXP)
    term = torch.where(p > 0, p * (logt - l), 0.0)
    e_term = torch.where(p > 0, p * (e_logt + 2 * F32 * (logt.abs() + l.abs()))
                         + term.abs() * (4 * EXP + e_logt), 0.0)
    loss = loss + term.sum(1)
    e_loss = e_loss + e_term.sum(1) + 10 * F32 * term.abs().sum(1)
    gone = ~used[:, 0]
    loss, e_loss = m * loss, m.abs() * (e_loss + 4 * F32 * loss.abs())
    d = scale * m[:, None] * slope
    e_d = abs(scale) * m.abs()[:, None] * e_slope + 4 * F32 * d.abs()
    off = ~here
    return {"loss": (loss.masked_fill(gone, 0.0), e_loss.masked_fill(gone, 0.0) + 1e-37),
            "dlogp": (d.masked_fill(off, 0.0), e_d.masked_fill(off, 0.0) + 1e-37)}
