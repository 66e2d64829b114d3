"""Cases of the operators around the output head: dropout from a counter-based
generator, and the gated feed-forward block that produces the head's input H.

Dropout. Element e (counted row by row, from 0) has 32 random bits: with z the
SplitMix64 output number e >> 1 of the stream of `seed`, the low 32 bits of z
where e is even and the high 32 where it is odd. It is dropped where the bits
are below floor(p 2^32); what is kept is multiplied by 1 / (1 - p):
    y = residual + (keep ? x / (1 - p) : 0)        dx = keep ? dy / (1 - p) : 0

Feed-forward block, weights as a linear layer holds them, Wg, Wu [F, D] and
Wd [D, F]:
    G = X Wg^T    U = X Wu^T    A = act(G) U    Z = A Wd^T
    Y = residual + dropout(Z)
and its gradients from dY and the saved G, U, A:
    dZ = dropout'(dY)           dA = dZ Wd
    dG = dA U act'(G)           dU = dA act(G)
    dX = dG Wg + dU Wu          dWg = dG^T X    dWu = dU^T X    dWd = dZ^T A
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
SQRT_2_OVER_PI = math.sqrt(2.0 / math.pi)


# --------------------------------------------------------------------- cases

def _ffn(name, op, T, D, F, act="silu", p=0.0, residual=False):
    return {"name": name, "op": op, "T": T, "D": D, "F": F, "act": act, "p": p,
            "residual": residual}


def _drop(name, op, rows, cols, p, dtype="bf16", residual=False):
    return {"name": name, "op": op, "rows": rows, "cols": cols, "p": p, "dtype": dtype,
            "residual": residual}


def listed():
    return [
        # one token's hidden state: launch latency
        _drop("dropout_token", "dropout", 1, 768, 0.1),
        # the residual branch in front of the head, at the largest batch the head is timed on
        _drop("dropout_residual", "dropout", 65536, 768, 0.1, residual=True),
        # odd width, fp32 gradients
        _drop("dropout_backward_odd_f32", "dropout_backward", 16411, 1021, 0.25, "f32"),
        # the backward of dropout over a block's inner activations
        _drop("dropout_backward_wide", "dropout_backward", 65536, 2048, 0.5),
        # decoding one token at the head's model width
        _ffn("ffn_token", "ffn_forward", 1, 768, 2048, residual=True),
        # decoding a small batch in a wide model: bound by the weights' bytes
        _ffn("ffn_decode_wide", "ffn_forward", 16, 4096, 12288, residual=True),
        # a ragged prompt, sizes that fill no tile
        _ffn("ffn_prompt_ragged", "ffn_forward", 1003, 1096, 2952, "gelu_tanh", residual=True),
        # a training step's forward at the head's ordinary batch, activations saved
        _ffn("ffn_train_forward", "ffn_train_forward", 16384, 768, 2048, p=0.1, residual=True),
        # backward of the head's smallest batch
        _ffn("ffn_backward_small", "ffn_backward", 256, 768, 2048),
        # backward with ragged sizes
        _ffn("ffn_backward_ragged", "ffn_backward", 3001, 1352, 3640, "gelu"),
        # backward of the head's largest batch
        _ffn("ffn_backward_large", "ffn_backward", 65536, 768, 2048, p=0.1),
        # forward and backward as a training step calls them, a wider model
        _ffn("ffn_step", "ffn_step", 8192, 2048, 5504, p=0.1, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.4:
        op = rng.choice(["dropout", "dropout_backward"])
        cols = _log(rng, 1, 4096)
        rows = max(1, min(_log(rng, 1, 65536), 65536 * 2048 // cols))
        return {"op": op, "rows": rows, "cols": cols,
                "p": rng.choice([0.05, 0.1, 0.25, 0.5, round(rng.random() * 0.9, 3)]),
                "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "residual": op == "dropout" and rng.random() < 0.5}
    op = rng.choice(["ffn_forward", "ffn_forward", "ffn_train_forward", "ffn_backward",
                     "ffn_backward", "ffn_step"])
    most = 12.0 * 65536 * 768 * 2048  # the largest listed backward
    flops = {"ffn_forward": 6, "ffn_train_forward": 6, "ffn_backward": 12, "ffn_step": 18}[op]
    D = 8 * _log(rng, 8, 512)
    F = 8 * min(_log(rng, 8, 1536), 4 * D // 8)
    T = _log(rng, 1, 65536)
    T = max(1, min(T, int(most / (flops * D * F)), (1 << 27) // F))
    forward = op != "ffn_backward"
    return {"op": op, "T": T, "D": D, "F": F,
            "act": rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]),
            "p": rng.choice([0.0, 0.1, 0.2]), "residual": forward and rng.random() < 0.7}


def work(case):
    if case["op"].startswith("dropout"):
        n = case["rows"] * case["cols"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * size * (3 if case["residual"] else 2), "flops": 2.0 * n}
    T, D, F = case["T"], case["D"], case["F"]
    x, a, w, r = T * D, T * F, 3 * F * D, T * D if case["residual"] else 0
    values = {"ffn_forward": 2 * x + w + r,                   # X, W -> Y
              "ffn_train_forward": 2 * x + w + r + 3 * a,     # ... and G, U, A
              "ffn_backward": 3 * x + 2 * w + 3 * a,          # X, dY, W, G, U, A -> dX, dW
              "ffn_step": 4 * x + 2 * w + r}[case["op"]]      # X, dY, W -> Y, dX, dW
    flops = {"ffn_forward": 6, "ffn_train_forward": 6, "ffn_backward": 12, "ffn_step": 18}
    return {"bytes": 2 * values, "flops": float(flops[case["op"]]) * T * D * F}


# -------------------------------------------------------------------- inputs

def _seed64(seed):
    return (seed * 0x2545F4914F6CDD1D + 0x1234567) % 2**64


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=BF16):
        t = torch.randn(*shape, generator=gen, device="cuda", dtype=F32)
        return t.mul_(scale).to(dtype)

    s = {"case": case, "seed": _seed64(seed)}
    if case["op"].startswith("dropout"):
        dtype = BF16 if case["dtype"] == "bf16" else F32
        shape = (case["rows"], case["cols"])
        # gradients reach the backward small: a mean over tokens divides them
        s["x"] = normal(*shape, scale=1.0 if case["op"] == "dropout" else 1e-3, dtype=dtype)
        s["residual"] = normal(*shape, dtype=dtype) if case["residual"] else None
        return s
    T, D, F = case["T"], case["D"], case["F"]
    s["X"] = normal(T, D)  # a normalised hidden state
    s["Wg"] = normal(F, D, scale=D ** -0.5)
    s["Wu"] = normal(F, D, scale=D ** -0.5)
    s["Wd"] = normal(D, F, scale=F ** -0.5)
    s["residual"] = normal(T, D) if case["residual"] else None
    if case["op"] in ("ffn_backward", "ffn_step"):
        s["dY"] = normal(T, D, scale=1e-2)
    if case["op"] == "ffn_backward":  # what the forward of this batch left behind
        X = s["X"].float()
        G, U = X @ s["Wg"].float().T, X @ s["Wu"].float().T
        s["saved"] = (G.to(BF16), U.to(BF16), _act(G, case["act"]).mul_(U).to(BF16))
    return s


# ---------------------------------------------------------------- plain form

def _signed(v):
    v %= 2**64
    return v - 2**64 if v >= 2**63 else v


def _keep(shape, p, seed, device):
    """The elements that stay: truth values of `shape`."""
    n = math.prod(shape)
    e = torch.arange(n, device=device, dtype=torch.int64)
    z = ((e >> 1) + 1) * _signed(0x9E3779B97F4A7C15) + _signed(seed)
    z = (z ^ ((z >> 30) & (2**34 - 1))) * _signed(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & (2**37 - 1))) * _signed(0x94D049BB133111EB)
    z = z ^ ((z >> 31) & (2**33 - 1))
    bits = (z >> ((e & 1) * 32)) & (2**32 - 1)
    return (bits >= int(p * 2**32)).view(shape)


def _dropped(x, p, seed):
    """dropout(x) in 32 bits."""
    if p == 0.0:
        return x
    return torch.where(_keep(x.shape, p, seed, x.device), x * (1.0 / (1.0 - p)), 0.0)


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    if act == "gelu":
        return 0.5 * g * (1.0 + torch.erf(g * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * g * (1.0 + torch.tanh(SQRT_2_OVER_PI * (g + 0.044715 * g * g * g)))
    return torch.clamp(g, min=0.0)


def _act_slope(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
                + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        t = torch.tanh(SQRT_2_OVER_PI * (g + 0.044715 * g * g * g))
        return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * SQRT_2_OVER_PI * (
            1.0 + 3 * 0.044715 * g * g)
    return (g > 0).to(g.dtype)


def _plain_forward(s, c):
    X = s["X"].float()
    G, U = X @ s["Wg"].float().T, X @ s["Wu"].float().T
    A = _act(G, c["act"]) * U
    Y = _dropped(A @ s["Wd"].float().T, c["p"], s["seed"])
    if s["residual"] is not None:
        Y = Y + s["residual"].float()
    return Y, G, U, A


def _plain_backward(s, c, G, U, A):
    X = s["X"].float()
    dZ = _dropped(s["dY"].float(), c["p"], s["seed"])
    dWd = dZ.T @ A
    dA = dZ @ s["Wd"].float()
    dG, dU = dA * U * _act_slope(G, c["act"]), dA * _act(G, c["act"])
    dX = dG @ s["Wg"].float() + dU @ s["Wu"].float()
    return {"dX": dX.to(BF16), "dWg": (dG.T @ X).to(BF16), "dWu": (dU.T @ X).to(BF16),
            "dWd": dWd.to(BF16)}


def _run_plain(s, c):
    op = c["op"]
    if op == "dropout":
        y = _dropped(s["x"].float(), c["p"], s["seed"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return y.to(s["x"].dtype)
    if op == "dropout_backward":
        return _dropped(s["x"].float(), c["p"], s["seed"]).to(s["x"].dtype)
    if op == "ffn_backward":
        return _plain_backward(s, c, *(t.float() for t in s["saved"]))
    Y, G, U, A = _plain_forward(s, c)
    if op == "ffn_forward":
        return Y.to(BF16)
    if op == "ffn_train_forward":
        return {"Y": Y.to(BF16), "G": G.to(BF16), "U": U.to(BF16), "A": A.to(BF16)}
    return {"Y": Y.to(BF16), **_plain_backward(s, c, G, U, A)}


# ------------------------------------------------------- the framework's calls

_workspaces = {}  # one per problem size, as a training or serving loop holds it


def _run_own(s, c):
    import sampled_softmax_output_gb300 as ss
    op = c["op"]
    if op == "dropout":
        return ss.dropout(s["x"], c["p"], s["seed"], residual=s["residual"])
    if op == "dropout_backward":
        return ss.dropout_backward(s["x"], c["p"], s["seed"])
    size = (c["T"], c["D"], c["F"])
    if size not in _workspaces:
        _workspaces.clear()
        _workspaces[size] = ss.ffn_workspace(*size)
    ws = _workspaces[size]
    weights = (s["Wg"], s["Wu"], s["Wd"])
    opts = {"act": c["act"], "p": c["p"], "seed": s["seed"]}
    if op == "ffn_backward":
        return ss.ffn_backward(s["dY"], s["X"], *weights, s["saved"], ws, dw_dtype=BF16, **opts)
    if op == "ffn_forward":
        return ss.ffn_forward(s["X"], *weights, ws, residual=s["residual"], **opts)
    Y, saved = ss.ffn_forward(s["X"], *weights, ws, residual=s["residual"], save=True, **opts)
    if op == "ffn_train_forward":
        return {"Y": Y, "G": saved[0], "U": saved[1], "A": saved[2]}
    grads = ss.ffn_backward(s["dY"], s["X"], *weights, saved, ws, dw_dtype=BF16, **opts)
    return {"Y": Y, **grads}


def run(state):
    return _run_own(state, state["case"]) if own else _run_plain(state, state["case"])


# --------------------------------------------------------------- in 64 bits

def _factor64(shape, p, seed):
    """1 / (1 - p) where an element stays, else 0, from unsigned integers on the host."""
    if p == 0.0:
        return None
    n = math.prod(shape)
    out = np.empty(n + (n & 1), np.bool_)
    u = np.uint64
    for lo in range(0, (n + 1) // 2, 1 << 22):
        k = np.arange(lo, min(lo + (1 << 22), (n + 1) // 2), dtype=u)
        with np.errstate(over="ignore"):
            z = u(seed) + (k + u(1)) * u(0x9E3779B97F4A7C15)
            z = (z ^ (z >> u(30))) * u(0xBF58476D1CE4E5B9)
            z = (z ^ (z >> u(27))) * u(0x94D049BB133111EB)
            z = z ^ (z >> u(31))
        words = np.stack([z & u(0xFFFFFFFF), z >> u(32)], axis=1).reshape(-1)
        out[2 * lo:2 * lo + words.size] = words >= u(int(p * 2**32))
    stays = torch.from_numpy(out[:n]).cuda().view(shape)
    return stays.to(F64) / (1.0 - p)


def _gate64(g, act):
    """(act(g), act'(g)) in 64 bits."""
    if act == "silu":
        s = torch.special.expit(g)
        return g * s, s + g * s * torch.special.expit(-g)
    if act == "gelu":
        cdf = torch.special.ndtr(g)
        return g * cdf, cdf + g * torch.exp(g.square() / -2) * (2 * math.pi) ** -0.5
    if act == "gelu_tanh":
        # (1 + tanh(v)) / 2 = expit(2 v)
        v2 = 2 * SQRT_2_OVER_PI * (g + 0.044715 * g.pow(3))
        s = torch.special.expit(v2)
        dv2 = 2 * SQRT_2_OVER_PI * (1 + 0.134145 * g.square())
        return g * s, s + g * s * torch.special.expit(-v2) * dv2
    on = torch.heaviside(g, torch.zeros((), dtype=F64, device=g.device))
    return g * on, on


def exact(case, seed):
    s = prepare(case, seed)
    op, r = case["op"], s["residual"] if "residual" in s else None
    if op.startswith("dropout"):
        x = s["x"].to(F64)
        f = _factor64(x.shape, case["p"], s["seed"])
        y = x if f is None else x * f
        return y if r is None else y + r.to(F64)
    X, Wg, Wu, Wd = (s[k].to(F64) for k in ("X", "Wg", "Wu", "Wd"))
    f = _factor64((case["T"], case["D"]), case["p"], s["seed"])
    out = {}
    if op == "ffn_backward":
        G, U, A = (t.to(F64) for t in s["saved"])
    else:
        G, U = torch.einsum("td,fd->tf", X, Wg), torch.einsum("td,fd->tf", X, Wu)
        A = _gate64(G, case["act"])[0] * U
        Y = torch.einsum("tf,df->td", A, Wd)
        Y = Y if f is None else Y * f
        out["Y"] = Y if r is None else Y + r.to(F64)
    if op == "ffn_forward":
        return out["Y"]
    if op == "ffn_train_forward":
        return {**out, "G": G, "U": U, "A": A}
    dZ = s["dY"].to(F64)
    dZ = dZ if f is None else dZ * f
    dA = torch.einsum("td,df->tf", dZ, Wd)
    a, slope = _gate64(G, case["act"])
    dG, dU = dA * U * slope, dA * a
    out["dX"] = torch.einsum("tf,fd->td", dG, Wg) + torch.einsum("tf,fd->td", dU, Wu)
    out["dWg"], out["dWu"] = torch.einsum("tf,td->fd", dG, X), torch.einsum("tf,td->fd", dU, X)
    out["dWd"] = torch.einsum("td,tf->df", dZ, A)
    return out
