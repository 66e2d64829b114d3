"""Cases of the head's token log-probabilities and the losses made of them:
distillation from a teacher's top logits, a clipped policy loss with a KL term,
and losses of preference pairs.

Log-probabilities. H [T, D] hidden states, W [V, D] vocabulary rows, ids [T, K]
(-1: absent), z = H W^T or, with a cap, z = cap / (1 + exp(-H W^T / tau)):
    lse[t] = log sum_j exp(z[t, j])        logp[t, k] = z[t, ids[t, k]] - lse[t]
and with w = d objective / d logp (0 where an id is absent), a[t] = -sum_k w[t, k],
    G[t, j] = (a[t] exp(z[t, j] - lse[t]) + sum_k w[t, k] [ids[t, k] = j]) dz/ds
    dH = G W        dW = G^T H

Policy. r = exp(logp - old), A the advantage, d = ref - logp, m a weight per token:
    kl = exp(d) - d - 1
    loss = m (-min(r A, clip(r, 1 - lo, 1 + hi) A) + beta kl)
Tokens of weight 0 give 0.

Preference. Pair i is the sequences 2i (chosen) and 2i + 1 (rejected) of a packed
batch, R the sum (or the mean) of m (logp - ref) over a sequence, x = R_c - R_r:
    sigmoid: -(1 - e) log s(beta x) - e log s(-beta x)     ipo: (x - 1 / (2 beta))^2
and the reward of a sequence is beta R. Tokens outside every sequence have gradient 0.

Distillation. From the teacher's values at its top ids, either p = softmax over
those K, loss = m sum_k p (log p - logp), or, with a tail, p = exp(value),
    p' = max(1 - sum p, 0)       q' = max(1 - sum_k exp(logp), 2^-12)
    loss = m (sum_k p (log p - logp) + p' (log p' - log q'))
Where 2^-12 holds, the tail's gradient is 0.

Every loss comes with its gradient: dlogp = scale d loss / d logp.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
TAIL_FLOOR = 2.0 ** -12
LOGIT_STD = 3.0  # the next token's entropy is then 6 nats, as early in training


# --------------------------------------------------------------------- cases

def _score(name, T, D, V, K=1, cap=0.0):
    return {"name": name, "op": "score", "T": T, "D": D, "V": V, "K": K, "cap": cap}


def _policy(name, T, D=0, V=0, cap=0.0, kl=0.05):
    """D = 0: the loss alone, its log-probabilities at hand."""
    return {"name": name, "op": "policy", "T": T, "D": D, "V": V, "cap": cap, "kl": kl}


def _preference(name, pairs, T, D=0, V=0, kind="sigmoid", average=False, cap=0.0):
    return {"name": name, "op": "preference", "pairs": pairs, "T": T, "D": D, "V": V,
            "kind": kind, "average": average, "cap": cap}


def _distill(name, T, K, D=0, V=0, tail=False, teacher="f32", cap=0.0):
    return {"name": name, "op": "distill", "T": T, "K": K, "D": D, "V": V, "tail": tail,
            "teacher": teacher, "cap": cap}


def listed():
    return [
        # a served model reports one token's log-probability
        _score("score_token", 1, 768, 50304),
        # a prompt's log-probabilities at 20 alternatives a position, sizes that fill no tile
        _score("score_prompt_ragged", 1003, 1088, 50257, K=20),
        # the policy loss of one short answer: launch latency
        _policy("policy_rows_small", 256),
        # the policy loss of a whole rollout: bound by memory
        _policy("policy_rows_rollout", 1 << 24),
        # a policy step on a short answer: the head's smallest batch
        _policy("policy_step_small", 256, 768, 50304),
        # a policy step at the head's ordinary batch
        _policy("policy_step", 16384, 768, 50304),
        # four short pairs
        _preference("preference_rows_small", 4, 1003),
        # 64 pairs of long answers
        _preference("preference_rows_long", 64, 1 << 21, kind="ipo", average=True),
        # a preference step of a wider model
        _preference("preference_step", 8, 8192, 2048, 50304),
        # distillation rows alone, the teacher's values kept in bf16
        _distill("distill_rows", 65536, 128, tail=True, teacher="bf16"),
        # distillation into the soft-capped head, an odd number of tokens
        _distill("distill_step_capped", 3001, 32, 1024, 24576, cap=30.0),
        # distillation at the head's ordinary batch
        _distill("distill_step", 16384, 64, 768, 50304, tail=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["score", "policy", "policy", "preference", "preference", "distill", "distill"])
    K = _log(rng, 1, 128)
    if op != "score" and rng.random() < 0.4:  # the loss alone
        if op == "policy":
            c = _policy("", _log(rng, 8, 1 << 24), kl=rng.choice([0.0, 0.05, 0.2]))
        elif op == "preference":
            pairs = _log(rng, 1, 512)
            c = _preference("", pairs, _log(rng, 8 * pairs, 1 << 21),
                            kind=rng.choice(["sigmoid", "ipo"]), average=rng.random() < 0.4)
        else:
            c = _distill("", _log(rng, 8, 65536), K, tail=rng.random() < 0.5,
                         teacher=rng.choice(["f32", "bf16"]))
    else:
        D = 64 * _log(rng, 1, 32)
        V = _log(rng, 300, 131072)
        T = max(8, min(_log(rng, 8, 16384), int(8192 * 50304 * 2048 / (V * D)),
                       16384 * 50304 // V))
        cap = rng.choice([0.0, 0.0, 30.0])
        if op == "score":
            c = _score("", T, D, V, K, cap)
        elif op == "policy":
            c = _policy("", T, D, V, cap, rng.choice([0.0, 0.05]))
        elif op == "preference":
            c = _preference("", _log(rng, 1, max(1, min(64, T // 2))), T, D, V,
                            rng.choice(["sigmoid", "ipo"]), rng.random() < 0.4, cap)
        else:
            c = _distill("", T, K, D, V, rng.random() < 0.5, rng.choice(["f32", "bf16"]), cap)
    c.pop("name")
    return c


def work(case):
    T, D, V, op, K = case["T"], case["D"], case["V"], case["op"], case.get("K", 1)
    if op == "score":
        return {"bytes": 2 * (T + V) * D + 8 * T * K + 4 * T, "flops": 2.0 * T * V * D}
    # what the loss reads and writes beside the log-probabilities
    if op == "policy":       # old, A, m (, ref) -> loss (, kl)
        rows, flops = T * (4 * 4 + (8 if case["kl"] else 0)), 20.0 * T
    elif op == "preference":  # ref, m, offsets -> loss, rewards
        rows, flops = T * 8 + 20 * case["pairs"], 6.0 * T
    else:                     # values, ids, m -> loss
        rows = T * (K * ((4 if case["teacher"] == "f32" else 2) + 4) + 8)
        flops = 20.0 * T * K
    if not D:
        return {"bytes": rows + 8 * T * K, "flops": flops}
    ids = 0 if op == "distill" else 4 * T * K
    return {"bytes": rows + ids + 4 * (T + V) * D + 4 * T * K, "flops": flops + 6.0 * T * V * D}


# -------------------------------------------------------------------- inputs

TAU = 7.5
CLIP = (0.2, 0.28)
BETA, SMOOTHING = 0.1, 0.05


def _logit_chunks(H, W, cap):
    """(first row, logits) of 2048 rows at a time, in 32 bits."""
    Wt = W.float().T
    for t0 in range(0, H.shape[0], 2048):
        z = H[t0:t0 + 2048].float() @ Wt
        yield t0, (cap * torch.sigmoid(z / TAU) if cap else z)


def _sampled(H, W, cap, gen):
    """Tokens drawn from the head's own distribution, as a rollout has them, and their
    log-probabilities."""
    ids, logp = [], []
    for _, z in _logit_chunks(H, W, cap):
        gumbel = torch.empty_like(z).exponential_(generator=gen).clamp_(min=1e-30).log_()
        at = (z - gumbel).argmax(1, keepdim=True)
        ids.append(at)
        logp.append(z.gather(1, at) - torch.logsumexp(z, 1, keepdim=True))
    return torch.cat(ids).view(-1).int(), torch.cat(logp).view(-1)


def _teacher_top(H, W, cap, K, gen):
    """A teacher near the student: its K largest log-probabilities and their ids."""
    ids, values = [], []
    for _, z in _logit_chunks(H, W, cap):
        z = z.add_(torch.randn(z.shape, generator=gen, device="cuda"), alpha=0.7)
        top = z.topk(min(K, z.shape[1]), 1)
        ids.append(top.indices)
        values.append(top.values - torch.logsumexp(z, 1, keepdim=True))
    return torch.cat(ids).int(), torch.cat(values)


def _offsets(pairs, T, rng):
    """2 pairs sequences of uneven lengths, and a padded end in longer batches."""
    end = T - T // 64
    cuts = torch.randint(0, end + 1, (2 * pairs - 1,), generator=rng, device="cuda").sort().values
    edge = torch.tensor([0, end], device="cuda")
    return torch.cat([edge[:1], cuts, edge[1:]]).int()


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, D, V, op, cap = case["T"], case["D"], case["V"], case["op"], case.get("cap", 0.0)
    K = min(case.get("K", 1), V) if V else case.get("K", 1)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(scale)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = {"case": case}
    if D:
        s["H"] = normal(T, D).to(BF16)  # a normalised hidden state
        s["W"] = normal(V, D, scale=LOGIT_STD * D ** -0.5).to(BF16)
    if op == "score":
        s["ids"] = torch.randint(0, V, (T, K), generator=gen, device="cuda").int()
        return s
    # the prompt's tokens have weight 0; a mean over the others
    weight = (uniform(T) >= 0.25).float()
    s["weight"] = weight / weight.sum().clamp(min=1.0) if op != "preference" else weight
    if op == "distill":
        if D:
            ids, values = _teacher_top(s["H"], s["W"], cap, K, gen)
        else:
            ids = torch.argsort(uniform(1, 4 * K)).int()[:, :K].repeat(T, 1)
            # the ids beyond the list hold as much as e^4 of it
            tail = torch.tensor([0.0] * K + [4.0], device="cuda")
            values, s["logp"] = (
                torch.log_softmax(normal(T, K + 1, scale=2.0) + tail, 1)[:, :K].contiguous()
                for _ in range(2))
        # some rows of the teacher's list are shorter
        short = (uniform(T, 1) < 0.06) & (torch.arange(K, device="cuda") >= (K + 1) // 2)
        s["ids"] = torch.where(short, -1, ids).contiguous()
        s["teacher"] = torch.where(short, 0.0, values).to(F32 if case["teacher"] == "f32" else BF16)
        if not D:
            s["logp"] = torch.where(short, 0.0, s["logp"])
        return s
    if D:
        s["ids"], logp = _sampled(s["H"], s["W"], cap, gen)
    else:
        logp = normal(T).exp_().neg_()
        s["logp"] = logp
    if op == "policy":
        s["advantage"] = normal(T)
        step = normal(T, scale=0.2)
        for edge in (math.log(1 - CLIP[0]), math.log(1 + CLIP[1])):
            # which side of the clip's edge a value on it falls on is rounding's choice
            step = torch.where((step - edge).abs() < 1e-4, 0.0, step)
        s["old"] = logp - step
        s["ref"] = logp + normal(T, scale=0.5) if case["kl"] else None
    else:
        s["ref"] = logp + normal(T)
        s["offsets"] = _offsets(case["pairs"], T, gen)
    return s


# ---------------------------------------------------------------- plain form

def _plain_logits(s, cap):
    z = s["H"].float() @ s["W"].float().T
    return torch.sigmoid_(z.div_(TAU)).mul_(cap) if cap else z


def _plain_logprobs(z, ids):
    top = z.amax(1, keepdim=True)
    lse = torch.exp(z - top).sum(1, keepdim=True).log_().add_(top)
    here = ids >= 0
    logp = torch.where(here, z.gather(1, ids.clamp(min=0).long()) - lse, 0.0)
    return logp, lse


def _plain_grads(s, z, lse, ids, dlogp, cap):
    w = torch.where(ids >= 0, dlogp, 0.0)
    G = torch.exp(z - lse).mul_(-w.sum(1, keepdim=True))
    G.scatter_add_(1, ids.clamp(min=0).long(), w)
    if cap:
        G.mul_(z.mul(cap - z).div_(cap * TAU))
    return {"dH": (G @ s["W"].float()).to(BF16), "dW": (G.T @ s["H"].float()).to(BF16)}


def _plain_policy(s, c, logp):
    lo, hi = CLIP
    m, A = s["weight"], s["advantage"]
    r = torch.exp(logp - s["old"])
    held = torch.clamp(r, 1 - lo, 1 + hi)
    free = r * A <= held * A
    loss = torch.where(free, -r * A, -held * A)
    slope = torch.where(free, -r * A, 0.0)
    out = {}
    if c["kl"]:
        d = s["ref"] - logp
        out["kl"] = torch.where(m != 0, torch.expm1(d) - d, 0.0)
        loss = loss + c["kl"] * out["kl"]
        slope = slope - c["kl"] * torch.expm1(d)
    return {**out, "loss": torch.where(m != 0, m * loss, 0.0),
            "dlogp": torch.where(m != 0, m * slope, 0.0)}


def _sequence_of(offsets, T):
    """The sequence of each token, -1 outside every one."""
    seq = torch.searchsorted(offsets.long(), torch.arange(T, device="cuda"), right=True) - 1
    return torch.where(seq < offsets.numel() - 1, seq, -1)


def _plain_preference(s, c, logp):
    T, n = logp.numel(), 2 * c["pairs"]
    seq = _sequence_of(s["offsets"], T)
    inside, at = seq >= 0, seq.clamp(min=0)
    m = torch.where(inside, s["weight"], 0.0)
    # long sums: in 64 bits
    R = torch.zeros(n, dtype=F64, device="cuda").index_add_(0, at, (m * (logp - s["ref"])).double())
    if c["average"]:
        size = torch.zeros(n, dtype=F64, device="cuda").index_add_(0, at, m.double())
        share = torch.where(size > 0, 1.0 / size, 0.0)
        R = R * share
    x = R[0::2] - R[1::2]
    if c["kind"] == "sigmoid":
        h, e = BETA * x, SMOOTHING
        loss = (1 - e) * torch.log1p(torch.exp(-h)) + e * torch.log1p(torch.exp(h))
        slope = BETA * (e - 1.0 / (1.0 + torch.exp(h)))
    else:
        loss = (x - 1 / (2 * BETA)) ** 2
        slope = 2 * (x - 1 / (2 * BETA))
    slope = torch.stack([slope, -slope], 1).view(-1) / c["pairs"]
    if c["average"]:
        slope = slope * share
    return {"loss": loss.float(), "reward": (BETA * R).float().view(-1, 2),
            "dlogp": torch.where(inside, m * slope[at].float(), 0.0)}


def _plain_distill(s, c, logp, ids):
    here = ids >= 0
    m = s["weight"].unsqueeze(1)
    x = s["teacher"].float()
    if not c["tail"]:
        e = torch.where(here, torch.exp(x - torch.where(here, x, -1e30).amax(1, keepdim=True)), 0.0)
        total = e.sum(1, keepdim=True)
        p = torch.where(total > 0, e / total, 0.0)
        loss = torch.where(p > 0, p * (torch.log(p) - logp), 0.0).sum(1, keepdim=True)
        slope = -p
    else:
        # what is left of 1: in 64 bits
        p = torch.where(here, torch.exp(x.double()), 0.0)
        q = torch.where(here, torch.exp(logp.double()), 0.0)
        p1 = torch.clamp(1.0 - p.sum(1, keepdim=True), min=0.0).float()
        q1 = (1.0 - q.sum(1, keepdim=True)).float()
        p, q = p.float(), q.float()
        floor = q1 <= TAIL_FLOOR
        q1 = torch.where(floor, TAIL_FLOOR, q1)
        loss = torch.where(p > 0, p * (x - logp), 0.0).sum(1, keepdim=True)
        loss = loss + torch.where(p1 > 0, p1 * (torch.log(p1) - torch.log(q1)), 0.0)
        slope = torch.where(floor, 0.0, p1 / q1) * q - p
    some = (m != 0) & here.any(1, keepdim=True)
    return {"loss": torch.where(some, m * loss, 0.0).view(-1),
            "dlogp": torch.where(some, m * slope, 0.0)}


_PLAIN = {"policy": _plain_policy, "preference": _plain_preference}


def _run_plain(s, c):
    op = c["op"]
    if not c["D"]:
        return _plain_distill(s, c, s["logp"], s["ids"]) if op == "distill" else \
            _PLAIN[op](s, c, s["logp"])
    ids = s["ids"] if s["ids"].dim() == 2 else s["ids"].unsqueeze(1)
    z = _plain_logits(s, c["cap"])
    logp, lse = _plain_logprobs(z, ids)
    if op == "score":
        return {"logp": logp, "lse": lse.view(-1)}
    out = _plain_distill(s, c, logp, ids) if op == "distill" else _PLAIN[op](s, c, logp.view(-1))
    dlogp = out.pop("dlogp").view(logp.shape)
    return {**out, "logp": logp.view(s["ids"].shape),
            **_plain_grads(s, z, lse, ids, dlogp, c["cap"])}


# ------------------------------------------------------- the framework's calls

_workspaces = {}  # one per problem size, as a training or serving loop holds it


def _workspace(*size):
    import sampled_softmax_output_gb300 as ss
    if size not in _workspaces:
        _workspaces.clear()
        _workspaces[size] = ss.logprob_workspace(*size)
    return _workspaces[size]


def _own_loss(ss, s, c, logp, ws):
    if c["op"] == "policy":
        return ss.policy_loss(logp, s["old"], s["advantage"], ref_logp=s["ref"],
                              weight=s["weight"], clip=CLIP, kl=c["kl"])
    if c["op"] == "preference":
        return ss.preference_loss(logp, s["offsets"], ws, ref_logp=s["ref"], weight=s["weight"],
                                  beta=BETA, kind=c["kind"],
                                  smoothing=SMOOTHING if c["kind"] == "sigmoid" else 0.0,
                                  average=c["average"], scale=1.0 / c["pairs"])
    return ss.distill_loss(logp, s["teacher"], ids=s["ids"], weight=s["weight"], tail=c["tail"])


def _run_own(s, c):
    import sampled_softmax_output_gb300 as ss
    if not c["D"]:
        # a preference loss records errors in a workspace of any size
        return _own_loss(ss, s, c, s["logp"], _workspace(0, 1, 64))
    ws = _workspace(c["T"], c["V"], c["D"])
    head = {"cap": c["cap"], "tau": TAU} if c["cap"] else {}
    if c["op"] == "score":
        logp, lse = ss.logprobs(s["H"], s["W"], s["ids"], ws, **head)
        return {"logp": logp, "lse": lse}
    logp, lse = ss.logprobs(s["H"], s["W"], s["ids"], ws, **head)
    out = _own_loss(ss, s, c, logp, ws)
    dH, dW = ss.logprobs_backward(out.pop("dlogp"), s["H"], s["W"], s["ids"], logp, lse, ws,
                                  dw_dtype=BF16, **head)
    return {**out, "logp": logp, "dH": dH, "dW": dW}


def run(state):
    return _run_own(state, state["case"]) if own else _run_plain(state, state["case"])


# --------------------------------------------------------------- in 64 bits

def _loss64(s, c, logp, ids):
    """The loss and d loss / d logp (of the scaled sum) in 64 bits, one row of logp a token."""
    m = s["weight"].to(F64)
    used = m != 0
    if c["op"] == "policy":
        x, A = logp.view(-1), s["advantage"].to(F64)
        ratio = torch.exp(x - s["old"].to(F64))
        out_hi = (A > 0) & (ratio > 1 + CLIP[1])
        out_lo = (A < 0) & (ratio < 1 - CLIP[0])
        gain = torch.where(out_hi, (1 + CLIP[1]) * A, torch.where(out_lo, (1 - CLIP[0]) * A,
                                                                ratio * A))
        slope = torch.where(out_hi | out_lo, 0.0, -ratio * A)
        loss, more = -gain, {}
        if c["kl"]:
            d = s["ref"].to(F64) - x
            kl = torch.exp(d) - d - 1
            more["kl"] = torch.where(used, kl, 0.0)
            loss, slope = loss + c["kl"] * kl, slope + c["kl"] * (1 - torch.exp(d))
        zero = torch.zeros((), dtype=F64, device="cuda")
        return {**more, "loss": torch.where(used, m * loss, zero),
                "dlogp": torch.where(used, m * slope, zero)}
    if c["op"] == "preference":
        x = logp.view(-1)
        gap = m * (x - s["ref"].to(F64))
        edges = s["offsets"].tolist()
        cum = torch.cat([gap.new_zeros(1), gap.cumsum(0)])
        mass = torch.cat([m.new_zeros(1), m.cumsum(0)])
        at = s["offsets"].long()
        R, size = cum[at[1:]] - cum[at[:-1]], mass[at[1:]] - mass[at[:-1]]
        per = torch.ones_like(R)
        if c["average"]:
            per = torch.where(size > 0.5, 1 / size.clamp(min=0.5), 0.0)
        R = R * per
        margin = R.view(-1, 2) @ torch.tensor([1.0, -1.0], dtype=F64, device="cuda")
        if c["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            loss = -(1 - SMOOTHING) * ls(BETA * margin) - SMOOTHING * ls(-BETA * margin)
            slope = BETA * (SMOOTHING - torch.special.expit(-BETA * margin))
        else:
            loss = (margin - 0.5 / BETA).square()
            slope = 2 * margin - 1 / BETA
        slope = torch.stack([slope, -slope], 1).view(-1) * per / c["pairs"]
        spread = torch.repeat_interleave(slope, at[1:] - at[:-1])
        dlogp = torch.zeros_like(x)
        dlogp[edges[0]:edges[-1]] = spread
        return {"loss": loss, "reward": BETA * R.view(-1, 2), "dlogp": dlogp * m}
    x, here = s["teacher"].to(F64), ids >= 0
    x = torch.where(here, x, -math.inf)
    q = torch.where(here, logp.exp(), 0.0)
    if c["tail"]:
        logt = x
        p = torch.exp(logt)
        p1 = (1 - p.sum(1)).clamp(min=0.0)
        q1 = (1 - q.sum(1)).clamp(min=TAIL_FLOOR)
        ratio = torch.where(q1 > TAIL_FLOOR, p1 / q1, 0.0)
        loss = torch.special.xlogy(p1, p1) - p1 * q1.log()
    else:
        logt = torch.log_softmax(torch.where(here.any(1, keepdim=True), x, 0.0), 1)
        p = torch.where(here, logt.exp(), 0.0)
        ratio = torch.zeros_like(m)
        loss = torch.zeros_like(m)
    loss = loss + torch.where(p > 0, p * (torch.where(here, logt, 0.0) - logp), 0.0).sum(1)
    used = used & here.any(1)
    return {"loss": torch.where(used, m * loss, 0.0),
            "dlogp": torch.where(used.unsqueeze(1), m.unsqueeze(1) * (ratio.unsqueeze(1) * q - p),
                                 0.0)}


def exact(case, seed):
    s = prepare(case, seed)
    c, op, cap = case, case["op"], case.get("cap", 0.0)
    if not c["D"]:
        return _loss64(s, c, s["logp"].to(F64), s.get("ids"))
    H, W = s["H"].to(F64), s["W"].to(F64)
    T, step = H.shape[0], 2048
    ids = s["ids"].long().view(T, -1)

    def head(t0):
        raw = torch.einsum("td,vd->tv", H[t0:t0 + step], W)
        if not cap:
            return raw, None
        share = torch.special.expit(raw / TAU)
        return cap * share, cap / TAU * share * torch.special.expit(-raw / TAU)

    logp, lse = [], []
    for t0 in range(0, T, step):
        z, at = head(t0)[0], ids[t0:t0 + step]
        lse.append(torch.logsumexp(z, 1))
        picked = torch.gather(z, 1, at.clamp(min=0)) - lse[-1].unsqueeze(1)
        logp.append(picked.masked_fill(at < 0, 0.0))
    logp, lse = torch.cat(logp), torch.cat(lse)
    if op == "score":
        return {"logp": logp, "lse": lse}
    out = _loss64(s, c, logp, ids)
    w = out.pop("dlogp").view(T, -1).masked_fill(ids < 0, 0.0)
    dH, dW = torch.empty_like(H), torch.zeros_like(W)
    for t0 in range(0, T, step):
        rows = slice(t0, min(t0 + step, T))
        z, slope = head(t0)
        P = torch.softmax(z, 1)
        G = torch.zeros_like(P).scatter_add_(1, ids[rows].clamp(min=0), w[rows])
        G -= P * w[rows].sum(1, keepdim=True)
        if slope is not None:
            G *= slope
        dH[rows] = torch.einsum("tv,vd->td", G, W)
        dW += torch.einsum("tv,td->vd", G, H[rows])
    return {**out, "logp": logp.view(s["ids"].shape), "dH": dH, "dW": dW}
