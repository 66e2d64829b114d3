"""The losses of log-probabilities where a term has no weight or a value is no number,
infinite or near its limit."""
import math

import pytest
import torch

import sampled_softmax_output_gb300 as ss
from logprob_util import F32, F64, assert_within, preference64

pytestmark = pytest.mark.gpu
I32 = torch.int32
NAN, INF = float("nan"), float("inf")


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _policy_inputs(n, seed=0):
    g = _gen(seed)
    logp = -torch.randn(n, generator=g, device="cuda").exp()
    old = logp - 0.1 * torch.randn(n, generator=g, device="cuda")
    return logp, old, torch.randn(n, generator=g, device="cuda")


# ------------------------------------------------------------ distillation

@pytest.mark.parametrize("K", [1, 2, 7, 33, 128])
@pytest.mark.parametrize("rest", ["nothing", "-infinity", "absent"])
def test_distill_row_without_any_number(K, rest):
    """The teacher's values that count are NaN and nothing else, or -infinity beside it:
    a NaN, not a loss of 0; of that row alone."""
    g = _gen(K)
    s, t = (torch.log_softmax(torch.randn(9, K + 1, generator=g, device="cuda"), 1)[:, :K]
            .contiguous() for _ in range(2))
    ids = torch.arange(K, device="cuda", dtype=I32).repeat(9, 1)
    want = ss.distill_loss(s, t, ids)
    t[4] = NAN
    if rest == "-infinity":
        t[4, 1:] = -INF
    elif rest == "absent":
        ids[4, 1:] = -1
    got = ss.distill_loss(s, t, ids)
    assert got["loss"][4].isnan()
    here = ids[4] >= 0
    assert got["dlogp"][4][here].isnan().all() and (got["dlogp"][4][~here] == 0).all()
    others = torch.arange(9, device="cuda") != 4
    for k in ("loss", "dlogp"):
        assert torch.equal(got[k][others], want[k][others])


# ------------------------------------------------------------------ policy

def test_policy_kl_of_an_impossible_token():
    """A token that the policy gives no probability at all and the reference some: its KL
    is infinite, not a NaN."""
    logp = torch.tensor([-INF, -1.0, -INF], device="cuda")
    ref = torch.tensor([-2.0, -2.0, 1e30], device="cuda")
    A = torch.zeros(3, device="cuda")
    out = ss.policy_loss(logp, torch.full_like(logp, -1.0), A, ref_logp=ref, kl=0.1)
    assert out["kl"][0] == INF and out["kl"][2] == INF and out["kl"][1].isfinite()
    assert out["loss"][0] == INF and out["dlogp"][0] == -INF


@pytest.mark.parametrize("ref", [-INF, INF, NAN, 100.0, -5000.0])
def test_policy_reference_of_no_weight(ref):
    """kl = 0 with a reference: its KL is written, and touches neither loss nor gradient,
    whatever it is."""
    logp, old, A = _policy_inputs(103)
    plain = ss.policy_loss(logp, old, A)
    far = logp + ref
    out = ss.policy_loss(logp, old, A, ref_logp=far, kl=0.0)
    assert torch.equal(out["loss"], plain["loss"])
    assert torch.equal(out["dlogp"], plain["dlogp"])
    if not math.isnan(ref):
        assert (out["kl"] > 90).all()


def test_policy_kl_of_a_near_reference():
    """exp(d) - d - 1 is d^2 / 2 near 0: all its digits are there, and it is never negative.
    The difference d of the two is exact here; 12 half steps of the KL: below |d| = 1/2
    some 8 roundings of its series, above 1 step of expm1 (2 |expm1(d)| / kl <= 8.8 half
    steps) and the subtraction's."""
    g = _gen(5)
    n = 20001
    size = torch.logspace(-7, 1, n, device="cuda")
    sign = (torch.rand(n, generator=g, device="cuda") < 0.5).float() * 2 - 1
    logp = torch.full((n,), -1.0, device="cuda")
    # (both on one grid of 2^-23, so that their difference is exact up to 2)
    d = torch.where(size < 2, torch.round(sign * size * 2.0 ** 23) * 2.0 ** -23, 0.0)
    ref = torch.where(size < 2, logp + d, logp + torch.round(sign * size))
    old, A = logp.clone(), torch.zeros(n, device="cuda")
    out = ss.policy_loss(logp, old, A, ref_logp=ref, kl=0.5)
    x = ref.to(F64) - logp.to(F64)
    # (64 bits lose 2e-16 / |d| of it themselves: 2e-9 at 1e-7)
    want = torch.expm1(x) - x
    assert (out["kl"] >= 0).all() and (out["kl"][x != 0] > 0).all()
    assert_within(out["kl"], (want, 12 * F32 * want), "kl")
    assert_within(out["loss"], (0.5 * want, 13 * F32 * 0.5 * want), "loss")
    same = ss.policy_loss(logp, old, A, ref_logp=logp, kl=0.5)
    assert (same["kl"] == 0).all() and (same["dlogp"] == 0).all()


# -------------------------------------------------------------- preference

@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
def test_preference_gradient_of_no_number(kind):
    """A NaN that counts is in its pair's loss and gradient, and in no other's."""
    logp = -torch.rand(40, generator=_gen(6), device="cuda")
    at = torch.tensor([0, 9, 20, 27, 40], dtype=I32, device="cuda")
    ws = ss.logprob_workspace(0, 1, 64)
    want = ss.preference_loss(logp, at, ws, kind=kind)
    logp[13] = NAN
    got = ss.preference_loss(logp, at, ws, kind=kind)
    assert got["loss"][0].isnan() and got["dlogp"][:20].isnan().all()
    assert torch.equal(got["loss"][1], want["loss"][1])
    assert torch.equal(got["dlogp"][20:], want["dlogp"][20:])


def _preference_call(logp, at, dlogp, ws):
    """The C entry, so that dlogp may be any buffer."""
    pairs = at.numel() // 2
    loss, reward = torch.zeros(pairs, device="cuda"), torch.zeros(pairs, 2, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    status = ss.lib().ss_preference_loss(
        logp.data_ptr(), None, None, at.data_ptr(), pairs, logp.numel(), 0, 0.1, 0.0, 0, 1.0,
        loss.data_ptr(), reward.data_ptr(), dlogp.data_ptr(), ws.data_ptr(), ws.numel(), s)
    assert status == 0
    torch.cuda.synchronize()
    return loss, reward


# offsets in, the pairs that are bad and those that are good
BAD = {"before all": ([40000, 4, 900, 20000, 39000], [0], [1]),
       "above": ([0, 40001, 900, 20000, 39000], [0], [1]),
       "negative": ([-5, 900, 1000, 20000, 39000], [0], [1]),
       "falling": ([900, 1000, 800, 20000, 39000], [0], [1]),
       "last below": ([0, 900, 30000, 39000, 3], [1], [0]),
       "last negative": ([0, 900, 30000, 39000, -3], [1], [0]),
       "last above": ([0, 900, 30000, 39000, 2 ** 31 - 1], [1], [0]),
       "between": ([0, 900, 9000, 8000, 9500, 20000, 39000], [1], [0, 2])}


@pytest.mark.parametrize("offsets,bad,good", BAD.values(), ids=BAD.keys())
@pytest.mark.parametrize("in_place", [False, True])
def test_preference_other_pairs_beside_a_bad_one(offsets, bad, good, in_place):
    """The good pairs' losses, rewards and gradients are there, with the gradient in the
    place of the log-probabilities too, and nothing is written around it."""
    n, guard = 40000, 64
    logp = -torch.rand(n, generator=_gen(7), device="cuda")
    at = torch.tensor(offsets, dtype=I32, device="cuda")
    own = logp.clone()
    for _ in range(10):
        buffer = torch.full((n + 2 * guard,), 7.0, device="cuda")
        dlogp = buffer[guard:guard + n]
        dlogp.copy_(logp)
        ws = ss.logprob_workspace(0, 1, 64)
        loss, reward = _preference_call(dlogp if in_place else logp, at, dlogp, ws)
        assert ss.read_status(ws)[0] == 8
        assert (buffer[:guard] == 7).all() and (buffer[guard + n:] == 7).all()
        assert torch.equal(logp, own)
        for i in bad:
            assert loss[i].isnan() and reward[i].isnan().all()
        for i in good:
            part = at[2 * i:2 * i + 3]
            want = preference64(logp, part, beta=torch.tensor(0.1).item())
            assert_within(loss[i:i + 1], want["loss"], "loss")
            assert_within(reward[i:i + 1], want["reward"], "reward")
            a, b = offsets[2 * i], offsets[2 * i + 2]
            assert_within(dlogp[a:b], tuple(t[a:b] for t in want["dlogp"]), "dlogp")
