"""The losses of log-probabilities where a term has no weight or a value is no number,
infinite or near its limit."""
import math

import pytest
import torch

import sampled_softmax_output_gb300 as ss

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
