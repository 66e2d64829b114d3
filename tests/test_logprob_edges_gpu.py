"""The head's log-probabilities where logits are infinite, on one token, two and more:
the kernels for few tokens and for many give what the formulas give."""
import pytest
import torch

import sampled_softmax_output_gb300 as ss
from logprob_util import F32, F64, assert_within, logprobs64

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
NAN, INF = float("nan"), float("inf")
AT = 5  # the column of H and W that holds the infinities


def _inputs(T, V, D=128, K=6, seed=0):
    """H positive in column AT, so that a row of W has a logit of its entry's sign there."""
    g = torch.Generator("cuda").manual_seed(seed)
    H = torch.randn(T, D, generator=g, device="cuda")
    H[:, AT] = H[:, AT].abs() + 0.5
    W = (torch.randn(V, D, generator=g, device="cuda") * 3.0 * D ** -0.5).to(BF16)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").to(I32)
    return H.to(BF16), W, ids


def _without(V, rows):
    """The other rows of the vocabulary, and the place of each among them."""
    kept = torch.tensor([j for j in range(V) if j not in rows], dtype=torch.long, device="cuda")
    place = torch.full((V,), -1, dtype=I32, device="cuda")
    place[kept] = torch.arange(len(kept), dtype=I32, device="cuda")
    return kept, place


ROWS = {"first": [0], "second": [1], "middle": [152], "last": [299],
        "each warp's first": list(range(0, 300, 4)), "a warp's": [8, 9, 10, 11],
        "a tile's half": list(range(128, 256)), "all but one": [j for j in range(300) if j != 77]}


@pytest.mark.parametrize("T", [1, 2, 3, 130])
@pytest.mark.parametrize("rows", ROWS.values(), ids=ROWS.keys())
def test_logits_of_minus_infinity(T, rows):
    """They add nothing to the sum, wherever they stand in the vocabulary."""
    H, W, ids = _inputs(T, 300)
    W[rows, AT] = -INF
    ids[:, 0] = rows[0]
    kept, place = _without(300, rows)
    logp, lse = ss.logprobs(H, W, ids, ss.logprob_workspace(T, 300, 128))
    ref = logprobs64(H, W[kept], place[ids.long()])
    assert_within(lse, ref["lse"], "lse")
    gone = place[ids.long()] < 0
    assert (logp[gone] == -INF).all()
    assert_within(logp.masked_fill(gone, 0.0), ref["logp"], "logp")


@pytest.mark.parametrize("T", [1, 2, 3, 130])
@pytest.mark.parametrize("rows", [[0], [152], [299], [0, 299], [150, 151], list(range(300))],
                         ids=lambda r: f"{len(r)} from {r[0]}")
def test_logits_of_plus_infinity(T, rows):
    """Such a token's sum is infinite: log-probabilities of -infinity, and no number for
    the ids that are infinite themselves. A token whose logit there is -infinity is as
    without those rows."""
    H, W, ids = _inputs(T, 300, seed=1)
    W[rows, AT] = INF
    ids[:, 0] = rows[0]
    other = torch.arange(T, device="cuda") % 3 == 1
    H[other] = -H[other]
    logp, lse = ss.logprobs(H, W, ids, ss.logprob_workspace(T, 300, 128))
    kept, place = _without(300, rows)
    infinite = place[ids.long()] < 0
    assert (lse[~other] == INF).all()
    assert logp[~other][infinite[~other]].isnan().all()
    assert (logp[~other][~infinite[~other]] == -INF).all()
    if len(kept) and other.any():
        ref = logprobs64(H[other], W[kept], place[ids.long()][other])
        assert_within(lse[other], ref["lse"], "lse")
        assert_within(logp[other].masked_fill(infinite[other], 0.0), ref["logp"], "logp")


@pytest.mark.parametrize("T", [1, 2, 3, 130])
def test_a_row_with_an_infinity(T):
    """H's infinity makes every logit infinite, of the sign of W's entry; a NaN beside it
    makes them all NaN. The other tokens are as without it."""
    H, W, ids = _inputs(T, 300, seed=2)
    ws = ss.logprob_workspace(T, 300, 128)
    clean = ss.logprobs(H, W, ids, ws)
    H[T - 1, AT] = INF
    logp, lse = ss.logprobs(H, W, ids, ws)
    assert (W[:, AT] > 0).any() and (W[:, AT] != 0).all()
    assert lse[T - 1] == INF
    up = W[ids[T - 1].long(), AT] > 0
    assert logp[T - 1][up].isnan().all() and (logp[T - 1][~up] == -INF).all()
    assert torch.equal(logp[:T - 1], clean[0][:T - 1])
    assert torch.equal(lse[:T - 1], clean[1][:T - 1])
    H[T - 1, AT + 1] = NAN
    logp, lse = ss.logprobs(H, W, ids, ws)
    assert lse[T - 1].isnan() and logp[T - 1].isnan().all()


@pytest.mark.parametrize("T", [1, 2, 3, 130])
@pytest.mark.parametrize("cap", [30.0, 200.0])
def test_a_row_with_an_infinity_under_a_cap(T, cap):
    """Its logits are the cap or 0: the log-sum-exp of n of one and the rest of the other."""
    H, W, ids = _inputs(T, 300, seed=3)
    H[T - 1, AT] = INF
    logp, lse = ss.logprobs(H, W, ids, ss.logprob_workspace(T, 300, 128), cap=cap, tau=7.5)
    z = torch.where(W[:, AT].to(F64) > 0, cap, 0.0)
    want = torch.logsumexp(z, 0)
    # the reciprocal that makes z is 2^-18 off at most; the sum as logprobs64 counts it
    tol = 2.0 ** -18 * cap + (4 * cap + 64 + 8 + 2 * cap) * 2 * F32 + 2.0 ** -21
    assert abs(float(lse[T - 1]) - float(want)) <= tol
    assert ((logp[T - 1].to(F64) - (z[ids[T - 1].long()] - want)).abs()
            <= 2 * tol + 2 * F32 * cap).all()


@pytest.mark.parametrize("T", [1, 2, 3, 130])
@pytest.mark.parametrize("log_size", [20, 27, 32, 33, 34, 90, 120])
def test_large_finite_logits(T, log_size):
    """However large the logits are, a finite sum of them is a finite number: the largest
    logit, to fp32's digits of it."""
    H, W, ids = _inputs(T, 300, seed=4)
    W = (W.float() * 2.0 ** log_size).to(BF16)
    logp, lse = ss.logprobs(H, W, ids, ss.logprob_workspace(T, 300, 128))
    ref = logprobs64(H, W, ids)
    assert_within(lse, ref["lse"], "lse")
    assert_within(logp, ref["logp"], "logp")
