"""The head's log-probabilities where logits are infinite, on one token, two and more:
the kernels for few tokens and for many give what the formulas give."""
import pytest
import torch

import sampled_softmax_output_gb300 as ss
from logprob_util import assert_within, logprobs64

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
INF = float("inf")
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
    kept = torch.tensor([j for j in range(V) if j not in rows], device="cuda")
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
