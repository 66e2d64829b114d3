"""The losses of include/ss_logprob.h on the GPU against 64 bits, every element within
the bound that logprob_util counts, and their chain with the head."""
import math

import pytest
import torch

import sampled_softmax_output_gb300 as ss
from logprob_util import EXP, F32, F64, assert_within, distill64, policy64, preference64

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
NAN, INF = float("nan"), float("inf")
LENGTHS = [1, 2, 3, 4, 5, 127, 256, 1021, 4096, 100003]


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _check(got, ref):
    assert set(got) == set(ref)
    for k, v in ref.items():
        assert_within(got[k], v, k)


# ------------------------------------------------------------------ policy

def _policy_inputs(n, seed=0, clip=(0.2, 0.2)):
    g = _gen(seed)
    logp = -_randn(g, n).exp()
    step = 0.3 * _randn(g, n)
    for edge in (math.log1p(-clip[0]), math.log1p(clip[1])):
        step = torch.where((step - edge).abs() < 1e-4, 0.0, step)
    m = (torch.rand(n, generator=g, device="cuda") > 0.3).float() * (0.5 + torch.rand(
        n, generator=g, device="cuda"))
    return {"logp": logp, "old": logp - step, "A": _randn(g, n), "ref": logp + 0.5 * _randn(g, n),
            "m": m}


def _policy(x, ref=True, weight=True, clip=(0.2, 0.2), kl=0.1, scale=1.0):
    r = x["ref"] if ref else None
    m = x["m"] if weight else None
    kl = kl if ref else 0.0
    got = ss.policy_loss(x["logp"], x["old"], x["A"], ref_logp=r, weight=m, clip=clip, kl=kl,
                         scale=scale)
    shape = x["logp"].shape
    assert all(t.shape == shape for t in got.values())
    flat = {k: v.reshape(-1) for k, v in x.items()}
    _check({k: v.view(-1) for k, v in got.items()},
           policy64(flat["logp"], flat["old"], flat["A"], flat["ref"] if ref else None,
                    flat["m"] if weight else None, clip, kl, scale))
    return got


@pytest.mark.parametrize("n", LENGTHS)
@pytest.mark.parametrize("ref,weight", [(True, True), (False, False), (True, False)])
def test_policy(n, ref, weight):
    _policy(_policy_inputs(n), ref, weight, scale=1.0 / n)


def test_policy_of_another_shape_and_clip():
    x = {k: v.view(30, 70) for k, v in _policy_inputs(2100, clip=(0.1, 0.4)).items()}
    _policy(x, clip=(0.1, 0.4), kl=0.0)
    one = ss.policy_loss(x["logp"], x["old"], x["A"], clip=0.2)
    two = ss.policy_loss(x["logp"], x["old"], x["A"], clip=(0.2, 0.2))
    assert torch.equal(one["loss"], two["loss"]) and set(one) == {"loss", "dlogp"}


def test_policy_on_views_off_16_bytes():
    x = {k: torch.cat([v[:1], v])[1:] for k, v in _policy_inputs(1000).items()}
    assert x["logp"].data_ptr() % 16 != 0
    got = _policy(x)
    aligned = _policy({k: v.clone() for k, v in x.items()})
    assert all(torch.equal(got[k], aligned[k]) for k in got)


def test_policy_clipping_by_hand():
    # ratios 2 and 1/2, both signs of the advantage; 1 within the clip
    old = torch.tensor([-1.0] * 5, device="cuda")
    logp = old + torch.tensor([math.log(2), math.log(2), -math.log(2), -math.log(2), 0.0],
                              device="cuda")
    A = torch.tensor([3.0, -3.0, 3.0, -3.0, 3.0], device="cuda")
    out = ss.policy_loss(logp, old, A, clip=(0.2, 0.3))
    loss = torch.tensor([-3.9, 6.0, -1.5, 2.4, -3.0], device="cuda")
    grad = torch.tensor([0.0, 6.0, -1.5, 0.0, -3.0], device="cuda")
    assert torch.allclose(out["loss"], loss, rtol=1e-6) and torch.allclose(out["dlogp"], grad,
                                                                           rtol=1e-6)


def test_policy_masked_and_extreme_values():
    n = 64
    x = _policy_inputs(n)
    want = ss.policy_loss(x["logp"], x["old"], x["A"], x["ref"], x["m"], kl=0.1)
    bad = {k: v.clone() for k, v in x.items()}
    gone = x["m"] == 0
    assert gone.any()
    for k, v in zip(("logp", "old", "A", "ref"), (NAN, INF, -INF, NAN)):
        bad[k][gone] = v
    got = ss.policy_loss(bad["logp"], bad["old"], bad["A"], bad["ref"], bad["m"], kl=0.1)
    assert all(torch.equal(got[k], want[k]) for k in want)
    # the ratio overflows: clipped, no gradient; and no advantage, no term
    t = torch.tensor([0.0, 0.0], device="cuda")
    out = ss.policy_loss(t, t - 200, torch.tensor([1.0, 0.0], device="cuda"), clip=0.2)
    assert out["loss"].tolist() == [-torch.tensor(1.2).item(), 0.0]
    assert out["dlogp"].tolist() == [0.0, 0.0]
    # no clipping above
    out = ss.policy_loss(t + 3, t, torch.ones_like(t), clip=(0.2, INF))
    assert torch.allclose(out["dlogp"], -torch.exp(t + 3))
    # a NaN where it counts stays one
    out = ss.policy_loss(t * NAN, t, torch.ones_like(t))
    assert out["loss"].isnan().all() and out["dlogp"].isnan().all()


def test_policy_gradient_by_differences():
    """In 64 bits, of the loss as the formulas give it, at points off the clip's ends."""
    x = _policy_inputs(400)
    got = ss.policy_loss(x["logp"], x["old"], x["A"], x["ref"], x["m"], kl=0.1)["dlogp"]
    f = {k: v.to(F64) for k, v in x.items()}
    h = 1e-6

    def loss(l):
        r = torch.exp(l - f["old"])
        d = f["ref"] - l
        return f["m"] * (-torch.minimum(r * f["A"], r.clamp(0.8, 1.2) * f["A"])
                         + 0.1 * (torch.exp(d) - d - 1))

    slope = (loss(f["logp"] + h) - loss(f["logp"] - h)) / (2 * h)
    # 64-bit differences are good to 1e-8 here, the kernel to fp32
    assert ((slope - got).abs() <= 1e-5 * (1 + slope.abs())).all()


def test_policy_refusals():
    x = _policy_inputs(8)
    with pytest.raises(ss.SSError):
        ss.policy_loss(x["logp"], x["old"], x["A"], kl=0.1)  # a KL term without a reference
    with pytest.raises(ss.SSError):
        ss.policy_loss(x["logp"], x["old"], x["A"], clip=1.5)
    with pytest.raises(ValueError):
        ss.policy_loss(x["logp"], x["old"][:4], x["A"])
    with pytest.raises(ValueError):
        ss.policy_loss(x["logp"].view(2, 4).T, x["old"], x["A"])
    with pytest.raises(TypeError):
        ss.policy_loss(x["logp"], x["old"], x["A"], weight=x["m"] != 0)
    empty = torch.empty(0, device="cuda")
    assert ss.policy_loss(empty, empty, empty)["loss"].shape == (0,)


# -------------------------------------------------------------- preference

def _pref_inputs(lengths, seed=0, before=0, after=0):
    n = before + sum(lengths) + after
    g = _gen(seed)
    logp = -_randn(g, n).exp()
    m = (torch.rand(n, generator=g, device="cuda") > 0.2).float()
    at = torch.tensor([before] + lengths, device="cuda").cumsum(0).to(I32)
    return logp, at, logp + _randn(g, n), m


def _ws():
    return ss.logprob_workspace(0, 1, 64)


SETS = [[1, 1], [0, 5], [0, 0], [3, 2, 0, 7], [100, 513, 512, 511, 1, 0], [5000, 3],
        [40000, 90001], [7] * 700]


@pytest.mark.parametrize("lengths", SETS, ids=lambda s: f"{len(s) // 2}x{max(s)}")
@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("average", [False, True])
def test_preference(lengths, kind, average):
    logp, at, ref, m = _pref_inputs(lengths, before=3, after=9)
    ws = _ws()
    e = 0.1 if kind == "sigmoid" else 0.0
    beta = 0.1 if kind != "hinge" else 0.01
    for r, w in ((ref, m), (None, None)):
        got = ss.preference_loss(logp, at, ws, ref_logp=r, weight=w, beta=beta, kind=kind,
                                 smoothing=e, average=average, scale=0.5)
        want = preference64(logp, at, r, w, torch.tensor(beta).item(), kind,
                            torch.tensor(e).item(), average, 0.5)
        _check(got, want)
    assert ss.read_status(ws)[0] == 0


def test_preference_far_margins():
    """Margins where one side's logistic function underflows."""
    logp = torch.tensor([0.0, -5000.0, -5000.0, 0.0], device="cuda")
    at = torch.arange(5, device="cuda", dtype=I32)
    got = ss.preference_loss(logp, at, _ws(), beta=1.0)
    assert got["loss"].tolist() == [0.0, 5000.0]
    assert got["dlogp"].tolist() == [0.0, 0.0, -1.0, 1.0]
    got = ss.preference_loss(logp, at, _ws(), beta=1.0, kind="hinge")
    assert got["loss"].tolist() == [0.0, 5001.0]


@pytest.mark.parametrize("average", [False, True])
def test_preference_of_an_impossible_token(average):
    """A log-probability of -infinity that counts: an infinite margin, not a NaN."""
    logp = torch.tensor([-1.0, -2.0, -3.0, -INF, -1.0, -1.0, -INF, -1.0], device="cuda")
    at = torch.tensor([0, 2, 4, 6, 8], dtype=I32, device="cuda")
    got = ss.preference_loss(logp, at, _ws(), average=average)
    assert got["loss"].tolist() == [0.0, 0.0] and got["reward"][:, 1].tolist() == [-INF, -INF]
    assert (got["dlogp"] == 0).all()
    swapped = torch.cat([logp[2:4], logp[:2]])
    got = ss.preference_loss(swapped, at[:3], _ws(), average=average)
    assert got["loss"].tolist() == [INF] and got["reward"][0, 0] == -INF
    assert got["dlogp"].isfinite().all()


def test_preference_masked_values_and_padding():
    logp, at, ref, m = _pref_inputs([50, 70, 0, 33], before=5, after=20)
    ws = _ws()
    want = ss.preference_loss(logp, at, ws, ref_logp=ref, weight=m)
    bad, bad_ref = logp.clone(), ref.clone()
    out = torch.ones_like(m, dtype=torch.bool)
    out[5:158] = m[5:158] == 0
    bad[out], bad_ref[out] = NAN, -INF
    got = ss.preference_loss(bad, at, ws, ref_logp=bad_ref, weight=m)
    assert all(torch.equal(got[k], want[k]) for k in want)
    assert (got["dlogp"][out] == 0).all()
    # a sequence whose weights are all 0 has no mean: 0
    m[5:55] = 0
    got = ss.preference_loss(logp, at, ws, ref_logp=ref, weight=m, average=True)
    assert got["reward"][0, 0] == 0 and (got["dlogp"][5:55] == 0).all()


def test_preference_of_nothing():
    ws = _ws()
    x = torch.randn(50, device="cuda")
    got = ss.preference_loss(x, torch.zeros(1, dtype=I32, device="cuda"), ws)
    assert got["loss"].shape == (0,) and (got["dlogp"] == 0).all()
    got = ss.preference_loss(x[:0], torch.zeros(5, dtype=I32, device="cuda"), ws)
    assert torch.allclose(got["loss"], torch.full((2,), math.log(2), device="cuda"))


@pytest.mark.parametrize("bad", [[0, 9, 4], [0, 4, 41], [-1, 4, 8], [8, 4, 0]])
def test_preference_bad_offsets(bad):
    """Only reads and writes within the batch, an error in the status word; the other
    pair's loss is there."""
    logp = -torch.rand(40, device="cuda")
    good = [12, 15, 20] if bad[2] <= 12 else [bad[2], bad[2], bad[2]]
    at = torch.tensor(bad + good[1:], dtype=I32, device="cuda")
    ws = _ws()
    got = ss.preference_loss(logp, at, ws)
    assert ss.read_status(ws)[0] == 8
    assert got["loss"][0].isnan() and got["reward"][0].isnan().all()


def test_preference_refusals():
    logp, at, ref, m = _pref_inputs([3, 4])
    ws = _ws()
    with pytest.raises(ValueError):
        ss.preference_loss(logp, at[:2], ws)
    with pytest.raises(ValueError):
        ss.preference_loss(logp, at, ws, kind="other")
    with pytest.raises(ValueError):
        ss.preference_loss(logp.view(1, 7), at, ws)
    with pytest.raises(TypeError):
        ss.preference_loss(logp, at.long(), ws)
    with pytest.raises(ss.SSError):
        ss.preference_loss(logp, at, ws, kind="ipo", smoothing=0.1)
    with pytest.raises(ss.SSError):
        ss.preference_loss(logp, at, ws, beta=0.0)
    with pytest.raises(ValueError):
        ss.preference_loss(logp, at, ws, ref_logp=ref[:3])


# ------------------------------------------------------------ distillation

def _distill_inputs(T, K, seed=0, teacher=torch.float32):
    g = _gen(seed)
    tail = torch.zeros(K + 1, device="cuda")
    tail[K] = 3.0
    s, t = (torch.log_softmax(2 * _randn(g, T, K + 1) + tail, 1)[:, :K].contiguous()
            for _ in range(2))
    ids = torch.arange(K, device="cuda", dtype=I32).repeat(T, 1)
    short = (torch.rand(T, 1, generator=g, device="cuda") < 0.3) & (
        torch.arange(K, device="cuda") >= (K + 1) // 2)
    none = torch.rand(T, generator=g, device="cuda") < 0.1
    ids[short] = -1
    ids[none] = -1
    m = (torch.rand(T, generator=g, device="cuda") > 0.2).float() * 1.7
    return s, t.to(teacher), ids, m


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 8, 13, 16, 20, 32, 33, 64, 100, 127, 128])
@pytest.mark.parametrize("tail", [False, True])
def test_distill(K, tail):
    for T, dt in ((1, torch.float32), (37, BF16), (1003, torch.float32), (515, BF16)):
        s, t, ids, m = _distill_inputs(T, K, teacher=dt)
        _check(ss.distill_loss(s, t, ids, m, tail, 0.7), distill64(s, t, ids, m, tail, 0.7))
        _check(ss.distill_loss(s, t, tail=tail), distill64(s, t, tail=tail))


def test_distill_on_views_off_16_bytes():
    s, t, ids, m = _distill_inputs(50, 8)
    want = ss.distill_loss(s, t, ids, m)

    def off(v):
        return torch.cat([v.reshape(-1)[:1], v.reshape(-1)])[1:].view(v.shape)

    got = ss.distill_loss(off(s), off(t), off(ids), off(m))
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["dlogp"], want["dlogp"])


def test_distill_teacher_in_logits():
    """Without a tail a shift of the teacher's values changes nothing."""
    s, t, ids, m = _distill_inputs(200, 16)
    a = ss.distill_loss(s, t, ids, m)
    b = ss.distill_loss(s, t + 1000.0, ids, m)
    # t + 1000 is rounded to 2^-14
    assert torch.allclose(a["dlogp"], b["dlogp"], rtol=2.0 ** -12)
    same = ss.distill_loss(torch.log_softmax(t, 1), t)
    assert same["loss"].abs().max() < 1e-5


@pytest.mark.parametrize("tail", [False, True])
def test_distill_values_of_minus_infinity_and_garbage(tail):
    s, t, ids, m = _distill_inputs(64, 10)
    t[:, 3] = -INF                      # of probability 0, not absent
    _check(ss.distill_loss(s, t, ids, m, tail), distill64(s, t, ids, m, tail))
    want = ss.distill_loss(s, t, ids, m, tail)
    gone = (ids < 0) | (m == 0)[:, None]
    s[gone], t[gone] = NAN, INF
    got = ss.distill_loss(s, t, ids, m, tail)
    assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["dlogp"], want["dlogp"])
    assert (got["dlogp"][gone] == 0).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("which", ["teacher", "student"])
def test_distill_nan_of_an_entry_that_counts(tail, which):
    """It is in the row's sums: the loss is NaN, of that row alone, and so is the gradient
    where those sums are its factor."""
    s, t, _, _ = _distill_inputs(64, 10)
    want = ss.distill_loss(s, t, tail=tail)
    (t if which == "teacher" else s)[5, 3] = NAN
    if which == "student" and tail:
        t[5, 3] = -INF                  # its share of the tail counts all the same
    got = ss.distill_loss(s, t, tail=tail)
    assert got["loss"][5].isnan()
    # (without a tail the student's values are no factor of the gradient)
    assert got["dlogp"][5].isnan().all() or (which == "student" and not tail)
    rest = torch.arange(64, device="cuda") != 5
    for k in ("loss", "dlogp"):
        assert torch.equal(got[k][rest], want[k][rest])


def test_distill_without_a_teacher_value():
    """A row whose values are all -infinity is no distribution: nothing without a tail,
    everything in the tail with one."""
    s = torch.full((2, 4), -2.0, device="cuda")
    t = torch.full((2, 4), -INF, device="cuda")
    got = ss.distill_loss(s, t)
    assert (got["loss"] == 0).all() and (got["dlogp"] == 0).all()
    got = ss.distill_loss(s, t, tail=True)
    rest = 1 - 4 * math.exp(-2)
    assert torch.allclose(got["loss"], torch.full((2,), -math.log(rest), device="cuda"), rtol=1e-5)
    assert torch.allclose(got["dlogp"], torch.full((2, 4), math.exp(-2) / rest, device="cuda"),
                          rtol=1e-5)


def test_distill_tail_at_its_floor():
    """The student leaves less than 2^-12: the tail's loss is there, its gradient not."""
    s = torch.log(torch.tensor([[0.6, 0.39999]], device="cuda"))
    t = torch.log(torch.tensor([[0.5, 0.3]], device="cuda"))
    got = ss.distill_loss(s, t, tail=True)
    p = torch.exp(t.to(F64))
    rest = 1 - float(p.sum())
    want = float((p * (t.to(F64) - s.to(F64))).sum()) + rest * (math.log(rest) + 12 * math.log(2))
    assert abs(float(got["loss"]) - want) < 1e-5
    assert torch.allclose(got["dlogp"], -p.float(), rtol=1e-6)
    # a student sure of them all: q' is the floor, not 0 and not below it
    got = ss.distill_loss(torch.log(torch.tensor([[0.75, 0.26]], device="cuda")), t, tail=True)
    assert got["loss"].isfinite().all()


def test_distill_tail_keeps_its_digits():
    """A student that leaves 2^-10 to the tail: its slope has the digits that sums in
    fp32 would lose (2^-24 beside 2^-10 is 6e-5)."""
    K = 128
    g = _gen(3)
    q = torch.rand(300, K, generator=g, device="cuda", dtype=F64)
    q = q / q.sum(1, keepdim=True) * (1 - 2.0 ** -10)
    s = torch.log(q).float()
    t = torch.log_softmax(_randn(g, 300, K + 1), 1)[:, :K].contiguous()
    got = ss.distill_loss(s, t, tail=True)
    want = distill64(s, t, tail=True)
    _check(got, want)
    p, q = torch.exp(t.to(F64)), torch.exp(s.to(F64))
    p1, rest = 1 - p.sum(1, keepdim=True), 1 - q.sum(1, keepdim=True)
    ratio = p1 / rest
    slope = (got["dlogp"].to(F64) + p) / q
    # p' and q' are 2^-27 off and rounded; dlogp = ratio q - p has p's own error and
    # half a step of both terms, which the division by q shows as p / q
    tol = 2.0 ** -27 * (1 / p1 + 1 / rest) + (EXP + 6 * F32) * (1 + p / (ratio * q))
    assert ((slope / ratio - 1).abs() < tol).all()
    # 2^-27 beside 2^-10 is 7.6e-6, beside p' near 0.003 2.5e-6
    assert tol.median() < 2e-5


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_by_differences(tail):
    s, t, ids, m = _distill_inputs(80, 12)
    got = ss.distill_loss(s, t, ids, m, tail)["dlogp"]
    l = s.to(F64)
    h = 1e-6
    for k in (0, 5, 11):
        u = torch.zeros_like(l)
        u[:, k] = h
        up, down = (distill64(l + d, t, ids, m, tail)["loss"][0] for d in (u, -u))
        slope = (up - down) / (2 * h)
        assert ((slope - got[:, k]).abs() <= 1e-5 * (1 + slope.abs())).all()


def test_distill_refusals():
    s, t, ids, m = _distill_inputs(8, 4)
    with pytest.raises(TypeError):
        ss.distill_loss(s, t.half())
    with pytest.raises(ValueError):
        ss.distill_loss(s, t[:4])
    with pytest.raises(ValueError):
        ss.distill_loss(s.view(-1), t.view(-1))
    with pytest.raises(TypeError):
        ss.distill_loss(s, t, ids.long())
    with pytest.raises(ValueError):
        ss.distill_loss(s, t, weight=m[:3])
    big = torch.zeros(2, 129, device="cuda")
    with pytest.raises(ss.SSError) as e:
        ss.distill_loss(big, big)
    assert e.value.name == "SS_ERR_UNSUPPORTED"


# ---------------------------------------------------------------- together

def _head_inputs(T, V, D, seed=0):
    g = _gen(seed)
    H = _randn(g, T, D).to(BF16)
    W = (3 * D ** -0.5 * _randn(g, V, D)).to(BF16)
    return H, W, g


def _chain_slopes(loss64, H, W, dH, dW, tol=2 ** -7):
    """d loss along a direction of H and of W in 64 bits, against the gradients, which
    are two bf16 roundings of at most 2^-8 off."""
    h = 1e-5
    H, W = H.to(F64), W.to(F64)
    for grad, at in ((dH, 0), (dW, 1)):
        u = torch.randn_like((H, W)[at])
        u /= u.norm()
        points = [((H + d * u, W) if at == 0 else (H, W + d * u)) for d in (h, -h)]
        slope = (loss64(*points[0]) - loss64(*points[1])) / (2 * h)
        assert abs(slope - float((grad.to(F64) * u).sum())) <= tol * float(grad.norm()) + 1e-7


def test_policy_step_by_differences():
    T, V, D = 90, 400, 128
    H, W, g = _head_inputs(T, V, D)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(I32)
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)
    step = 0.3 * _randn(g, T)
    old = logp - torch.where((step.exp() - 1).abs() < 0.19, step, 0.5)  # off the clip's ends
    A, ref, m = _randn(g, T), logp + 0.4 * _randn(g, T), torch.rand(T, generator=g, device="cuda")
    out = ss.policy_loss(logp, old, A, ref, m, kl=0.2)
    dH, dW = ss.logprobs_backward(out["dlogp"], H, W, ids, logp, lse, ws)

    def loss(h, v):
        z = h @ v.T
        l = z.gather(1, ids.long()[:, None])[:, 0] - torch.logsumexp(z, 1)
        r = torch.exp(l - old)
        d = ref - l
        return float((m * (-torch.minimum(r * A, r.clamp(0.8, 1.2) * A)
                           + 0.2 * (torch.exp(d) - d - 1))).sum())

    _chain_slopes(loss, H, W, dH, dW)


def test_preference_step_by_differences():
    T, V, D = 120, 400, 128
    H, W, g = _head_inputs(T, V, D, 1)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(I32)
    at = torch.tensor([0, 30, 65, 65, 110], dtype=I32, device="cuda")
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)
    ref = logp + 0.3 * _randn(g, T)
    out = ss.preference_loss(logp, at, ws, ref_logp=ref, beta=0.2, smoothing=0.1)
    dH, dW = ss.logprobs_backward(out["dlogp"], H, W, ids, logp, lse, ws)
    assert (dH[110:] == 0).all()

    def loss(h, v):
        z = h @ v.T
        gap = z.gather(1, ids.long()[:, None])[:, 0] - torch.logsumexp(z, 1) - ref
        total = 0.0
        for a, b, c in ((0, 30, 65), (65, 65, 110)):
            x = 0.2 * float(gap[a:b].sum() - gap[b:c].sum())
            total += 0.9 * math.log1p(math.exp(-x)) + 0.1 * math.log1p(math.exp(x))
        return total

    _chain_slopes(loss, H, W, dH, dW)


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("tail", [False, True])
def test_distill_step_by_differences(cap, tail):
    T, V, D, K = 70, 400, 128, 9
    H, W, g = _head_inputs(T, V, D, 2)
    head = {"cap": cap, "tau": 7.5} if cap else {}
    z = 3 * _randn(g, T, V)
    top = z.topk(K, 1)
    ids = top.indices.to(I32)
    t = (top.values - torch.logsumexp(z, 1, keepdim=True)).contiguous()
    ids[::5, 6:] = -1
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws, **head)
    out = ss.distill_loss(logp, t, ids, tail=tail)
    dH, dW = ss.logprobs_backward(out["dlogp"], H, W, ids, logp, lse, ws, **head)

    def loss(h, v):
        s = h @ v.T
        s = cap * torch.sigmoid(s / 7.5) if cap else s
        l = s.gather(1, ids.clamp(min=0).long()) - torch.logsumexp(s, 1, keepdim=True)
        return float(distill64(torch.where(ids >= 0, l, 0.0), t, ids, tail=tail)["loss"][0].sum())

    _chain_slopes(loss, H, W, dH, dW)


def test_whole_step_in_a_graph():
    T, V, D = 200, 500, 128
    H, W, g = _head_inputs(T, V, D, 3)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(I32)
    A, old = _randn(g, T), -torch.rand(T, generator=g, device="cuda") * 8
    ws = ss.logprob_workspace(T, V, D)

    def step():
        logp, lse = ss.logprobs(H, W, ids, ws)
        out = ss.policy_loss(logp, old, A, ref_logp=old, kl=0.1)
        return (logp, out["loss"]) + ss.logprobs_backward(out["dlogp"], H, W, ids, logp, lse, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    A.normal_()
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_behind_the_feed_forward_block():
    """The block's output as the head's H, and the head's dH as the block's dY."""
    T, D, F, V = 96, 128, 256, 300
    H0, W, g = _head_inputs(T, V, D, 4)
    Wg, Wu = ((D ** -0.5 * _randn(g, F, D)).to(BF16) for _ in range(2))
    Wd = (F ** -0.5 * _randn(g, D, F)).to(BF16)
    bws, ws = ss.ffn_workspace(T, D, F), ss.logprob_workspace(T, V, D)
    H, saved = ss.ffn_forward(H0, Wg, Wu, Wd, bws, residual=H0, save=True)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(I32)
    logp, lse = ss.logprobs(H, W, ids, ws)
    out = ss.policy_loss(logp, logp.clone(), _randn(g, T))
    dH, dW = ss.logprobs_backward(out["dlogp"], H, W, ids, logp, lse, ws)
    grads = ss.ffn_backward(dH, H0, Wg, Wu, Wd, saved, bws)
    assert all(t.isfinite().all() and t.abs().max() > 0 for t in (dH, dW, *grads.values()))


def test_agrees_with_the_sampled_head_over_the_whole_vocabulary():
    """Cross-entropy over all rows as candidates is -logp, and its gradient that of the
    mean of -logp. Both sides are within their stated tolerances of 64 bits: 1e-3 for
    the loss, 2e-2 of the norm for the gradients."""
    T, V, D = 300, 700, 128
    H, W, g = _head_inputs(T, V, D, 5)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda").to(I32)
    hws = ss.workspace(T, V, V, D)
    step = ss.step(H, W, ids, V, 1, hws, scale=1.0 / T)
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)
    assert torch.allclose(step["loss"], -logp, rtol=1e-3, atol=1e-5)
    dH, dW = ss.logprobs_backward(torch.full((T,), -1.0 / T, device="cuda"), H, W, ids, logp, lse,
                                  ws)
    for a, b in ((dH, step["dH"]), (dW, step["dW"])):
        assert (a.float() - b.float()).norm() <= 2e-2 * b.float().norm()
