"""The head's log-probabilities on the GPU against 64 bits, every element within the
bound that logprob_util counts from the stated roundings."""
import pytest
import torch

import sampled_softmax_output_gb300 as ss
from logprob_util import F64, assert_within, grads64, logits64, logprobs64

pytestmark = pytest.mark.gpu
BF16, F32T, I32 = torch.bfloat16, torch.float32, torch.int32

# one token and one row of the vocabulary, sizes around the tiles of 128 and 256, K of
# one k-block, of a run and a part of one, several runs
SIZES = [(1, 1, 64, 1), (1, 1000, 768, 1), (2, 257, 64, 3), (31, 300, 192, 5), (33, 129, 256, 1),
         (100, 255, 320, 7), (128, 256, 128, 1), (129, 1023, 832, 20), (255, 127, 576, 32),
         (257, 513, 1088, 1), (300, 3001, 768, 128), (513, 2049, 64, 2), (1003, 777, 448, 4),
         # the widest model, the largest vocabulary
         (2, 70, 16384, 1), (3, 300, 16384, 2), (40, 524288, 64, 3), (1, 524288, 64, 128)]


def _inputs(T, V, D, K, seed=0, std=3.0):
    g = torch.Generator("cuda").manual_seed(seed)
    H = torch.randn(T, D, generator=g, device="cuda").to(BF16)
    W = (torch.randn(V, D, generator=g, device="cuda") * std * D ** -0.5).to(BF16)
    ids = torch.randint(0, V, (T, K), generator=g, device="cuda").to(I32)
    dlogp = torch.randn(T, K, generator=g, device="cuda")
    return H, W, ids, dlogp


def _head(cap):
    return {"cap": cap, "tau": 7.5} if cap else {}


def _forward(H, W, ids, cap=0.0, ws=None):
    T, D = H.shape
    ws = ss.logprob_workspace(T, W.shape[0], D, backward=False) if ws is None else ws
    logp, lse = ss.logprobs(H, W, ids, ws, **_head(cap))
    assert logp.shape == ids.shape and lse.shape == (T,)
    ref = logprobs64(H, W, ids.view(T, -1), **_head(cap))
    assert_within(lse, ref["lse"], "lse")
    assert_within(logp.view(T, -1), ref["logp"], "logp")
    assert ss.read_status(ws)[0] == 0
    return logp, lse


def _backward(dlogp, H, W, ids, logp, lse, cap=0.0, ws=None, dw_dtype=F32T):
    T, D = H.shape
    ws = ss.logprob_workspace(T, W.shape[0], D) if ws is None else ws
    dH, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, dw_dtype=dw_dtype, **_head(cap))
    assert dH.dtype == BF16 and dW.dtype == dw_dtype
    two = [t.view(T, -1) for t in (dlogp, ids, logp)]
    ref = grads64(two[0], H, W, two[1], two[2], lse, fp32_dw=dw_dtype == F32T, **_head(cap))
    assert_within(dH, ref["dH"], "dH")
    assert_within(dW, ref["dW"], "dW")
    assert ss.read_status(ws)[0] == 0
    return dH, dW


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_forward(size, cap):
    _forward(*_inputs(*size)[:3], cap=cap)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_backward(size, cap):
    H, W, ids, dlogp = _inputs(*size, seed=1)
    logp, lse = _forward(H, W, ids, cap)
    _backward(dlogp, H, W, ids, logp, lse, cap, dw_dtype=F32T)
    _backward(dlogp, H, W, ids, logp, lse, cap, dw_dtype=BF16)


def test_one_id_per_token_in_one_dimension():
    H, W, ids, dlogp = _inputs(200, 700, 128, 1)
    flat = _forward(H, W, ids.view(-1))
    both = _forward(H, W, ids)
    assert torch.equal(flat[0], both[0].view(-1))
    a = _backward(dlogp.view(-1), H, W, ids.view(-1), *flat)
    b = _backward(dlogp, H, W, ids, *both)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("K", [1, 6])
def test_absent_and_repeated_ids(K):
    T, V, D = 130, 400, 192
    H, W, ids, dlogp = _inputs(T, V, D, K, seed=2)
    ids[::3] = -1                      # tokens without any id
    ids[1::3, K // 2:] = -1
    ids[2::3] = ids[2::3, :1]          # the same id K times
    logp, lse = _forward(H, W, ids)
    assert (logp[ids < 0] == 0).all()
    dlogp[ids < 0] = float("nan")      # not looked at
    dH, dW = _backward(dlogp, H, W, ids, logp, lse)
    assert (dH[::3] == 0).all()


def test_ids_that_hit_every_column():
    """Every id of the vocabulary in every token: the softmax itself."""
    T, V, D = 40, 128, 64
    H, W, _, _ = _inputs(T, V, D, 1)
    ids = torch.stack([torch.randperm(V, device="cuda") for _ in range(T)]).to(I32)
    logp, lse = _forward(H, W, ids)
    assert (logp.exp().sum(1) - 1).abs().max() < 1e-5
    # a gradient of ones moves the softmax by 1 - V P: its own sum is 0
    _backward(torch.ones_like(logp), H, W, ids, logp, lse)


def test_many_ids_in_one_tile():
    """More of a warp's ids in its 128 columns than it has lanes."""
    T, V, D = 64, 1500, 128
    H, W, _, _ = _inputs(T, V, D, 1)
    ids = torch.randint(256, 384, (T, 100), device="cuda").to(I32)
    _forward(H, W, ids)


def test_cap_above_the_plain_range():
    """A cap so large that exp(cap) overflows."""
    H, W, ids, dlogp = _inputs(100, 500, 128, 3, std=40.0)
    ws = ss.logprob_workspace(100, 500, 128)
    logp, lse = ss.logprobs(H, W, ids, ws, cap=200.0, tau=20.0)
    ref = logprobs64(H, W, ids, cap=200.0, tau=20.0)
    assert_within(lse, ref["lse"], "lse")
    assert_within(logp, ref["logp"], "logp")
    dH, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, cap=200.0, tau=20.0)
    ref = grads64(dlogp, H, W, ids, logp, lse, cap=200.0, tau=20.0)
    assert_within(dH, ref["dH"], "dH")
    assert_within(dW, ref["dW"], "dW")


def test_few_tokens_again_and_again():
    """One workspace for one token and two in turn, after an id out of range too, and the
    same bits each time."""
    V, D = 50257, 128
    H, W, ids, _ = _inputs(2, V, D, 5)
    ws = ss.logprob_workspace(2, V, D, backward=False)
    want = [_forward(H[:T], W, ids[:T].contiguous(), ws=ws) for T in (1, 2)]
    bad = ids.clone()
    bad[1, 3] = V
    for _ in range(20):
        for T in (1, 2):
            logp, lse = ss.logprobs(H[:T], W, ids[:T], ws)
            assert torch.equal(logp, want[T - 1][0]) and torch.equal(lse, want[T - 1][1])
        ss.logprobs(H, W, bad, ws)
        ss.logprobs(H, W, ids, ws)  # does nothing
        assert ss.read_status(ws)[0] != 0
        ws[:ss.WORKSPACE_HEADER_BYTES].zero_()


@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_no_shift_of_sampled_tokens(cap):
    """What is off by the same amount for every token adds up over a sequence. Each of
    these log-probabilities is within 1.5e-6 (rms) of its value, their mean within 4 of
    its own standard deviations, and the log-sum-exp's corrections leave some 3e-8."""
    T, V, D = 4096, 4000, 128
    H, W, _, _ = _inputs(T, V, D, 1)
    z = logits64(H, W, **_head(cap))[0]
    want = torch.log_softmax(z, 1)
    gen = torch.Generator("cuda").manual_seed(5)
    ids = torch.multinomial(want.exp(), 1, generator=gen)
    logp, _ = _forward(H, W, ids.to(I32), cap)
    off = logp.to(F64) - want.gather(1, ids)
    assert off.std() < 1.5e-6
    assert off.mean().abs() < 4 * 1.5e-6 / T ** 0.5 + 3e-8


def test_least_cap():
    """The smallest cap that the backward pass takes."""
    head = {"cap": 2.0 ** -6, "tau": 2.0 ** -8}
    for K in (1, 3):
        H, W, ids, dlogp = _inputs(100, 500, 128, K, std=2.0 ** -8)
        ws = ss.logprob_workspace(100, 500, 128)
        logp, lse = ss.logprobs(H, W, ids, ws, **head)
        ref = logprobs64(H, W, ids.view(100, -1), **head)
        assert_within(lse, ref["lse"], "lse")
        assert_within(logp.view(100, -1), ref["logp"], "logp")
        dH, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, **head)
        two = [t.view(100, -1) for t in (dlogp, ids, logp)]
        ref = grads64(two[0], H, W, two[1], two[2], lse, **head)
        assert_within(dH, ref["dH"], "dH")
        assert_within(dW, ref["dW"], "dW")


@pytest.mark.parametrize("std", [0.0, 60.0])
def test_flat_and_peaked_softmax(std):
    H, W, ids, dlogp = _inputs(150, 600, 128, 1, std=std)
    logp, lse = _forward(H, W, ids)
    _backward(dlogp, H, W, ids, logp, lse)


@pytest.mark.parametrize("K", [1, 4])
def test_gradient_by_differences(K):
    """The objective's own change along a direction of W and of H, in 64 bits, against
    the kernel's gradient: both from the same bf16 H and W. dH and dW are within
    2^-7 of their norm (two bf16 roundings of at most 2^-8 each), so their product
    with a direction is within that of the product of the norms."""
    T, V, D = 60, 300, 128
    H, W, ids, dlogp = _inputs(T, V, D, K, seed=3)
    logp, lse = _forward(H, W, ids)
    dH, dW = _backward(dlogp, H, W, ids, logp, lse)
    H, W, w = H.to(F64), W.to(F64), dlogp.to(F64)

    def objective(h, v):
        z = h @ v.T
        return float((w * (z.gather(1, ids.long()) - torch.logsumexp(z, 1, keepdim=True))).sum())

    step = 1e-5
    for grad, at in ((dH, 0), (dW, 1)):
        u = torch.randn_like((H, W)[at])
        u /= u.norm()
        up = (H + step * u, W) if at == 0 else (H, W + step * u)
        down = (H - step * u, W) if at == 0 else (H, W - step * u)
        slope = (objective(*up) - objective(*down)) / (2 * step)
        assert abs(slope - float((grad.to(F64) * u).sum())) < 2 ** -7 * float(grad.norm()) + 1e-6


def test_accumulate():
    H, W, ids, dlogp = _inputs(140, 333, 128, 2)
    ws = ss.logprob_workspace(140, 333, 128)
    logp, lse = ss.logprobs(H, W, ids, ws)
    for dt in (F32T, BF16):
        _, once = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, dw_dtype=dt)
        total = torch.ones_like(once)
        _, got = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, dw_dtype=dt,
                                      accumulate=True, dW=total)
        assert got is total
        # one addition (and for bf16 the rounding of `once`)
        tol = torch.finfo(dt).eps * (1 + once.float().abs())
        assert ((total.float() - 1 - once.float()).abs() <= tol).all()
        _, fresh = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, dw_dtype=dt,
                                        accumulate=True)
        assert torch.equal(fresh, once)


def test_no_tokens():
    H, W, _, _ = _inputs(0, 50, 64, 1)
    ids = torch.zeros(0, 3, dtype=I32, device="cuda")
    ws = ss.logprob_workspace(0, 50, 64)
    logp, lse = ss.logprobs(H, W, ids, ws)
    assert logp.shape == (0, 3) and lse.shape == (0,)
    kept = torch.ones(50, 64, device="cuda")
    ss.logprobs_backward(logp, H, W, ids, logp, lse, ws, dW=kept, accumulate=True)
    assert (kept == 1).all()
    for dt in (F32T, BF16):
        _, dW = ss.logprobs_backward(logp, H, W, ids, logp, lse, ws, dw_dtype=dt)
        assert (dW == 0).all()


@pytest.mark.parametrize("K", [1, 3])
def test_garbage_in_tokens_without_a_gradient(K):
    """Padding's hidden states may hold anything: a token whose coefficients are 0, or
    that has no id, adds nothing anywhere."""
    T, V, D = 150, 400, 128
    H, W, ids, dlogp = _inputs(T, V, D, K, seed=4)
    pad = torch.arange(T, device="cuda") % 4 == 1
    gone = torch.arange(T, device="cuda") % 4 == 2
    dlogp[pad] = 0
    ids[gone] = -1
    clean = H.clone()
    clean[pad | gone] = 0
    H[pad] = float("nan")
    H[gone] = float("inf")
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)
    ref_logp, ref_lse = ss.logprobs(clean, W, ids, ws)
    live = ~(pad | gone)
    assert torch.equal(logp[live], ref_logp[live]) and torch.equal(lse[live], ref_lse[live])
    assert not lse[pad].isfinite().any() and not logp[pad].isfinite().any()
    dH, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws)
    ref_dH, ref_dW = ss.logprobs_backward(dlogp, clean, W, ids, ref_logp, ref_lse, ws)
    assert torch.equal(dW, ref_dW) and torch.equal(dH, ref_dH)
    assert (dH[~live] == 0).all()


def test_coefficients_of_very_different_size():
    """One id per token: the backward scales its operands by the largest of them."""
    T, V, D = 200, 300, 128
    H, W, ids, _ = _inputs(T, V, D, 1, seed=5)
    logp, lse = _forward(H, W, ids)
    g = torch.Generator("cuda").manual_seed(6)
    size = torch.exp2(torch.randint(-30, 1, (T, 1), generator=g, device="cuda").float())
    dlogp = size * torch.randn(T, 1, generator=g, device="cuda")
    _backward(dlogp, H, W, ids, logp, lse)
    _backward(dlogp * 2.0 ** -60, H, W, ids, logp, lse)
    _backward(torch.full_like(dlogp, 1.0 / 3), H, W, ids, logp, lse)
    ws = ss.logprob_workspace(T, V, D)
    dH, dW = ss.logprobs_backward(torch.zeros_like(dlogp), H, W, ids, logp, lse, ws)
    assert (dH == 0).all() and (dW == 0).all()


def test_a_shared_coefficient_is_not_rounded_with_its_tokens():
    """All tokens of one coefficient c = 1 + 2^-8, half a step between bf16 values. G
    as it is would be 2^-8 off at every id; here (1 - P) is what rounds, and a row of
    dW from one token is c (1 - P) h."""
    T, V, D = 64, 2000, 128
    H, W, _, _ = _inputs(T, V, D, 1, std=1.0)
    ids = torch.randperm(V, device="cuda")[:T].to(I32)
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)
    dlogp = torch.full((T,), 1 + 2.0 ** -8, device="cuda")
    _, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws)
    ref = grads64(dlogp[:, None], H, W, ids[:, None], logp[:, None], lse)["dW"][0]
    rows = ids.long()
    off = (dW[rows].to(F64) - ref[rows]).norm() / ref[rows].norm()
    # P is near 1 / V: 1 - P rounds to 1 (0.5e-3 off); the other tokens' terms are
    # small beside it
    assert off < 1.5e-3


def test_same_bits_every_time():
    H, W, ids, dlogp = _inputs(700, 5000, 256, 9, seed=7)
    ws = ss.logprob_workspace(700, 5000, 256)
    first = None
    for _ in range(3):
        logp, lse = ss.logprobs(H, W, ids, ws)
        out = (logp, lse) + ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws)
        first = out if first is None else first
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_smaller_batches_on_one_workspace():
    ws = ss.logprob_workspace(600, 700, 192)
    for T, V, D, K in ((600, 700, 192, 2), (7, 700, 192, 1), (250, 300, 64, 5)):
        H, W, ids, dlogp = _inputs(T, V, D, K)
        logp, lse = _forward(H, W, ids, ws=ws)
        _backward(dlogp, H, W, ids, logp, lse, ws=ws)


def test_bad_ids_are_recorded():
    H, W, ids, dlogp = _inputs(50, 90, 64, 2)
    for bad in (90, -2, 2 ** 31 - 1):
        ws = ss.logprob_workspace(50, 90, 64)
        logp, lse = ss.logprobs(H, W, ids, ws)
        wrong = ids.clone()
        wrong[17, 1] = bad
        ss.logprobs(H, W, wrong, ws)
        assert ss.read_status(ws)[0] == 4
        # nothing runs on that workspace until its header is zeroed
        keep = torch.full_like(logp, 7.0)
        ss.logprobs(H, W, ids, ws, logp=keep)
        assert (keep == 7).all()
        ws[:1024].zero_()
        ss.logprobs_backward(dlogp, H, W, wrong, logp, lse, ws)
        assert ss.read_status(ws)[0] == 4
    one = ids[:, :1].contiguous()
    one[3] = 90
    ws = ss.logprob_workspace(50, 90, 64)
    ss.logprobs_backward(dlogp[:, :1].contiguous(), H, W, one, logp[:, :1].contiguous(), lse, ws)
    assert ss.read_status(ws)[0] == 4


def test_refusals():
    H, W, ids, dlogp = _inputs(50, 90, 64, 2)
    ws = ss.logprob_workspace(50, 90, 64)
    logp, lse = ss.logprobs(H, W, ids, ws)
    with pytest.raises(ValueError):
        ss.logprobs(H.T, W, ids, ws)
    with pytest.raises(ValueError):
        ss.logprobs(H, W[:, :32], ids, ws)
    with pytest.raises(ValueError):
        ss.logprobs(H, W, ids[:49], ws)
    with pytest.raises(ValueError):
        ss.logprobs(H, W, ids[None], ws)
    with pytest.raises(TypeError):
        ss.logprobs(H, W, ids.long(), ws)
    with pytest.raises(ss.SSError) as e:
        ss.logprobs(H, W, torch.zeros(50, 129, dtype=I32, device="cuda"), ws)
    assert e.value.name == "SS_ERR_UNSUPPORTED"
    with pytest.raises(ss.SSError) as e:
        ss.logprobs_backward(dlogp, H, W, ids, logp, lse,
                             ss.logprob_workspace(40, 90, 64)[:-1024])
    assert e.value.name == "SS_ERR_WORKSPACE"
    with pytest.raises(ValueError):
        ss.logprobs_backward(dlogp[:, 0].contiguous(), H, W, ids, logp, lse, ws)
    with pytest.raises(TypeError):
        ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws, dw_dtype=torch.float16)
    with pytest.raises(ss.SSError) as e:  # rows off a 16-byte boundary
        off = torch.empty(51 * 64, dtype=BF16, device="cuda")[1:50 * 64 + 1].view(50, 64)
        ss.logprobs(off, W, ids, ws)
    assert e.value.name == "SS_ERR_INVALID"


def test_another_stream_and_a_graph():
    H, W, ids, dlogp = _inputs(300, 900, 128, 2)
    ws = ss.logprob_workspace(300, 900, 128)
    logp, lse = ss.logprobs(H, W, ids, ws)
    dH, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        on = ss.logprobs(H, W, ids, ws)
        back = ss.logprobs_backward(dlogp, H, W, ids, *on, ws)
    torch.cuda.synchronize()
    assert torch.equal(on[0], logp) and torch.equal(back[1], dW)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_logp, g_lse = ss.logprobs(H, W, ids, ws)
        g_dH, g_dW = ss.logprobs_backward(dlogp, H, W, ids, g_logp, g_lse, ws)
    new = _inputs(300, 900, 128, 2, seed=8)
    for t, n in zip((H, W, ids, dlogp), new):
        t.copy_(n)
    want = ss.logprobs(H, W, ids, ws)
    want += ss.logprobs_backward(dlogp, H, W, ids, *want, ws)
    for t in (g_logp, g_lse, g_dH, g_dW):
        t.fill_(float("nan"))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got, w in zip((g_logp, g_lse, g_dH, g_dW), want):
        assert torch.equal(got, w)


def test_two_graphs_at_once():
    """Each on a workspace of its own, replayed together on two streams."""
    jobs = []
    for seed in (11, 12):
        H, W, ids, dlogp = _inputs(500, 3000, 256, 3, seed=seed)
        ws = ss.logprob_workspace(500, 3000, 256)
        want = ss.logprobs(H, W, ids, ws)
        want += ss.logprobs_backward(dlogp, H, W, ids, *want, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = ss.logprobs(H, W, ids, ws)
            got += ss.logprobs_backward(dlogp, H, W, ids, *got, ws)
        jobs.append((g, got, want, torch.cuda.Stream(), (H, W, ids, dlogp, ws)))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, _, _, s, _ in jobs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, got, want, _, _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_past_two_to_the_32_logits():
    """T V past 2^32: G's rows lie behind 8 GB. Checked on the last rows and on the
    vocabulary rows that only they have as ids."""
    T, V, D = 90000, 50304, 64
    H, W, ids, dlogp = _inputs(T, V, D, 1, std=1.0)
    ids.clamp_(max=V - 1001)
    last = slice(T - 1000, T)
    ids[last, 0] = torch.arange(V - 1000, V, device="cuda", dtype=I32)
    ws = ss.logprob_workspace(T, V, D)
    logp, lse = ss.logprobs(H, W, ids, ws)
    ref = logprobs64(H[last], W, ids[last])
    assert_within(lse[last], ref["lse"], "lse")
    assert_within(logp[last], ref["logp"], "logp")
    dH, dW = ss.logprobs_backward(dlogp, H, W, ids, logp, lse, ws)
    part = grads64(dlogp[last], H[last], W, ids[last], logp[last], lse[last])
    assert_within(dH[last], part["dH"], "dH")
    # the first rows' dH too (their G lies at the start), and dW of the last rows:
    # every token's probability term, in 64 bits, from those columns alone
    first = slice(0, 500)
    assert_within(dH[first], grads64(dlogp[first], H[first], W, ids[first], logp[first],
                                     lse[first])["dH"], "dH")
    cols = slice(V - 64, V)
    P = torch.exp(H.to(F64) @ W[cols].to(F64).T - lse.to(F64)[:, None]) * -dlogp.to(F64)
    rows = torch.arange(T - 64, T, device="cuda")
    P[rows, torch.arange(64, device="cuda")] += dlogp[rows, 0].to(F64)
    want = P.T @ H.to(F64)
    # two roundings of at most 2^-8, 1e-4 for a sum of 90000 in fp32
    assert (dW[cols].to(F64) - want).norm() <= (2 ** -7 + 1e-4) * want.norm()


def test_more_tokens_than_one_block_scales():
    """One id per token, and more tokens than one block looks through for the largest
    coefficient."""
    T, V, D = 5000, 200, 64
    H, W, ids, dlogp = _inputs(T, V, D, 1, seed=9)
    dlogp[3:4000:7] = 0
    logp, lse = _forward(H, W, ids)
    _backward(dlogp, H, W, ids, logp, lse)


@pytest.mark.parametrize("T", [1, 2, 5])
def test_a_row_that_is_no_number(T):
    H, W, ids, _ = _inputs(T, 300, 128, 2)
    H[T - 1] = float("nan")
    logp, lse = ss.logprobs(H, W, ids, ss.logprob_workspace(T, 300, 128))
    assert lse[T - 1].isnan() and logp[T - 1].isnan().all()
    assert lse[:T - 1].isfinite().all() and logp[:T - 1].isfinite().all()
