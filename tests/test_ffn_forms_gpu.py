"""The feed-forward block in every form that its choice of kernels has, against 64
bits (test_ffn_plan_host.py: that these sizes reach them all)."""
import concurrent.futures

import pytest
import torch

import sampled_softmax_output_gb300 as ss
from block_util import BF, keep_mask, refined
from ffn_plan import ACT_SIZES, FORM_SIZES
from test_ffn_gpu import _backward_check, _forward_check, _inputs, _weights

pytestmark = pytest.mark.gpu
ACTS = sorted(ss.ACTS)


@pytest.mark.parametrize("k,size", list(enumerate(FORM_SIZES)))
def test_forms(k, size):
    x = _inputs(*size, seed=40 + k)
    act = ACTS[k % 4]
    ws = ss.ffn_workspace(*size)
    Y, saved = _forward_check(x, act, p=0.1, seed=k, ws=ws)
    only, _ = _forward_check(x, act, p=0.1, seed=k, save=False, ws=ws)
    assert torch.equal(only, Y)
    _backward_check(x, saved, act, p=0.1, seed=k, ws=ws)


@pytest.mark.parametrize("T", [17, 24, 31, 32])
@pytest.mark.parametrize("D,F", [(264, 520), (1096, 392), (768, 2048)])
@pytest.mark.parametrize("dw_dtype", [torch.float32, torch.bfloat16])
def test_17_to_32_tokens(T, D, F, dw_dtype):
    """With and without low bits, with and without dropout."""
    x = _inputs(T, D, F, seed=T)
    ws = ss.ffn_workspace(T, D, F)
    _, saved = _forward_check(x, "silu", ws=ws)
    _backward_check(x, saved, "silu", dw_dtype=dw_dtype, ws=ws)
    _backward_check(x, tuple(t.clone() for t in saved), "silu", p=0.3, seed=2, offset=5,
                    dw_dtype=dw_dtype, ws=ws)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("size", ACT_SIZES)
def test_activations_on_pairs(act, size):
    x = _inputs(*size, seed=3)
    x["Wg"] *= 4  # gates far out on both sides
    ws = ss.ffn_workspace(*size)
    _, saved = _forward_check(x, act, ws=ws)
    _backward_check(x, saved, act, ws=ws)
    _backward_check(x, tuple(t.clone() for t in saved), act, ws=ws)


@pytest.mark.parametrize("size", [(2, 16384, 8), (2, 8, 65536), (300, 16384, 8), (300, 8, 65536)])
def test_widest(size):
    """SS_MAX_D and SS_MAX_F."""
    x = _inputs(*size, seed=41)
    _, saved = _forward_check(x, "gelu", p=0.1, seed=1)
    _backward_check(x, saved, "gelu", p=0.1, seed=1)


@pytest.mark.parametrize("T", [5, 300, 2100])
def test_kept_values_are_those_of_dropout(T):
    """The block's dropout against ss.dropout over the undropped output, value by
    value. The sums are the same; Z is rounded, its dropout once more, and Y once:
    three half steps."""
    x = _inputs(T, 264, 392, seed=5, residual=False)
    ws = ss.ffn_workspace(T, 264, 392)
    Z = ss.ffn_forward(*_weights(x), ws)
    Y = ss.ffn_forward(*_weights(x), ws, p=0.3, seed=6).double()
    want = ss.dropout(Z, 0.3, 6).double()
    kept = torch.from_numpy(keep_mask(Z.numel(), 0.3, 6)).cuda().view(Z.shape)
    assert torch.equal(Y[~kept], want[~kept])
    assert ((Y - want).abs() <= 3.1 * BF * torch.maximum(Y.abs(), want.abs()) + 1e-37).all()


@pytest.mark.parametrize("size", [(512, 2048, 24320), (339, 4040, 11680)])
def test_more_than_2048_units(size):
    """dX and dW in one launch of CTA pairs: few long units beside thousands of
    short ones."""
    x = _inputs(*size, seed=42)
    ws = ss.ffn_workspace(*size)
    _, saved = ss.ffn_forward(*_weights(x), ws, save=True)
    want = _backward_check(x, saved, "silu", ws=ws)
    for _ in range(3):
        g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws)
        assert all(torch.equal(g[k], want[k]) for k in want)


@pytest.mark.parametrize("T", [3, 2100])
def test_low_bits_around_zero(T):
    """Sums of either sign that round to a zero or to bf16's smallest values: with
    their low bits they are off by half a 16th of a step of 2^-133, but half a step
    above an even bf16 (a tie, rounded down) is 16 16ths' place in a half byte that
    ends at 15: there by a whole 16th, 2^-137. (The 256th more of (n - 8) 16ths
    that the second half byte adds is below 2^-141: 1.01 covers it.) Or nothing is
    left out where the products themselves were flushed to zero."""
    D, F = 8, 256
    X, W = torch.zeros(T, D, device="cuda"), torch.zeros(F, D, device="cuda")
    X[:, 0] = 2.0 ** -60
    # sums k 2^-137, k = -128 .. 127: up to four steps
    k = torch.arange(F, device="cuda") - F // 2
    W[:, 0] = k * 2.0 ** -77
    W = W.to(torch.bfloat16)
    _, saved = ss.ffn_forward(X.to(torch.bfloat16), W, W, torch.ones(D, F, device="cuda").to(
        torch.bfloat16), ss.ffn_workspace(T, D, F), save=True)
    exact = k.double() * 2.0 ** -137
    bound = torch.where(k.abs() % 32 == 8, 2.0 ** -137, 2.0 ** -138)
    G, U, _ = refined(saved)
    for fine, bf in ((G, saved[0]), (U, saved[1])):
        off = (fine.double() - exact).abs()
        flushed = (bf == 0) & (fine == 0)
        assert ((off <= 1.01 * bound) | flushed).all()


def test_two_host_threads():
    """Calls of two threads at once, a stream and a workspace each."""
    sizes = [(300, 264, 392), (2100, 776, 1288)]
    blocks = [(_inputs(*s, seed=43), ss.ffn_workspace(*s), torch.cuda.Stream()) for s in sizes]

    def step(x, ws):
        Y, saved = ss.ffn_forward(*_weights(x), ws, residual=x["residual"], p=0.1, seed=4,
                                  save=True)
        g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, p=0.1, seed=4)
        return [ss.dropout(Y, 0.2, 5), *g.values()]

    want = [step(x, ws) for x, ws, _ in blocks]
    torch.cuda.synchronize()

    def run(block):
        x, ws, stream = block
        with torch.cuda.stream(stream):
            outs = [step(x, ws) for _ in range(30)]
            stream.synchronize()
        return outs

    with concurrent.futures.ThreadPoolExecutor(2) as ex:
        got = list(ex.map(run, blocks))
    for (_, ws, _), outs, ref in zip(blocks, got, want):
        assert ss.read_status(ws)[0] == 0
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
