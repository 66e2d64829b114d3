"""The gated feed-forward block on the GPU against 64 bits, every element within
the bound that block_util counts from the stated roundings."""
import os
import subprocess
import sys

import pytest
import torch

import sampled_softmax_output_gb300 as ss
from block_util import (ACT, BF, F32, act64, assert_within, backward64, forward64, keep_factor,
                        keep_mask, refined)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

# one token to several tiles, single features, sizes just off a tile's edge, K
# shorter than one k-block and ragged
SIZES = [(1, 8, 8), (1, 768, 2048), (2, 72, 136), (7, 64, 64), (16, 1096, 520), (33, 256, 768),
         (64, 520, 1000), (127, 136, 264), (128, 128, 128), (129, 768, 256), (200, 1032, 2056),
         (255, 256, 264), (256, 768, 2048), (257, 264, 520), (513, 1352, 904), (1003, 392, 2952)]
LARGE = [(4099, 768, 2048), (2050, 2048, 1032), (16384, 264, 520), (70001, 16, 24),
         (1500, 1096, 1280)]


def _inputs(T, D, F, seed=0, residual=True):
    g = torch.Generator("cuda").manual_seed(seed)

    def n(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF16)

    return {"X": n(T, D), "Wg": n(F, D, scale=2 * D ** -0.5), "Wu": n(F, D, scale=D ** -0.5),
            "Wd": n(D, F, scale=F ** -0.5), "residual": n(T, D) if residual else None,
            "dY": n(T, D)}


def _weights(x):
    return x["X"], x["Wg"], x["Wu"], x["Wd"]


def _forward_check(x, act, p=0.0, seed=0, offset=0, save=True, ws=None):
    T, D = x["X"].shape
    F = x["Wg"].shape[0]
    ws = ss.ffn_workspace(T, D, F) if ws is None else ws
    got = ss.ffn_forward(*_weights(x), ws, act=act, residual=x["residual"], p=p, seed=seed,
                         offset=offset, save=save)
    ref = forward64(*_weights(x), act, x["residual"], keep_factor((T, D), p, seed, offset))
    Y, saved = got if save else (got, ())
    assert_within(Y, ref["Y"], "Y")
    for t, name in zip(saved, "GUA"):
        assert_within(t, ref[name], name)
    if save:
        # with their low bits: half a 16th of a step off, a whole one at the end
        # of the nibble's range, next to the sums' own error in `dg`
        G, U, _ = refined(saved)
        for t, name in ((G, "G"), (U, "U")):
            value, bound = ref[name]
            fine = (bound - BF * value.abs()) * 1.01 + BF / 8 * value.abs()
            assert_within(t, (value, fine), name + " with low bits")
    assert ss.read_status(ws)[0] == 0
    return Y, saved


def _backward_check(x, saved, act, p=0.0, seed=0, offset=0, dw_dtype=torch.float32, ws=None):
    T, D = x["X"].shape
    F = x["Wg"].shape[0]
    ws = ss.ffn_workspace(T, D, F) if ws is None else ws
    g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, act=act, p=p, seed=seed, offset=offset,
                        dw_dtype=dw_dtype)
    used = refined(saved) if isinstance(saved, ss.FfnSaved) else saved
    ref = backward64(x["dY"], *_weights(x), used, act, keep_factor((T, D), p, seed, offset),
                     dw_dtype == torch.float32)
    for k in ("dX", "dWg", "dWu", "dWd"):
        assert g[k].dtype == (BF16 if k == "dX" else dw_dtype)
        assert_within(g[k], ref[k], k)
    assert ss.read_status(ws)[0] == 0
    return g


@pytest.mark.parametrize("size", SIZES)
def test_forward(size):
    x = _inputs(*size)
    Y, _ = _forward_check(x, "silu")
    only, _ = _forward_check(x, "silu", save=False)  # nothing kept: the same result
    assert torch.equal(only, Y)


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dw_dtype", [torch.float32, BF16])
def test_backward(size, dw_dtype):
    x = _inputs(*size, seed=1)
    T, D, F = size
    _, saved = ss.ffn_forward(*_weights(x), ss.ffn_workspace(T, D, F), save=True)
    _backward_check(x, saved, "silu", dw_dtype=dw_dtype)


@pytest.mark.parametrize("size", [(3, 72, 136), (130, 264, 392), (1500, 768, 1288),
                                  (1500, 1096, 1280)])
def test_backward_from_plain_tensors(size):
    """Any G, U and A, without low bits."""
    x = _inputs(*size, seed=20)
    _, saved = ss.ffn_forward(*_weights(x), ss.ffn_workspace(*size), save=True)
    plain = tuple(t.clone() for t in saved)
    _backward_check(x, plain, "gelu")
    with_low = _backward_check(x, saved, "gelu")
    stacked = torch.stack(plain)
    again = ss.ffn_backward(x["dY"], *_weights(x), stacked, ss.ffn_workspace(*size), act="gelu")
    ref = backward64(x["dY"], *_weights(x), plain, "gelu")
    assert_within(again["dX"], ref["dX"], "dX")
    assert not torch.equal(again["dWg"], with_low["dWg"])


def test_step_is_nearer_to_64_bits_with_low_bits():
    """A bf16 rounding is spread evenly over a step of 2^-8 to 2^-7 of the value:
    an error of at most 2^-7 / sqrt(12) of the norm. With the low bits dG's is the
    only one in dWg (fp32); without them U's, as large and independent, comes on
    top: sqrt(2) times that and more."""
    T, D, F = 600, 264, 392
    x = _inputs(T, D, F, seed=21)
    ws = ss.ffn_workspace(T, D, F)
    _, saved = ss.ffn_forward(*_weights(x), ws, save=True)
    exact = forward64(*_weights(x), "silu")
    ref = backward64(x["dY"], *_weights(x), [exact[k][0] for k in "GUA"], "silu")["dWg"][0]

    def err(s):
        g = ss.ffn_backward(x["dY"], *_weights(x), s, ws)["dWg"].double()
        return float((g - ref).norm() / ref.norm())

    assert err(saved) < 2.0 ** -7 / 12 ** 0.5 and err(tuple(saved)) > 1.2 * err(saved)


@pytest.mark.parametrize("size", LARGE)
def test_large(size):
    x = _inputs(*size, seed=2)
    ws = ss.ffn_workspace(*size)
    _, saved = _forward_check(x, "gelu_tanh", p=0.1, seed=5, ws=ws)
    _backward_check(x, saved, "gelu_tanh", p=0.1, seed=5, ws=ws)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("size", [(5, 72, 200), (300, 264, 392), (2100, 776, 1288)])
def test_activations(act, size):
    x = _inputs(*size, seed=3)
    x["Wg"] *= 4  # gates far out on both sides
    _, saved = _forward_check(x, act)
    _backward_check(x, saved, act)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("T", [1, 300])
def test_tails(act, T):
    """act(g) to its own digits where it is tiny. With X, Wd and one column of dY of
    ones in row 0, dWu is act(G) and dWg act'(G), rounded to bf16 once. An
    exponential's argument of size E has three roundings: 3 F32 E of the value."""
    D, F = 8, 2048
    G = torch.zeros(T, F, dtype=BF16, device="cuda")
    G[0] = torch.linspace(-13, 13, F, device="cuda").to(BF16)
    X, dY = torch.ones(T, D, dtype=BF16, device="cuda"), torch.zeros(T, D, device="cuda")
    dY[0, 3] = 1
    W, Wd = torch.ones(F, D, dtype=BF16, device="cuda"), torch.ones(D, F, dtype=BF16, device="cuda")
    g = ss.ffn_backward(dY.to(BF16), X, W, W, Wd, (G, torch.ones_like(G), G),
                        ss.ffn_workspace(T, D, F), act=act)
    x = G[0].double()
    a, d = act64(x, act)
    E = {"silu": x.abs(), "gelu": x * x / 2, "relu": 0 * x,
         "gelu_tanh": 1.6 * (x + 0.044715 * x ** 3).abs()}[act]
    rel = ACT + 3 * F32 * E
    for k in range(D):
        assert_within(g["dWu"][:, k], (a, (BF + 1.01 * rel) * a.abs()), "act")
        # the slope: two terms of at most 1 + |g|
        fine = 2 * ACT * (1 + x.abs())
        assert_within(g["dWg"][:, k], (d, BF * d.abs() + 1.01 * fine), "slope")


@pytest.mark.parametrize("size", [(3, 64, 72), (130, 264, 392), (1500, 768, 1288)])
@pytest.mark.parametrize("p,offset", [(0.1, 0), (0.5, 7), (1.0, 0), (0.25, 2 ** 40 + 1)])
def test_dropout(size, p, offset):
    x = _inputs(*size, seed=4)
    _, saved = _forward_check(x, "silu", p, 9, offset)
    _backward_check(x, saved, "silu", p, 9, offset)
    x["residual"] = None
    _forward_check(x, "silu", p, 9, offset, save=False)


def test_dropout_is_that_of_the_operator():
    """The block's dropout equals ss.dropout over the undropped output."""
    x = _inputs(300, 264, 392, seed=5, residual=False)
    ws = ss.ffn_workspace(300, 264, 392)
    Z = ss.ffn_forward(*_weights(x), ws)
    Y = ss.ffn_forward(*_weights(x), ws, p=0.3, seed=6)
    kept = torch.from_numpy(keep_mask(Z.numel(), 0.3, 6)).cuda().view(Z.shape)
    assert torch.equal(Y == 0, ss.dropout(Z, 0.3, 6) == 0)
    assert (Y[~kept] == 0).all()


def test_poison_in_dropped_gradients_stays_out():
    x = _inputs(200, 264, 392, seed=6)
    ws = ss.ffn_workspace(200, 264, 392)
    _, saved = ss.ffn_forward(*_weights(x), ws, p=0.4, seed=3, save=True)
    clean = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, p=0.4, seed=3)
    gone = torch.from_numpy(~keep_mask(200 * 264, 0.4, 3)).cuda().view(200, 264)
    for bad in (float("nan"), float("inf")):
        dY = x["dY"].masked_fill(gone, bad)
        g = ss.ffn_backward(dY, *_weights(x), saved, ws, p=0.4, seed=3)
        for k in g:
            assert torch.equal(g[k], clean[k]), k


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("T", [4, 700])
def test_extreme_gates(act, T):
    """Gates up to the edge of bf16: the slope is finite there, no 0 times infinity."""
    D, F = 64, 136
    x = _inputs(T, D, F, seed=7, residual=False)
    ws = ss.ffn_workspace(T, D, F)
    # (in 64 bits: the range itself is past what 32 hold)
    G = torch.linspace(-3e38, 3e38, T * F, device="cuda", dtype=torch.float64).view(T, F).to(BF16)
    G[0, :4] = torch.tensor([0.0, -0.0, 1e30, -1e30])
    U = torch.ones_like(G)
    A = torch.zeros_like(G)
    g = ss.ffn_backward(x["dY"], *_weights(x), (G, U, A), ws, act=act)
    assert torch.isfinite(g["dWg"]).all()


@pytest.mark.parametrize("size", [(3, 72, 136), (260, 264, 392), (1100, 768, 1288)])
def test_accumulate(size):
    T, D, F = size
    x = _inputs(*size, seed=8)
    ws = ss.ffn_workspace(*size)
    _, saved = ss.ffn_forward(*_weights(x), ws, save=True)
    for dt in (torch.float32, BF16):
        once = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, dw_dtype=dt)
        base = {k: torch.randn_like(once[k].float()).to(dt) for k in ("dWg", "dWu", "dWd")}
        into = {k: v.clone() for k, v in base.items()}
        g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, dw_dtype=dt, accumulate=True, **into)
        f32 = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, dw_dtype=torch.float32)
        for k in base:
            assert g[k] is into[k]
            want = base[k].double() + f32[k].double()
            step = torch.finfo(dt).eps / 2
            assert ((g[k].double() - want).abs() <= 1.01 * step * want.abs() + 1e-6).all(), k
        new = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, dw_dtype=dt, accumulate=True)
        for k in base:
            assert torch.equal(new[k], once[k])


def test_deterministic():
    x = _inputs(777, 520, 1032, seed=9)
    ws = ss.ffn_workspace(777, 520, 1032)
    runs = []
    for _ in range(3):
        Y, saved = ss.ffn_forward(*_weights(x), ws, p=0.1, seed=1, save=True)
        g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, p=0.1, seed=1)
        runs.append([Y, *saved, *g.values()])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("T", [1, 5, 100, 130, 600, 2100])
@pytest.mark.parametrize("shift", [0, 8])
@pytest.mark.parametrize("D,F", [(264, 392), (272, 1040)])
def test_rows_behind_the_last_stay(T, shift, D, F):
    """Rows behind the batch keep what they held; buffers on 16-byte boundaries
    that are no 32-byte ones give the same results (shift = 8 values)."""
    x = _inputs(T, D, F, seed=10)
    ws = ss.ffn_workspace(T, D, F)
    L = ss.lib()
    bufs = {k: torch.full(((T + 300) * w + 8,), 7.0, dtype=BF16, device="cuda")[shift:][
        :(T + 300) * w].view(T + 300, w)
            for k, w in (("Y", D), ("G", F), ("U", F), ("A", F), ("dX", D))}
    ptr = {k: v.data_ptr() for k, v in {**x, **bufs}.items()}
    s = torch.cuda.current_stream().cuda_stream
    assert L.ss_ffn_forward(ptr["X"], ptr["Wg"], ptr["Wu"], ptr["Wd"], ptr["residual"], T, D, F, 0,
                            None, ptr["Y"], ptr["G"], ptr["U"], ptr["A"], None, ws.data_ptr(),
                            ws.numel(), s) == 0
    dW = [torch.empty(F * D, device="cuda") for _ in range(3)]
    assert L.ss_ffn_backward(ptr["dY"], ptr["X"], ptr["Wg"], ptr["Wu"], ptr["Wd"], ptr["G"],
                             ptr["U"], ptr["A"], None, T, D, F, 0, None, 1, 0, ptr["dX"],
                             *(w.data_ptr() for w in dW), ws.data_ptr(), ws.numel(), s) == 0
    torch.cuda.synchronize()
    for k, b in bufs.items():
        assert (b[T:] == 7).all(), k
    saved = [bufs[k][:T] for k in "GUA"]
    ref = forward64(*_weights(x), "silu", x["residual"])
    for k in "YGUA":
        assert_within(bufs[k][:T], ref[k], k)
    ref = backward64(x["dY"], *_weights(x), saved, "silu")
    assert_within(bufs["dX"][:T], ref["dX"], "dX")
    for w, k, shape in zip(dW, ("dWg", "dWu", "dWd"), ((F, D), (F, D), (D, F))):
        assert_within(w.view(shape), ref[k], k)


def test_residual_in_place_and_empty_batch():
    x = _inputs(100, 264, 392, seed=11)
    ws = ss.ffn_workspace(100, 264, 392)
    want = ss.ffn_forward(*_weights(x), ws, residual=x["residual"], p=0.1, seed=2)
    r = x["residual"].clone()
    assert ss.ffn_forward(*_weights(x), ws, residual=r, p=0.1, seed=2, out=r) is r
    assert torch.equal(r, want)
    e = _inputs(0, 264, 392)
    Y, saved = ss.ffn_forward(*_weights(e), ws, residual=e["residual"], save=True)
    assert Y.shape == (0, 264) and saved[0].shape == (0, 392)
    g = ss.ffn_backward(e["dY"], *_weights(e), saved, ws)
    assert g["dX"].shape == (0, 264)
    assert all((g[k] == 0).all() for k in ("dWg", "dWu", "dWd"))
    kept = torch.ones(392, 264, device="cuda")
    g = ss.ffn_backward(e["dY"], *_weights(e), saved, ws, accumulate=True, dWg=kept)
    assert (g["dWg"] == 1).all()


@pytest.mark.parametrize("T", [3, 260, 1100])
def test_captured_step_draws_new_masks(T):
    """Forward and backward in one graph, replayed with other seeds and inputs."""
    D, F = 264, 392
    x = _inputs(T, D, F, seed=12)
    ws, ws2 = ss.ffn_workspace(T, D, F), ss.ffn_workspace(T, D, F)
    seed = torch.tensor([1], dtype=torch.int64, device="cuda")

    def step(s, w):
        Y, saved = ss.ffn_forward(*_weights(x), w, residual=x["residual"], p=0.2, seed=s, save=True)
        g = ss.ffn_backward(x["dY"], *_weights(x), saved, w, p=0.2, seed=s)
        return [Y, *g.values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(seed, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(seed, ws)
    for k in (2, 3):
        seed.fill_(k)
        fresh = _inputs(T, D, F, seed=12 + k)
        x["X"].copy_(fresh["X"])
        x["dY"].copy_(fresh["dY"])
        graph.replay()
        want = step(k, ws2)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_first_call_of_a_process_may_be_captured():
    """No warm-up: the kernels are loaded while the stream is being captured."""
    code = """
import torch, sampled_softmax_output_gb300 as ss
g = torch.Generator("cuda").manual_seed(1)
n = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
for T, D, F in ((3, 64, 72), (2100, 272, 1040)):
    X, Wg, Wu, Wd, dY = n(T, D), n(F, D), n(F, D), n(D, F), n(T, D)
    ws = ss.ffn_workspace(T, D, F)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y, saved = ss.ffn_forward(X, Wg, Wu, Wd, ws, p=0.1, seed=2, save=True)
        out = ss.ffn_backward(dY, X, Wg, Wu, Wd, saved, ws, p=0.1, seed=2)
        Z = ss.dropout(Y, 0.5, 3)
    graph.replay()
    Y2, saved2 = ss.ffn_forward(X, Wg, Wu, Wd, ws, p=0.1, seed=2, save=True)
    out2 = ss.ffn_backward(dY, X, Wg, Wu, Wd, saved2, ws, p=0.1, seed=2)
    assert torch.equal(Y, Y2) and torch.equal(Z, ss.dropout(Y2, 0.5, 3))
    assert all(torch.equal(out[k], out2[k]) for k in out)
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_smaller_batches_share_a_workspace_and_other_streams():
    D, F = 264, 392
    ws = ss.ffn_workspace(700, D, F)
    s = torch.cuda.Stream()
    for T in (700, 1, 130, 16, 699):
        x = _inputs(T, D, F, seed=T)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            _, saved = _forward_check(x, "silu", ws=ws)
            _backward_check(x, saved, "silu", ws=ws)
        torch.cuda.current_stream().wait_stream(s)


@pytest.mark.parametrize("size,passes", [((8192, 1024, 5504), 6), ((3001, 1352, 3640), 20),
                                         ((8192, 768, 5504), 6)])
def test_many_tiles_to_a_pair(size, passes):
    """Long runs of tiles, buffers that are used again and again under the load of
    the products: within the bounds, and the same bits every time."""
    x = _inputs(*size, seed=24)
    ws = ss.ffn_workspace(*size)
    _, saved = _forward_check(x, "silu", p=0.1, seed=6, ws=ws)
    want = _backward_check(x, saved, "silu", p=0.1, seed=6, ws=ws)
    for _ in range(passes):
        _, again = ss.ffn_forward(*_weights(x), ws, p=0.1, seed=6, save=True)
        assert all(torch.equal(a, b) for a, b in zip([*again, again.low_bits()],
                                                     [*saved, saved.low_bits()]))
        for kept in (saved, again):
            g = ss.ffn_backward(x["dY"], *_weights(x), kept, ws, p=0.1, seed=6)
            assert all(torch.equal(g[k], want[k]) for k in want)


def test_past_32_bits():
    """[T, F] of more than 2^32 values: the first and the last rows. dY is zero
    between them, so that they alone make the weight gradients."""
    T, D, F, n = 600_001, 64, 8192, 150
    x = _inputs(T, D, F, seed=22)
    x["dY"][n:-n] = 0
    ws = ss.ffn_workspace(T, D, F)
    Y, saved = ss.ffn_forward(*_weights(x), ws, residual=x["residual"], p=0.1, seed=3, save=True)
    g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, p=0.1, seed=3)
    assert ss.read_status(ws)[0] == 0
    ends = torch.cat([torch.arange(n), torch.arange(T - n, T)]).cuda()
    factor = torch.cat([keep_factor((n, D), 0.1, 3), keep_factor((n, D), 0.1, 3, (T - n) * D)])
    part = {k: x[k][ends] for k in ("X", "residual", "dY")}
    part.update({k: x[k] for k in ("Wg", "Wu", "Wd")})
    kept = [t[ends] for t in saved]
    ref = forward64(*_weights(part), "silu", part["residual"], factor)
    assert_within(Y[ends], ref["Y"], "Y")
    for t, name in zip(kept, "GUA"):
        assert_within(t, ref[name], name)
    low = saved.low_bits()[ends]
    ref = backward64(part["dY"], *_weights(part), refined(kept, low), "silu", factor)
    assert_within(g["dX"][ends], ref["dX"], "dX")
    assert (g["dX"][n:-n] == 0).all()
    for k in ("dWg", "dWu", "dWd"):
        assert_within(g[k], ref[k], k)


@pytest.mark.parametrize("sizes", [((3, 264, 392), (5, 264, 392)),
                                   ((300, 264, 392), (2100, 776, 1288)),
                                   ((2100, 1096, 1288), (16, 2048, 1032))])
@pytest.mark.parametrize("graphs", [False, True])
def test_two_at_once(sizes, graphs):
    """Two blocks on two streams, eager or as captured graphs, a workspace each:
    what each gives alone."""
    blocks, streams = [], [torch.cuda.Stream() for _ in sizes]
    for size in sizes:
        x = _inputs(*size, seed=23)
        blocks.append((x, ss.ffn_workspace(*size)))

    def step(x, ws):
        Y, saved = ss.ffn_forward(*_weights(x), ws, residual=x["residual"], p=0.1, seed=4,
                                  save=True)
        g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, p=0.1, seed=4)
        return [ss.dropout(Y, 0.2, 5), *g.values()]

    want = [[t.clone() for t in step(*b)] for b in blocks]
    torch.cuda.synchronize()
    got = [None, None]
    if graphs:
        made = []
        for b, s in zip(blocks, streams):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                made.append((graph, step(*b)))
        got = [out for _, out in made]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if graphs:
                    made[i][0].replay()
                else:
                    got[i] = step(*blocks[i])
    torch.cuda.synchronize()
    for (x, ws), outs, ref in zip(blocks, got, want):
        assert ss.read_status(ws)[0] == 0
        assert all(torch.equal(a, b) for a, b in zip(outs, ref))


def test_gradients_against_differences():
    """<gradient, direction> against central differences of the forward in 64
    bits. The differences are off by the third derivative's h^2 (h = 1e-4: below
    1e-6 of the slope here); the gradients are bf16 results within 2^-7 of
    their norms, and a random direction is near the gradient's own."""
    T, D, F = 40, 72, 136
    x = _inputs(T, D, F, seed=13, residual=False)
    ws = ss.ffn_workspace(T, D, F)
    _, saved = ss.ffn_forward(*_weights(x), ws, act="gelu", p=0.2, seed=4, save=True)
    g = ss.ffn_backward(x["dY"], *_weights(x), saved, ws, act="gelu", p=0.2, seed=4)
    factor = keep_factor((T, D), 0.2, 4)
    names = ("X", "Wg", "Wu", "Wd")

    def loss(w):
        return float((forward64(*w, "gelu", None, factor)["Y"][0] * x["dY"].double()).sum())

    for i, k in enumerate(names):
        v = g["d" + k].double()
        v = v / v.norm()
        h = 1e-4
        w = [x[n].double() for n in names]
        up, down = list(w), list(w)
        up[i], down[i] = w[i] + h * v, w[i] - h * v
        slope = (loss(up) - loss(down)) / (2 * h)
        assert abs(slope - float(g["d" + k].double().norm())) <= 2.0 ** -7 * abs(slope), k


def test_block_in_front_of_the_head():
    """Block, head and back, as a training step runs them: the block's output is
    the head's H, the head's dH the block's dY; the loss's slope along the
    gradient against differences of the whole in 64 bits."""
    T, D, F, V, C = 96, 128, 264, 500, 300
    x = _inputs(T, D, F, seed=14)
    g = torch.Generator("cuda").manual_seed(15)
    W = (torch.randn(V, D, generator=g, device="cuda") * 0.2).to(BF16)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    ws, head_ws = ss.ffn_workspace(T, D, F), ss.workspace(T, V, C, D)
    H, saved = ss.ffn_forward(*_weights(x), ws, residual=x["residual"], p=0.1, seed=16, save=True)
    out = ss.step(H, W, targets, C, 17, head_ws, scale=1.0)
    grads = ss.ffn_backward(out["dH"], *_weights(x), saved, ws, p=0.1, seed=16)
    torch.cuda.synchronize()
    assert ss.read_status(ws)[0] == 0 and ss.read_status(head_ws)[0] == 0
    factor = keep_factor((T, D), 0.1, 16)
    Wc = W[out["cand"].long()].double()
    slot = out["slot"].long()

    def loss(X):
        Y = forward64(X, x["Wg"], x["Wu"], x["Wd"], "silu", x["residual"], factor)["Y"][0]
        S = Y @ Wc.T
        return float((torch.logsumexp(S, 1) - S.gather(1, slot[:, None])[:, 0]).sum())

    assert abs(float(out["loss"].double().sum()) - loss(x["X"].double())) <= 1e-2 * abs(
        loss(x["X"].double()))
    v = grads["dX"].double()
    n = float(v.norm())
    h = 1e-4
    X = x["X"].double()
    slope = (loss(X + h * v / n) - loss(X - h * v / n)) / (2 * h)
    # H, dH, dG, dU and dX are each rounded to bf16: five half steps of 2^-8
    assert abs(slope - n) <= 5 * 2.0 ** -8 * abs(slope)


def test_refusals():
    x = _inputs(16, 64, 72)
    ws = ss.ffn_workspace(16, 64, 72)
    X, Wg, Wu, Wd = _weights(x)
    with pytest.raises(ValueError):
        ss.ffn_forward(X, Wg, Wu, Wd, ws, act="tanh")
    with pytest.raises(ValueError):
        ss.ffn_forward(X, Wg, Wu[:64], Wd, ws)
    with pytest.raises(ValueError):
        ss.ffn_forward(X, Wg, Wu, Wd.T, ws)
    with pytest.raises(ValueError):
        ss.ffn_forward(X.view(2, 8, 64), Wg, Wu, Wd, ws)
    with pytest.raises(TypeError):
        ss.ffn_forward(X, Wg, Wu, Wd, ws, residual=X.float())
    with pytest.raises(ss.SSError):
        ss.ffn_forward(X, Wg, Wu, Wd, ws[:-1024])
    with pytest.raises(ss.SSError):
        ss.ffn_forward(X, Wg, Wu, Wd, ws, p=2.0)
    with pytest.raises(ss.SSError):
        w = torch.zeros(70, 64, dtype=BF16, device="cuda")
        ss.ffn_forward(X, w, w, torch.zeros(64, 70, dtype=BF16, device="cuda"), ws)
    _, saved = ss.ffn_forward(X, Wg, Wu, Wd, ws, save=True)
    with pytest.raises(ValueError):
        ss.ffn_backward(x["dY"][:8], X, Wg, Wu, Wd, saved, ws)
    with pytest.raises(ValueError):
        ss.ffn_backward(x["dY"], X, Wg, Wu, Wd, (saved[0], saved[1], saved[2][:, :64]), ws)
    _, other = ss.ffn_forward(X[:8], Wg, Wu, Wd, ws, save=True)
    with pytest.raises(ValueError):
        ss.ffn_backward(x["dY"], X, Wg, Wu, Wd, other, ws)
    with pytest.raises(IndexError):
        saved[3]
    with pytest.raises(TypeError):
        ss.ffn_backward(x["dY"], X, Wg, Wu, Wd, saved, ws, dw_dtype=torch.float16)
    with pytest.raises(TypeError):
        ss.ffn_backward(x["dY"], X, Wg, Wu, Wd, saved, ws, dWg=torch.zeros_like(Wg))
