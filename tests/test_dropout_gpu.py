"""Dropout on the GPU against its definition in 64 bits. What is kept is one
fp32 product (and one addition), then one rounding to the output's type, so a
value is off by at most half a step of that type and two of fp32; what is
dropped is exact."""
import numpy as np
import pytest
import torch

import sampled_softmax_output_gb300 as ss
from block_util import BF, F32, F64, keep_factor, keep_mask

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]


def _x(n, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(n, generator=g, device="cuda").to(dtype)


def _check(y, x, p, seed, residual=None, offset=0):
    f = keep_factor((x.numel(),), p, seed, offset).view(x.shape)
    kept = x.to(F64) * f
    want = kept + (0 if residual is None else residual.to(F64))
    step = BF if y.dtype == torch.bfloat16 else F32
    bound = 1.01 * (step * want.abs() + 3 * F32 * (kept.abs() + want.abs()))
    assert ((y.to(F64) - want).abs() <= bound).all()
    gone = f == 0
    exact = torch.zeros_like(x) if residual is None else residual
    assert torch.equal(y[gone], exact[gone])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 768, 4095, 4097, 100003, 1 << 20])
@pytest.mark.parametrize("p", [0.1, 0.5, 0.999])
def test_values(dtype, n, p):
    x, r = _x(n, dtype, 1), _x(n, dtype, 2)
    _check(ss.dropout(x, p, 11), x, p, 11)
    _check(ss.dropout(x, p, 12, residual=r), x, p, 12, r)
    # the backward makes the same mask
    assert torch.equal(ss.dropout_backward(x, p, 11), ss.dropout(x, p, 11))


@pytest.mark.parametrize("dtype", DTYPES)
def test_ends_of_p(dtype):
    x, r = _x(1003, dtype, 3), _x(1003, dtype, 4)
    assert torch.equal(ss.dropout(x, 0.0, 5), x)
    assert torch.equal(ss.dropout(x, 1.0, 5), torch.zeros_like(x))
    assert torch.equal(ss.dropout(x, 1.0, 5, residual=r), r)
    _check(ss.dropout(x, 2.0 ** -40, 5), x, 2.0 ** -40, 5)  # keeps everything, scale 1
    _check(ss.dropout(x, 1.0 - 2.0 ** -20, 5), x, 1.0 - 2.0 ** -20, 5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset", [1, 2, 5, 8, 2 ** 32 + 3, 2 ** 63 + 2])
def test_pieces_get_the_whole_tensors_mask(dtype, offset):
    x = _x(1000, dtype, 6)
    whole = ss.dropout(x, 0.3, 7, offset=offset)
    _check(whole, x, 0.3, 7, offset=offset)
    for cut in (1, 8, 333):  # pieces that start unaligned, too
        a = ss.dropout(x[:cut], 0.3, 7, offset=offset)
        b = ss.dropout(x[cut:], 0.3, 7, offset=offset + cut)
        assert torch.equal(torch.cat([a, b]), whole)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_alignment_and_neighbours(dtype, shift):
    """Views that start off a 16-byte boundary; nothing beside the output is written."""
    n = 4099
    x, r = _x(n + 8, dtype, 8), _x(n + 8, dtype, 9)
    out = torch.full((n + 16,), 7.0, dtype=dtype, device="cuda")
    ss.dropout(x[shift:shift + n], 0.25, 10, residual=r[shift:shift + n], out=out[shift:shift + n])
    _check(out[shift:shift + n], x[shift:shift + n], 0.25, 10, r[shift:shift + n])
    assert (out[:shift] == 7).all() and (out[shift + n:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place(dtype):
    x, r = _x(5001, dtype, 11), _x(5001, dtype, 12)
    want = ss.dropout(x, 0.2, 13, residual=r)
    y = x.clone()
    assert ss.dropout(y, 0.2, 13, residual=r, out=y) is y and torch.equal(y, want)
    z = r.clone()
    ss.dropout(x, 0.2, 13, residual=z, out=z)
    assert torch.equal(z, want)
    d = x.clone()
    assert torch.equal(ss.dropout_backward(d, 0.2, 13, out=d), ss.dropout_backward(x, 0.2, 13))


def test_nothing_of_a_dropped_element_comes_through():
    n = 4096
    gone = torch.from_numpy(~keep_mask(n, 0.4, 3)).cuda()
    for bad in (float("inf"), float("-inf"), float("nan")):
        x = _x(n, torch.bfloat16, 14)
        x[gone] = bad
        y = ss.dropout(x, 0.4, 3)
        assert (y[gone] == 0).all() and torch.isfinite(y).all()
        kept = x.clone()
        kept[~gone] = bad  # what is kept comes through as it is
        z = ss.dropout(kept, 0.4, 3)[~gone].float()
        assert torch.isnan(z).all() if bad != bad else (z == bad).all()


def test_share_and_independence_of_seeds():
    n = 1 << 22
    x = torch.ones(n, device="cuda")
    masks = [ss.dropout(x, 0.1, s) == 0 for s in (0, 1, 2, 2 ** 64 - 1)]
    for m in masks:  # a binomial's share: 6 standard deviations
        assert abs(m.double().mean().item() - 0.1) < 6 * (0.09 / n) ** 0.5
    for i in range(3):  # both dropped: 0.01
        both = (masks[i] & masks[i + 1]).double().mean().item()
        assert abs(both - 0.01) < 6 * (0.0099 / n) ** 0.5
    pairs = (masks[0][0::2] & masks[0][1::2]).double().mean().item()
    assert abs(pairs - 0.01) < 6 * (0.0099 * 2 / n) ** 0.5


def test_seed_tensor_and_graph_replay():
    x = _x(70001, torch.bfloat16, 15)
    seed = torch.tensor([21], dtype=torch.int64, device="cuda")
    assert torch.equal(ss.dropout(x, 0.1, seed), ss.dropout(x, 0.1, 21))
    out = torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ss.dropout(x, 0.1, seed, out=out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ss.dropout(x, 0.1, seed, out=out)
    for s in (22, -1, 2 ** 62):
        seed.fill_(s)
        g.replay()
        assert torch.equal(out, ss.dropout(x, 0.1, s))


def test_other_stream_and_shapes():
    s = torch.cuda.Stream()
    x = _x(3 * 5 * 7, torch.float32, 16).view(3, 5, 7)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = ss.dropout(x, 0.5, 17)
    s.synchronize()
    assert y.shape == x.shape
    _check(y, x, 0.5, 17)
    assert ss.dropout(x[:0], 0.5, 17).shape == (0, 5, 7)


def test_past_32_bits():
    """More than 2^31 elements: the ends of the tensor against the definition."""
    n = (1 << 31) + 1029
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = ss.dropout(x, 0.5, 18, out=x)
    for lo in (0, (1 << 31) - 512, n - 1029):
        keep = torch.from_numpy(keep_mask(1029, 0.5, 18, lo)).cuda()
        assert torch.equal(y[lo:lo + 1029], keep.to(torch.bfloat16) * 2)


def test_refusals():
    x = _x(64, torch.bfloat16, 19).view(8, 8)
    with pytest.raises(ValueError):
        ss.dropout(x.T, 0.1, 0)  # not contiguous
    with pytest.raises(TypeError):
        ss.dropout(x, 0.1, 0, residual=x.float())
    with pytest.raises(ValueError):
        ss.dropout(x, 0.1, 0, residual=x[:4])
    with pytest.raises(ValueError):
        ss.dropout(x, 0.1, 0, offset=-1)
    with pytest.raises(TypeError):
        ss.dropout(x, 0.1, torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        ss.dropout(x, 0.1, torch.zeros(2, dtype=torch.int64, device="cuda"))
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ss.SSError):
            ss.dropout(x, p, 0)
