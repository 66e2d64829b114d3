"""A workspace whose status word holds an error: calls of the feed-forward block
write none of their outputs until its header is zeroed, on either family of
kernels. (The word is set from the host; no device wait runs out here.)"""
import pytest
import torch

import sampled_softmax_output_gb300 as ss
from test_ffn_gpu import _backward_check, _forward_check, _inputs, _weights

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
TIMEOUT = 7


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("size", [(1, 768, 2048), (24, 264, 392), (130, 768, 1032),
                                  (257, 768, 2048), (2100, 1096, 1280), (2100, 776, 1288)])
def test_outputs_stay_until_the_header_is_zeroed(size, p):
    T, D, F = size
    x = _inputs(T, D, F, seed=30)
    ws = ss.ffn_workspace(T, D, F)
    _, saved = ss.ffn_forward(*_weights(x), ws, p=p, seed=1, save=True)
    word = ws[:4].view(torch.int32)
    word.fill_(TIMEOUT)

    # Y in the residual's place: an input that must survive
    residual = x["residual"].clone()
    ss.ffn_forward(*_weights(x), ws, residual=residual, p=p, seed=1, out=residual)
    assert torch.equal(residual, x["residual"])
    kept = {k: torch.full((T + 1, w), 7.0, dtype=BF16, device="cuda")
            for k, w in (("Y", D), ("G", F), ("U", F), ("A", F))}
    low = torch.full((T, ss.lib().ss_ffn_low_bits_pitch(F)), 7, dtype=torch.uint8, device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    assert ss.lib().ss_ffn_forward(*(t.data_ptr() for t in _weights(x)), None, T, D, F, 0, None,
                                   kept["Y"].data_ptr(), kept["G"].data_ptr(),
                                   kept["U"].data_ptr(), kept["A"].data_ptr(), low.data_ptr(),
                                   ws.data_ptr(), ws.numel(), s) == 0
    for k, t in kept.items():
        assert (t == 7).all(), k
    assert (low == 7).all()

    for dt in (torch.float32, BF16):
        for accumulate in (False, True):
            out = {"dX": torch.full((T, D), 3.0, dtype=BF16, device="cuda")}
            for k, shape in (("dWg", (F, D)), ("dWu", (F, D)), ("dWd", (D, F))):
                out[k] = torch.full(shape, 3.0, dtype=dt, device="cuda")
            ss.ffn_backward(x["dY"], *_weights(x), saved, ws, p=p, seed=1, dw_dtype=dt,
                            accumulate=accumulate, **out)
            for k, t in out.items():
                assert (t == 3).all(), k
    assert ss.read_status(ws)[0] == TIMEOUT

    ws[:ss.WORKSPACE_HEADER_BYTES].zero_()
    _, saved = _forward_check(x, "silu", p=p, seed=1, ws=ws)
    _backward_check(x, saved, "silu", p=p, seed=1, ws=ws)
