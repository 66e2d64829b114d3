"""Host-side checks of include/ss_logprob.h: exported symbols, workspace sizes, and
arguments refused before the device is touched (the fake device addresses are never
dereferenced)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sampled_softmax_output_gb300 as ss

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
FAKE = 0x7F0000000000
p = ctypes.c_void_p


def test_exports_every_declared_symbol():
    names = ss.header_symbols(ss.HEADER_LOGPROB)
    assert set(names) == {"ss_logprob_workspace_size", "ss_logprob_forward",
                          "ss_logprob_backward", "ss_policy_loss", "ss_preference_loss",
                          "ss_distill_loss"}
    for n in names:
        assert hasattr(ss.lib(), n), n


def test_workspace_size():
    f = ss.lib().ss_logprob_workspace_size
    n = f(1000, 50257, 768, 1)
    assert n >= 1024 + 1000 * 50304 * 2 + 1000 * 768 * 2 and n % 1024 == 0
    small = f(1000, 50257, 768, 0)
    assert 1000 * 2 * 197 * 8 < small < n // 10
    assert f(0, 1, 64, 1) == 1024 and f(999, 50257, 768, 1) <= n
    for bad in ((-1, 10, 64), (1, 0, 64), (1, 10, 0), (1, 10, 96), (1, 10, 16448),
                (1, 524289, 64), (1 << 31, 10, 64), (1 << 30, 524288, 64)):
        assert f(*bad, 1) == 0, bad
    with pytest.raises(ss.SSError):
        ss.logprob_workspace_size(1, 10, 96)


FWD = ("H", "W", "ids", "K", "T", "V", "D", "head", "logp", "lse", "ws", "wsb")
BWD = ("dlogp", "H", "W", "ids", "logp", "lse", "K", "T", "V", "D", "head", "dw", "acc", "dH",
       "dW", "ws", "wsb")
PLAIN = ("K", "T", "V", "D", "dw", "acc", "wsb")


def _call(fn, names, **kw):
    a = {n: FAKE for n in names}
    a.update(K=1, T=64, V=1000, D=128, head=None, dw=1, acc=0, wsb=1 << 40)
    a.update(kw)
    args = [a[n] if n in PLAIN else (None if a[n] is None else ctypes.byref(a[n]))
            if n == "head" else p(a[n]) for n in names]
    return getattr(ss.lib(), fn)(*args, None)


def _fwd(**kw):
    return _call("ss_logprob_forward", FWD, **kw)


def _bwd(**kw):
    return _call("ss_logprob_backward", BWD, **kw)


@pytest.mark.parametrize("fn,backward", [(_fwd, 0), (_bwd, 1)])
def test_logprob_argument_errors(fn, backward):
    assert fn(T=-1) == INVALID and fn(V=0) == INVALID and fn(D=0) == INVALID and fn(K=0) == INVALID
    assert fn(T=1 << 31) == UNSUPPORTED and fn(V=524289) == UNSUPPORTED
    assert fn(D=100) == UNSUPPORTED and fn(D=16448) == UNSUPPORTED and fn(K=129) == UNSUPPORTED
    assert fn(head=ss.Head(0.0, 1.0, 1)) == UNSUPPORTED
    assert fn(head=ss.Head(0.0, 1.0, 3)) == INVALID
    for cap, tau in ((-1.0, 1.0), (math.nan, 1.0), (math.inf, 1.0), (30.0, 0.0), (30.0, math.nan)):
        assert fn(head=ss.Head(cap, tau, 0)) == INVALID, (cap, tau)
    need = ss.lib().ss_logprob_workspace_size(64, 1000, 128, backward)
    assert fn(wsb=need - 1) == WORKSPACE
    for k in ("H", "W", "ws"):
        assert fn(**{k: 0}) == INVALID and fn(**{k: FAKE + 8}) == INVALID, k
    for k in ("ids", "logp", "lse"):
        assert fn(**{k: 0}) == INVALID and fn(**{k: FAKE + 2}) == INVALID, k


def test_logprob_forward_of_nothing():
    assert _fwd(T=0, H=0, ids=0, logp=0, lse=0) == OK


def test_logprob_backward_argument_errors():
    for k in ("dH", "dW"):
        assert _bwd(**{k: 0}) == INVALID and _bwd(**{k: FAKE + 8}) == INVALID, k
    assert _bwd(dlogp=0) == INVALID and _bwd(dlogp=FAKE + 1) == INVALID
    assert _bwd(head=ss.Head(2.0 ** -6 * 0.99, 1.0, 0)) == UNSUPPORTED
    assert _bwd(dw=2) == INVALID and _bwd(dw=-1) == INVALID and _bwd(acc=2) == INVALID
    assert _bwd(T=0, dlogp=0, H=0, ids=0, logp=0, lse=0, dH=0, acc=1) == OK


def _policy(**kw):
    a = dict(logp=FAKE, old=FAKE, adv=FAKE, ref=FAKE, w=FAKE, n=8, lo=0.2, hi=0.2, klc=0.1,
             scale=1.0, loss=FAKE, kl=FAKE, d=FAKE)
    a.update(kw)
    return ss.lib().ss_policy_loss(p(a["logp"]), p(a["old"]), p(a["adv"]), p(a["ref"]), p(a["w"]),
                                   a["n"], a["lo"], a["hi"], a["klc"], a["scale"], p(a["loss"]),
                                   p(a["kl"]), p(a["d"]), None)


def test_policy_argument_errors():
    assert _policy(n=0) == OK and _policy(n=0, logp=0, loss=0) == OK
    assert _policy(n=-1) == INVALID and _policy(n=1 << 62) == UNSUPPORTED
    for bad in (dict(lo=-0.1), dict(lo=1.1), dict(lo=math.nan), dict(hi=-0.1), dict(hi=math.nan),
                dict(klc=-1.0), dict(klc=math.inf), dict(klc=math.nan), dict(scale=math.inf),
                dict(scale=math.nan), dict(ref=0), dict(ref=0, klc=0.0)):
        assert _policy(**bad) == INVALID, bad
    for k in ("logp", "old", "adv", "loss", "d"):
        assert _policy(**{k: 0}) == INVALID, k
    for k in ("logp", "old", "adv", "ref", "w", "loss", "kl", "d"):
        assert _policy(**{k: FAKE + 2}) == INVALID, k


def _pref(**kw):
    a = dict(logp=FAKE, ref=FAKE, w=FAKE, off=FAKE, pairs=2, n=8, kind=0, beta=0.1, e=0.0, avg=0,
             scale=1.0, loss=FAKE, reward=FAKE, d=FAKE, ws=FAKE, wsb=1024)
    a.update(kw)
    return ss.lib().ss_preference_loss(p(a["logp"]), p(a["ref"]), p(a["w"]), p(a["off"]),
                                       a["pairs"], a["n"], a["kind"], a["beta"], a["e"], a["avg"],
                                       a["scale"], p(a["loss"]), p(a["reward"]), p(a["d"]),
                                       p(a["ws"]), a["wsb"], None)


def test_preference_argument_errors():
    assert _pref(n=0, pairs=0, logp=0, off=0, ws=0, wsb=0) == OK
    assert _pref(n=-1) == INVALID and _pref(pairs=-1) == INVALID
    assert _pref(n=1 << 31) == UNSUPPORTED and _pref(pairs=1 << 29) == UNSUPPORTED
    for bad in (dict(kind=-1), dict(kind=3), dict(beta=0.0), dict(beta=-1.0), dict(beta=math.nan),
                dict(beta=math.inf), dict(e=-0.1), dict(e=0.6), dict(e=0.1, kind=1),
                dict(e=0.1, kind=2), dict(avg=2), dict(scale=math.nan), dict(wsb=1024, ws=0)):
        assert _pref(**bad) == INVALID, bad
    assert _pref(wsb=1023) == WORKSPACE
    for k in ("logp", "off", "loss", "reward", "d"):
        assert _pref(**{k: 0}) == INVALID, k
    for k in ("logp", "ref", "w", "off", "loss", "reward", "d"):
        assert _pref(**{k: FAKE + 2}) == INVALID, k


def _dist(**kw):
    a = dict(logp=FAKE, t=FAKE, dt=1, ids=FAKE, w=FAKE, T=4, K=8, tail=0, scale=1.0, loss=FAKE,
             d=FAKE)
    a.update(kw)
    return ss.lib().ss_distill_loss(p(a["logp"]), p(a["t"]), a["dt"], p(a["ids"]), p(a["w"]),
                                    a["T"], a["K"], a["tail"], a["scale"], p(a["loss"]),
                                    p(a["d"]), None)


def test_distill_argument_errors():
    assert _dist(T=0) == OK and _dist(T=0, logp=0) == OK
    assert _dist(T=-1) == INVALID and _dist(K=0) == INVALID
    assert _dist(T=1 << 31) == UNSUPPORTED and _dist(K=129) == UNSUPPORTED
    assert _dist(dt=2) == INVALID and _dist(tail=2) == INVALID and _dist(scale=math.inf) == INVALID
    for k in ("logp", "t", "loss", "d"):
        assert _dist(**{k: 0}) == INVALID, k
    for k in ("logp", "t", "ids", "w", "loss", "d"):
        assert _dist(**{k: FAKE + 2}) == INVALID, k
    assert _dist(t=FAKE + 1, dt=0) == INVALID


def test_python_refusals_on_host_tensors():
    H, W = torch.zeros(4, 64).bfloat16(), torch.zeros(9, 64).bfloat16()
    ids, ws = torch.zeros(4, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    x = torch.zeros(4)
    with pytest.raises(ValueError):
        ss.logprobs(H, W, ids, ws)
    with pytest.raises(TypeError):
        ss.logprobs(H.float(), W, ids, ws)
    with pytest.raises(TypeError):
        ss.logprobs_backward(x, H.numpy, W, ids, x, x, ws)
    with pytest.raises(ValueError):
        ss.policy_loss(x, x, x)
    with pytest.raises(TypeError):
        ss.policy_loss(x.double(), x, x)
    with pytest.raises(ValueError):
        ss.preference_loss(x, torch.zeros(3, dtype=torch.int32), ws)
    with pytest.raises(TypeError):
        ss.distill_loss(np.zeros((2, 2)), x)
