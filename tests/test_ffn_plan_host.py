"""The feed-forward block's choice of kernels over its sizes, on the CPU."""
import heapq
import math
import random

import pytest

import ffn_plan
from test_ffn_gpu import LARGE, SIZES


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    return ffn_plan.compile_plan(str(tmp_path_factory.mktemp("plan")))


def _sizes(n, seed):
    rng = random.Random(seed)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    for _ in range(n):
        T, D, F = log(1, 65536), 8 * log(1, 2048), 8 * log(1, 8192)
        if T * D * F <= 4e11 and T * F <= 6e8:
            yield T, D, F


def test_the_gpu_tests_reach_every_form(plan):
    """A form is a kernel with its tile and cluster. What sizes over the whole range
    choose, the GPU tests' sizes choose too."""
    tested = set()
    for size in SIZES + LARGE + ffn_plan.FORM_SIZES:
        tested |= ffn_plan.forms(plan, *size)
    for size in _sizes(120_000, 1):
        new = ffn_plan.forms(plan, *size) - tested
        assert not new, (size, new)
    # 17 to 32 tokens have their tiles to themselves
    assert {f for f in tested if "split" in f[0] and f[1] == 32} == {
        (k + " split", 32, s) for k in ("up", "down", "act", "x") for s in (1, 2, 4, 8)
        if (k, s) != ("x", 1)}  # dX has two k-blocks at least, and then two CTAs


def test_every_activation_meets_every_epilogue_on_pairs(plan):
    reached = set()
    for size in ffn_plan.ACT_SIZES:
        reached |= ffn_plan.forms(plan, *size)
    assert {(k + " pair", how, bn) for k in ("up", "act") for how in ("registers", "staged")
            for bn in (192, 256)} <= reached


def _dealt(n_a, kb_a, n_b, kb_b, pairs):
    """Each unit, the longer kind first, to the pair that is free first."""
    free = [(0, p) for p in range(pairs)]
    out = [[] for _ in range(pairs)]
    a, b = [(u, kb_a) for u in range(n_a)], [(n_a + u, kb_b) for u in range(n_b)]
    for u, kb in a + b if kb_a >= kb_b else b + a:
        t, p = heapq.heappop(free)
        out[p].append(u)
        heapq.heappush(free, (t + kb, p))
    return out, max(t for t, _ in free)


def test_units_go_to_the_pair_that_is_free_first(plan):
    rng = random.Random(3)
    cases = [(n, 5, 0, 5, 76) for n in (1, 75, 76, 77, 5000)]
    cases += [(2304, 8, 32, 384, 76), (1, 1, 1, 1, 2), (3, 1024, 64, 8, 67), (76, 4, 76, 4, 76)]
    for _ in range(600):
        n_a, n_b = (int(math.exp(rng.uniform(0, 8.5))) for _ in range(2))
        kb_a, kb_b = (int(math.exp(rng.uniform(0, 7))) for _ in range(2))
        cases.append((n_a, kb_a, n_b, kb_b, min(n_a + n_b, rng.choice([1, 2, 66, 74, 76]))))
    for case in cases:
        assert ffn_plan.deal(plan, *case) == _dealt(*case), case


@pytest.mark.parametrize("T,D,F", [(512, 4096, 12288), (512, 4096, 14336), (500, 4096, 11008),
                                   (339, 4040, 11680)])
def test_many_units_are_shared_evenly(plan, T, D, F):
    """Past 2048 units: no pair has more than a unit of the shorter kind above the
    even share, or one of the longer kind where there are fewer of them than pairs."""
    n_w, n_x = 3 * -(-F // 256) * -(-D // 256), -(-T // 256) * -(-D // 256)
    k_w, k_x = -(-T // 64), 2 * -(-F // 64)
    assert n_w + n_x > 2048
    _, most = ffn_plan.deal(plan, n_w, k_w, n_x, k_x, 76)
    assert n_x < 76 and k_x > k_w
    assert most <= max((n_w * k_w + n_x * k_x) / 76 + k_w, k_x)
