"""The feed-forward block's choice of kernels over its sizes, on the CPU."""
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
