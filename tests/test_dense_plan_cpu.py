"""The choice of the dense operators' kernels, which the host makes: the cases that
the GPU tests run hold every kernel that any size takes, and no other."""
import ctypes as C
import math
import random

import pytest

from routed_expert_execution_amd import moe
from tests import dense_cases as D

torch = pytest.importorskip("torch")
BF16, F32 = torch.bfloat16, torch.float32
TYPES = {True: BF16, False: F32}


@pytest.mark.parametrize("gated,bf16,plan,half,whole", D.LINEAR)
def test_linear_cases_take_their_kernel(gated, bf16, plan, half, whole):
    if half:
        T, K, N, group = half
        assert group == 32 and K % 64 == 32
        assert moe.moe_linear_plan(T, N, K, group, TYPES[bf16], TYPES[bf16], gated) == plan + (1, 1)
    T, K, N, _ = whole
    assert K % 128 == 0
    for group in (64, 128):
        assert moe.moe_linear_plan(T, N, K, group, TYPES[bf16], TYPES[bf16], gated) == plan + (1, 1)


def _gated_cases():
    for bf16, plan, aligned, odd in D.GATED:
        yield bf16, aligned, False, plan + (1, 1)
        yield bf16, odd, False, plan + (1, 1)
    for bf16, tile, parts, aligned, odd in D.BACKWARD:
        yield bf16, aligned, True, (tile, parts)
        yield bf16, odd, True, (tile, parts)


@pytest.mark.parametrize("bf16,sizes,backward,plan", list(_gated_cases()))
def test_gated_cases_take_their_kernel(bf16, sizes, backward, plan):
    p = moe.moe_gated_plan(*sizes, TYPES[bf16], backward)
    if backward:
        assert p[0] == moe.MOE_PLAN_TILES and p[1:3] == plan[0] and p[3] == 1 and (p[4] > 1, p[5] > 1) == plan[1]
    else:
        assert p == plan


def test_no_size_takes_a_kernel_that_the_cases_lack():
    """Random sizes over what the operators take (the number of waves of the rows
    kernels, a launch's size and no kernel of its own, aside)."""
    def kernel(p):
        return p[:3] + ((p[3],) if p[0] != D.ROWS else ())

    linear = {(g, b, kernel(p), n == 32) for g, b, p, *sizes in D.LINEAR for *_, n in filter(None, sizes)}
    gated = {(b, kernel(p)) for b, p, *_ in D.GATED}
    backward = {(b, t, s) for b, t, s, *_ in D.BACKWARD}
    seen = (set(), set(), set())
    rng = random.Random(2)

    def log(low, high):
        return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))

    for _ in range(60000):
        T, group, bf16, g = log(1, 1 << 15), rng.choice((32, 64, 128)), rng.random() < 0.6, rng.random() < 0.5
        K = group * log(1, 16384 // group)
        y = rng.choice((BF16, F32))
        p = moe.moe_linear_plan(T, log(1, 1 << 17), K, group, TYPES[bf16], y, g)
        assert y == TYPES[bf16] == BF16 or p[0] != D.TILES
        seen[0].add((g, bf16, kernel(p), group == 32))
        d, f = log(1, 8192), log(1, 16384)
        seen[1].add((bf16, kernel(moe.moe_gated_plan(T, d, f, TYPES[bf16]))))
        p = moe.moe_gated_plan(T, d, f, TYPES[bf16], True)
        seen[2].add((bf16, p[1:3], (p[4] > 1, p[5] > 1)))
    assert not seen[0] - linear and not seen[1] - gated and not seen[2] - backward, (seen[0] - linear, seen[1] - gated, seen[2] - backward)


def test_plans_refuse():
    out = (C.c_int32 * 6)()
    lib = moe.library()
    assert lib.moe_linear_plan(1, 32, 128, 32, 0, 0, 0, out) == moe.MOE_OK and lib.moe_gated_plan(1, 8, 8, 0, 0, out) == moe.MOE_OK
    assert lib.moe_linear_plan(1, 32, 128, 32, 0, 0, 0, None) == moe.MOE_EINVAL and lib.moe_gated_plan(1, 8, 8, 0, 0, None) == moe.MOE_EINVAL
    for bad in ((0, 32, 128, 32, 0, 0), (1, 0, 128, 32, 0, 0), (1, 32, 100, 32, 0, 0), (1, 32, 128, 48, 0, 0), (1, 32, 128, 32, 2, 0),
                (1, 32, 128, 32, 0, -1), ((1 << 20) + 1, 32, 128, 32, 0, 0)):
        assert lib.moe_linear_plan(*bad, 0, out) == moe.MOE_EINVAL, bad
    for bad in ((0, 8, 8, 0), (1, 0, 8, 0), (1, 8, 0, 0), (1, 8, 8, 2), (1, (1 << 20) + 1, 8, 0), ((1 << 20) + 1, 8, 8, 0)):
        assert lib.moe_gated_plan(*bad, 1, out) == moe.MOE_EINVAL, bad
    with pytest.raises(moe.MoeError):
        moe.moe_linear_plan(1, 32, 128, 32, torch.float16, F32)
    with pytest.raises(moe.MoeError):
        moe.moe_gated_plan(1, 8, 8, torch.float16)
