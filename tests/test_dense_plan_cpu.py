"""The choice of the dense operators' kernels, which the host makes: the cases that
the GPU tests run hold every kernel that any size takes, and no other."""
import ctypes as C
import math
import random
import re
import shutil
import subprocess

import pytest

from routed_expert_execution_amd import build, moe
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


def test_no_kernel_is_compiled_that_no_size_takes():
    """The kernels in the library's symbols against those of the cases."""
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm")
    text = subprocess.run([nm, "-C", build.LIB], check=True, capture_output=True, text=True).stdout
    built = {}
    for name, args in re.findall(r"(?<!__device_stub__)\b(\w+_kernel)<([^>]*)>", text):
        built.setdefault(name, set()).add(tuple({"true": True, "false": False}.get(a, a if not a.isdigit() else int(a)) for a in args.split(", ")))
    rows, shared, tiles = set(), set(), set()
    for gated, bf16, (kind, tokens, n, parts), half, whole in D.LINEAR:
        for s in (4, 2, 1):
            if kind == D.ROWS:
                rows.add((bf16, 1 if tokens == 4 else 4, n // 16, s, gated))
            elif kind == D.SHARED:
                shared.add((bf16, tokens // 16, n // 16, parts, s, gated))
            elif s < 4 or half:
                tiles |= {(tokens, n * (2 if gated else 1), gated, s == 4, fast, parts) for fast in (False, True)}
    assert built["rows_kernel"] == rows and built["shared_rows_kernel"] == shared
    assert {t[:2] + t[4:] for t in built["quant_tile_kernel"]} == tiles
    forward = {(b, p[1], 2 * p[2], fast, p[3]) for b, p, *_ in D.GATED if p[0] == D.TILES for fast in (False, True)}
    assert {t[:3] + t[8:] for t in built["tile_kernel"]} == forward
    few = {(b, max(1, p[1] // 16), 1 if p[1] == 4 else 4) for b, p, *_ in D.GATED if p[0] == D.ROWS}
    assert built["gated_rows_kernel"] == few
    assert {t[:3] + t[5:] for t in built["backward_tiles_kernel"]} == {(b, *tile, fast) for b, tile, *_ in D.BACKWARD for fast in (False, True)}
