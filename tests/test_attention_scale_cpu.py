"""Scales so large that their product with log2(e), which the kernels use, would not be finite in fp32 are refused, on the host."""
import ctypes as C

import pytest

from routed_expert_execution_amd import moe
from tests import test_attention_cpu as T


@pytest.fixture(scope="module")
def ctx():
    return moe.Context(1, 4, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)


@pytest.mark.parametrize("scale,text", [(1.6e38, "host-only"), (2.0 ** 127, "scale"), (2.4e38, "scale"), (3.4e38, "scale"), (1e-45, "host-only")])
def test_largest_scale(ctx, scale, text):
    T._refused(ctx, T._cached(ctx, scale=scale), text)
    T._refused(ctx, T._forward(ctx, T._attn(scale=scale)), text)
    T._refused(ctx, T._backward(ctx, T._attn(scale=scale)), text)
    assert C.c_float(scale).value > 0
