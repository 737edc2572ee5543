"""The dense operators' checks of arguments, without a GPU: a host-only context
judges the arguments first and refuses the call for its device last, so each
refusal is told by its message."""
import ctypes as C

import numpy as np
import pytest

from routed_expert_execution_amd import moe

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def ctx():
    return moe.Context(1, 4, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)


# Host buffers stand for device memory: no call here gets past the checks.
BUF = np.zeros(1 << 20, dtype=np.uint8)
BASE = (BUF.ctypes.data + 255) // 256 * 256


def _qmat(rows=32, cols=128, group=32, affine=0, data=BASE):
    return moe.moe_qmat(rows, cols, group, affine, data)


def _refused(ctx, status, text):
    assert status == moe.MOE_EINVAL
    assert text in moe.library().moe_last_error(ctx.handle).decode(), moe.library().moe_last_error(ctx.handle)


def _linear(ctx, w=None, x=BASE, xd=0, ldx=128, T=2, y=BASE, yd=0, ldy=32):
    w = _qmat() if w is None else w
    return moe.library().moe_linear(ctx.handle, x, xd, ldx, T, C.byref(w), y, yd, ldy, None)


def test_linear_bytes():
    # tiles of 16 x 128: 1024 bytes of codes, 32 or 48 more for each of a row's groups in the tile
    f = moe.library().moe_linear_bytes
    assert f(16, 128, 128, 0) == 1024 + 32
    assert f(16, 128, 32, 1) == 1024 + 4 * 48
    assert f(17, 160, 32, 1) == 4 * (1024 + 4 * 48)
    for bad in ((0, 128, 32, 0), (16, 0, 32, 0), (16, 100, 32, 0), (16, 96, 64, 0), (16, 128, 16, 0), (16, 256, 256, 0),
                (16, 128, 32, 2), (-1, 128, 32, 0), ((1 << 24) + 1, 128, 32, 0), (16, (1 << 24) + 128, 128, 0)):
        assert f(*bad) == 0, bad


def test_linear_good_arguments_reach_the_device_check(ctx):
    _refused(ctx, _linear(ctx), "host-only")
    _refused(ctx, _linear(ctx, T=0, x=None, y=None), "host-only")
    _refused(ctx, _linear(ctx, T=1, ldx=0, ldy=0), "host-only")  # one row has no stride


@pytest.mark.parametrize("kw,text", [
    (dict(w=_qmat(data=None)), "null matrix"), (dict(w=_qmat(rows=0)), "bad matrix"), (dict(w=_qmat(cols=100)), "bad matrix"),
    (dict(w=_qmat(group=48)), "bad matrix"), (dict(w=_qmat(affine=3)), "bad matrix"), (dict(w=_qmat(data=BASE + 8)), "16-byte"),
    (dict(x=None), "null x"), (dict(y=None), "null the result"), (dict(xd=2), "type of x"), (dict(yd=-1), "type of the result"),
    (dict(x=BASE + 2), "misaligned x"), (dict(xd=1, x=BASE + 1), "misaligned x"), (dict(y=BASE + 1), "misaligned the result"),
    (dict(ldx=127), "rows of x"), (dict(ldy=31), "rows of the result"), (dict(ldx=-128), "rows of x"),
    (dict(ldx=(1 << 40) + 1), "rows of x"), (dict(T=-1), "outside"), (dict(T=(1 << 20) + 1), "outside")])
def test_linear_refuses(ctx, kw, text):
    _refused(ctx, _linear(ctx, **kw), text)


def test_linear_null_context_and_matrix(ctx):
    lib = moe.library()
    w = _qmat()
    assert lib.moe_linear(None, BASE, 0, 128, 2, C.byref(w), BASE, 0, 32, None) == moe.MOE_EINVAL
    assert lib.moe_linear_gated(None, BASE, 0, 128, 2, C.byref(w), C.byref(w), BASE, 0, 32, None) == moe.MOE_EINVAL
    assert lib.moe_linear_pack(None, BASE, BASE, None, C.byref(w), None) == moe.MOE_EINVAL
    assert lib.moe_linear_dequant(None, C.byref(w), BASE, None) == moe.MOE_EINVAL
    _refused(ctx, lib.moe_linear(ctx.handle, BASE, 0, 128, 2, None, BASE, 0, 32, None), "null matrix")
    _refused(ctx, lib.moe_linear_gated(ctx.handle, BASE, 0, 128, 2, C.byref(w), None, BASE, 0, 32, None), "null matrix")
    _refused(ctx, lib.moe_linear_gated(ctx.handle, BASE, 0, 128, 2, None, C.byref(w), BASE, 0, 32, None), "null matrix")


@pytest.mark.parametrize("other", [dict(rows=48), dict(cols=256), dict(group=64), dict(affine=1)])
def test_linear_gated_refuses_unlike_matrices(ctx, other):
    a, b = _qmat(), _qmat(**other)
    _refused(ctx, moe.library().moe_linear_gated(ctx.handle, BASE, 0, 256, 2, C.byref(a), C.byref(b), BASE, 0, 64, None), "differ")


def test_pack_and_dequant_refuse(ctx):
    lib = moe.library()
    w, wa = _qmat(), _qmat(affine=1)
    _refused(ctx, lib.moe_linear_pack(ctx.handle, None, BASE, None, C.byref(w), None), "null argument")
    _refused(ctx, lib.moe_linear_pack(ctx.handle, BASE, None, None, C.byref(w), None), "null argument")
    _refused(ctx, lib.moe_linear_pack(ctx.handle, BASE, BASE, None, C.byref(wa), None), "null argument")
    _refused(ctx, lib.moe_linear_pack(ctx.handle, BASE, BASE + 1, None, C.byref(w), None), "misaligned")
    _refused(ctx, lib.moe_linear_pack(ctx.handle, BASE, BASE, None, C.byref(w), None), "host-only")
    _refused(ctx, lib.moe_linear_dequant(ctx.handle, C.byref(w), None, None), "null")
    _refused(ctx, lib.moe_linear_dequant(ctx.handle, C.byref(w), BASE, None), "host-only")


GATED = dict(x=BASE, dtype=0, ldx=64, T=2, d=64, F=96, wg=BASE, wu=BASE, h=BASE, gate=None, up=None)
BACK = dict(dh=BASE, lddh=96, x=BASE, dtype=0, ldx=64, T=2, d=64, F=96, wg=BASE, wu=BASE, gate=BASE, up=BASE, dx=BASE,
            dwg=BASE, dwu=BASE, ws=BASE, n=1 << 20)


def _gated(ctx, **kw):
    return moe.library().moe_gated(ctx.handle, *{**GATED, **kw}.values(), None)


def _back(ctx, **kw):
    return moe.library().moe_gated_backward(ctx.handle, *{**BACK, **kw}.values(), None)


@pytest.mark.parametrize("kw,text", [
    ({}, "host-only"), (dict(T=0, x=None, wg=None, wu=None, h=None), "host-only"), (dict(gate=BASE, up=BASE), "host-only"),
    (dict(d=0), "outside"), (dict(F=0), "outside"), (dict(T=-1), "outside"), (dict(d=(1 << 20) + 1), "outside"),
    (dict(dtype=7), "type of x"), (dict(ldx=63), "rows of x"), (dict(x=None), "null x"), (dict(wg=None), "null"),
    (dict(wu=None), "null"), (dict(h=None), "null"), (dict(gate=BASE), "null"), (dict(up=BASE), "null"),
    (dict(wg=BASE + 2), "misaligned"), (dict(h=BASE + 1), "misaligned"), (dict(gate=BASE + 2, up=BASE), "misaligned")])
def test_gated_refuses(ctx, kw, text):
    _refused(ctx, _gated(ctx, **kw), text)


@pytest.mark.parametrize("kw,text", [
    ({}, "host-only"), (dict(dx=None), "host-only"), (dict(dwg=None, dwu=None), "host-only"),
    (dict(T=0, dh=None, x=None, gate=None, up=None, wg=None, wu=None), "host-only"),
    (dict(d=0), "outside"), (dict(T=(1 << 20) + 1), "outside"), (dict(dtype=2), "type of x"), (dict(ldx=63), "rows of x"),
    (dict(lddh=95), "rows of dh"), (dict(dh=None), "null dh"), (dict(x=None), "null x"), (dict(gate=None), "null"),
    (dict(up=None), "null"), (dict(wg=None), "null"), (dict(wu=None), "null"), (dict(dwg=None), "null"),
    (dict(dwu=None), "null"), (dict(ws=None), "null"), (dict(ws=BASE + 128), "256-byte"), (dict(n=255), "needed"),
    (dict(dx=BASE + 1), "misaligned"), (dict(dwu=BASE + 2), "misaligned")])
def test_gated_backward_refuses(ctx, kw, text):
    _refused(ctx, _back(ctx, **kw), text)


def test_gated_workspace_sizes():
    f = moe.library().moe_gated_workspace
    for T, d, F in ((0, 1, 1), (1, 64, 96), (333, 1000, 1411), (4096, 2048, 8192)):
        for dtype, e in ((moe.MOE_F32, 4), (moe.MOE_BF16, 2)):
            assert f(T, d, F, dtype) >= max(256, 2 * T * F * e)  # dg and du at least
    assert f(1, 0, 1, 0) == 0 and f(1, 1, 0, 0) == 0 and f(-1, 1, 1, 0) == 0 and f(1, 1, 1, 2) == 0


def test_binding_refuses_before_the_library(ctx):
    codes = torch.zeros(32, 64, dtype=torch.uint8)
    scales = torch.zeros(32, 4, dtype=torch.float16)
    for c, s, z in ((codes.int(), scales, None), (codes, scales.float(), None), (codes, scales[:16], None),
                    (codes, scales, torch.zeros(32, 2, dtype=torch.uint8)), (codes, scales, torch.zeros(32, 4)),
                    (codes, scales, None),  # (the last: not on the context's device)
                    (codes, scales.repeat(1, 2), None)):
        with pytest.raises(ValueError):
            moe.QuantMatrix(ctx, c, s, z)
    x, w = torch.zeros(2, 64), torch.zeros(96, 64)
    h = torch.zeros(2, 96)
    for bad in ((x.half(), w, w, h), (x, w.bfloat16(), w, h), (x, w, w[:95], h), (x, w, w, h[:1]), (x, w, w, h.bfloat16()),
                (x.t().contiguous().t(), w, w, h), (x[:1].expand(2, 64), w, w, h), (x, w, w, h)):
        with pytest.raises(ValueError):
            moe.moe_gated(ctx, *bad)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    for bad in ((h.bfloat16(), x, w, w, h, h), (h, x, w, w, h[:1], h), (h, x, w, w, h, h.bfloat16()), (h[:, :95], x, w, w, h, h),
                (h, x, w, w, h, h)):
        with pytest.raises(ValueError):
            moe.moe_gated_backward(ctx, *bad, dx=x, workspace=ws)
    with pytest.raises(ValueError):
        moe.moe_gated_workspace(ctx, 1, 1, 1, torch.float16)
