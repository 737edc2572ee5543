"""GPU: every kernel of the dense operators (dense_cases.py), with rows of x that
can and cannot be loaded 16 bytes a lane, against the 64-bit formulas.  Bounds as
in test_gpu_dense.py; those of the 4-bit products as in test_gpu_dense_precision.py
(no weight is rounded)."""
import pytest

from tests import dense_cases as D
from tests import harness as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not H.gpu_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

from routed_expert_execution_amd import moe  # noqa: E402
from tests import test_gpu_dense as G  # noqa: E402

TYPES = {True: torch.bfloat16, False: torch.float32}
ctx = G.ctx


def _linear_sizes():
    for gated, bf16, plan, half, whole in D.LINEAR:
        if half:
            yield gated, bf16, plan, half
        for group in (64, 128):
            yield gated, bf16, plan, whole[:3] + (group,)


@pytest.mark.parametrize("gated,bf16,plan,sizes", list(_linear_sizes()))
def test_linear_kernels(ctx, gated, bf16, plan, sizes):
    T, K, N, group = sizes
    dt = TYPES[bf16]
    assert moe.moe_linear_plan(T, N, K, group, dt, dt, gated) == plan + (1, 1)
    for pad, affine in ((0, True), (0, False), (5, True)):
        print("linear", gated, bf16, plan, sizes, pad, affine, flush=True)
        gen = G._gen(T + K + N + pad)
        x = G._normal(gen, T, K, dt, pad=pad)
        q, r = G._quantised(gen, N, K, group, affine), G._quantised(gen, N, K, group, affine)
        y = torch.full((T, N + pad), 777.0, dtype=dt, device="cuda")
        X = x.double()
        (w, mw), (v, mv) = G._values(q, group), G._values(r, group)
        D_ = (3 * 128 + K / 32 + 16) * G.U
        g = X @ w.t()
        tg = D_ * (X.abs() @ mw.t())
        if gated:
            moe.moe_linear_gated(ctx, x, moe.QuantMatrix(ctx, *q), moe.QuantMatrix(ctx, *r), y[:, :N])
            u, tu = X @ v.t(), D_ * (X.abs() @ mv.t())
            ref = G._silu(g) * u
            # (2 |g| steps more of the logistic function's argument, far below zero)
            G._close(y[:, :N], ref, G._gated_tol(g, u, tg, tu, ref, dt) + 2 * g.abs() * G.U * ref.abs())
        else:
            moe.moe_linear(ctx, x, moe.QuantMatrix(ctx, *q), y[:, :N])
            G._close(y[:, :N], g, tg + G._half_step(g, dt) + 1e-30)
        assert (y[:, N:] == 777.0).all()


def _gated_sizes():
    for bf16, plan, aligned, odd in D.GATED:
        yield bf16, plan, aligned
        yield bf16, plan, odd


@pytest.mark.parametrize("bf16,plan,sizes", list(_gated_sizes()))
def test_gated_kernels(ctx, bf16, plan, sizes):
    T, d, F = sizes
    dt = TYPES[bf16]
    assert moe.moe_gated_plan(T, d, F, dt) == plan + (1, 1)
    for pad in (0, 8):
        print("gated", bf16, plan, sizes, pad, flush=True)
        x, wg, wu = G._block(G._gen(T + d + F + pad), T, d, F, dt, pad)
        h, g_out, u_out = (torch.full((T, F), 777.0, dtype=dt, device="cuda") for _ in range(3))
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=g_out, up_out=u_out)
        X, A, B = x.double(), wg.double(), wu.double()
        g, u = X @ A.t(), X @ B.t()
        tg, tu = (G._chain(d, dt) * (X.abs() @ m.abs().t()) for m in (A, B))
        ref = G._silu(g) * u
        G._close(h, ref, G._gated_tol(g, u, tg, tu, ref, dt) + 2 * g.abs() * G.U * ref.abs(), "h")
        G._close(g_out, g, tg + G._half_step(g, dt) + 1e-30, "gate")
        G._close(u_out, u, tu + G._half_step(u, dt) + 1e-30, "up")


def _backward_sizes():
    for bf16, tile, parts, aligned, odd in D.BACKWARD:
        yield bf16, tile, parts, aligned
        yield bf16, tile, parts, odd


@pytest.mark.parametrize("bf16,tile,parts,sizes", list(_backward_sizes()))
def test_backward_kernels(ctx, bf16, tile, parts, sizes):
    T, d, F = sizes
    dt = TYPES[bf16]
    p = moe.moe_gated_plan(T, d, F, dt, True)
    assert p[1:3] == tile and (p[4] > 1, p[5] > 1) == parts
    print("backward", bf16, tile, parts, sizes, flush=True)
    gen = G._gen(T + d + F)
    x, wg, wu = G._block(gen, T, d, F, dt)
    dh = G._normal(gen, T, F, dt)
    gate, up = G._cancels((x.float() @ wg.float().t()).to(dt)), (x.float() @ wu.float().t()).to(dt)
    got = G._backward(ctx, dh, x, wg, wu, gate, up)
    for name, y, (ref, tol) in zip(("dx", "dw_gate", "dw_up"), got, G._backward_ref(dh, x, wg, wu, gate, up, dt)):
        G._close(y, ref, tol, name)
