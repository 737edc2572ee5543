"""GPU: an infinity or NaN in one token or one row of weights changes nothing else,
bit for bit, in every kernel of the dense operators (dense_cases.py): ragged last
tiles and half steps read lines past the end again, whose results are not stored."""
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


def _but(n, bad):
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[bad] = False
    return keep


def _linear_sizes():
    for gated, bf16, plan, half, whole in D.LINEAR:
        if half:
            yield gated, bf16, half
        yield gated, bf16, whole


@pytest.mark.parametrize("gated,bf16,sizes", list(_linear_sizes()))
def test_linear_keeps_bad_rows_apart(ctx, gated, bf16, sizes):
    T, K, N, group = sizes
    dt = TYPES[bf16]
    for pad in (0, 5):
        print("linear", gated, bf16, sizes, pad, flush=True)
        gen = G._gen(T + K + N + pad)
        x = G._normal(gen, T, K, dt, pad=pad)
        (codes, scales, zeros), r = G._quantised(gen, N, K, group, True), G._quantised(gen, N, K, group, True)
        up = moe.QuantMatrix(ctx, *r)

        def product(x, scales):
            w = moe.QuantMatrix(ctx, codes, scales, zeros)
            y = torch.empty(T, N, dtype=dt, device="cuda")
            moe.moe_linear_gated(ctx, x, w, up, y) if gated else moe.moe_linear(ctx, x, w, y)
            return y

        clean = product(x, scales)
        bad_t = {T // 2, T - 1}
        bad_n = [N // 2, N - 2, N - 1]
        x2, s2 = x.clone(), scales.clone()
        x2[T // 2, 3] = float("inf")
        x2[T - 1, K - 1] = float("nan")
        s2[N // 2, 1], s2[N - 2, 0], s2[N - 1] = float("nan"), float("inf"), 0.0
        y = product(x2, s2)
        rows, cols = _but(T, sorted(bad_t)), _but(N, bad_n)
        assert torch.equal(y[rows][:, cols].view(torch.uint8), clean[rows][:, cols].view(torch.uint8))
        if T > 2:
            assert not torch.isfinite(y[rows][:, N // 2]).any()
            assert (y[rows][:, N - 1] == 0).all()
            # (an infinite gate of the one sign has a silu of 0 or NaN, of the other an infinity)
            assert gated or not torch.isfinite(y[rows][:, N - 2]).any()
            # (the infinity is x times q - z, which may be zero: then NaN)
            assert not torch.isfinite(y[T // 2, cols]).all() if gated else not torch.isfinite(y[T // 2, cols]).any()
        assert torch.isnan(y[T - 1, cols]).all()


def _gated_sizes():
    for bf16, plan, *sizes in D.GATED:
        for s in sizes:
            yield bf16, s


@pytest.mark.parametrize("bf16,sizes", list(_gated_sizes()) + [(b, (70, 136, 140)) for b in (True, False)])
def test_gated_keeps_bad_rows_apart(ctx, bf16, sizes):
    T, d, F = sizes
    dt = TYPES[bf16]
    print("gated", bf16, sizes, flush=True)
    x, wg, wu = G._block(G._gen(T), T, d, F, dt)

    def block(x, wg):
        h, g, u = (torch.empty(T, F, dtype=dt, device="cuda") for _ in range(3))
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
        return h, g, u

    clean = block(x, wg)
    x2, wg2 = x.clone(), wg.clone()
    x2[T - 1, 0], wg2[F - 1, d - 1], wg2[F // 2, 0] = float("nan"), float("inf"), float("nan")
    rows, cols = _but(T, [T - 1]), _but(F, [F - 1, F // 2])
    for y, c in zip(block(x2, wg2), clean):
        assert torch.equal(y[rows][:, cols], c[rows][:, cols])
        assert torch.isnan(y[T - 1]).all()
    assert torch.equal(block(x2, wg2)[2][rows], clean[2][rows])


def _backward_sizes():
    for bf16, tile, parts, *sizes in D.BACKWARD:
        for s in sizes:
            yield bf16, s


@pytest.mark.parametrize("bf16,sizes", list(_backward_sizes()))
def test_backward_keeps_bad_rows_apart(ctx, bf16, sizes):
    T, d, F = sizes
    dt = TYPES[bf16]
    print("backward", bf16, sizes, flush=True)
    gen = G._gen(T + 1)
    x, wg, wu = G._block(gen, T, d, F, dt)
    dh, gate, up = (G._normal(gen, T, F, dt) for _ in range(3))
    clean = G._backward(ctx, dh, x, wg, wu, gate, up)
    # a token: its row of dx, and of the gradients the rows whose dg or du it spoils
    dh2 = dh.clone()
    dh2[T - 1, F - 1] = float("nan")
    dx, dwg, dwu = G._backward(ctx, dh2, x, wg, wu, gate, up)
    rows = _but(T, [T - 1])
    assert torch.equal(dx[rows], clean[0][rows]) and torch.isnan(dx[T - 1]).all()
    for y, c in ((dwg, clean[1]), (dwu, clean[2])):
        assert torch.equal(y[:F - 1], c[:F - 1]) and torch.isnan(y[F - 1]).all()
    # a column of x: that column of the weights' gradients; of the weights: that column of dx
    x2, wu2 = x.clone(), wu.clone()
    x2[T // 2, d - 1], wu2[F // 2, d - 1] = float("nan"), float("nan")
    dx, dwg, dwu = G._backward(ctx, dh, x2, wg, wu2, gate, up)
    for y, c in zip((dx, dwg, dwu), clean):
        assert torch.equal(y[:, :d - 1], c[:, :d - 1]) and torch.isnan(y[:, d - 1]).all()
