"""GPU: the dense operators (4-bit linear and gated block, the gated block in
bf16 and fp32 and its backward pass) against plain 64-bit formulas.

Tolerances are first-order bounds of the arithmetic that the interface
documents, element by element, with u = 2^-24 (fp32) and half a step of bf16,
2^-8 of the value:
  - a sum of n products added in fp32 in any order differs from the exact sum by
    at most D u sum |a b|, D the longest chain of additions a term passes through.
    The 4-bit products add a group (128 columns at most, three terms for fp32 x)
    on the matrix cores, then 2 roundings for scale and zero point, then the
    groups of a wave and the waves: D <= 3 * 128 + cols / 32 + 16.  Their terms
    are (16 + q) x and (16 + z) x, times the scale.
    The bf16 products add all of k in some order: D <= k + 16.  The fp32 ones are
    six products of bf16 terms (24 bits of each factor in three terms, what is
    left out below 2^-25 of the product), all added to one sum: D <= 6 k + 32.
  - h = silu(g) u: |silu'| <= 1.1, and 8 u for the logistic function itself
  - dg and du are rounded to the type before the products: the reference rounds
    its 64-bit values in the same way, and where one lies within 32 u of the
    middle between two neighbours, the other neighbour is allowed for.
"""
import ctypes as C

import pytest

from tests import harness as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not H.gpu_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import synth  # noqa: E402
from routed_expert_execution_amd import moe  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _say(*a):
    print(*a, flush=True)


def _ctx():
    cfg = moe.make_config(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)
    pool = torch.zeros(moe.moe_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    return moe.Context(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=0, slot_pool=pool)


@pytest.fixture(scope="module")
def ctx():
    return _ctx()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, rows, cols, dtype, scale=1.0, pad=0):
    return (torch.randn(rows, cols + pad, generator=gen, device="cuda") * scale).to(dtype)[:, :cols]


def _quantised(gen, N, K, group, affine):
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.randn(N, K // group, generator=gen, device="cuda") * 0.01).to(torch.float16)
    zeros = torch.randint(0, 16, (N, K // group), generator=gen, device="cuda", dtype=torch.uint8) if affine else None
    return codes, scales, zeros


def _values(q, group):
    """(w, sum of magnitudes' factor) in 64 bits: s (q - z), |s| (32 + q + z)."""
    codes, scales, zeros = q
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).double()
    z = torch.full_like(scales, 8.0, dtype=torch.float64) if zeros is None else zeros.double()
    z, s = z.repeat_interleave(group, 1), scales.double().repeat_interleave(group, 1)
    return s * (c - z), s.abs() * (32 + c + z)


def _chain(k, dtype):
    return (k + 16 if dtype == torch.bfloat16 else 6 * k + 32) * U


def _half_step(ref, dtype):
    return ref.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U)


def _close(y, ref, tol, what=""):
    y = y.double()
    bad = ~((y - ref).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4].tolist(), ref[bad][:4].tolist(),
                           tol[bad][:4].tolist())


def _linear_tol(x, mag, ref, y_dtype):
    K = x.shape[1]
    D = 3 * 128 + K / 32 + 16
    return D * U * (x.double().abs() @ mag.t()) + _half_step(ref, y_dtype) + 1e-30


def _silu(g):
    return g * torch.sigmoid(g)


def _gated_tol(g, u, dg, du, h, dtype):
    """Bound of h = silu(g) u for |error| <= dg, du of g, u."""
    return 1.1 * dg * (u.abs() + du) + _silu(g).abs() * du + 8 * U * h.abs() + _half_step(h, dtype) + 1e-30


# ---- 4-bit matrices ----

@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("N,K,group", [(1, 32, 32), (16, 128, 128), (17, 160, 32), (100, 192, 64), (33, 896, 128), (256, 2048, 32)])
def test_pack_holds_every_value(ctx, N, K, group, affine):
    gen = _gen(N + K)
    q = _quantised(gen, N, K, group, affine)
    if affine:
        q[2][0, 0] = 255  # any byte is a zero point
    w = moe.QuantMatrix(ctx, *q)
    out = torch.full((N, K), float("nan"), device="cuda")
    moe.moe_linear_dequant(ctx, w, out)
    ref = _values(q, group)[0]
    assert torch.equal(out.double(), ref)


LINEAR = [  # T, K, N, group, affine, x, y, pad
    (1, 32, 1, 32, False, "bf16", "bf16", 0), (1, 2048, 2048, 32, False, "bf16", "bf16", 0), (1, 96, 7, 32, True, "f32", "f32", 0),
    (2, 160, 40, 32, True, "bf16", "f32", 5), (3, 8192, 50, 128, True, "bf16", "f32", 0), (4, 192, 64, 64, False, "f32", "bf16", 1),
    (5, 384, 33, 128, True, "bf16", "bf16", 3), (8, 1024, 272, 64, True, "f32", "f32", 0), (16, 2112, 515, 64, True, "bf16", "bf16", 8),
    (17, 128, 16, 32, True, "f32", "f32", 7), (31, 640, 100, 128, False, "bf16", "f32", 0), (37, 4096, 300, 64, True, "bf16", "bf16", 0),
    (64, 512, 129, 32, True, "f32", "f32", 0), (65, 288, 65, 32, False, "bf16", "f32", 1), (100, 1280, 200, 128, True, "f32", "f32", 4),
    (129, 256, 257, 64, True, "bf16", "bf16", 8), (200, 1344, 384, 64, True, "bf16", "bf16", 1), (513, 1024, 640, 128, True, "bf16", "bf16", 0),
    (700, 416, 530, 32, True, "bf16", "bf16", 8), (1024, 2048, 1024, 128, False, "bf16", "bf16", 0), (600, 768, 700, 64, False, "bf16", "f32", 0),
    (530, 512, 300, 128, True, "f32", "bf16", 0), (2, 128, 70001, 128, False, "bf16", "f32", 0),
    # every tile shape, rows of x that can and cannot be loaded 16 bytes a lane, a last step of half the columns
    (2000, 544, 4100, 32, True, "bf16", "bf16", 0), (2000, 544, 4100, 32, False, "bf16", "bf16", 5), (1500, 1088, 2050, 64, True, "bf16", "bf16", 0),
    (1500, 320, 2050, 64, True, "bf16", "bf16", 3), (3000, 416, 147, 32, False, "bf16", "bf16", 0), (70, 4096, 30000, 128, True, "bf16", "bf16", 0)]


def _weights_rounded(T, x_dtype, y_dtype):
    """Whether the call may round a weight to bf16 (more than 64 tokens, everything bf16)."""
    return T > 64 and x_dtype == y_dtype == torch.bfloat16


@pytest.mark.parametrize("T,K,N,group,affine,xd,yd,pad", LINEAR)
def test_linear(ctx, T, K, N, group, affine, xd, yd, pad):
    _say("linear", T, K, N, group, affine, xd, yd, pad)
    gen = _gen(T * 31 + K + N)
    x = _normal(gen, T, K, DT[xd], pad=pad)
    q = _quantised(gen, N, K, group, affine)
    y = torch.full((T, N + pad), 777.0, dtype=DT[yd], device="cuda")
    moe.moe_linear(ctx, x, moe.QuantMatrix(ctx, *q), y[:, :N])
    w, mag = _values(q, group)
    ref = x.double() @ w.t()
    tol = _linear_tol(x, mag, ref, DT[yd])
    if _weights_rounded(T, DT[xd], DT[yd]):
        tol = tol + 2.0 ** -8 * (x.double().abs() @ w.abs().t())
    _close(y[:, :N], ref, tol)
    assert (y[:, N:] == 777.0).all()  # the columns between the rows are the caller's


@pytest.mark.parametrize("T,K,N,group,affine,xd,yd,pad", LINEAR)
def test_linear_gated(ctx, T, K, N, group, affine, xd, yd, pad):
    _say("linear_gated", T, K, N, group, affine, xd, yd, pad)
    gen = _gen(T * 37 + K + N)
    x = _normal(gen, T, K, DT[xd], pad=pad)
    q, r = _quantised(gen, N, K, group, affine), _quantised(gen, N, K, group, affine)
    h = torch.full((T, N + pad), 777.0, dtype=DT[yd], device="cuda")
    moe.moe_linear_gated(ctx, x, moe.QuantMatrix(ctx, *q), moe.QuantMatrix(ctx, *r), h[:, :N])
    X = x.double()
    (wg, mg), (wu, mu) = _values(q, group), _values(r, group)
    g, u = X @ wg.t(), X @ wu.t()
    D = (3 * 128 + K / 32 + 16) * U
    tg, tu = D * (X.abs() @ mg.t()), D * (X.abs() @ mu.t())
    if _weights_rounded(T, DT[xd], DT[yd]):
        tg, tu = tg + 2.0 ** -8 * (X.abs() @ wg.abs().t()), tu + 2.0 ** -8 * (X.abs() @ wu.abs().t())
    ref = _silu(g) * u
    _close(h[:, :N], ref, _gated_tol(g, u, tg, tu, ref, DT[yd]))
    assert (h[:, N:] == 777.0).all()


@pytest.mark.parametrize("T,K,N", [(1024, 2048, 1024), (300, 1024, 520)])
def test_linear_rounds_weights_at_most_once(ctx, T, K, N):
    """The bound of test_linear for rounded weights is the worst case, far above
    what independent roundings give.  Here the weights are bf16 values already
    (scales powers of two, codes below 2^8), so rounding them changes nothing
    and the fp32 bound alone holds."""
    gen = _gen(K)
    x = _normal(gen, T, K, torch.bfloat16)
    codes, scales, zeros = _quantised(gen, N, K, 128, True)
    scales = torch.exp2(torch.randint(-9, -4, scales.shape, generator=gen, device="cuda").float()).half()
    q = (codes, scales, zeros)
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear(ctx, x, moe.QuantMatrix(ctx, *q), y)
    w, mag = _values(q, 128)
    ref = x.double() @ w.t()
    D = K + 16
    _close(y, ref, D * U * (x.double().abs() @ mag.t()) + _half_step(ref, torch.bfloat16))


@pytest.mark.parametrize("T", [1, 4, 9, 40, 300])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_linear_keeps_bad_rows_apart(ctx, T, xd):
    """A token with an infinity or a NaN, a row of weights with a zero, infinite
    or NaN scale: nothing else changes, bit for bit."""
    K, N, group = 256, 80, 64
    gen = _gen(T)
    x = _normal(gen, T, K, DT[xd])
    codes, scales, zeros = _quantised(gen, N, K, group, True)
    yd = torch.float32
    clean = torch.empty(T, N, dtype=yd, device="cuda")
    moe.moe_linear(ctx, x, moe.QuantMatrix(ctx, codes, scales, zeros), clean)
    x2, s2 = x.clone(), scales.clone()
    x2[T // 2, 3] = float("inf")
    if T > 2:
        x2[T - 1, K - 1] = float("nan")
    s2[5, 1], s2[17, 0], s2[79] = float("nan"), float("inf"), 0.0
    y = torch.empty(T, N, dtype=yd, device="cuda")
    moe.moe_linear(ctx, x2, moe.QuantMatrix(ctx, codes, s2, zeros), y)
    good_t = [t for t in range(T) if t != T // 2 and not (T > 2 and t == T - 1)]
    good_n = [n for n in range(N) if n not in (5, 17, 79)]
    assert torch.equal(y[good_t][:, good_n].view(torch.int32), clean[good_t][:, good_n].view(torch.int32))
    assert (y[good_t][:, 79] == 0).all()
    assert not torch.isfinite(y[good_t][:, 5]).any() and not torch.isfinite(y[good_t][:, 17]).any()
    # (a zero scale's row is 0 * inf there, or 0 where the infinity meets no code)
    assert not torch.isfinite(y[T // 2, good_n]).any()
    if T > 2:
        assert torch.isnan(y[T - 1, good_n]).all()


def test_linear_of_zeros_and_of_no_tokens(ctx):
    gen = _gen(3)
    w = moe.QuantMatrix(ctx, *_quantised(gen, 40, 256, 32, True))
    for xd in DT.values():
        y = torch.full((3, 40), 9.0, dtype=xd, device="cuda")
        moe.moe_linear(ctx, torch.zeros(3, 256, dtype=xd, device="cuda"), w, y)
        assert (y == 0).all()
        y = torch.full((3, 40), 9.0, dtype=xd, device="cuda")
        moe.moe_linear(ctx, torch.empty(0, 256, dtype=xd, device="cuda"), w, y[:0])
        moe.moe_linear_gated(ctx, torch.empty(0, 256, dtype=xd, device="cuda"), w, w, y[:0])
        assert (y == 9).all()


# ---- the gated block ----

GATED = [  # T, d, F
    (1, 1, 1), (1, 128, 512), (1, 2048, 512), (2, 65, 33), (4, 2048, 512), (5, 96, 130), (16, 200, 48), (17, 256, 264), (33, 1000, 65),
    (64, 512, 192), (65, 127, 129), (100, 72, 300), (128, 256, 256), (130, 264, 520), (300, 1024, 640), (257, 333, 1411), (600, 2048, 512),
    (513, 8, 8), (1030, 320, 1100),
    # the largest tiles: whole and partial last steps, aligned and not
    (2048, 520, 4100), (2050, 513, 4096), (1030, 2048, 1026), (4100, 256, 264)]


def _block(gen, T, d, F, dtype, pad=0):
    x = _normal(gen, T, d, dtype, pad=pad)
    return x, _normal(gen, F, d, dtype, d ** -0.5), _normal(gen, F, d, dtype, d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,F", GATED)
def test_gated(ctx, T, d, F, dtype):
    _say("gated", T, d, F, dtype)
    dt = DT[dtype]
    for pad, save in ((0, True), (3, False), (8, True)):
        x, wg, wu = _block(_gen(T + d + F + pad), T, d, F, dt, pad)
        h = torch.full((T, F), 777.0, dtype=dt, device="cuda")
        g_out, u_out = (torch.full_like(h, 777.0), torch.full_like(h, 777.0)) if save else (None, None)
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=g_out, up_out=u_out)
        X, G, W = x.double(), wg.double(), wu.double()
        g, u = X @ G.t(), X @ W.t()
        D = _chain(d, dt)
        tg, tu = D * (X.abs() @ G.abs().t()), D * (X.abs() @ W.abs().t())
        ref = _silu(g) * u
        _close(h, ref, _gated_tol(g, u, tg, tu, ref, dt), "h")
        if save:
            _close(g_out, g, tg + _half_step(g, dt) + 1e-30, "gate")
            _close(u_out, u, tu + _half_step(u, dt) + 1e-30, "up")


def _rounded(v, dt):
    """(v rounded to dt, how far the other neighbour may be where v is within 32 u of the middle)."""
    r = v.to(dt).double()
    if dt == torch.float32:
        return v, 32 * U * v.abs()
    # the middle is half a step from the value: 2^-8 relative to the power of two below
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(1e-300)))) * 2.0 ** -7
    near = (step / 2 - (v - r).abs()) <= 32 * U * v.abs()
    return r, torch.where(near, step, torch.zeros_like(step))


def _backward_ref(dh, x, wg, wu, gate, up, dt):
    """Gradients and their tolerances."""
    dh, X, G, W, g, u = (t.double() for t in (dh, x, wg, wu, gate, up))
    s = torch.sigmoid(g)
    dg, slack_g = _rounded(dh * u * s * (1 + g * (1 - s)), dt)
    du, slack_u = _rounded(dh * g * s, dt)
    # fp32 evaluation of the factors before the rounding: 1 + g (1 - s) cancels for
    # g near its zero, so its error is relative to 1 + |g|
    slack_g = slack_g + (0 if dt == torch.bfloat16 else 32 * U * (dh * u * s).abs() * (1 + g.abs()))
    T, F = dh.shape
    dx = dg @ G + du @ W
    tx = _chain(2 * F, dt) * (dg.abs() @ G.abs() + du.abs() @ W.abs()) + slack_g @ G.abs() + slack_u @ W.abs() + _half_step(dx, dt)
    out = [(dx, tx)]
    for v, sl in ((dg, slack_g), (du, slack_u)):
        dw = v.t() @ X
        out.append((dw, _chain(T, dt) * (v.abs().t() @ X.abs()) + sl.t() @ X.abs() + _half_step(dw, dt)))
    return [(a, b + 1e-30) for a, b in out]


def _cancels(g):
    """bf16: a dg whose factor 1 + g (1 - s) nearly vanishes is not within 32 u of
    its 64-bit value; such g (near -1.278) are moved."""
    s = torch.sigmoid(g.double())
    return torch.where((1 + g.double() * (1 - s)).abs() < 0.02, torch.ones_like(g), g)


def _backward(ctx, dh, x, wg, wu, gate, up, need=("dx", "dw"), workspace=None):
    T, d, F = x.shape[0], x.shape[1], wg.shape[0]
    dt = x.dtype
    n = moe.moe_gated_workspace(ctx, T, d, F, dt)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda") if workspace is None else workspace  # (NaN in every type)
    dx = torch.full((T, d), 777.0, dtype=dt, device="cuda") if "dx" in need else None
    dwg, dwu = (torch.full((F, d), 777.0, dtype=dt, device="cuda") for _ in range(2)) if "dw" in need else (None, None)
    moe.moe_gated_backward(ctx, dh, x, wg, wu, gate, up, dx=dx, dw_gate=dwg, dw_up=dwu, workspace=ws)
    return dx, dwg, dwu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,F", GATED)
def test_gated_backward(ctx, T, d, F, dtype):
    _say("gated_backward", T, d, F, dtype)
    dt = DT[dtype]
    for pad in (0, 3, 8):
        gen = _gen(T * 3 + d + F + pad)
        x, wg, wu = _block(gen, T, d, F, dt, pad)
        dh = _normal(gen, T, F, dt, pad=pad)
        gate, up = _cancels((x.float() @ wg.float().t()).to(dt)), (x.float() @ wu.float().t()).to(dt)
        got = _backward(ctx, dh, x, wg, wu, gate, up)
        for name, y, (ref, tol) in zip(("dx", "dw_gate", "dw_up"), got, _backward_ref(dh, x, wg, wu, gate, up, dt)):
            _close(y, ref, tol, name)
        # each gradient alone: the same bits
        dx, _, _ = _backward(ctx, dh, x, wg, wu, gate, up, need=("dx",))
        _, dwg, dwu = _backward(ctx, dh, x, wg, wu, gate, up, need=("dw",))
        for a, b in zip(got, (dx, dwg, dwu)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_backward_of_no_tokens_is_zero(ctx, dtype):
    dt = DT[dtype]
    e = lambda *s: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    wg = torch.ones(70, 50, dtype=dt, device="cuda")
    dx, dwg, dwu = _backward(ctx, e(0, 70), e(0, 50), wg, wg, e(0, 70), e(0, 70))
    assert dx.shape == (0, 50) and (dwg == 0).all() and (dwu == 0).all()
    moe.moe_gated(ctx, e(0, 50), wg, wg, e(0, 70))


@pytest.mark.parametrize("g", [0.0, -200.0, 200.0, -1e30, 1e30])
def test_gated_saturates(ctx, g):
    """Far gates: silu is 0 or g, its slope 0 or 1, and no NaN comes of exp's overflow."""
    T, d, F = 3, 64, 40
    for dt in DT.values():
        x = torch.zeros(T, d, dtype=dt, device="cuda")
        x[:, 0] = 1
        wg, wu = torch.zeros(F, d, dtype=dt, device="cuda"), torch.zeros(F, d, dtype=dt, device="cuda")
        wg[:, 0], wu[:, 0] = g, 2.0
        h, gate, up = (torch.empty(T, F, dtype=dt, device="cuda") for _ in range(3))
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=gate, up_out=up)
        assert torch.equal(h, (2 * wg[:, 0].clamp_min(0)).expand(T, F).contiguous() if g else torch.zeros_like(h)) and (up == 2).all()
        dx, dwg, dwu = _backward(ctx, torch.ones_like(h), x, wg, wu, gate, up)
        slope = {True: 1.0, False: 0.0}[g > 0] if g else 0.5
        assert (dwg[:, 0] == T * 2 * slope).all() and (dwg[:, 1:] == 0).all()
        assert torch.isfinite(dwu).all() and torch.isfinite(dx).all()


def test_gated_keeps_bad_rows_apart(ctx):
    """A token with an infinity or NaN changes its own row of h and dx, a row of
    weights its own column of h; the last columns and rows (in ragged tiles too)
    see nothing of what lies behind them."""
    for dt in DT.values():
        for T, d, F in ((3, 100, 50), (70, 130, 140)):
            x, wg, wu = _block(_gen(T), T, d, F, dt)
            h, g, u = (torch.empty(T, F, dtype=dt, device="cuda") for _ in range(3))
            moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
            x2, wg2 = x.clone(), wg.clone()
            x2[1, 0], wg2[7, d - 1] = float("nan"), float("inf")
            h2 = torch.empty_like(h)
            moe.moe_gated(ctx, x2, wg2, wu, h2)
            rows = [t for t in range(T) if t != 1]
            cols = [f for f in range(F) if f != 7]
            assert torch.equal(h2[rows][:, cols], h[rows][:, cols])
            assert torch.isnan(h2[1]).all() and not torch.isfinite(h2[rows][:, 7]).all()
            dh = _normal(_gen(5), T, F, dt)
            dx, _, _ = _backward(ctx, dh, x, wg, wu, g, u)
            dh2 = dh.clone()
            dh2[1, F - 1] = float("nan")
            dx2, dwg2, _ = _backward(ctx, dh2, x, wg, wu, g, u)
            assert torch.equal(dx2[rows], dx[rows]) and torch.isnan(dx2[1]).all()
            assert torch.isnan(dwg2[F - 1]).all() and torch.isfinite(dwg2[:F - 1]).all()


def test_gradient_against_differences(ctx):
    """<gradient, v> against central differences of the 64-bit block along random
    directions of x and the weights.  fp32 kernel, step 1e-3: the differences are
    good to their step's square (1e-6 times a third derivative of order one) and
    the gradient to fp32, so 1e-4 of the magnitudes leaves two orders."""
    T, d, F = 37, 48, 70
    gen = _gen(11)
    x, wg, wu = _block(gen, T, d, F, torch.float32)
    dh = _normal(gen, T, F, torch.float32)
    h, g, u = (torch.empty(T, F, device="cuda") for _ in range(3))
    moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
    dx, dwg, dwu = _backward(ctx, dh, x, wg, wu, g, u)

    def loss(x, wg, wu):
        return (_silu(x @ wg.t()) * (x @ wu.t()) * dh.double()).sum()

    base = [t.double() for t in (x, wg, wu)]
    for i, grad in enumerate((dx, dwg, dwu)):
        v = torch.randn(grad.shape, generator=gen, device="cuda").double()
        e = 1e-3
        hi = loss(*[t + e * v if j == i else t for j, t in enumerate(base)])
        lo = loss(*[t - e * v if j == i else t for j, t in enumerate(base)])
        want = float((hi - lo) / (2 * e))
        have = float((grad.double() * v).sum())
        scale = float((grad.double().abs() * v.abs()).sum()) / grad.numel() ** 0.5
        assert abs(have - want) <= 1e-4 * max(scale, abs(want)), (i, have, want, scale)


# ---- as they are used ----

def test_far_rows(ctx):
    """Rows further apart than 32 bits of bytes and of elements."""
    ld = (1 << 31) + 64
    big = torch.empty(ld + 4096, dtype=torch.bfloat16, device="cuda")
    gen = _gen(9)
    T, K, N = 2, 256, 48
    near = _normal(gen, T, K, torch.bfloat16)
    x = torch.as_strided(big, (T, K), (ld, 1))
    x.copy_(near)
    w = moe.QuantMatrix(ctx, *_quantised(gen, N, K, 64, True))
    a, b = (torch.empty(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_linear(ctx, near, w, a)
    out = torch.as_strided(big, (T, N), (ld, 1), 1024)
    moe.moe_linear(ctx, x, w, out)
    assert torch.equal(a, out.contiguous())
    _, wg, wu = _block(gen, T, K, N, torch.bfloat16)
    moe.moe_gated(ctx, near, wg, wu, a)
    moe.moe_gated(ctx, x, wg, wu, b)
    assert torch.equal(a, b)
    gate, up = _normal(gen, T, N, torch.bfloat16), _normal(gen, T, N, torch.bfloat16)
    dh = torch.as_strided(big, (T, N), (ld, 1), 2048)
    dh.copy_(_normal(gen, T, N, torch.bfloat16))
    for p, q in zip(_backward(ctx, dh, x, wg, wu, gate, up), _backward(ctx, dh.contiguous(), near, wg, wu, gate, up)):
        assert torch.equal(p, q)


def test_a_matrix_of_more_tiles_than_a_launch_has_workgroups(ctx):
    """The passes over a matrix go round where it has more than 2^20 tiles."""
    N, K, group = (1 << 20) + 5, 2080, 32
    gen = _gen(10)
    codes, scales, zeros = _quantised(gen, N, K, group, True)
    w = moe.QuantMatrix(ctx, codes, scales, zeros)
    out = torch.full((N, K), float("nan"), device="cuda")
    moe.moe_linear_dequant(ctx, w, out)
    x = _normal(gen, 1, K, torch.bfloat16)
    y = torch.empty(1, N, device="cuda")
    moe.moe_linear(ctx, x, w, y)
    for n in range(0, N, 1 << 15):
        e = slice(n, min(n + (1 << 15), N))
        ref, mag = _values((codes[e], scales[e], zeros[e]), group)
        assert torch.equal(out[e].double(), ref), n
        dot = x.double() @ ref.t()
        _close(y[:, e], dot, _linear_tol(x, mag, dot, torch.float32), n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_most_tokens(ctx, dtype):
    T, d, F, dt = 1 << 20, 32, 24, DT[dtype]
    gen = _gen(11)
    x, wg, wu = _block(gen, T, d, F, dt)
    X = x.double()
    q, r = _quantised(gen, F, d, 32, True), _quantised(gen, F, d, 32, True)
    p, s = moe.QuantMatrix(ctx, *q), moe.QuantMatrix(ctx, *r)
    (w, mag), (v, mag_v) = _values(q, 32), _values(r, 32)
    a, b = X @ w.t(), X @ v.t()
    D = (3 * 128 + d / 32 + 16) * U
    for yd in DT.values():
        extra = 2.0 ** -8 if _weights_rounded(T, dt, yd) else 0.0
        y = torch.empty(T, F, dtype=yd, device="cuda")
        moe.moe_linear(ctx, x, p, y)
        _close(y, a, _linear_tol(x, mag, a, yd) + extra * (X.abs() @ w.abs().t()))
        moe.moe_linear_gated(ctx, x, p, s, y)
        ta, tb = (D * (X.abs() @ m.t()) + extra * (X.abs() @ k.abs().t()) for m, k in ((mag, w), (mag_v, v)))
        h = _silu(a) * b
        _close(y, h, _gated_tol(a, b, ta, tb, h, yd))
    h, gate, up = (torch.empty(T, F, dtype=dt, device="cuda") for _ in range(3))
    moe.moe_gated(ctx, x, wg, wu, h, gate_out=gate, up_out=up)
    g, u = X @ wg.double().t(), X @ wu.double().t()
    tg, tu = (_chain(d, dt) * (X.abs() @ m.double().abs().t()) for m in (wg, wu))
    ref = _silu(g) * u
    _close(h, ref, _gated_tol(g, u, tg, tu, ref, dt))
    gate, dh = _cancels(gate), _normal(gen, T, F, dt)
    for name, y, (ref, tol) in zip(("dx", "dw_gate", "dw_up"), _backward(ctx, dh, x, wg, wu, gate, up),
                                   _backward_ref(dh, x, wg, wu, gate, up, dt)):
        _close(y, ref, tol, name)


def _step_buffers(gen, T, d, F, dt):
    x, wg, wu = _block(gen, T, d, F, dt)
    dh = _normal(gen, T, F, dt)
    h, g, u = (torch.empty(T, F, dtype=dt, device="cuda") for _ in range(3))
    return x, wg, wu, dh, h, g, u


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_step(ctx, dtype):
    """Forward and backward pass in a graph, replayed on new inputs with eager
    work between the replays, each replay against the eager result."""
    dt = DT[dtype]
    T, d, F = 70, 136, 200
    x, wg, wu, dh, h, g, u = _step_buffers(_gen(1), T, d, F, dt)
    q = moe.QuantMatrix(ctx, *_quantised(_gen(2), 96, 256, 32, True))
    xq, yq = torch.empty(3, 256, dtype=dt, device="cuda"), torch.empty(3, 96, dtype=dt, device="cuda")
    ws = torch.empty(moe.moe_gated_workspace(ctx, T, d, F, dt), dtype=torch.uint8, device="cuda")
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    xq.zero_()

    def step():
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
        moe.moe_gated_backward(ctx, dh, x, wg, wu, g, u, dx=dx, dw_gate=dwg, dw_up=dwu, workspace=ws)
        moe.moe_linear(ctx, xq, q, yq)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        gen = _gen(100 + i)
        x.copy_(_normal(gen, T, d, dt))
        dh.copy_(_normal(gen, T, F, dt))
        xq.copy_(_normal(gen, 3, 256, dt))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (h, dx, dwg, dwu, yq)]
        for t in (h, dx, dwg, dwu, yq):
            t.zero_()
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (h, dx, dwg, dwu, yq)):
            assert torch.equal(a, b)


def test_given_streams(ctx):
    """stream= as a torch stream and as its handle: the work is on that stream."""
    gen = _gen(4)
    w = moe.QuantMatrix(ctx, *_quantised(gen, 64, 256, 32, False))
    x, wg, wu, dh, h, g, u = _step_buffers(gen, 9, 256, 72, torch.bfloat16)
    want = torch.empty(9, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear(ctx, x, w, want)
    moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
    grads = _backward(ctx, dh, x, wg, wu, g, u)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for given in (s, s.cuda_stream):
        with torch.cuda.stream(s):
            torch.cuda._sleep(10_000_000)  # the buffers are filled late on that stream
            y, h2 = torch.zeros_like(want), torch.zeros_like(h)
            out = [torch.zeros_like(t) for t in grads]
            ws = torch.zeros(moe.moe_gated_workspace(ctx, 9, 256, 72, torch.bfloat16), dtype=torch.uint8, device="cuda")
        moe.moe_linear(ctx, x, w, y, stream=given)
        moe.moe_gated(ctx, x, wg, wu, h2, stream=given)
        moe.moe_gated_backward(ctx, dh, x, wg, wu, g, u, dx=out[0], dw_gate=out[1], dw_up=out[2], workspace=ws, stream=given)
        s.synchronize()
        assert torch.equal(y, want) and torch.equal(h2, h) and all(torch.equal(a, b) for a, b in zip(out, grads))


def test_two_streams_at_once(ctx):
    """Calls of one context on two streams, a workspace each, against the same calls in turn."""
    sizes = [(300, 512, 640), (260, 768, 384)]
    sets = [_step_buffers(_gen(i), *s, torch.bfloat16) for i, s in enumerate(sizes)]
    q = [moe.QuantMatrix(ctx, *_quantised(_gen(7 + i), 512, s[1], 32, True)) for i, s in enumerate(sizes)]

    def one(i):
        x, wg, wu, dh, h, g, u = sets[i]
        y = torch.empty(x.shape[0], 512, dtype=torch.bfloat16, device="cuda")
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
        moe.moe_linear(ctx, x, q[i], y)
        return [h.clone(), y, *_backward(ctx, dh, x, wg, wu, g, u)]

    want = [one(0), one(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(3):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = one(i)
    torch.cuda.synchronize()
    for i in (0, 1):
        for a, b in zip(want[i], got[i]):
            assert torch.equal(a, b)


def test_tune_quantise_serve_beside_the_experts():
    """A dense block as it is used: a step of tuning changes the weights along
    their gradient, the result is held in 4 bits (nearest code, a scale and zero
    point for 64 columns) and serves a token next to a routed layer of the same
    context; every stage against its 64-bit formula on the stage's own inputs."""
    wl = dict(synth.workload("tiny"))
    cx = H.make_ctx(wl, n_slots=wl["E"])
    d, F, T = wl["d"], 320, 24
    dt = torch.bfloat16
    x, wg, wu, dh, h, g, u = _step_buffers(_gen(21), T, d, F, dt)
    moe.moe_gated(cx, x, wg, wu, h, gate_out=g, up_out=u)
    g.copy_(_cancels(g))
    dx, dwg, dwu = _backward(cx, dh, x, wg, wu, g, u)
    for y, (ref, tol) in zip((dx, dwg, dwu), _backward_ref(dh, x, wg, wu, g, u, dt)):
        _close(y, ref, tol)
    wg, wu = (wg.float() - 1e-3 * dwg.float()).to(dt), (wu.float() - 1e-3 * dwu.float()).to(dt)
    wd = _normal(_gen(22), d, F, dt, F ** -0.5)

    def quantise(w, group=64):
        v = w.float().reshape(w.shape[0], -1, group)
        lo, hi = v.amin(-1).clamp_max(0), v.amax(-1).clamp_min(0)
        s = ((hi - lo) / 15).clamp_min(1e-4).half()
        z = (-lo / s.float()).round().clamp(0, 15)
        c = (v / s.float().unsqueeze(-1) + z.unsqueeze(-1)).round().clamp(0, 15).reshape(w.shape).to(torch.uint8)
        return (c[:, 0::2] | c[:, 1::2] << 4).contiguous(), s, z.to(torch.uint8)

    qs = [quantise(w) for w in (wg, wu, wd)]
    mats = [moe.QuantMatrix(cx, *q) for q in qs]
    for w, q in zip((wg, wu, wd), qs):  # within half a step of the weights (a code more where both ends are clamped)
        step = q[1].double().repeat_interleave(64, 1)
        assert ((_values(q, 64)[0] - w.double()).abs() <= 1.01 * step).all()

    # one token: the routed layer and the dense block, then their sum
    tok = H.torch_x(synth.activations(wl["seed"], 1, d, "bf16"), "bf16")
    recs = [synth.expert_record(wl["seed"], 0, e, wl["qtype"], d, wl["f"]) for e in range(wl["E"])]
    for e in range(wl["E"]):
        H.put_expert(cx, e, recs[e])
        moe.moe_slot_bind(cx, 0, e, e)
    ids = torch.empty(1, wl["k"], dtype=torch.int32, device="cuda")
    tw = torch.empty(1, wl["k"], dtype=torch.float32, device="cuda")
    plan = moe.Plan(cx, 1)
    y_routed, y_dense = torch.empty(1, d, device="cuda"), torch.empty(1, d, device="cuda")
    wr = torch.from_numpy(synth.router_weights(wl["seed"], wl["E"], d)).cuda()
    hid = torch.empty(1, F, dtype=dt, device="cuda")
    moe.moe_route_ffn(cx, 0, tok, ids, tw, plan, y_routed, w_router=wr)
    moe.moe_linear_gated(cx, tok, mats[0], mats[1], hid)
    moe.moe_linear(cx, hid, mats[2], y_dense)
    assert moe.moe_check(cx) == moe.MOE_OK and torch.isfinite(y_routed).all()
    X = tok.double()
    (a, ma), (b, mb), (c, mc) = (_values(q, 64) for q in qs)
    gg, uu = X @ a.t(), X @ b.t()
    D = (3 * 128 + d / 32 + 16) * U
    ref = _silu(gg) * uu
    _close(hid, ref, _gated_tol(gg, uu, D * (X.abs() @ ma.t()), D * (X.abs() @ mb.t()), ref, dt), "hidden")
    ref = hid.double() @ c.t()
    _close(y_dense, ref, _linear_tol(hid, mc, ref, torch.float32), "down")
