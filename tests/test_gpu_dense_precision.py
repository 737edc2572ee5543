"""GPU: what the dense operators' sums are taken in, pinned where a rounding to
fewer bits would show.

Products with 4-bit weights round neither weights nor x, whatever the number of
tokens and the types: y is fp32's sum, rounded to y's type once.  The sum of one
group (128 columns at most) is exact products added in fp32; a term passes
through 128 additions there, as 16 + q or q - z with its correction for z, then
2 roundings for scale and zero point, then at most cols / 32 + 16 additions over
groups, waves and parts: |error| <= (3 * 128 + cols / 32 + 16) 2^-24 sum |s| (32 + q + z) |x|,
and half a step of y's type.
"""
import pytest

from tests import harness as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not H.gpu_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

from routed_expert_execution_amd import moe  # noqa: E402

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ctx():
    cfg = moe.make_config(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)
    pool = torch.zeros(moe.moe_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    return moe.Context(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=0, slot_pool=pool)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantised(gen, N, K, group, affine):
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.randn(N, K // group, generator=gen, device="cuda") * 0.01).to(torch.float16)
    zeros = torch.randint(0, 256, (N, K // group), generator=gen, device="cuda", dtype=torch.uint8) if affine else None
    return codes, scales, zeros


def _values(q, group):
    """s (q - z) and |s| (32 + q + z) in 64 bits."""
    codes, scales, zeros = q
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).double()
    z = torch.full_like(scales, 8.0, dtype=torch.float64) if zeros is None else zeros.double()
    z, s = z.repeat_interleave(group, 1), scales.double().repeat_interleave(group, 1)
    return s * (c - z), s.abs() * (32 + c + z)


def _bound(x, mag):
    return (3 * 128 + x.shape[1] / 32 + 16) * U * (x.double().abs() @ mag.t())


def _within(y, ref, tol):
    bad = ~((y.double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs() + 1e-30)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), y[bad][:4].tolist(), ref[bad][:4].tolist(), tol[bad][:4].tolist())


# T, K, N: few and many tiles of every shape, whole and half last steps, rows that
# can and cannot be loaded 16 bytes a lane (pad)
EXACT = [(128, 1024, 4096, 0), (300, 2048, 520, 0), (106, 2304, 3360, 0), (130, 1056, 2000, 0), (1000, 1024, 5504, 0), (2048, 1024, 4096, 0),
         (2000, 544, 4100, 5), (1500, 1120, 2050, 3), (147, 1792, 1988, 4), (70, 160, 9000, 0), (4096, 512, 333, 8)]


@pytest.mark.parametrize("group,affine", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("T,K,N,pad", EXACT)
def test_many_tokens_round_no_weight(ctx, T, K, N, pad, group, affine):
    K = (K + group - 1) // group * group
    print("exact", T, K, N, pad, group, affine, flush=True)
    gen = _gen(T + K + N + group)
    x = torch.randn(T, K + pad, generator=gen, device="cuda").to(BF16)[:, :K]
    q, r = _quantised(gen, N, K, group, affine), _quantised(gen, N, K, group, affine)
    p, s = moe.QuantMatrix(ctx, *q), moe.QuantMatrix(ctx, *r)
    y = torch.full((T, N + pad), 777.0, dtype=BF16, device="cuda")
    moe.moe_linear(ctx, x, p, y[:, :N])
    (w, mw), (v, mv) = _values(q, group), _values(r, group)
    X = x.double()
    g, u = X @ w.t(), X @ v.t()
    tg, tu = _bound(x, mw), _bound(x, mv)
    _within(y[:, :N], g, tg)
    moe.moe_linear_gated(ctx, x, p, s, y[:, :N])
    # |silu'| <= 1.1, and 8 steps of fp32 for the logistic function (at g far
    # below zero 2 |g| more, of its argument, where silu itself vanishes)
    h = g * torch.sigmoid(g) * u
    _within(y[:, :N], h, 1.1 * tg * (u.abs() + tu) + (g * torch.sigmoid(g)).abs() * tu + (8 + 2 * g.abs()) * U * h.abs())
    assert (y[:, N:] == 777.0).all()


# ---- fp32 factors as three bf16 terms ----
#
# Against the identity a product is its other factor, so that the terms' sum shows:
# all 24 bits of a value from 2^-110 up (two terms would leave 2^-17 of it), and at
# most 2^-134, half of bf16's least value, off below that.

def _whole(gen, rows, cols, e):
    """fp32 values of 24 bits and both signs in [2^e, 2^(e + 1))."""
    m = 1 + torch.rand(rows, cols, generator=gen, device="cuda", dtype=torch.float64)
    return (m * torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 0.5, -1.0, 1.0) * 2.0 ** e).float()


def _same(y, x, e, what):
    if e >= -110:
        assert torch.equal(y, x), (what, e, (y - x).abs().max())
    else:
        assert ((y.double() - x.double()).abs() <= 2.0 ** -134).all(), (what, e)


EXPONENTS = [-130, -120, -111, -110, -60, -1, 0, 40, 110]


@pytest.mark.parametrize("T,N", [(1, 128), (9, 128), (9, 4224), (40, 128)])
def test_fp32_x_is_whole_in_4_bit_products(ctx, T, N):
    """Codes of 9 on the diagonal and of 8, the zero point, elsewhere."""
    K = 128
    c = torch.full((N, K), 8, dtype=torch.uint8, device="cuda")
    c[:K].fill_diagonal_(9)
    w = moe.QuantMatrix(ctx, (c[:, 0::2] | c[:, 1::2] << 4).contiguous(), torch.ones(N, 1, dtype=torch.float16, device="cuda"))
    for e in EXPONENTS:
        x = _whole(_gen(e + 200), T, K, e)
        y = torch.empty(T, N, device="cuda")
        moe.moe_linear(ctx, x, w, y)
        _same(y[:, :K], x, e, "x")
        assert (y[:, K:] == 0).all()


# (T, d, F) of the rows kernels, and of each tile
@pytest.mark.parametrize("T,F,kind", [(3, 130, 0), (16, 130, 0), (40, 130, 0), (18, 4365, 2), (21, 8949, 2), (4099, 132, 2)])
def test_fp32_factors_are_whole_in_the_gated_block(ctx, T, F, kind):
    d = 128 if F < 4000 else 132
    assert moe.moe_gated_plan(T, d, F, F32)[0] == kind
    n = min(d, F)
    eye = torch.zeros(F, d, device="cuda")
    eye[:n].fill_diagonal_(1.0)
    for e in EXPONENTS:
        x = _whole(_gen(e + 300), T, d, e)
        wg, wu = eye, 2 * eye
        h, gate, up = (torch.empty(T, F, device="cuda") for _ in range(3))
        moe.moe_gated(ctx, x, wg, wu, h, gate_out=gate, up_out=up)
        _same(gate[:, :n], x[:, :n], e, "gate")
        _same(up[:, :n] / 2, x[:, :n], e, "up")
        # the weights' bits: tokens that are unit vectors
        tokens = torch.zeros(T, d, device="cuda")
        tokens[:min(T, d)].fill_diagonal_(1.0)
        m = min(T, d)
        wg, wu = _whole(_gen(e + 400), F, d, e), _whole(_gen(e + 500), F, d, e)
        moe.moe_gated(ctx, tokens, wg, wu, h, gate_out=gate, up_out=up)
        _same(gate[:m], wg[:, :m].t(), e, "w_gate")
        _same(up[:m], wu[:, :m].t(), e, "w_up")


@pytest.mark.parametrize("T,d,F", [(129, 2384, 115), (107, 116, 105), (141, 916, 1051), (145, 2373, 121)])
def test_fp32_factors_are_whole_in_the_backward_pass(ctx, T, d, F):
    """With gate 0 and up 2, dg is dh and du is 0: against identities dx is dh and
    dw_gate its transpose; against unit vectors they are the weights and x."""
    ws = torch.empty(moe.moe_gated_workspace(ctx, T, d, F, F32), dtype=torch.uint8, device="cuda")
    zero, two = torch.zeros(T, F, device="cuda"), torch.full((T, F), 2.0, device="cuda")
    dx, dwg, dwu = (torch.empty(s, device="cuda") for s in ((T, d), (F, d), (F, d)))

    def backward(dh, x, wg):
        moe.moe_gated_backward(ctx, dh, x, wg, wg, zero, two, dx=dx, dw_gate=dwg, dw_up=dwu, workspace=ws)

    eye_w, eye_x, eye_h = torch.zeros(F, d, device="cuda"), torch.zeros(T, d, device="cuda"), torch.zeros(T, F, device="cuda")
    a, b, c = min(F, d), min(T, d), min(T, F)
    eye_w[:a].fill_diagonal_(1.0), eye_x[:b].fill_diagonal_(1.0), eye_h[:c].fill_diagonal_(1.0)
    for e in EXPONENTS:
        dh, x, wg = (_whole(_gen(e + i), *s, e) for i, s in ((600, (T, F)), (700, (T, d)), (800, (F, d))))
        backward(dh, eye_x, eye_w)
        _same(dx[:, :a], dh[:, :a], e, "dx")
        _same(dwg[:, :b], dh[:b].t(), e, "dw_gate")
        backward(eye_h, x, wg)
        _same(dx[:c], wg[:c], e, "w_gate")
        _same(dwg[:c], x[:c], e, "x")


def test_fp32_products_of_whole_factors(ctx):
    """One product a sum: what the six products of terms leave out is below 2^-24 of
    it, and its additions round 6 times: 16 steps of 2^-24 hold, of which the two
    terms of a shorter splitting would leave 2^7 of those out."""
    for T, F, d in ((18, 4365, 132), (21, 8949, 132), (4099, 132, 132)):
        assert moe.moe_gated_plan(T, d, F, F32)[0] == moe.MOE_PLAN_TILES
        x = _whole(_gen(T), T, d, 0)
        diagonal = _whole(_gen(F), 1, d, 0)[0]
        w = torch.zeros(F, d, device="cuda")
        w[:d] = torch.diag(diagonal)
        h, gate, up = (torch.empty(T, F, device="cuda") for _ in range(3))
        moe.moe_gated(ctx, x, w, w, h, gate_out=gate, up_out=up)
        want = x.double() * diagonal.double()
        assert ((gate[:, :d].double() - want).abs() <= 16 * U * want.abs()).all()


# ---- large x ----

@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("T,N", [(1, 4160), (9, 4160), (24, 4160), (40, 4160), (60, 4160), (300, 20800)])
def test_x_below_2_to_112(ctx, T, N, group):
    """The largest codes and zero points and x of one sign near the documented end:
    (16 + 255) * 128 * 2^112 < 2^128, so no sum on the way to a result in range
    overflows; the tiles (T = 300) sum q - z."""
    K = 256
    codes = torch.full((N, K // 2), 0xFF, dtype=torch.uint8, device="cuda")
    scales = torch.full((N, K // group), 2.0 ** -12, device="cuda").half()
    zeros = torch.full((N, K // group), 255, dtype=torch.uint8, device="cuda")
    zeros[::2] = 0
    w = moe.QuantMatrix(ctx, codes, scales, zeros)
    for dt in (BF16, F32):
        x = torch.full((T, K), 2.0 ** 112 * (1 - 2.0 ** -8), device="cuda").to(dt)
        ref = x.double() @ _values((codes, scales, zeros), group)[0].t()
        for yd in (BF16, F32):
            y = torch.empty(T, N, dtype=yd, device="cuda")
            moe.moe_linear(ctx, x, w, y)
            tol = _bound(x, _values((codes, scales, zeros), group)[1]) + ref.abs() * (2.0 ** -8 if yd == BF16 else U)
            assert ((y.double() - ref).abs() <= tol).all()
