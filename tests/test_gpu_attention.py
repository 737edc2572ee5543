"""GPU: attention over packed sequences and its backward pass against their formulas in 64 bits."""
import math

import pytest

from tests import harness as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not H.gpu_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

from routed_expert_execution_amd import moe  # noqa: E402
from tests import attention_cases as A  # noqa: E402
from tests.attention_cases import BF16, F32  # noqa: E402


@pytest.fixture(scope="module")
def ctx():
    return A.context()


def _inputs(seed, lq, lk, heads, Hkv, D, dtype, gap=0, tail=0):
    g = A.gen(seed)
    q = A.normal(g, sum(lq) + tail, heads, D, dtype, gap)
    k, v = (A.normal(g, sum(lk) + tail, Hkv, D, dtype, gap) for _ in range(2))
    return q, k, v, A.offsets(lq), A.offsets(lk)


def _forward(ctx, q, k, v, oq, ok, **kw):
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    moe.moe_attention(ctx, q, k, v, oq, out, lse=lse, offsets_k=ok, **kw)
    return out, lse


def _backward(ctx, dout, q, k, v, out, lse, oq, ok, gap=0, **kw):
    grads = []
    for t in (q, k, v):
        T, heads, D = t.shape
        grads.append(torch.full((T, heads * D + gap), 7.0, dtype=t.dtype, device="cuda")[:, : heads * D].unflatten(1, (heads, D)))
    ws = torch.empty(moe.moe_attention_workspace(ctx, q), dtype=torch.uint8, device="cuda")
    moe.moe_attention_backward(ctx, dout, q, k, v, out, lse, oq, dq=grads[0], dk=grads[1], dv=grads[2], workspace=ws, offsets_k=ok, **kw)
    return grads


def _sequences(lq, lk):
    a = b = 0
    for n, m in zip(lq, lk):
        yield slice(a, a + n), slice(b, b + m), n, m
        a, b = a + n, b + m


def _term(dtype):
    """What an exponential, or dS, loses on its way into the second product: rounded to bf16, or three bf16 terms."""
    return A.HALF[BF16] if dtype == BF16 else 2 * A.U


def _score_error(q, k, scale):
    """A score is a sum of D products in fp32 (D + 4 half steps of the sum of their
    magnitudes); its product with scale / ln 2, the maximum's, and their difference
    are four more.  An exponential is 2^-21 off, relative."""
    return (q.shape[-1] + 8) * A.U * scale * (q.abs() @ k.abs().t().contiguous())


def _check_forward(q, k, v, out, lse, lq, lk, scale, causal=True, window=0):
    per = q.shape[1] // k.shape[1]
    for rq, rk, n, m in _sequences(lq, lk):
        if not n:
            continue
        seen = A.visible(n, m, causal, window)
        for h in range(q.shape[1]):
            qd, kd, vd = q[rq, h].double(), k[rk, h // per].double(), v[rk, h // per].double()
            ref, p, s = A.attend(qd, kd, vd, scale, seen) if m else (torch.zeros_like(qd), None, None)
            if not m:
                assert (out[rq, h] == 0).all() and (lse[rq, h] == -math.inf).all()
                continue
            score = torch.where(seen, _score_error(qd, kd, scale), torch.zeros_like(s)).amax(-1)
            rel = 2 * score + 2.0 ** -20
            mag = p @ vd.abs()
            tol = 2 * rel.unsqueeze(-1) * mag + _term(q.dtype) * mag + (m / 16 + 8) * A.U * mag + A.HALF[q.dtype] * ref.abs() + 1e-30
            A.close(out[rq, h], ref, tol)
            want = torch.logsumexp(s, -1)
            empty = ~seen.any(-1)
            assert (lse[rq, h][empty] == -math.inf).all() and (out[rq, h][empty] == 0).all()
            A.close(lse[rq, h][~empty], want[~empty], (2 * score + 2.0 ** -19 + 4 * A.U * want.abs() + m * A.U)[~empty])


def _check_backward(dout, q, k, v, out, lse, grads, lq, lk, scale, causal=True, window=0):
    per, D, dtype = q.shape[1] // k.shape[1], q.shape[2], q.dtype
    half, term = A.HALF[dtype], _term(dtype)
    for rq, rk, n, m in _sequences(lq, lk):
        seen = A.visible(n, m, causal, window) if n and m else None
        for kh in range(k.shape[1]):
            kd, vd = k[rk, kh].double(), v[rk, kh].double()
            dk, dv = torch.zeros_like(kd), torch.zeros_like(vd)
            tk, tv = torch.zeros_like(kd), torch.zeros_like(vd)
            for h in range(kh * per, (kh + 1) * per):
                qd, od, gd = q[rq, h].double(), out[rq, h].double(), dout[rq, h].double()
                if not n or not m:
                    assert (grads[0][rq, h] == 0).all()
                    continue
                L = lse[rq, h].double().unsqueeze(-1)
                s = (qd @ kd.t()) * scale
                p = torch.where(seen, torch.exp(torch.where(seen, s - L, torch.zeros_like(s))), torch.zeros_like(s))
                rel = _score_error(qd, kd, scale) + 4 * A.U * torch.where(L.isfinite(), L.abs(), torch.zeros_like(L)) + 2.0 ** -20
                dp, delta = gd @ vd.t(), (gd * od).sum(-1, keepdim=True)
                ds = p * (dp - delta)
                e_dp = (D + 8) * A.U * (gd.abs() @ vd.abs().t() + (gd * od).abs().sum(-1, keepdim=True))
                e_ds = p * e_dp * (1 + rel) + (rel + term) * ds.abs()
                passes = (max(n, m) * per / 16 + 16) * A.U
                ref = scale * (ds @ kd)
                A.close(grads[0][rq, h], ref, scale * (e_ds @ kd.abs() + passes * (ds.abs() @ kd.abs())) + half * ref.abs() + 1e-30)
                dk += scale * (ds.t() @ qd)
                tk += scale * (e_ds.t() @ qd.abs() + passes * (ds.abs().t() @ qd.abs()))
                dv += p.t() @ gd
                tv += (rel * p + (term + passes) * p).t() @ gd.abs()
            if m:
                A.close(grads[1][rk, kh], dk, tk + half * dk.abs() + 1e-30)
                A.close(grads[2][rk, kh], dv, tv + half * dv.abs() + 1e-30)


CASES = [
    # queries, keys (None: the same), heads, key heads, D, causal, window, dtype, gap
    ([1], None, 1, 1, 64, True, 0, BF16, 0), ([2], None, 3, 1, 96, True, 0, F32, 0), ([31, 32, 33], None, 4, 2, 64, True, 0, BF16, 0),
    ([127, 128, 129], None, 2, 1, 128, True, 0, BF16, 8), ([300], None, 4, 2, 128, False, 0, BF16, 0), ([65, 1, 0, 200], None, 6, 2, 192, True, 0, BF16, 5),
    ([257], None, 2, 2, 256, True, 0, BF16, 0), ([100, 61], None, 2, 1, 64, True, 0, F32, 3), ([130], None, 2, 2, 128, False, 0, F32, 0),
    ([90], None, 3, 3, 192, True, 0, F32, 0), ([140], None, 2, 1, 256, True, 0, F32, 0), ([200, 33], None, 2, 1, 64, True, 50, BF16, 0),
    ([333], None, 4, 4, 128, True, 1, BF16, 0), ([150], None, 2, 1, 96, True, 64, F32, 0), ([40, 7], [170, 300], 4, 2, 128, True, 0, BF16, 0),
    ([170, 5], [40, 5], 4, 2, 128, True, 0, BF16, 0), ([170, 5], [40, 9], 2, 1, 96, False, 0, F32, 0), ([3, 4, 0], [0, 70, 9], 2, 2, 64, True, 0, BF16, 0),
    ([100], [300], 2, 1, 64, True, 130, F32, 0), ([500], [130], 2, 1, 64, True, 40, BF16, 0), ([700], None, 7, 1, 64, True, 0, BF16, 0),
    ([5] * 70, None, 2, 1, 64, True, 0, BF16, 0), ([1, 700], [400, 3], 2, 2, 256, False, 0, BF16, 0), ([161], None, 2, 2, 96, False, 0, BF16, 0),
    # long enough for steps without a mask, an odd and an even number of them, between others
    ([1100, 70], None, 6, 2, 128, True, 0, BF16, 0), ([900], None, 4, 4, 96, False, 0, BF16, 8), ([777], None, 8, 1, 64, True, 300, BF16, 0),
    ([640], [1000], 3, 1, 128, True, 0, BF16, 5), ([900, 450], None, 2, 1, 128, True, 500, BF16, 3), ([1000], [300], 4, 2, 64, False, 0, BF16, 0),
    ([400], None, 4, 2, 192, True, 0, F32, 0), ([300, 100], None, 2, 1, 256, True, 0, F32, 3), ([520], None, 4, 1, 128, True, 200, F32, 0), ([600], None, 2, 1, 256, True, 0, BF16, 0),
    # workgroups enough for dK and dV by one each, in fp32
    ([700, 333], None, 16, 8, 64, True, 0, F32, 0), ([600, 500], None, 16, 8, 96, False, 0, F32, 4),
    # more rows than go by parts of the keys: bf16 from 64 tiles of 128 rows times heads on, fp32 from 200
    ([130] * 5, None, 12, 4, 64, True, 0, BF16, 0), ([260, 40], [300, 90], 32, 8, 128, True, 90, BF16, 3), ([400, 20], None, 16, 2, 192, True, 0, BF16, 0),
    ([333], None, 24, 4, 256, False, 0, BF16, 8), ([130] * 9, None, 12, 4, 64, True, 0, F32, 0), ([260, 40], [300, 90], 64, 8, 128, True, 90, F32, 3),
    ([140] * 4, None, 26, 2, 192, True, 0, F32, 0), ([300], None, 80, 4, 256, True, 0, F32, 0)]


@pytest.mark.parametrize("lq,lk,heads,Hkv,D,causal,window,dtype,gap", CASES)
def test_attention(ctx, lq, lk, heads, Hkv, D, causal, window, dtype, gap):
    lk = lk or lq
    q, k, v, oq, ok = _inputs(sum(lq) + D, lq, lk, heads, Hkv, D, dtype, gap, tail=3)
    kw = dict(causal=causal, window=window)
    out, lse = _forward(ctx, q, k, v, oq, ok, **kw)
    n, m = sum(lq), sum(lk)
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()  # the rows behind the last sequence
    _check_forward(q, k, v, out, lse, lq, lk, D ** -0.5, **kw)
    dout = A.normal(A.gen(9), n + 3, heads, D, dtype, gap)
    grads = _backward(ctx, dout, q, k, v, out, lse, oq, ok, gap, **kw)
    assert (grads[0][n:] == 7).all() and (grads[1][m:] == 7).all() and (grads[2][m:] == 7).all()
    _check_backward(dout, q, k, v, out, lse, grads, lq, lk, D ** -0.5, **kw)
    assert moe.moe_check(ctx) == moe.MOE_OK
    again, lse2 = _forward(ctx, q, k, v, oq, ok, **kw)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    for a, b in zip(grads, _backward(ctx, dout, q, k, v, out, lse, oq, ok, gap, **kw)):
        assert torch.equal(a, b)
    alone = torch.empty_like(out[:n])
    moe.moe_attention(ctx, q[:n], k[:m], v[:m], oq, alone, offsets_k=ok, **kw)  # without lse
    assert torch.equal(alone, out[:n])


@pytest.mark.parametrize("heads", [2, 100])  # few rows, and many
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_and_sharp_rows(ctx, dtype, heads):
    """Scores far apart, all equal, and a scale of its own."""
    for factor, scale in ((40.0, 1.0), (0.0, 1.0), (1.0, 2.5), (1.0, 1e-20)):
        q, k, v, oq, ok = _inputs(5, [150], [150], heads, 1, 64, dtype)
        q = (q * factor).contiguous()
        out, lse = _forward(ctx, q, k, v, oq, ok, scale=scale)
        _check_forward(q, k, v, out, lse, [150], [150], scale)
        dout = A.normal(A.gen(2), 150, heads, 64, dtype)
        _check_backward(dout, q, k, v, out, lse, _backward(ctx, dout, q, k, v, out, lse, oq, ok, scale=scale), [150], [150], scale)


def test_gradients_are_differences(ctx):
    """Central differences of <dout, out> in 64 bits, along directions of each input."""
    lq, lk, D, scale = [37, 20], [50, 20], 64, 0.2
    q, k, v, oq, ok = _inputs(11, lq, lk, 4, 2, D, F32)
    dout = A.normal(A.gen(3), sum(lq), 4, D, F32)
    out, lse = _forward(ctx, q, k, v, oq, ok, scale=scale)
    grads = _backward(ctx, dout, q, k, v, out, lse, oq, ok, scale=scale)

    def value(q, k, v):
        total = 0.0
        for rq, rk, n, m in _sequences(lq, lk):
            for h in range(4):
                o, _, _ = A.attend(q[rq, h], k[rk, h // 2], v[rk, h // 2], scale, A.visible(n, m))
                total = total + (o * dout[rq, h].double()).sum()
        return total

    x, step = [t.double() for t in (q, k, v)], 1e-5
    for i in range(3):
        for seed in range(3):
            way = A.normal(A.gen(20 + seed), *x[i].shape, F32).double()
            there = [t + step * way if j == i else t for j, t in enumerate(x)]
            back = [t - step * way if j == i else t for j, t in enumerate(x)]
            diff = (value(*there) - value(*back)) / (2 * step)
            got = (grads[i].double() * way).sum()
            # differences: step^2 of third derivatives, and 2^-53 / step; gradients: 1e-5 of their magnitudes (fp32 sums of this size, checked above)
            assert abs(got - diff) <= 1e-5 * (grads[i].double() * way).abs().sum() + 1e-6


def test_packed_is_one_by_one(ctx):
    """Sequences packed give what each gives alone, bit for bit, wherever it lies."""
    lengths = [130, 1, 64, 200]
    q, k, v, oq, ok = _inputs(4, lengths, lengths, 4, 2, 128, BF16)
    out, lse = _forward(ctx, q, k, v, oq, ok)
    dout = A.normal(A.gen(6), sum(lengths), 4, 128, BF16)
    grads = _backward(ctx, dout, q, k, v, out, lse, oq, ok)
    for r, _, n, _ in _sequences(lengths, lengths):
        one = A.ints([0, n])
        o, s = _forward(ctx, q[r], k[r], v[r], one, one)
        assert torch.equal(o, out[r]) and torch.equal(s, lse[r])
        for a, b in zip(grads, _backward(ctx, dout[r], q[r], k[r], v[r], o, s, one, one)):
            assert torch.equal(a[r], b)


@pytest.mark.parametrize("heads", [2, 80])  # few rows, and many
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_adds_nothing(ctx, dtype, value, heads):
    """Infinities and NaN in keys, values, queries and gradients: rows and keys that do
    not see them keep their bits, those that see them are NaN (in the value's channel)."""
    n, at, D, window = 150, 70, 64, 20
    for win in (0, window):
        kw = dict(window=win)
        q, k, v, oq, ok = _inputs(8, [n, 40], [n, 40], heads, 1, D, dtype)
        dout = A.normal(A.gen(1), n + 40, heads, D, dtype)
        out, lse = _forward(ctx, q, k, v, oq, ok, **kw)
        grads = _backward(ctx, dout, q, k, v, out, lse, oq, ok, **kw)
        row = torch.arange(n + 40, device="cuda")
        sees = (row >= at) & (row < n) & ((row < at + win) if win else True)  # the rows that see key `at`
        seen = (row <= at) & ((row > at - win) if win else True)              # the keys that row `at` sees

        w = v.clone()
        w[at, 0, 5] = value
        o, s = _forward(ctx, q, k, w, oq, ok, **kw)
        assert torch.equal(s, lse) and torch.equal(o[~sees], out[~sees])
        assert not o[sees][..., 5].isfinite().any()
        others = torch.arange(D, device="cuda") != 5
        assert torch.equal(o[..., others], out[..., others])

        x = k.clone()
        x[at, 0, 5] = value
        o, s = _forward(ctx, q, x, v, oq, ok, **kw)
        assert torch.equal(o[~sees], out[~sees]) and torch.equal(s[~sees], lse[~sees])
        bad = _backward(ctx, dout, q, x, v, out, lse, oq, ok, **kw)
        assert torch.equal(bad[0][~sees], grads[0][~sees]) and not bad[0][sees][..., 5].isfinite().any()

        for which in ("q", "dout"):
            y, g = q.clone(), dout.clone()
            (y if which == "q" else g)[at, 1, 5] = value
            bad = _backward(ctx, g, y, k, v, out, lse, oq, ok, **kw)
            for a, b in zip(bad[1:], grads[1:]):
                assert torch.equal(a[~seen], b[~seen])
            for a, b in zip(bad[:1], grads[:1]):
                keep = torch.ones(n + 40, heads, dtype=torch.bool, device="cuda")
                keep[at, 1] = False
                assert torch.equal(a[keep], b[keep])
            assert not bad[1][seen][..., 5].isfinite().any() if which == "q" else not bad[2][seen][..., 5].isfinite().any()


@pytest.mark.parametrize("heads", [2, 20])  # few rows, and many
def test_offsets_that_cannot_be(ctx, heads):
    """NaN for that sequence, error word, the others as ever, nothing outside."""
    q, k, v, good, _ = _inputs(2, [40, 50, 60], [40, 50, 60], heads, 1, 64, BF16, tail=10)
    out, lse = _forward(ctx, q, k, v, good, good)
    dout = A.normal(A.gen(1), 160, heads, 64, BF16)
    grads = _backward(ctx, dout, q, k, v, out, lse, good, good)
    assert moe.moe_check(ctx) == moe.MOE_OK
    for off, keep in (([0, 40, 90, 161], slice(0, 90)), ([-3, 40, 90, 150], slice(40, 150)), ([0, 40, 90, 2 ** 31 - 1], slice(0, 90))):
        bad = A.ints(off)
        o, s = _forward(ctx, q, k, v, bad, bad)
        assert moe.moe_check(ctx) == moe.MOE_EINVAL and moe.moe_check(ctx) == moe.MOE_OK
        assert torch.equal(o[keep], out[keep]) and torch.equal(s[keep], lse[keep])
        gone = [i for i in range(150) if not keep.start <= i < keep.stop]
        assert o[gone].isnan().all() and s[gone].isnan().all()
        b = _backward(ctx, dout, q, k, v, out, lse, bad, bad)
        assert moe.moe_check(ctx) == moe.MOE_EINVAL
        for x, y in zip(b, grads):
            assert torch.equal(x[keep], y[keep]) and x[gone].isnan().all()
    # descending: in bounds, and said
    _backward(ctx, dout, q, k, v, out, lse, A.ints([0, 90, 40, 150]), A.ints([0, 90, 40, 150]))
    assert moe.moe_check(ctx) == moe.MOE_EINVAL


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [128, 256])
def test_keys_without_queries(ctx, dtype, D):
    """No queries at all, or no keys at all: gradients of zero, rows of zero."""
    k, v = (A.normal(A.gen(6), 70, 2, D, dtype) for _ in range(2))
    none, off, empty = torch.empty(0, 4, D, dtype=dtype, device="cuda"), A.ints([0, 30, 70]), A.ints([0, 0, 0])
    dk, dv = torch.full_like(k, 7), torch.full_like(v, 7)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    moe.moe_attention(ctx, none, k, v, empty, none, offsets_k=off)
    moe.moe_attention_backward(ctx, none, none, k, v, none, torch.empty(0, 4, device="cuda"), empty, dq=none, dk=dk, dv=dv, workspace=ws, offsets_k=off)
    assert not dk.any() and not dv.any()
    q, nothing = A.normal(A.gen(7), 70, 4, D, dtype), torch.empty(0, 2, D, dtype=dtype, device="cuda")
    out, lse = _forward(ctx, q, nothing, nothing, off, empty)
    assert not out[:70].any() and (lse[:70] == -math.inf).all()
    dq = torch.full_like(q, 7)
    ws = torch.empty(moe.moe_attention_workspace(ctx, q), dtype=torch.uint8, device="cuda")
    moe.moe_attention_backward(ctx, q, q, nothing, nothing, out, lse, off, dq=dq, dk=nothing, dv=nothing, workspace=ws, offsets_k=empty)
    assert not dq.any() and moe.moe_check(ctx) == moe.MOE_OK


def test_a_tuning_step_captured(ctx):
    """Rotate, attend and back, captured once; each replay on new inputs and other lengths
    against the eager calls; and both on two streams at once."""
    D, heads, Hkv, T = 128, 4, 2, 300
    g = A.gen(12)
    off = A.ints([0, 100, 300])
    positions, rotary = torch.arange(T, dtype=torch.int32, device="cuda"), moe.Rotary(ctx, A.frequencies(D))
    fused, dout = (torch.zeros(T, n, D, dtype=BF16, device="cuda") for n in (heads + 2 * Hkv, heads))

    class Side:
        def __init__(self):
            self.q, self.out, self.dq = (torch.empty(T, heads, D, dtype=BF16, device="cuda") for _ in range(3))
            self.k = torch.empty(T, Hkv, D, dtype=BF16, device="cuda")
            self.lse = torch.empty(T, heads, device="cuda")
            self.grad = torch.zeros(T, heads + 2 * Hkv, D, dtype=BF16, device="cuda")
            self.ws = torch.empty(moe.moe_attention_workspace(ctx, self.q), dtype=torch.uint8, device="cuda")

        def step(self):
            v = fused[:, heads + Hkv:]
            moe.moe_rotate(ctx, fused[:, :heads], positions, rotary, self.q)
            moe.moe_rotate(ctx, fused[:, heads:heads + Hkv], positions, rotary, self.k)
            moe.moe_attention(ctx, self.q, self.k, v, off, self.out, lse=self.lse)
            dq, dk, dv = self.grad[:, :heads], self.grad[:, heads:heads + Hkv], self.grad[:, heads + Hkv:]
            moe.moe_attention_backward(ctx, dout, self.q, self.k, v, self.out, self.lse, off, dq=dq, dk=dk, dv=dv, workspace=self.ws)
            moe.moe_rotate(ctx, dq, positions, rotary, dq, inverse=True)
            moe.moe_rotate(ctx, dk, positions, rotary, dk, inverse=True)

    sides = [Side() for _ in range(3)]
    for side in sides:
        side.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sides[0].step()
    for i in range(4):
        fused.copy_(A.normal(g, T, heads + 2 * Hkv, D, BF16))
        dout.copy_(A.normal(g, T, heads, D, BF16))
        off[1] += 13 * i
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        with torch.cuda.stream(streams[0]):
            graph.replay()
        with torch.cuda.stream(streams[1]):
            sides[1].step()
        torch.cuda.synchronize()
        sides[2].step()
        torch.cuda.synchronize()
        for side in sides[:2]:
            same = [torch.equal(side.out, sides[2].out), torch.equal(side.grad, sides[2].grad)]
            assert same == [True, True]
    assert sides[2].grad.isfinite().all() and sides[2].grad.any()


def test_prompt_then_decode(ctx):
    """A prompt by moe_attention on the values that the cache keeps is the cached attention of its tokens."""
    n, heads, Hkv, D = 90, 4, 2, 64
    g = A.gen(14)
    q, k, v = A.normal(g, n, heads, D, F32), A.normal(g, n, Hkv, D, F32), A.normal(g, n, Hkv, D, F32)
    cache = moe.KvCache(ctx, 6, 16, Hkv, D, 32)
    batch = moe.KvBatch(ctx, A.ints([0, n]), A.ints([n]), A.ints([[5, 2, 0, 1, 4, 3]]), tokens=n)
    turned, kept = torch.empty_like(q), [torch.empty_like(k) for _ in range(2)]
    moe.moe_kv_append(ctx, cache, batch, k, v, rotary=moe.Rotary(ctx, A.frequencies(D)), q=q, q_out=turned)
    moe.moe_kv_read(ctx, cache, batch, *kept)
    a, b = torch.empty_like(q), torch.empty_like(q)
    moe.moe_attention(ctx, turned, *kept, A.ints([0, n]), a)
    ws = torch.empty(moe.moe_attention_cached_workspace(ctx, cache, batch, heads), dtype=torch.uint8, device="cuda")
    moe.moe_attention_cached(ctx, cache, batch, turned, b, workspace=ws)
    # both within 1e-5 of the values' magnitude (up to 4) of the formula: scores' sums of 64 products, twice
    A.close(a, b.double(), torch.full_like(a, 1e-4, dtype=torch.float64))


@pytest.mark.parametrize("heads", [2, 64])  # few rows, and many
def test_tokens_far_apart(ctx, heads):
    """Tokens so far apart that a tile spans more than 2^32 bytes."""
    q, k, v, oq, _ = _inputs(3, [70], [70], heads, 1, 64, BF16)
    ld = (1 << 32) // 2 // 64 + 8

    def apart(t):
        far = torch.as_strided(torch.empty((t.shape[0] - 1) * ld + t.shape[1] * t.shape[2], dtype=t.dtype, device="cuda"), t.shape, (ld, t.shape[2], 1))
        far.copy_(t)
        return far
    out, lse = _forward(ctx, q, k, v, oq, oq)
    dout = A.normal(A.gen(4), 70, heads, 64, BF16)
    grads = _backward(ctx, dout, q, k, v, out, lse, oq, oq)
    far = [apart(t) for t in (q, k, v)]
    o, s = _forward(ctx, *far, oq, oq)
    assert torch.equal(o, out) and torch.equal(s, lse)
    for a, b in zip(grads, _backward(ctx, dout, *far, out, lse, oq, oq)):
        assert torch.equal(a, b)
