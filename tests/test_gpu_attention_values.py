"""GPU: attention where memory holds what no call has written, and where values are not finite."""
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


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,lengths,page,D,group,window", [
    ([1], [400], 16, 64, 32, 50), ([3, 1], [1000, 333], 16, 128, 64, 17), ([40], [700], 32, 96, 32, 100), ([1], [129], 64, 256, 128, 1), ([1], [5000], 16, 128, 128, 1000),
    ([2, 1, 5], [77, 47, 300], 16, 192, 64, 30)])
def test_unwritten_pages_and_a_window(ctx, new, lengths, page, D, group, window, dtype):
    """Pages that no call has written hold fp16 infinities or NaN, page 0 among them; so do
    those that lie before the windows, which the table no longer names."""
    g, Hkv, heads = A.gen(31), 2, 4
    table, total = A.page_table(g, lengths, page, spare=1)
    table = torch.where(table >= 0, table + 1, table)  # page 0 is no sequence's
    whole = moe.KvBatch(ctx, A.offsets(lengths), A.ints(lengths), table, tokens=sum(lengths))
    x = [A.normal(g, sum(lengths), Hkv, D, F32) for _ in range(2)]
    q = A.normal(g, sum(new), heads, D, dtype)
    within = table.clone()
    for s, (n, length) in enumerate(zip(new, lengths)):
        within[s, :max(0, length - n - window + 1) // page] = -1
    batch = moe.KvBatch(ctx, A.offsets(new), A.ints(lengths), within, tokens=sum(new), most_new=max(new))

    def outcome(fill):
        cache = moe.KvCache(ctx, total + 1, page, Hkv, D, group)
        cache.data.view(torch.int16).fill_(fill)
        moe.moe_kv_append(ctx, cache, whole, *x)
        for s in range(len(lengths)):
            for p in table[s][(within[s] < 0) & (table[s] >= 0)].tolist():
                cache.data.view(cache.pages, -1)[p].view(torch.int16).fill_(fill)
        out = torch.empty_like(q)
        ws = torch.empty(moe.moe_attention_cached_workspace(ctx, cache, batch, heads), dtype=torch.uint8, device="cuda")
        moe.moe_attention_cached(ctx, cache, batch, q, out, window=window, workspace=ws)
        assert moe.moe_check(ctx) == moe.MOE_OK
        return out

    want = outcome(0)
    assert want.isfinite().all()
    for fill in (0x7C00, 0xFC00 - 0x10000, 0x7E00, -1):
        assert torch.equal(outcome(fill), want), hex(fill & 0xFFFF)


def _forward(ctx, q, k, v, off, **kw):
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
    moe.moe_attention(ctx, q, k, v, off, out, lse=lse, **kw)
    return out, lse


@pytest.mark.parametrize("heads", [2, 80])  # few rows, and many
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window", [0, 20])
def test_log_sums_of_rows_that_see_nan(ctx, dtype, heads, window):
    """NaN, as the row itself: minus infinity is a row's that sees no key."""
    lengths, D = [150, 40, 7], 64  # the last two fit into one tile
    off, T = A.offsets(lengths), sum(lengths)
    g = A.gen(8)
    q, k, v = A.normal(g, T, heads, D, dtype), A.normal(g, T, 1, D, dtype), A.normal(g, T, 1, D, dtype)
    out, lse = _forward(ctx, q, k, v, off, window=window)
    assert lse.isfinite().all()
    at = 0
    for n in lengths:
        key = at + n // 3
        x = k.clone()
        x[key, 0, 5] = math.nan
        o, s = _forward(ctx, q, x, v, off, window=window)
        row = torch.arange(T, device="cuda")
        sees = (row >= key) & (row < at + n) & ((row < key + window) if window else True)
        assert s[sees].isnan().all() and o[sees].isnan().all()
        assert torch.equal(s[~sees], lse[~sees]) and torch.equal(o[~sees], out[~sees])
        y = q.clone()
        y[key, 1, 9] = math.nan
        o, s = _forward(ctx, y, k, v, off, window=window)
        keep = torch.ones(T, heads, dtype=torch.bool, device="cuda")
        keep[key, 1] = False
        assert s[key, 1].isnan() and o[key, 1].isnan().all()
        assert torch.equal(s[keep], lse[keep]) and torch.equal(o[keep], out[keep])
        at += n


@pytest.mark.parametrize("heads", [2, 80])  # few rows, and many
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 192])
@pytest.mark.parametrize("causal,window,at", [(False, 0, 100), (True, 0, 100), (True, 300, 200), (False, 0, 399), (True, 0, 399), (False, 0, 0)])
def test_infinite_values(ctx, dtype, heads, D, causal, window, at):
    """A value that is not finite makes the rows that see it NaN in its channel, wherever in
    the sequence it lies: in a tile that all rows see whole, or in one that is masked."""
    n = 400
    off, g = A.ints([0, n]), A.gen(5)
    q, k, v = A.normal(g, n, heads, D, dtype), A.normal(g, n, 1, D, dtype), A.normal(g, n, 1, D, dtype)
    out, lse = _forward(ctx, q, k, v, off, causal=causal, window=window)
    row = torch.arange(n, device="cuda")
    sees = ((row >= at) | (not causal)) & ((row < at + window) if window else True)
    others = torch.arange(D, device="cuda") != 5
    for value in (math.inf, -math.inf, math.nan):
        w = v.clone()
        w[at, 0, 5] = value
        o, s = _forward(ctx, q, k, w, off, causal=causal, window=window)
        assert o[sees][..., 5].isnan().all()
        assert torch.equal(s, lse) and torch.equal(o[~sees], out[~sees]) and torch.equal(o[..., others], out[..., others])


@pytest.mark.parametrize("offset,spread,dtype", [(0.0, 1.0, F32), (100.0, 1.0, F32), (1000.0, 1.0, F32), (10000.0, 1.0, F32), (-10000.0, 6.0, F32), (30000.0, 20.0, F32), (1000.0, 30.0, BF16), (3000.0, 5.0, BF16)])
def test_codes_of_far_keys(ctx, offset, spread, dtype):
    """Rotated keys that lie far from zero for how far they lie apart: the codes are those
    of the exact values."""
    g, T, Hkv, D, group = A.gen(17), 1024, 8, 128, 32
    want = (offset + spread * torch.rand(T, Hkv, D, generator=g, device="cuda", dtype=torch.float64))
    positions, freqs = torch.arange(T, dtype=torch.int32, device="cuda") * 37, A.frequencies(D)
    k = A.rotated(want, positions, freqs, False, inverse=True).to(dtype)
    v = want.to(dtype)
    table = torch.arange(T // 64, dtype=torch.int32, device="cuda").unsqueeze(0)
    batch = moe.KvBatch(ctx, A.ints([0, T]), A.ints([T]), table, tokens=T)
    cache = moe.KvCache(ctx, T // 64, 64, Hkv, D, group)
    moe.moe_kv_append(ctx, cache, batch, k, v, rotary=moe.Rotary(ctx, freqs), positions=positions)
    got = [torch.empty(T, Hkv, D, device="cuda") for _ in range(2)]
    moe.moe_kv_read(ctx, cache, batch, *got)
    for held, x in zip(got, (A.rotated(k, positions, freqs, False), v.double())):
        x = x.unflatten(-1, (-1, group))
        low = x.amin(-1, keepdim=True).float().half().double()
        step = ((x.amax(-1, keepdim=True) - low) / 15).float().half().double()
        place = torch.where(step > 0, (x - low) / step.clamp_min(1e-30), torch.zeros_like(x))
        value = low + step * place.round().clamp(0, 15)
        # the sum's rounding to fp32; next to a border (1e-9 of a step: cosines differ in their last bits) either code
        border = (place - place.floor() - 0.5).abs() < 1e-9
        tol = A.U * value.abs() + torch.where(border, step, torch.zeros_like(step))
        off = (held.unflatten(-1, (-1, group)).double() - value).abs() > tol
        assert not off.any(), f"{int(off.sum())} of {off.numel()} codes"
