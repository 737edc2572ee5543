"""GPU: rotary positions, and keys and values into a paged 4-bit cache and back,
against their formulas in 64 bits."""
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


def _rotation_tol(x, ref, half, interleaved, scale, dtype):
    """Two products and a sum in fp32 of a cosine and a sine rounded to fp32 (3 half
    steps of each product, 2^-24), and the result's own rounding."""
    y = x.double().abs()
    other = y.clone()
    if interleaved:
        other[..., 0:2 * half:2], other[..., 1:2 * half:2] = y[..., 1:2 * half:2], y[..., 0:2 * half:2]
    else:
        other[..., :half], other[..., half:2 * half] = y[..., half:2 * half], y[..., :half]
    return 4 * A.U * abs(scale) * (y + other) + A.HALF[dtype] * ref.abs() + 1e-37


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,heads,D,rot,interleaved,pad,far", [
    (1, 1, 64, 64, False, 0, 1), (1, 16, 128, 128, False, 0, 2000000), (7, 3, 96, 96, True, 5, 100), (33, 2, 128, 64, False, 64, 9000),
    (5, 5, 192, 100, False, 3, 70000), (5, 5, 192, 100, True, 3, 70000), (300, 40, 256, 256, True, 0, 40000), (40, 1, 64, 2, False, 0, 50),
    (17, 129, 256, 30, False, 0, 50), (9, 4, 128, 16, True, 8, 2 ** 31 - 64)])
def test_rotate(ctx, T, heads, D, rot, interleaved, pad, far, inverse, dtype):
    g = A.gen(T + D + rot)
    x = A.normal(g, T, heads, D, dtype, pad)
    positions = (far - torch.randint(0, min(far + 1, 64), (T,), generator=g, device="cuda")).to(torch.int32)
    freqs, scale = A.frequencies(rot), 1.25
    y = A.normal(g, T, heads, D, dtype, pad and 11)
    beside = y.as_strided((T, 11), (y.stride(0), 1), heads * D).clone() if pad else None
    moe.moe_rotate(ctx, x, positions, moe.Rotary(ctx, freqs, interleaved, scale), y, inverse=inverse)
    ref = A.rotated(x, positions, freqs, interleaved, inverse, scale)
    tol = _rotation_tol(x, ref, rot // 2, interleaved, scale, dtype)
    if far > 2 ** 30:
        tol = tol + 1e-6 * x.double().abs().amax()  # 2^31 times an angle's last of 53 bits, for both sides
    A.close(y, ref, tol)
    assert torch.equal(y[..., rot:], x[..., rot:])
    if pad:
        assert torch.equal(beside, y.as_strided((T, 11), (y.stride(0), 1), heads * D))
    # in place, the same bits
    z = x.clone().as_strided(x.shape, x.clone().stride()) if pad == 0 else A.normal(g, T, heads, D, dtype, pad)
    z.copy_(x)
    moe.moe_rotate(ctx, z, positions, moe.Rotary(ctx, freqs, interleaved, scale), z, inverse=inverse)
    assert torch.equal(z, y)


def test_rotate_and_back(ctx):
    """The inverse is the gradient: <g, R x> = <R^T g, x>, and R^T R x = x."""
    g = A.gen(3)
    x, dy = A.normal(g, 50, 4, 128, F32), A.normal(g, 50, 4, 128, F32)
    positions, r = torch.arange(50, dtype=torch.int32, device="cuda") * 977, moe.Rotary(ctx, A.frequencies(96))
    y, dx, back = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    moe.moe_rotate(ctx, x, positions, r, y)
    moe.moe_rotate(ctx, dy, positions, r, dx, inverse=True)
    moe.moe_rotate(ctx, y, positions, r, back, inverse=True)
    A.close(back, x.double(), 16 * A.U * (x.double().abs().amax(-1, keepdim=True) * 2 + 1e-30).expand_as(x))
    a, b = (dy.double() * y.double()).sum(), (dx.double() * x.double()).sum()
    assert abs(a - b) <= 8 * A.U * 2 * (dy.double().abs().sum(-1) * x.double().abs().amax(-1)).sum()


def test_rotate_no_tokens(ctx):
    x = torch.empty(0, 2, 64, device="cuda")
    moe.moe_rotate(ctx, x, torch.empty(0, dtype=torch.int32, device="cuda"), moe.Rotary(ctx, A.frequencies(64)), x.clone())


def _kept(x, group):
    """(value, lowest, step, place on the grid) of each x in 64 bits."""
    x = x.double().unflatten(-1, (-1, group))
    low = x.amin(-1, keepdim=True).float().half().double()
    step = ((x.amax(-1, keepdim=True) - low) / 15).float().half().double()
    place = torch.where(step > 0, (x - low) / step.clamp_min(1e-30), torch.zeros_like(x))
    value = low + step * place.round().clamp(0, 15)
    return [t.expand(x.shape).flatten(-2) for t in (value, low, step, place)]


def _check_kept(got, x, group):
    """fp32 values read back: those of the nearest code; next to a border (1e-9 of a
    step: cosines differ in their last bits) either code."""
    value, low, step, place = _kept(x, group)
    tol = 2 * A.U * (low.abs() + 15 * step)
    border = (place - place.floor() - 0.5).abs() < 1e-9
    A.close(got, value, torch.where(border, step + tol, tol) + 1e-37)


def _batch(ctx, new, before, page, g, tail=0):
    lengths = [n + b for n, b in zip(new, before)]
    table, pages = A.page_table(g, lengths, page)
    return moe.KvBatch(ctx, A.offsets(new), A.ints(lengths), table, tokens=sum(new) + tail, most_new=max(new)), pages


@pytest.mark.parametrize("new,before,page,H,Hkv,D,group,rot,interleaved,dtype", [
    ([1], [0], 16, 4, 1, 64, 32, 64, False, BF16), ([1, 1, 1], [0, 15, 4000], 16, 8, 8, 128, 128, 128, False, BF16),
    ([5, 0, 37, 1], [3, 9, 60, 0], 32, 6, 2, 96, 32, 96, True, BF16), ([70], [1], 64, 2, 2, 192, 64, 100, False, F32),
    ([70], [1], 64, 2, 2, 192, 32, 100, True, F32), ([130, 3], [0, 1022], 1024, 3, 3, 256, 128, 128, False, BF16),
    ([17, 16, 15], [16, 17, 15], 16, 5, 1, 256, 64, 256, True, F32), ([9] * 70, [0] * 70, 16, 1, 1, 64, 64, 32, False, BF16),
    # many tokens: a workgroup takes several, of one sequence or of neighbours
    ([1030, 2, 0, 1, 3063], [5, 0, 9, 1, 77], 64, 3, 1, 128, 64, 128, True, BF16), ([4100], [7], 16, 4, 2, 64, 32, 64, False, F32),
    ([1400, 1401, 1402], [0, 1, 2], 32, 2, 2, 192, 64, 100, False, BF16), ([3] * 1401, [2] * 1401, 16, 1, 2, 96, 32, 36, True, F32)])
def test_append_and_read(ctx, new, before, page, H, Hkv, D, group, rot, interleaved, dtype):
    g = A.gen(sum(new) + D)
    batch, pages = _batch(ctx, new, before, page, g, tail=3)
    cache = moe.KvCache(ctx, pages, page, Hkv, D, group)
    T = batch.tokens
    fused = A.normal(g, T, H + 2 * Hkv, D, dtype, 7)
    q, k, v = fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]
    freqs = A.frequencies(rot)
    q_out = torch.full((T, H, D), 7.0, dtype=dtype, device="cuda")
    moe.moe_kv_append(ctx, cache, batch, k, v, rotary=moe.Rotary(ctx, freqs, interleaved, 1.5), q=q, q_out=q_out)
    back = [torch.full((T, Hkv, D), 7.0, device="cuda") for _ in range(2)]
    moe.moe_kv_read(ctx, cache, batch, *back)
    used = T - 3
    positions = torch.cat([torch.arange(b, b + n, device="cuda") for n, b in zip(new, before)])
    ref = A.rotated(q[:used], positions, freqs, interleaved, scale=1.5)
    A.close(q_out[:used], ref, _rotation_tol(q[:used], ref, rot // 2, interleaved, 1.5, dtype))
    _check_kept(back[0][:used], A.rotated(k[:used], positions, freqs, interleaved, scale=1.5), group)
    _check_kept(back[1][:used], v[:used], group)
    for t in (q_out, *back):  # the rows behind the last sequence are left as they were
        assert (t[used:] == 7).all()
    rounded = [torch.empty((T, Hkv, D + 8), dtype=BF16, device="cuda").flatten(1)[:, :Hkv * D].unflatten(1, (Hkv, D)) for _ in range(2)]
    moe.moe_kv_read(ctx, cache, batch, *rounded)
    for a, b in zip(rounded, back):
        assert torch.equal(a[:used], b[:used].bfloat16())
    assert moe.moe_check(ctx) == moe.MOE_OK


def test_one_by_one_is_all_at_once(ctx):
    """The same bytes, whichever calls bring them; given positions; without a rotary; queries in place."""
    g, n, Hkv, D = A.gen(8), 41, 2, 128
    k, v, q = A.normal(g, n, Hkv, D, BF16), A.normal(g, n, Hkv, D, BF16), A.normal(g, n, 4, D, BF16)
    table = A.ints([[2, 0, 3, 1]])
    r = moe.Rotary(ctx, A.frequencies(D))
    caches = [moe.KvCache(ctx, 5, 16, Hkv, D, 32) for _ in range(2)]
    for c in caches:
        c.data.zero_()
    at_once = q.clone()
    moe.moe_kv_append(ctx, caches[0], moe.KvBatch(ctx, A.ints([0, n]), A.ints([n]), table, tokens=n), k, v, rotary=r, q=at_once, q_out=at_once)
    single = torch.empty_like(q)
    for i in range(n):
        moe.moe_kv_append(ctx, caches[1], moe.KvBatch(ctx, A.ints([0, 1]), A.ints([i + 1]), table, tokens=1), k[i:i + 1], v[i:i + 1], rotary=r, q=q[i:i + 1],
                          q_out=single[i:i + 1])
    assert torch.equal(caches[0].data, caches[1].data) and torch.equal(at_once, single)
    other, copied = moe.KvCache(ctx, 5, 16, Hkv, D, 32), torch.empty_like(q)
    other.data.zero_()
    whole = moe.KvBatch(ctx, A.ints([0, n]), A.ints([n]), table, tokens=n)
    moe.moe_kv_append(ctx, other, whole, k, v, rotary=r, positions=torch.arange(n, dtype=torch.int32, device="cuda"))
    assert torch.equal(other.data, caches[0].data)
    moe.moe_kv_append(ctx, other, whole, k, v, q=q, q_out=copied)
    assert torch.equal(copied, q)
    back = [torch.empty(n, Hkv, D, device="cuda") for _ in range(2)]
    moe.moe_kv_read(ctx, other, whole, *back)
    _check_kept(back[0], k, 32)
    # positions of their own: as of another place
    moe.moe_kv_append(ctx, other, whole, k, v, rotary=r, positions=torch.arange(n, dtype=torch.int32, device="cuda") + 100000)
    moe.moe_kv_read(ctx, other, whole, *back)
    _check_kept(back[0], A.rotated(k, torch.arange(n, device="cuda") + 100000, A.frequencies(D), False), 32)


def test_values_at_the_edges(ctx):
    """Equal values, zeros, exact halves, the smallest and largest fp16, beyond it, infinities and NaN: by group, the others untouched."""
    D, group = 128, 32
    x = torch.zeros(8, 1, D, device="cuda")
    x[0] = 0.3                                     # step 0
    x[1, 0, 1] = 15.0                              # codes of whole numbers
    x[2] = (torch.arange(D, device="cuda") % 16 + 0.5).clamp_max(15)
    x[2, 0, 0::32] = 0                             # halves: to the even code
    x[3, 0, ::2], x[3, 0, 1::2] = -65504, 65504
    x[4, 0, 5] = 65505.0
    x[5, 0, 40] = float("nan")
    x[6, 0, 70], x[6, 0, 100] = float("inf"), -float("inf")
    x[7] = torch.arange(D, device="cuda") * 1e-7   # steps below fp16's normal numbers
    batch = moe.KvBatch(ctx, A.ints([0, 8]), A.ints([8]), A.ints([[0]]), tokens=8)
    cache = moe.KvCache(ctx, 1, 16, 1, D, group)
    back = [torch.empty(8, 1, D, device="cuda") for _ in range(2)]
    moe.moe_kv_append(ctx, cache, batch, x, x)
    moe.moe_kv_read(ctx, cache, batch, *back)
    gone = {(4, 0), (5, 1), (6, 2), (6, 3)}
    for got in back:
        for t in range(8):
            for n in range(D // group):
                part, want = got[t, 0, n * group:(n + 1) * group], x[t, 0, n * group:(n + 1) * group]
                if (t, n) in gone:
                    assert part.isnan().all()
                else:
                    value, low, step, _ = _kept(want, group)
                    A.close(part, value, 2 * A.U * (low.abs() + 15 * step) + 1e-37)
    assert torch.equal(back[0][2, 0, 1:16], torch.tensor([2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14, 15.], device="cuda"))


def test_places_that_cannot_be(ctx):
    """Pages outside the cache, lengths and offsets that cannot be: left out, NaN read, error word; the others as ever."""
    D, Hkv = 64, 2
    g = A.gen(4)
    x = A.normal(g, 12, Hkv, D, F32)
    for off, lengths, table, lost in (([0, 4, 8, 12], [4, 4, 4], [[0], [-1], [2]], range(4, 8)), ([0, 4, 8, 12], [4, 4, 4], [[0], [3], [2]], range(4, 8)),
                                      ([0, 4, 8, 12], [4, 3, 4], [[0], [1], [2]], range(4, 8)), ([0, 4, 8, 12], [4, 17, 4], [[0], [1], [2]], range(7, 8)),
                                      ([0, 4, 8, 13], [4, 4, 5], [[0], [1], [2]], range(8, 12)), ([0, 4, 8, 12], [4, -5, 4], [[0], [1], [2]], range(4, 8))):
        cache = moe.KvCache(ctx, 3, 16, Hkv, D, 32)
        batch = moe.KvBatch(ctx, A.ints(off), A.ints(lengths), A.ints(table), tokens=12, most_new=5)
        back = [torch.full((12, Hkv, D), 7.0, device="cuda") for _ in range(2)]
        moe.moe_kv_append(ctx, cache, batch, x, x)
        assert moe.moe_check(ctx) == moe.MOE_EINVAL and moe.moe_check(ctx) == moe.MOE_OK
        moe.moe_kv_read(ctx, cache, batch, *back)
        assert moe.moe_check(ctx) == moe.MOE_EINVAL
        for got in back:
            for t in range(12):
                if t in lost:
                    assert got[t].isnan().all(), (off, lengths, table, t)
                else:
                    _check_kept(got[t], x[t], 32)


def test_places_that_cannot_be_among_many(ctx):
    """The same where a workgroup takes several tokens: a lost token leaves its neighbours as they are."""
    D, Hkv, n = 64, 1, 1440
    g = A.gen(11)
    x, q = A.normal(g, 3 * n, Hkv, D, F32), A.normal(g, 3 * n, 2, D, F32)
    lost = set(range(0, n, 7)) | {n - 1}
    table = A.ints([[-1 if s in lost else s] for s in range(n)])
    cache = moe.KvCache(ctx, n, 16, Hkv, D, 32)
    batch = moe.KvBatch(ctx, A.ints(list(range(0, 3 * n + 1, 3))), A.ints([3] * n), table, tokens=3 * n, most_new=3)
    q_out = torch.empty_like(q)
    moe.moe_kv_append(ctx, cache, batch, x, x, q=q, q_out=q_out)
    assert moe.moe_check(ctx) == moe.MOE_EINVAL and torch.equal(q_out, q)
    back = [torch.full((3 * n, Hkv, D), 7.0, device="cuda") for _ in range(2)]
    moe.moe_kv_read(ctx, cache, batch, *back)
    assert moe.moe_check(ctx) == moe.MOE_EINVAL
    gone = torch.tensor([s in lost for s in range(n)], device="cuda").repeat_interleave(3)
    for got in back:
        assert got[gone].isnan().all()
        _check_kept(got[~gone], x[~gone], 32)


def test_captured_and_on_two_streams(ctx):
    g, Hkv, H, D = A.gen(6), 2, 4, 96
    r = moe.Rotary(ctx, A.frequencies(D))
    k, v, q = (A.normal(g, 3, n, D, BF16) for n in (Hkv, Hkv, H))
    lengths = A.ints([1, 20, 33])
    table, pages = A.page_table(g, [16, 32, 48], 16)
    batch = moe.KvBatch(ctx, A.ints([0, 1, 2, 3]), lengths, table, tokens=3, most_new=1)
    caches = [moe.KvCache(ctx, pages, 16, Hkv, D, 32) for _ in range(2)]
    for c in caches:
        c.data.zero_()
    q_out, want = torch.empty_like(q), torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    moe.moe_kv_append(ctx, caches[1], batch, k, v, rotary=r, q=q, q_out=q_out)
    caches[1].data.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.moe_kv_append(ctx, caches[0], batch, k, v, rotary=r, q=q, q_out=q_out)
    for i in range(4):
        k.copy_(A.normal(g, 3, Hkv, D, BF16))
        q.copy_(A.normal(g, 3, H, D, BF16))
        lengths += 1
        graph.replay()
        torch.cuda.synchronize()
        moe.moe_kv_append(ctx, caches[1], batch, k, v, rotary=r, q=q, q_out=want)
        torch.cuda.synchronize()
        assert torch.equal(caches[0].data, caches[1].data) and torch.equal(q_out, want)
    # the two halves of the sequences on two streams
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    two = moe.KvCache(ctx, pages, 16, Hkv, D, 32)
    two.data.copy_(caches[1].data)
    lengths += 1
    torch.cuda.synchronize()
    for s, at in ((a, 0), (b, 2)):
        n = 2 if at == 0 else 1
        part = moe.KvBatch(ctx, torch.arange(n + 1, dtype=torch.int32, device="cuda"), lengths[at:at + n], table[at:at + n].contiguous(), tokens=n, most_new=1)
        torch.cuda.synchronize()
        moe.moe_kv_append(ctx, two, part, k[at:at + n], v[at:at + n], rotary=r, stream=s)
    moe.moe_kv_append(ctx, caches[1], batch, k, v, rotary=r)
    torch.cuda.synchronize()
    assert torch.equal(two.data, caches[1].data)


def test_offsets_past_32_bits(ctx):
    """A cache over 4 GiB: the last page's bytes are its own."""
    Hkv, D, page = 16, 256, 1024
    per_page = int(moe.library().moe_kv_bytes(1, page, Hkv, D, 32))
    pages = (1 << 32) // per_page + 3
    cache = moe.KvCache(ctx, pages, page, Hkv, D, 32)
    g = A.gen(2)
    x = [A.normal(g, 3, Hkv, D, F32) for _ in range(2)]
    first = moe.KvBatch(ctx, A.ints([0, 3]), A.ints([3]), A.ints([[0]]), tokens=3)
    last = moe.KvBatch(ctx, A.ints([0, 3]), A.ints([page]), A.ints([[pages - 1]]), tokens=3)
    over = moe.KvBatch(ctx, A.ints([0, 3]), A.ints([3]), A.ints([[(1 << 32) // per_page]]), tokens=3)
    for i, b in enumerate((first, last, over)):
        moe.moe_kv_append(ctx, cache, b, x[0] + i, x[1] - i)
    for i, b in enumerate((first, last, over)):
        back = [torch.empty(3, Hkv, D, device="cuda") for _ in range(2)]
        moe.moe_kv_read(ctx, cache, b, *back)
        _check_kept(back[0], x[0] + i, 32)
        _check_kept(back[1], x[1] - i, 32)
