"""GPU: attention over a paged 4-bit cache against softmax in 64 bits on the values that the cache holds."""
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


def _call(ctx, cache, batch, q, out=None, **kw):
    out = torch.empty_like(q) if out is None else out
    ws = torch.empty(moe.moe_attention_cached_workspace(ctx, cache, batch, q.shape[1]), dtype=torch.uint8, device="cuda")
    moe.moe_attention_cached(ctx, cache, batch, q, out, workspace=ws, **kw)
    return out


def _reference(held, table, length, q, dtype, scale, window=0, gap=0.0):
    """(out, tolerance) of one sequence's new rows q [n, H, D].

    A score is a sum of D products in fp32, grouped as step * (sum of (16 + code) q)
    + lowest * (sum of q): off by (D + 8) half steps of scale * sum |q| (47 step +
    |lowest|).  Twice that (the row's sum has it too) and the exponentials' 2^-21 go
    to each p.  p * step is rounded to bf16 (or kept to 2^-24 as three terms) and
    multiplies code - 8; sums are of fp32 terms up to p (|lowest| + 47 step), as many
    roundings as a wave takes steps, and a few; then the result's own rounding."""
    n, heads, D = q.shape
    rows = held.tokens(table, length)
    seen = A.visible(n, length, True, window)
    outs, tols = [], []
    Hkv = held.cache.heads
    for h in range(heads):
        kh = h * Hkv // heads
        k, v = held.values(0)[rows, kh], held.values(1)[rows, kh]
        ks, vs = held.steps(0)[rows, kh], held.steps(1)[rows, kh]
        qh = q[:, h].double()
        ref, p, _ = A.attend(qh, k, v, scale, seen)
        score = (D + 8) * A.U * scale * (qh.abs() @ (k.abs() + 60 * ks).t())
        rel = 2 * torch.where(seen, score, torch.zeros_like(score)).amax(-1, keepdim=True) + 2.0 ** -20
        term = A.HALF[BF16] if dtype == BF16 else 2 * A.U
        tol = rel * (p @ v.abs()) * 2 + term * (p @ (8 * vs)) + (length / 64 + 40) * A.U * (p @ (v.abs() + 60 * vs)) + A.HALF[dtype] * ref.abs() + 1e-30
        outs.append(ref)
        tols.append(tol)
    return torch.stack(outs, 1), torch.stack(tols, 1)


CASES = [
    # new, lengths, page, H, Hkv, D, group, window, dtype, gap between tokens
    ([1], [1], 16, 1, 1, 64, 32, 0, BF16, 0), ([1], [1], 16, 3, 1, 96, 32, 0, F32, 0), ([1], [777], 64, 16, 2, 128, 32, 0, BF16, 0),
    ([1, 1, 1, 1], [15, 16, 17, 129], 16, 8, 8, 64, 64, 0, BF16, 8), ([1], [5001], 32, 32, 8, 128, 128, 0, BF16, 0),
    ([1], [9000], 1024, 4, 1, 256, 32, 0, BF16, 0), ([3, 0, 1, 2], [40, 0, 260, 2], 16, 6, 3, 192, 64, 0, BF16, 5),
    ([2, 5], [300, 5], 16, 12, 4, 64, 32, 0, F32, 0), ([1], [3001], 64, 7, 1, 128, 64, 0, F32, 4), ([4], [700], 32, 40, 1, 128, 128, 0, BF16, 0),
    ([70], [100], 16, 2, 1, 64, 64, 0, BF16, 0), ([33, 1], [33, 900], 128, 10, 2, 256, 128, 0, F32, 0), ([1, 1], [2000, 100], 16, 8, 2, 128, 32, 100, BF16, 0),
    ([9, 2], [500, 37], 32, 4, 2, 96, 32, 33, F32, 0), ([5], [1000], 64, 8, 2, 192, 32, 1, BF16, 0), ([1] * 70, [i * 7 % 400 + 1 for i in range(70)], 16, 4, 2, 64, 32, 0, BF16, 0),
    ([1] * 130, [2000 if i == 77 else 9 for i in range(130)], 16, 4, 2, 128, 64, 0, BF16, 0), ([1], [6000], 16, 128, 1, 192, 32, 0, F32, 0),
    ([1, 300], [4000, 300], 64, 2, 1, 64, 32, 0, BF16, 0), ([1], [100000], 256, 2, 1, 64, 64, 0, BF16, 0), ([1], [40000], 64, 2, 1, 96, 32, 0, F32, 0),
    # a prompt's part beside single tokens, more sequences than a wave has lanes: a run is several sequences' tiles
    ([1] * 40 + [90] + [1] * 40 + [0, 17], [i * 37 % 700 + 1 for i in range(40)] + [2500] + [i * 53 % 900 + 1 for i in range(40)] + [5, 1700], 16, 8, 2, 64, 32, 0, BF16, 0),
    ([1] * 70 + [33, 2], [i * 29 % 500 + 1 for i in range(70)] + [1500, 800], 64, 12, 4, 128, 64, 200, F32, 0),
    ([1, 1, 1, 260, 1], [9000, 1, 128, 4000, 129], 32, 8, 2, 128, 128, 0, BF16, 0), ([500], [500], 16, 16, 16, 128, 32, 0, BF16, 0), ([500], [900], 16, 4, 4, 96, 32, 70, BF16, 0),
    ([i % 3 for i in range(700)], [i * 31 % 190 + 2 for i in range(700)], 16, 2, 1, 64, 32, 0, BF16, 0)]


@pytest.mark.parametrize("new,lengths,page,heads,Hkv,D,group,window,dtype,gap", CASES)
def test_attention_cached(ctx, new, lengths, page, heads, Hkv, D, group, window, dtype, gap):
    g = A.gen(sum(lengths) + D)
    table, pages = A.page_table(g, lengths, page)
    held = A.Held(ctx, g, pages, page, Hkv, D, group)
    T = sum(new)
    q = A.normal(g, T + 2, heads, D, dtype, gap)
    batch = moe.KvBatch(ctx, A.offsets(new), A.ints(lengths), table, tokens=T + 2, most_new=max(new))
    out = A.normal(g, T + 2, heads, D, dtype, gap)
    out.fill_(7)
    _call(ctx, held.cache, batch, q, out, window=window)
    assert (out[T:] == 7).all()
    at = 0
    for s, (n, length) in enumerate(zip(new, lengths)):
        if n:
            ref, tol = _reference(held, table[s], length, q[at:at + n], dtype, D ** -0.5, window)
            A.close(out[at:at + n], ref, tol)
        at += n
    assert moe.moe_check(ctx) == moe.MOE_OK
    again = _call(ctx, held.cache, batch, q, window=window)
    assert torch.equal(again[:T], out[:T])
    # another bound of the new tokens: cut otherwise, the same result within the tolerance
    loose = moe.KvBatch(ctx, A.offsets(new), A.ints(lengths), table, tokens=T + 2)
    other = _call(ctx, held.cache, loose, q, window=window)
    n, length = new[0], lengths[0]
    ref, tol = _reference(held, table[0], length, q[:n], dtype, D ** -0.5, window)
    A.close(other[:n], ref, tol)


def test_scale_and_sharp_rows(ctx):
    """Scores far apart (one key takes it all) and all equal; a scale of its own."""
    g = A.gen(1)
    table, pages = A.page_table(g, [600], 16)
    held = A.Held(ctx, g, pages, 16, 1, 128, 32)
    batch = moe.KvBatch(ctx, A.ints([0, 1]), A.ints([600]), table, tokens=1)
    for factor, scale in ((30.0, 1.0), (0.0, 1.0), (1.0, 3.5), (1.0, 1e-20), (300.0, 1.0)):
        q = (A.normal(g, 1, 2, 128, F32) * factor).contiguous()
        ref, tol = _reference(held, table[0], 600, q, F32, scale)
        A.close(_call(ctx, held.cache, batch, q, scale=scale), ref, tol)


def test_shared_pages_and_one_page_twice(ctx):
    """Two sequences with a common beginning, and one whose table names a page twice."""
    g = A.gen(2)
    held = A.Held(ctx, g, 6, 16, 2, 64, 32)
    table, lengths = A.ints([[0, 1, 2], [0, 1, 3], [4, 4, 5]]), [40, 45, 48]
    q = A.normal(g, 3, 4, 64, BF16)
    out = _call(ctx, held.cache, moe.KvBatch(ctx, A.ints([0, 1, 2, 3]), A.ints(lengths), table, tokens=3), q)
    for s in range(3):
        ref, tol = _reference(held, table[s], lengths[s], q[s:s + 1], BF16, 0.125)
        A.close(out[s:s + 1], ref, tol)


def test_nan_stays_where_it_is_seen(ctx):
    """A token kept as NaN: rows that do not see it are as without it; what lies behind a
    sequence's end in its last page, and NaN queries of other rows, change nothing."""
    g = A.gen(3)
    D, heads, length, n = 64, 2, 50, 6
    table = A.ints([[1, 0, 3, 2]])
    x = [A.normal(g, 64, 1, D, F32) for _ in range(2)]
    q = A.normal(g, n, heads, D, BF16)
    whole = moe.KvBatch(ctx, A.ints([0, 64]), A.ints([64]), table, tokens=64)
    batch = moe.KvBatch(ctx, A.ints([0, n]), A.ints([length]), table, tokens=n)

    def outcome(change, window=0):
        cache = moe.KvCache(ctx, 4, 16, 1, D, 32)
        y, p = [t.clone() for t in x], q.clone()
        change(*y, p)
        moe.moe_kv_append(ctx, cache, whole, *y)
        return _call(ctx, cache, batch, p, window=window)

    clean = outcome(lambda k, v, p: None)
    for which in (0, 1):
        def late(k, v, p, which=which):
            (k, v)[which][47, 0, 3] = float("nan")  # seen by the new tokens at 47, 48 and 49
        got = outcome(late)
        assert torch.equal(got[:3], clean[:3]) and got[3:].isnan().any(-1).all()

        def behind(k, v, p, which=which):
            (k, v)[which][50:] = float("inf")
        assert torch.equal(outcome(behind), clean)

        def before(k, v, p, which=which):
            (k, v)[which][:30] = float("nan")
        assert torch.equal(outcome(before, 10), outcome(lambda k, v, p: None, 10))

    def query(k, v, p):
        p[2, 1] = float("inf")
    got = outcome(query)
    assert got[2, 1].isnan().all()
    keep = torch.ones(n, heads, dtype=torch.bool, device="cuda")
    keep[2, 1] = False
    assert torch.equal(got[keep], clean[keep])


def test_uninitialised_memory_is_not_read(ctx):
    """Pages of NaN patterns wherever nothing was appended."""
    g = A.gen(5)
    for length in (1, 15, 16, 17, 33, 47):
        cache = moe.KvCache(ctx, 4, 16, 1, 64, 32)
        cache.data.fill_(0xFF)
        table = A.ints([[2, 0, 1]])
        x = [A.normal(g, length, 1, 64, F32) for _ in range(2)]
        batch = moe.KvBatch(ctx, A.ints([0, length]), A.ints([length]), table, tokens=length)
        moe.moe_kv_append(ctx, cache, batch, *x)
        out = _call(ctx, cache, batch, A.normal(g, length, 2, 64, F32))
        assert out.isfinite().all()


@pytest.mark.parametrize("new,lengths,page,window,dtype", [([1], [400], 16, 50, BF16), ([3, 1], [1000, 333], 16, 17, F32), ([40], [700], 32, 100, BF16), ([1], [129], 64, 1, BF16)])
def test_pages_before_the_window_may_be_gone(ctx, new, lengths, page, window, dtype):
    g = A.gen(21)
    table, pages = A.page_table(g, lengths, page)
    held = A.Held(ctx, g, pages, page, 1, 64, 32)
    q = A.normal(g, sum(new), 4, 64, dtype)
    out = _call(ctx, held.cache, moe.KvBatch(ctx, A.offsets(new), A.ints(lengths), table, tokens=sum(new), most_new=max(new)), q, window=window)
    for s, (n, length) in enumerate(zip(new, lengths)):
        table[s, :max(0, length - n - window + 1) // page] = -1
    gone = _call(ctx, held.cache, moe.KvBatch(ctx, A.offsets(new), A.ints(lengths), table, tokens=sum(new), most_new=max(new)), q, window=window)
    assert moe.moe_check(ctx) == moe.MOE_OK and torch.equal(gone, out)


def test_places_that_cannot_be(ctx):
    """Bad pages within what is read, lengths and offsets: NaN for that sequence, error word, the others as ever."""
    g = A.gen(4)
    D = 64
    held = A.Held(ctx, g, 60, 16, 2, D, 32)
    good = torch.arange(60, dtype=torch.int32, device="cuda").view(3, 20)
    q = A.normal(g, 6, 4, D, BF16)
    want = _call(ctx, held.cache, moe.KvBatch(ctx, A.ints([0, 2, 4, 6]), A.ints([300, 300, 300]), good, tokens=6, most_new=2), q)
    for off, lengths, page, lost in (([0, 2, 4, 6], [300, 300, 300], (1, 3, 60), (2, 4)), ([0, 2, 4, 6], [300, 300, 300], (1, 18, -1), (2, 4)),
                                     ([0, 2, 4, 6], [300, 1, 300], None, (2, 4)), ([0, 2, 4, 6], [300, 321, 300], None, (2, 4)),
                                     ([0, 2, 4, 6], [300, -7, 300], None, (2, 4)), ([0, 2, 4, 9], [300, 300, 300], None, (4, 6)),
                                     ([0, 2, 4, 6], [300, 2 ** 31 - 1, 300], None, (2, 4))):
        table = good.clone()
        if page:
            table[page[0], page[1]] = page[2]
        out = _call(ctx, held.cache, moe.KvBatch(ctx, A.ints(off), A.ints(lengths), table, tokens=6, most_new=2), q)
        assert moe.moe_check(ctx) == moe.MOE_EINVAL and moe.moe_check(ctx) == moe.MOE_OK
        keep = torch.ones(6, dtype=torch.bool, device="cuda")
        keep[lost[0]:lost[1]] = False
        assert out[~keep].isnan().all()
        A.close(out[keep], want[keep].double(), 2 * A.HALF[BF16] * want[keep].double().abs() + 0.02)
    # a bad entry that is not read: behind the length
    table = good.clone()
    table[1, 19] = 99
    out = _call(ctx, held.cache, moe.KvBatch(ctx, A.ints([0, 2, 4, 6]), A.ints([300, 300, 300]), table, tokens=6, most_new=2), q)
    assert torch.equal(out, want) and moe.moe_check(ctx) == moe.MOE_OK
    # more new tokens than the batch names
    out = _call(ctx, held.cache, moe.KvBatch(ctx, A.ints([0, 1, 4, 6]), A.ints([300, 300, 300]), good, tokens=6, most_new=2), q)
    assert out[1:4].isnan().all() and out[0].isfinite().all() and out[4:].isfinite().all() and moe.moe_check(ctx) == moe.MOE_EINVAL


def test_decoding_captured(ctx):
    """Rotate, append and attend as a decoding step, captured once; each replay on longer
    sequences with eager work between, against the eager calls; two graphs that share nothing."""
    g, D, H, Hkv, n = A.gen(7), 128, 8, 2, 3
    lengths = A.ints([5, 1500, 30])
    table, pages = A.page_table(g, [64, 1600, 64], 16)
    rotary = moe.Rotary(ctx, A.frequencies(D))
    batch = moe.KvBatch(ctx, A.ints([0, 1, 2, 3]), lengths, table, tokens=n, most_new=1)
    start = A.Held(ctx, g, pages, 16, Hkv, D, 32).cache.data
    fused = torch.zeros(n, H + 2 * Hkv, D, dtype=BF16, device="cuda")

    class Side:
        def __init__(self):
            self.cache = moe.KvCache(ctx, pages, 16, Hkv, D, 32)
            self.cache.data.copy_(start)
            self.q, self.out = (torch.empty(n, H, D, dtype=BF16, device="cuda") for _ in range(2))
            self.ws = torch.empty(moe.moe_attention_cached_workspace(ctx, self.cache, batch, H), dtype=torch.uint8, device="cuda")

        def step(self):
            moe.moe_kv_append(ctx, self.cache, batch, fused[:, H:H + Hkv], fused[:, H + Hkv:], rotary=rotary, q=fused[:, :H], q_out=self.q)
            moe.moe_attention_cached(ctx, self.cache, batch, self.q, self.out, workspace=self.ws)

    sides = [Side() for _ in range(3)]
    graphs = []
    for side in sides:
        side.step()
    torch.cuda.synchronize()
    for side in sides[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            side.step()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        fused.copy_(A.normal(g, n, H + 2 * Hkv, D, BF16))
        lengths += 1
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):  # both at once
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        sides[2].step()
        torch.cuda.synchronize()
        for side in sides[:2]:
            same = [torch.equal(side.out, sides[2].out), torch.equal(side.cache.data, sides[2].cache.data)]
            assert same == [True, True]
    assert sides[2].out.isfinite().all() and moe.moe_check(ctx) == moe.MOE_OK
