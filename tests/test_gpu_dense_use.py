"""GPU: the dense operators' tiles as programs use them: captured and replayed, on
two streams at once, on rows as far apart as one loading of them reaches and
further, with one matrix in both places."""
import pytest

from tests import harness as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not H.gpu_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

from routed_expert_execution_amd import moe  # noqa: E402
from tests import test_gpu_dense as G  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
ctx = G.ctx

# T, K, N, group, gated: a size of each tile
TILES = [(66, 416, 29777, 32, False), (131, 384, 18223, 128, False), (897, 416, 8415, 32, False), (69, 4736, 8071, 64, False),
         (68, 544, 12195, 32, True), (143, 416, 11737, 32, True), (131, 384, 17341, 64, True), (66, 4480, 19, 64, True)]


def _call(ctx, x, ws, y, gated):
    if gated:
        moe.moe_linear_gated(ctx, x, ws[0], ws[1], y)
    else:
        moe.moe_linear(ctx, x, ws[0], y)


def _matrices(ctx, gen, N, K, group):
    return [moe.QuantMatrix(ctx, *G._quantised(gen, N, K, group, True)) for _ in range(2)]


@pytest.mark.parametrize("T,K,N,group,gated", TILES)
def test_captured_tiles(ctx, T, K, N, group, gated):
    """Each replay on new x, with eager work between, against the eager call."""
    assert moe.moe_linear_plan(T, N, K, group, BF16, BF16, gated)[0] == moe.MOE_PLAN_TILES
    ws = _matrices(ctx, G._gen(1), N, K, group)
    x, y = torch.zeros(T, K, dtype=BF16, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda")
    _call(ctx, x, ws, y, gated)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _call(ctx, x, ws, y, gated)
    for i in range(4):
        x.copy_(G._normal(G._gen(10 + i), T, K, BF16))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        y.zero_()
        _call(ctx, x, ws, y, gated)
        torch.cuda.synchronize()
        assert torch.equal(got, y) and got.any()


def test_tiles_on_two_streams(ctx):
    """Calls of one context on two streams against the same calls in turn, and the same bits each time."""
    sets = []
    for i, (T, K, N, group, gated) in enumerate(TILES):
        gen = G._gen(20 + i)
        sets.append((G._normal(gen, T, K, BF16), _matrices(ctx, gen, N, K, group), torch.empty(T, N, dtype=BF16, device="cuda"), gated))
    want = []
    for x, ws, y, gated in sets:
        _call(ctx, x, ws, y, gated)
        want.append(y.clone())
        y.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for i, (x, ws, y, gated) in enumerate(sets):
            with torch.cuda.stream(streams[i % 2]):
                _call(ctx, x, ws, y, gated)
    torch.cuda.synchronize()
    for (_, _, y, _), w in zip(sets, want):
        assert torch.equal(y, w)


def _apart(t, ld):
    """The rows of t, ld elements apart."""
    far = torch.as_strided(torch.empty((t.shape[0] - 1) * ld + t.shape[1], dtype=t.dtype, device="cuda"), t.shape, (ld, 1))
    far.copy_(t)
    return far


# Offsets within a tile have 32 bits where rows are at most 2^31 / 256 bytes apart.
@pytest.mark.parametrize("past", [0, 8])
@pytest.mark.parametrize("T,K,N,group,gated", [(897, 416, 8415, 32, False), (143, 416, 11737, 32, True)])
def test_linear_rows_far_apart(ctx, T, K, N, group, gated, past):
    gen = G._gen(31)
    x, ws = G._normal(gen, T, K, BF16), _matrices(ctx, gen, N, K, group)
    a, b = (torch.empty(T, N, dtype=BF16, device="cuda") for _ in range(2))
    _call(ctx, x, ws, a, gated)
    _call(ctx, _apart(x, (1 << 22) + past), ws, b, gated)
    assert torch.equal(a, b)


@pytest.mark.parametrize("past", [0, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,F", [(600, 264, 2050), (300, 520, 136)])
def test_gated_rows_far_apart(ctx, T, d, F, dtype, past):
    dt = G.DT[dtype]
    ld = (1 << (22 if dt == BF16 else 21)) + past
    x, wg, wu, dh, h, g, u = G._step_buffers(G._gen(32), T, d, F, dt)
    far = _apart(x, ld)
    other = [torch.empty_like(t) for t in (h, g, u)]
    moe.moe_gated(ctx, x, wg, wu, h, gate_out=g, up_out=u)
    moe.moe_gated(ctx, far, wg, wu, other[0], gate_out=other[1], up_out=other[2])
    for a, b in zip((h, g, u), other):
        assert torch.equal(a, b)
    want = G._backward(ctx, dh, x, wg, wu, g, u)
    for a, b in zip(want, G._backward(ctx, _apart(dh, ld), far, wg, wu, g, u)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 9, 40, 66])
def test_one_matrix_as_gate_and_up(ctx, T):
    K, N, group = 384, 12195, 64
    gen = G._gen(41)
    q = G._quantised(gen, N, K, group, True)
    w = moe.QuantMatrix(ctx, *q)
    x = G._normal(gen, T, K, BF16)
    h, y = torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, N, device="cuda")
    moe.moe_linear_gated(ctx, x, w, w, h)
    moe.moe_linear(ctx, x, w, y)
    v, mag = G._values(q, group)
    g = x.double() @ v.t()
    t = (3 * 128 + K / 32 + 16) * G.U * (x.double().abs() @ mag.t())
    ref = G._silu(g) * g
    G._close(h, ref, G._gated_tol(g, g, t, t, ref, BF16) + 2 * g.abs() * G.U * ref.abs())
    G._close(y, g, t + G._half_step(g, F32) + 1e-30)
    # the block in bf16: its two gradients are of one matrix's places
    d, F = 72, 200
    x, wg, _, dh, h, g, u = G._step_buffers(gen, T, d, F, BF16)
    moe.moe_gated(ctx, x, wg, wg, h, gate_out=g, up_out=u)
    assert torch.equal(g, u)
    g.copy_(G._cancels(g))
    for y, (ref, tol) in zip(G._backward(ctx, dh, x, wg, wg, g, u), G._backward_ref(dh, x, wg, wg, g, u, BF16)):
        G._close(y, ref, tol)
