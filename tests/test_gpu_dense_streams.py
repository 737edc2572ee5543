"""GPU: a 4-bit matrix packed on another stream than the current one, while
either is late."""
import pytest

from tests import harness as H

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not H.gpu_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

from routed_expert_execution_amd import moe  # noqa: E402

N, K, GROUP = 512, 1024, 64


@pytest.fixture(scope="module")
def ctx():
    cfg = moe.make_config(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)
    pool = torch.zeros(moe.moe_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    return moe.Context(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=0, slot_pool=pool)


def _sources(affine):
    gen = torch.Generator(device="cuda").manual_seed(5)
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.rand(N, K // GROUP, generator=gen, device="cuda").to(torch.float16)
    zeros = torch.randint(0, 256, (N, K // GROUP), generator=gen, device="cuda", dtype=torch.uint8) if affine else None
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(1).float()
    z = 8.0 if zeros is None else zeros.float().repeat_interleave(GROUP, 1)
    return [codes, scales, zeros], (c - z) * scales.float().repeat_interleave(GROUP, 1)


def _values(ctx, w):
    out = torch.full((N, K), float("nan"), device="cuda")
    moe.moe_linear_dequant(ctx, w, out)
    return out


@pytest.mark.parametrize("affine", [False, True])
@pytest.mark.parametrize("given", ["stream", "handle", "default"])
def test_sources_dropped_while_the_packing_stream_is_late(ctx, given, affine):
    """The current stream takes and overwrites memory of the sources' sizes at once."""
    src, want = _sources(affine)
    late = torch.cuda.Stream()
    current = torch.cuda.Stream() if given == "default" else torch.cuda.current_stream()
    if given == "default":
        late = torch.cuda.default_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(late):
        torch.cuda._sleep(50_000_000)
    with torch.cuda.stream(current):
        w = moe.QuantMatrix(ctx, *src, stream=late if given == "stream" else late.cuda_stream)
        sizes = [(t.shape, t.dtype) for t in src if t is not None]
        src.clear()
        over = [torch.empty(s, dtype=t, device="cuda").fill_(7) for s, t in sizes for _ in range(3)]
    late.synchronize()
    assert torch.equal(_values(ctx, w), want)
    del over


def test_matrix_in_memory_that_the_current_stream_still_writes(ctx):
    src, want = _sources(True)
    n = int(moe.library().moe_linear_bytes(N, K, GROUP, 1))
    late = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = [torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(3)]
    torch.cuda._sleep(50_000_000)
    for t in before:
        t.fill_(0xFF)
    del t, before
    w = moe.QuantMatrix(ctx, *src, stream=late)
    late.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(_values(ctx, w), want)
