"""The attention layer's checks of arguments and its host functions, without a GPU: a
host-only context judges the arguments first and refuses the call for its device last,
so each refusal is told by its message."""
import ctypes as C
import math

import numpy as np
import pytest

from routed_expert_execution_amd import moe

torch = pytest.importorskip("torch")

# Host buffers stand for device memory: no call here gets past the checks.
BUF = np.zeros(1 << 16, dtype=np.uint8)
BASE = (BUF.ctypes.data + 255) // 256 * 256


@pytest.fixture(scope="module")
def ctx():
    return moe.Context(1, 4, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)


def _refused(ctx, status, text):
    assert status == moe.MOE_EINVAL
    assert text in moe.library().moe_last_error(ctx.handle).decode(), moe.library().moe_last_error(ctx.handle)


def _rotary(freqs=BASE, rot=64, interleaved=0, scale=1.0):
    return moe.moe_rotary(freqs, rot, interleaved, scale)


def _cache(pages=4, page_tokens=16, heads=2, head_dim=64, group=32, data=BASE):
    return moe.moe_kv_cache(pages, page_tokens, heads, head_dim, group, data)


def _batch(offsets=BASE, lengths=BASE, pages=BASE, n=2, max_pages=3, tokens=2, most_new=1):
    return moe.moe_kv_batch(offsets, lengths, pages, n, max_pages, tokens, most_new)


def _rotate(ctx, x=BASE, dtype=1, ldx=128, T=2, heads=2, head_dim=64, positions=BASE, rotary=None, inverse=0, y=BASE, ldy=128):
    r = _rotary() if rotary is None else rotary
    return moe.library().moe_rotate(ctx.handle, x, dtype, ldx, T, heads, head_dim, positions, C.byref(r), inverse, y, ldy, None)


@pytest.mark.parametrize("kw,text", [
    ({}, "host-only"), (dict(T=0, x=None, y=None, positions=None), "host-only"), (dict(T=1, ldx=0, ldy=0), "host-only"), (dict(y=BASE + 4096, ldy=300), "host-only"),
    (dict(T=-1), "outside"), (dict(T=(1 << 22) + 1), "outside"), (dict(heads=0), "heads"), (dict(heads=1025, ldx=1 << 20, ldy=1 << 20), "heads"), (dict(head_dim=80), "head_dim"),
    (dict(head_dim=0), "head_dim"), (dict(dtype=2), "bad type"), (dict(x=None), "null x"), (dict(y=None), "null y"), (dict(x=BASE + 1, y=BASE + 1), "misaligned x"),
    (dict(dtype=0, y=BASE + 2), "misaligned y"), (dict(ldx=127, ldy=127), "tokens of x"), (dict(y=BASE + 4096, ldy=127), "tokens of y"), (dict(ldx=-128), "tokens of x"),
    (dict(positions=None), "positions"), (dict(positions=BASE + 2), "positions"), (dict(inverse=2), "inverse"), (dict(ldx=130), "in place"),
    (dict(rotary=_rotary(freqs=None)), "frequencies"), (dict(rotary=_rotary(freqs=BASE + 2)), "frequencies"), (dict(rotary=_rotary(rot=0)), "rot="), (dict(rotary=_rotary(rot=63)), "rot="),
    (dict(rotary=_rotary(rot=66)), "rot="), (dict(rotary=_rotary(interleaved=2)), "interleaved"), (dict(rotary=_rotary(scale=float("nan"))), "finite")])
def test_rotate_refuses(ctx, kw, text):
    _refused(ctx, _rotate(ctx, **kw), text)


def test_null_contexts_and_structs(ctx):
    lib, r, m, b = moe.library(), _rotary(), _cache(), _batch()
    assert lib.moe_rotate(None, BASE, 1, 128, 2, 2, 64, BASE, C.byref(r), 0, BASE, 128, None) == moe.MOE_EINVAL
    _refused(ctx, lib.moe_rotate(ctx.handle, BASE, 1, 128, 2, 2, 64, BASE, None, 0, BASE, 128, None), "null rotary")
    assert lib.moe_kv_append(None, C.byref(m), C.byref(b), BASE, 128, BASE, 128, 1, None, None, None, 0, 0, None, 0, None) == moe.MOE_EINVAL
    assert lib.moe_kv_read(None, C.byref(m), C.byref(b), BASE, 128, BASE, 128, 1, None) == moe.MOE_EINVAL
    assert lib.moe_attention_cached(None, C.byref(m), C.byref(b), BASE, 128, 1, 2, 1.0, 0, BASE, 128, BASE, 1 << 16, None) == moe.MOE_EINVAL
    _refused(ctx, lib.moe_attention(ctx.handle, None, BASE, 256, BASE, 128, BASE, 128, BASE, 256, None, None), "null description")
    _refused(ctx, lib.moe_kv_read(ctx.handle, None, C.byref(b), BASE, 128, BASE, 128, 1, None), "null cache")
    _refused(ctx, lib.moe_kv_read(ctx.handle, C.byref(m), None, BASE, 128, BASE, 128, 1, None), "bad batch")
    assert lib.moe_attention_cached_workspace(None, C.byref(b), 2) == 0 and lib.moe_attention_cached_workspace(C.byref(m), None, 2) == 0


# (what all three calls on a cache refuse)
CACHE = [(dict(cache=_cache(data=None)), "null cache"), (dict(cache=_cache(data=BASE + 8)), "16-byte"), (dict(cache=_cache(pages=0)), "bad cache"),
         (dict(cache=_cache(pages=1 << 31)), "bad cache"), (dict(cache=_cache(page_tokens=8)), "bad cache"), (dict(cache=_cache(page_tokens=48)), "bad cache"),
         (dict(cache=_cache(page_tokens=2048)), "bad cache"), (dict(cache=_cache(heads=0)), "bad cache"), (dict(cache=_cache(head_dim=80)), "bad cache"),
         (dict(cache=_cache(group=16)), "bad cache"), (dict(cache=_cache(head_dim=96, group=64)), "bad cache"), (dict(cache=_cache(group=128)), "bad cache"),
         (dict(batch=_batch(n=-1)), "bad batch"), (dict(batch=_batch(n=65537)), "bad batch"), (dict(batch=_batch(max_pages=0)), "bad batch"),
         (dict(batch=_batch(max_pages=(1 << 26) + 1)), "bad batch"), (dict(batch=_batch(tokens=-1)), "bad batch"), (dict(batch=_batch(tokens=(1 << 22) + 1)), "bad batch"),
         (dict(batch=_batch(most_new=3)), "bad batch"), (dict(batch=_batch(most_new=-1)), "bad batch"), (dict(batch=_batch(offsets=None)), "null offsets"),
         (dict(batch=_batch(lengths=None)), "null offsets"), (dict(batch=_batch(pages=None)), "null offsets"), (dict(batch=_batch(pages=BASE + 2)), "misaligned offsets"),
         (dict(dtype=3), "bad type"), ({}, "host-only"), (dict(batch=_batch(n=0, offsets=None, lengths=None, pages=None)), "host-only")]


def _append(ctx, cache=None, batch=None, k=BASE, ldk=128, v=BASE, ldv=128, dtype=1, rotary=None, positions=None, q=None, ldq=256, q_heads=4, q_out=None, ldqo=256):
    cache, batch = cache or _cache(), batch or _batch()
    return moe.library().moe_kv_append(ctx.handle, C.byref(cache), C.byref(batch), k, ldk, v, ldv, dtype, C.byref(rotary) if rotary else None, positions, q, ldq, q_heads, q_out, ldqo, None)


@pytest.mark.parametrize("kw,text", CACHE + [
    (dict(batch=_batch(tokens=0, most_new=0), k=None, v=None), "host-only"), (dict(k=None), "null k"), (dict(v=None), "null v"), (dict(k=BASE + 1), "misaligned k"), (dict(ldk=127), "tokens of k"),
    (dict(ldv=0), "tokens of v"), (dict(positions=BASE + 1), "positions"), (dict(rotary=_rotary(rot=65)), "rot="), (dict(rotary=_rotary(scale=math.inf)), "finite"),
    (dict(q=BASE), "q_out"), (dict(q_out=BASE), "q_out"), (dict(q=BASE, q_out=BASE + 4096, q_heads=0), "q_heads"), (dict(q=BASE, q_out=BASE + 4096, ldq=255), "tokens of q"),
    (dict(q=BASE, q_out=BASE + 4096, ldqo=255), "tokens of q_out"), (dict(q=BASE, q_out=BASE, ldqo=300), "in place"), (dict(q=BASE, q_out=BASE, rotary=_rotary()), "host-only")])
def test_append_refuses(ctx, kw, text):
    _refused(ctx, _append(ctx, **kw), text)


def _read(ctx, cache=None, batch=None, k=BASE, ldk=128, v=BASE, ldv=128, dtype=0):
    cache, batch = cache or _cache(), batch or _batch()
    return moe.library().moe_kv_read(ctx.handle, C.byref(cache), C.byref(batch), k, ldk, v, ldv, dtype, None)


@pytest.mark.parametrize("kw,text", CACHE + [(dict(k=None), "null k"), (dict(v=BASE + 2), "misaligned v"), (dict(ldk=100), "tokens of k")])
def test_read_refuses(ctx, kw, text):
    _refused(ctx, _read(ctx, **kw), text)


def _cached(ctx, cache=None, batch=None, q=BASE, ldq=256, dtype=1, q_heads=4, scale=0.125, window=0, out=BASE, ldo=256, ws=BASE, n=1 << 30):
    cache, batch = cache or _cache(), batch or _batch()
    return moe.library().moe_attention_cached(ctx.handle, C.byref(cache), C.byref(batch), q, ldq, dtype, q_heads, scale, window, out, ldo, ws, n, None)


@pytest.mark.parametrize("kw,text", CACHE + [
    (dict(q_heads=3), "multiple"), (dict(q_heads=0), "multiple"), (dict(q_heads=1026), "multiple"), (dict(q=None), "null q"), (dict(out=None), "null out"), (dict(ldq=255), "tokens of q"),
    (dict(ldo=255), "tokens of out"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=math.inf), "scale"), (dict(scale=math.nan), "scale"),
    (dict(cache=_cache(heads=1024), batch=_batch(n=65536), q_heads=1024, ldq=1 << 20, ldo=1 << 20, n=1 << 40), "host-only"),
    (dict(batch=_batch(max_pages=1 << 20, tokens=1 << 18), n=1 << 40), "too many"), (dict(batch=_batch(max_pages=1 << 20, tokens=1 << 16), n=1 << 40), "host-only"),
    (dict(window=-1), "window"), (dict(window=1 << 40), "host-only"), (dict(ws=None), "workspace"), (dict(ws=BASE + 128), "256-byte"), (dict(n=255), "needed")])
def test_attention_cached_refuses(ctx, kw, text):
    _refused(ctx, _cached(ctx, **kw), text)


ATTN = dict(offsets_q=BASE, offsets_k=BASE, n=2, dtype=1, q_heads=4, kv_heads=2, head_dim=64, causal=1, scale=0.125, window=0, tokens_q=8, tokens_k=9)
PACKED = [(dict(n=-1), "n outside"), (dict(n=65537), "n outside"), (dict(tokens_q=-1), "tokens outside"), (dict(tokens_k=(1 << 22) + 1), "tokens outside"), (dict(offsets_q=None), "null offsets"),
          (dict(offsets_k=None), "null offsets"), (dict(offsets_k=BASE + 2), "misaligned offsets"), (dict(dtype=2), "bad type"), (dict(q_heads=3), "multiple"), (dict(q_heads=0), "multiple"),
          (dict(kv_heads=0), "multiple"), (dict(q_heads=2048, kv_heads=1), "multiple"), (dict(head_dim=80), "head_dim"), (dict(causal=2), "causal"), (dict(window=-1), "window"),
          (dict(causal=0, window=5), "window"), (dict(scale=0.0), "scale"), (dict(scale=-1.0), "scale"), (dict(scale=math.nan), "scale"), ({}, "host-only"), (dict(window=1 << 50), "host-only"),
          (dict(n=0, offsets_q=None, offsets_k=None), "host-only"), (dict(causal=0), "host-only"), (dict(n=65536, q_heads=1024, kv_heads=1024), "too many")]


def _attn(**kw):
    return moe.moe_attn(*(kw.get(name, ATTN[name]) for name, _ in moe.moe_attn._fields_))


def _forward(ctx, attn=None, q=BASE, ldq=1 << 20, k=BASE, ldk=1 << 20, v=BASE, ldv=1 << 20, out=BASE, ldo=1 << 20, lse=None):
    return moe.library().moe_attention(ctx.handle, C.byref(attn or _attn()), q, ldq, k, ldk, v, ldv, out, ldo, lse, None)


def _backward(ctx, attn=None, lse=BASE, ws=BASE, n=1 << 40, **kw):
    args = []
    for name in ("dout", "q", "k", "v", "out"):
        args += [kw.get(name, BASE), kw.get("ld" + name, 1 << 20)]
    args.append(lse)
    for name in ("dq", "dk", "dv"):
        args += [kw.get(name, BASE), kw.get("ld" + name, 1 << 20)]
    return moe.library().moe_attention_backward(ctx.handle, C.byref(attn or _attn()), *args, ws, n, None)


@pytest.mark.parametrize("kw,text", PACKED)
def test_packed_sequences_refused(ctx, kw, text):
    _refused(ctx, _forward(ctx, _attn(**kw)), text)
    _refused(ctx, _backward(ctx, _attn(**kw)), text)


@pytest.mark.parametrize("kw,text", [(dict(q=None), "null q"), (dict(k=None), "null k"), (dict(v=None), "null v"), (dict(out=None), "null out"), (dict(q=BASE + 1), "misaligned q"),
                                     (dict(ldq=255), "tokens of q"), (dict(ldk=127), "tokens of k"), (dict(ldv=0), "tokens of v"), (dict(ldo=255), "tokens of out"), (dict(lse=BASE + 2), "lse"),
                                     (dict(lse=BASE), "host-only"), (dict(attn=_attn(tokens_q=0, tokens_k=0), q=None, k=None, v=None, out=None), "host-only")])
def test_attention_refuses(ctx, kw, text):
    _refused(ctx, _forward(ctx, **kw), text)


@pytest.mark.parametrize("kw,text", [(dict(dout=None), "null dout"), (dict(lddout=255), "tokens of dout"), (dict(out=None), "null out"), (dict(dq=None), "null dq"), (dict(dk=None), "null dk"),
                                     (dict(dv=None), "null dv"), (dict(lddk=127), "tokens of dk"), (dict(dv=BASE + 1), "misaligned dv"), (dict(lse=None), "lse"), (dict(ws=None), "workspace"),
                                     (dict(ws=BASE + 16), "256-byte"), (dict(n=255), "needed"), (dict(q=None), "null q"), (dict(ldv=5), "tokens of v")])
def test_attention_backward_refuses(ctx, kw, text):
    _refused(ctx, _backward(ctx, **kw), text)


def test_attention_without_a_context():
    t = _attn()
    assert moe.library().moe_attention(None, C.byref(t), BASE, 256, BASE, 128, BASE, 128, BASE, 256, None, None) == moe.MOE_EINVAL
    assert moe.library().moe_attention_backward(None, C.byref(t), *[BASE, 256] * 5, BASE, *[BASE, 256] * 3, BASE, 1 << 20, None) == moe.MOE_EINVAL
    f = moe.library().moe_attention_workspace
    assert f(0, 1) == 256 and f(1000, 32) == 256000 and f(-1, 1) == 0 and f(1, 0) == 0 and f((1 << 22) + 1, 1) == 0


def test_sizes():
    f = moe.library().moe_kv_bytes
    # 16 tokens of a head: D / 2 bytes a token and a 4-byte pair a group, of keys and of values
    assert f(1, 16, 1, 64, 32) == 2 * 16 * (32 + 8) and f(3, 64, 5, 128, 128) == 3 * 5 * 64 * 2 * (64 + 4)
    assert f(0, 16, 1, 64, 32) == 0 and f(1, 24, 1, 64, 32) == 0 and f(1, 16, 1, 72, 32) == 0 and f(1, 16, 1, 64, 48) == 0
    ws = moe.library().moe_attention_cached_workspace
    assert ws(C.byref(_cache()), C.byref(_batch()), 4) == 256  # never longer than 48 tokens: not cut
    big = _batch(max_pages=10000)
    need = ws(C.byref(_cache()), C.byref(big), 4)
    assert 256 < need < 64 << 20
    for heads, most in ((2, 1), (8, 1), (64, 16), (128, 4)):
        assert ws(C.byref(_cache(head_dim=256)), C.byref(_batch(max_pages=10000, tokens=64, most_new=most)), heads) < 128 << 20
    assert ws(C.byref(_cache()), C.byref(big), 3) == 0 and ws(C.byref(_cache(pages=0)), C.byref(big), 4) == 0


def test_frequencies():
    plain, one = moe.moe_rotary_freqs(64)
    want = 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert one == 1.0 and np.allclose(plain, want, rtol=2 ** -23, atol=0)
    linear, _ = moe.moe_rotary_freqs(64, kind=moe.MOE_ROTARY_LINEAR, factor=4)
    assert np.allclose(linear, want / 4, rtol=2 ** -23, atol=0)
    base, _ = moe.moe_rotary_freqs(64, kind=moe.MOE_ROTARY_BASE, factor=4)
    assert base[0] == 1 and abs(base[-1] / (want[-1] / 4) - 1) < 1e-6 and (base <= plain).all()
    ramp, scale = moe.moe_rotary_freqs(64, kind=moe.MOE_ROTARY_RAMP, factor=8, context=2048, fast=32, slow=1)
    assert abs(scale - (0.1 * math.log(8) + 1)) < 1e-6
    turns = 2048 * want / (2 * math.pi)
    assert np.allclose(ramp[turns >= 40], want[turns >= 40], rtol=2 ** -23) and np.allclose(ramp[turns <= 0.7], want[turns <= 0.7] / 8, rtol=2 ** -23)
    between = (turns < 25) & (turns > 1.3)
    assert between.any() and (ramp[between] < plain[between]).all() and (ramp[between] > plain[between] / 8).all() and (np.diff(ramp) < 0).all()
    same, s = moe.moe_rotary_freqs(64, kind=moe.MOE_ROTARY_RAMP, factor=1)
    assert s == 1 and np.array_equal(same, plain)
    for bad in (dict(rot=0), dict(rot=63), dict(rot=258), dict(rot=64, base=1.0), dict(rot=64, base=math.nan), dict(rot=64, kind=4), dict(rot=64, kind=1, factor=0.5),
                dict(rot=2, kind=moe.MOE_ROTARY_BASE, factor=2), dict(rot=64, kind=3, factor=2, slow=0), dict(rot=64, kind=3, factor=2, fast=1), dict(rot=64, kind=3, factor=2, context=0)):
        with pytest.raises(ValueError):
            moe.moe_rotary_freqs(**bad)


def test_binding_refuses_before_the_library(ctx):
    x, p = torch.zeros(3, 2, 64), torch.zeros(3, dtype=torch.int32)
    for make in (lambda: moe.Rotary(ctx, torch.zeros(32)), lambda: moe.Rotary(ctx, torch.zeros(32, dtype=torch.float64)), lambda: moe.KvCache(ctx, 4, 16, 2, 64),
                 lambda: moe.KvCache(ctx, 4, 17, 2, 64), lambda: moe.KvBatch(ctx, p, p[:2], p.view(1, 3), tokens=3), lambda: moe.KvBatch(ctx, p, p, p, tokens=3),
                 lambda: moe._heads(ctx, x.half(), 3, 2, 64, "x"), lambda: moe._heads(ctx, x, 3, 2, 32, "x"), lambda: moe._heads(ctx, x.transpose(0, 1), 2, 3, 64, "x"),
                 lambda: moe._heads(ctx, x[:1].expand(3, 2, 64), 3, 2, 64, "x"), lambda: moe._heads(ctx, x, 3, 2, 64, "x"), lambda: moe._whole(ctx, p.long(), (3,), "p"),
                 lambda: moe._whole(ctx, p[::2], (2,), "p"), lambda: moe._whole(ctx, p, (3,), "p")):
        with pytest.raises(ValueError):
            make()
