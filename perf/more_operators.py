"""The operators of an attention layer in their plain form and as the library's users call them, with the sizes that they are timed at.

Five operators: rotary positions ("rotate"), keys and values appended to a paged cache held in 4 bits, rotated on the
way ("append"), attention over such a cache ("cached"), attention over packed prompts ("attention") and its backward
pass ("attention_backward").
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HEAD_DIMS = (64, 96, 128, 192, 256)


def listed():
    return [
        # the query heads of one decoded token far into a long context: latency
        {"name": "rotate_t1", "op": "rotate", "T": 1, "H": 16, "D": 128, "rot": 128, "interleaved": False, "inverse": False, "far": 1000000, "dtype": "bf16", "pad": 0},
        # a tuning step's gradients of the queries, half of each head rotated, columns of a wider buffer
        {"name": "rotate_t8192_inverse", "op": "rotate", "T": 8192, "H": 32, "D": 128, "rot": 64, "interleaved": True, "inverse": True, "far": 8192, "dtype": "bf16", "pad": 2048},
        # one token for each of 64 decoding requests
        {"name": "append_64x1", "op": "append", "seqs": 64, "new": 1, "ragged": False, "before": 4000, "page": 64, "H": 32, "Hkv": 8, "D": 128, "group": 32, "interleaved": False, "dtype": "bf16"},
        # prompts of different lengths
        {"name": "append_prompts", "op": "append", "seqs": 5, "new": 3001, "ragged": True, "before": 0, "page": 16, "H": 32, "Hkv": 8, "D": 128, "group": 64, "interleaved": True, "dtype": "bf16"},
        # one request in a short conversation: latency
        {"name": "cached_1x1", "op": "cached", "seqs": 1, "new": 1, "longest": 777, "page": 64, "H": 16, "Hkv": 2, "D": 128, "group": 32, "window": 0, "dtype": "bf16"},
        # one request with a long document: the axis of the cache has to be split
        {"name": "cached_1x1_long", "op": "cached", "seqs": 1, "new": 1, "longest": 130001, "page": 64, "H": 32, "Hkv": 8, "D": 128, "group": 32, "window": 0, "dtype": "bf16"},
        # a serving batch of different lengths: bandwidth
        {"name": "cached_64x1", "op": "cached", "seqs": 64, "new": 1, "longest": 16000, "page": 32, "H": 64, "Hkv": 8, "D": 128, "group": 128, "window": 0, "dtype": "bf16"},
        # three speculative tokens of several requests, kept in fp32
        {"name": "cached_5x3_f32", "op": "cached", "seqs": 5, "new": 3, "longest": 2501, "page": 16, "H": 12, "Hkv": 4, "D": 64, "group": 64, "window": 0, "dtype": "f32"},
        # short prompts packed, one pair of key heads
        {"name": "attention_packed", "op": "attention", "seqs": 9, "longest": 777, "H": 14, "Hkv": 2, "D": 64, "causal": True, "window": 0, "dtype": "bf16"},
        # one long prompt: matrix cores
        {"name": "attention_8192", "op": "attention", "seqs": 1, "longest": 8192, "H": 32, "Hkv": 8, "D": 128, "causal": True, "window": 0, "dtype": "bf16"},
        # a tuning step on packed sequences
        {"name": "attention_backward_packed", "op": "attention_backward", "seqs": 4, "longest": 4096, "H": 16, "Hkv": 4, "D": 128, "causal": True, "window": 0, "dtype": "bf16"},
        # a short odd sequence kept in fp32
        {"name": "attention_backward_f32", "op": "attention_backward", "seqs": 2, "longest": 611, "H": 6, "Hkv": 3, "D": 96, "causal": True, "window": 0, "dtype": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("rotate", "append", "cached", "cached", "attention", "attention_backward"))
    D, Hkv = rng.choice(HEAD_DIMS), _log(rng, 1, 16)
    H, dtype = Hkv * rng.choice((1, 2, 3, 4, 7, 8)), rng.choice(("bf16", "bf16", "f32"))
    group = rng.choice([g for g in (32, 64, 128) if D % g == 0])
    if op == "rotate":
        T = max(1, min(_log(rng, 1, 16384), 2 ** 25 // (H * D)))
        return {"op": op, "T": T, "H": H, "D": D, "rot": rng.choice((D, D, D // 2)), "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.5,
                "far": _log(rng, 1, 2000000), "dtype": dtype, "pad": rng.choice((0, 0, 64, 5))}
    if op == "append":
        seqs, ragged = _log(rng, 1, 128), rng.random() < 0.5
        new = max(1, min(_log(rng, 1, 4096) if ragged else _log(rng, 1, 8), 2 ** 24 // (H * D * seqs)))
        return {"op": op, "seqs": seqs, "new": new, "ragged": ragged, "before": _log(rng, 1, 4096) - 1, "page": rng.choice((16, 32, 64, 128)), "H": H, "Hkv": Hkv, "D": D,
                "group": group, "interleaved": rng.random() < 0.5, "dtype": dtype}
    window = rng.choice((0, 0, 0, _log(rng, 16, 2048)))
    if op == "cached":
        seqs, new = _log(rng, 1, 64), rng.choice((1, 1, 1, 2, 4, 16))
        longest = max(new, min(_log(rng, 16, 65536), 2 ** 29 // (seqs * Hkv * D), 2 ** 28 // (seqs * H * new)))
        return {"op": op, "seqs": seqs, "new": new, "longest": longest, "page": rng.choice((16, 32, 64, 128)), "H": H, "Hkv": Hkv, "D": D, "group": group, "window": window, "dtype": dtype}
    seqs = _log(rng, 1, 16)
    most = 2 ** ((36 if dtype == "bf16" else 33) - (op == "attention_backward"))
    longest = max(1, min(_log(rng, 16, 8192), int(math.sqrt(most / (seqs * H * D)))))
    causal = rng.random() < 0.8
    return {"op": op, "seqs": seqs, "longest": longest, "H": H, "Hkv": Hkv, "D": D, "causal": causal, "window": window if causal else 0, "dtype": dtype}


def _lengths(count, longest, least=1):
    """One sequence of the longest length and others of any length up to it: the same for every seed."""
    rng = random.Random(count * 1000003 + longest)
    return [longest] + [rng.randint(min(least, longest), longest) for _ in range(count - 1)]


def _new_lengths(case):
    return _lengths(case["seqs"], case["new"]) if case.get("ragged") else [case["new"]] * case["seqs"]


def _visible(queries, keys, causal, window):
    """How many keys the queries of one sequence see, all together: query i of n sees keys i + keys - n - window < j <= i + keys - n."""
    if not causal:
        return queries * keys
    return sum(min(window or keys, keys - queries + i + 1) for i in range(queries))


def work(case):
    e = {"bf16": 2, "f32": 4}[case["dtype"]]
    op, H, D = case["op"], case["H"], case["D"]
    if op == "rotate":
        return {"bytes": 2 * case["T"] * H * D * e + 4 * case["T"], "flops": 3 * case["T"] * H * case["rot"]}
    Hkv = case["Hkv"]
    if op == "append":
        T, held = sum(_new_lengths(case)), D // 2 + 4 * (D // case["group"])
        # keys, values and queries read, rotated queries written; the cache written, then read for the values it holds, written in bf16
        return {"bytes": T * (2 * H * D * e + 2 * Hkv * (D * e + 2 * held + 2 * D)), "flops": T * (3 * H * D + 8 * Hkv * D)}
    if op == "cached":
        lengths = _lengths(case["seqs"], case["longest"], case["new"])
        seen = [min(n, case["window"] + case["new"] - 1) if case["window"] else n for n in lengths]
        held = 2 * Hkv * (D // 2 + 4 * (D // case["group"]))
        pairs = sum(_visible(case["new"], n, True, case["window"]) for n in lengths)
        return {"bytes": sum(seen) * held + 2 * case["seqs"] * case["new"] * H * D * e, "flops": 4 * H * D * pairs}
    lengths = _lengths(case["seqs"], case["longest"])
    T, pairs = sum(lengths), sum(_visible(n, n, case["causal"], case["window"]) for n in lengths)
    if op == "attention":
        return {"bytes": T * ((2 * H + 2 * Hkv) * D * e + 4 * H), "flops": 4 * H * D * pairs}
    return {"bytes": T * ((4 * H + 4 * Hkv) * D * e + 4 * H), "flops": 10 * H * D * pairs}


def _normal(gen, *shape, dtype, pad=0):
    """Normal values of [T, heads, D]; with pad, the first columns of a wider buffer."""
    T, heads, D = shape
    return torch.randn(T, heads * D + pad, generator=gen, device="cuda").to(dtype)[:, : heads * D].unflatten(1, (heads, D))


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return _ints(at)


def _frequencies(rot):
    return (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float()


def _page_table(gen, lengths, page):
    """Pages of the sequences in random order over a pool with some to spare: (table [seqs, most], pages of the pool)."""
    each = [-(-n // page) for n in lengths]
    total = sum(each) + 3
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(lengths), max(1, max(each)), dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(each):
        table[i, :n] = order[at: at + n]
        at += n
    return table, total


def _held(gen, total, page, heads, D, group):
    """What a cache holds: two codes a byte (the even channel in the low half), fp16 steps and lows by group. Each group has a lowest and a highest code."""
    codes = torch.randint(0, 16, (total, page, heads, D // group, group), generator=gen, device="cuda", dtype=torch.uint8)
    at = torch.randint(0, group, (total, page, heads, D // group, 1), generator=gen, device="cuda")
    codes.scatter_(-1, at, 0)
    codes.scatter_(-1, (at + 1 + at % (group - 1)) % group, 15)
    codes = codes.flatten(-2)
    steps = (torch.rand(total, page, heads, D // group, generator=gen, device="cuda") * 0.3 + 0.15).to(torch.float16)
    lows = (-7.5 * steps.float() + 0.3 * torch.randn(steps.shape, generator=gen, device="cuda")).to(torch.float16)
    return codes[..., 0::2] | codes[..., 1::2] << 4, steps, lows


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, H, D, dtype = case["op"], case["H"], case["D"], DTYPES[case["dtype"]]
    if op == "rotate":
        positions = torch.randint(max(0, case["far"] - 4 * case["T"]), case["far"] + 1, (case["T"],), generator=gen, device="cuda", dtype=torch.int32)
        return {"x": _normal(gen, case["T"], H, D, dtype=dtype, pad=case["pad"]), "positions": positions, "freqs": _frequencies(case["rot"]), "interleaved": case["interleaved"],
                "inverse": case["inverse"]}
    Hkv = case["Hkv"]
    if op == "append":
        new = _new_lengths(case)
        lengths, T = [n + case["before"] for n in new], sum(new)
        table, total = _page_table(gen, lengths, case["page"])
        # the projections of a layer lie side by side: queries, keys, values
        fused = torch.randn(T, (H + 2 * Hkv) * D, generator=gen, device="cuda").to(dtype).unflatten(1, (H + 2 * Hkv, D))
        return {"q": fused[:, :H], "k": fused[:, H: H + Hkv], "v": fused[:, H + Hkv:], "offsets": _offsets(new), "lengths": _ints(lengths), "table": table, "pages": total,
                "freqs": _frequencies(D), "interleaved": case["interleaved"], "group": case["group"]}
    if op == "cached":
        lengths = _lengths(case["seqs"], case["longest"], case["new"])
        table, total = _page_table(gen, lengths, case["page"])
        return {"q": _normal(gen, case["seqs"] * case["new"], H, D, dtype=dtype), "offsets": _offsets([case["new"]] * case["seqs"]), "lengths": _ints(lengths), "table": table,
                "pages": total, "longest": case["longest"], "new": case["new"], "window": case["window"],
                "keys": _held(gen, total, case["page"], Hkv, D, case["group"]), "values": _held(gen, total, case["page"], Hkv, D, case["group"])}
    lengths = _lengths(case["seqs"], case["longest"])
    T = sum(lengths)
    inputs = {name: _normal(gen, T, heads, D, dtype=dtype) for name, heads in (("q", H), ("k", Hkv), ("v", Hkv))}
    inputs |= {"offsets": _offsets(lengths), "longest": case["longest"], "causal": case["causal"], "window": case["window"]}
    if op == "attention_backward":
        # what the forward pass has kept
        out, inputs["lse"] = _attend_packed(inputs)
        inputs["out"] = out.to(dtype)
        inputs["dout"] = _normal(gen, T, H, D, dtype=dtype)
    return inputs


def prepare(case, seed):
    state = {"op": case["op"], **_inputs(case, seed)}
    if own:
        _handles(case, state)
    return state


def _handles(case, state):
    """What a program of the library keeps between calls: its context, the cache, buffers for the results."""
    from routed_expert_execution_amd import moe

    cfg = moe.make_config(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)
    pool = torch.zeros(moe.moe_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    ctx = state["ctx"] = moe.Context(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=pool.device.index, slot_pool=pool)
    op = case["op"]
    if op in ("rotate", "append"):
        state["rotary"] = moe.Rotary(ctx, state["freqs"], interleaved=state["interleaved"])
    if op == "rotate":
        state["y"] = torch.empty(state["x"].shape, dtype=state["x"].dtype, device="cuda")
    elif op == "append":
        state["cache"] = moe.KvCache(ctx, state["pages"], case["page"], case["Hkv"], case["D"], case["group"])
        state["batch"] = moe.KvBatch(ctx, state["offsets"], state["lengths"], state["table"], tokens=state["q"].shape[0], most_new=case["new"])
        state["q_out"] = torch.empty(state["q"].shape, dtype=state["q"].dtype, device="cuda")
        state["k_held"], state["v_held"] = (torch.empty(state["k"].shape, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    elif op == "cached":
        cache = state["cache"] = moe.KvCache(ctx, state["pages"], case["page"], case["Hkv"], case["D"], case["group"])
        # the whole pool as sequences of one page each: appending the values that the codes stand for gives those codes
        pages, page = state["pages"], case["page"]
        every = moe.KvBatch(ctx, torch.arange(0, pages * page + 1, page, dtype=torch.int32, device="cuda"), torch.full((pages,), page, dtype=torch.int32, device="cuda"),
                            torch.arange(pages, dtype=torch.int32, device="cuda").unsqueeze(1), tokens=pages * page, most_new=page)
        moe.moe_kv_append(ctx, cache, every, _values(*state["keys"]).flatten(0, 1), _values(*state["values"]).flatten(0, 1))
        state["batch"] = moe.KvBatch(ctx, state["offsets"], state["lengths"], state["table"], tokens=state["q"].shape[0], most_new=case["new"])
        state["out"] = torch.empty_like(state["q"])
        state["workspace"] = torch.empty(moe.moe_attention_cached_workspace(ctx, cache, state["batch"], case["H"]), dtype=torch.uint8, device="cuda")
    elif op == "attention":
        state["out"], state["lse"] = torch.empty_like(state["q"]), torch.empty(state["q"].shape[:2], dtype=torch.float32, device="cuda")
    else:
        for name in ("q", "k", "v"):
            state["d" + name] = torch.empty_like(state[name])
        state["workspace"] = torch.empty(moe.moe_attention_workspace(ctx, state["q"], state["k"]), dtype=torch.uint8, device="cuda")


def _rotated(x, positions, freqs, interleaved, inverse=False):
    """x in its own type or wider; angles in 64 bits, since a position may be far."""
    angles = positions.double().unsqueeze(1) * freqs.double()
    c, s = torch.cos(angles).to(x.dtype).unsqueeze(1), torch.sin(angles).to(x.dtype).unsqueeze(1)
    s = -s if inverse else s
    half, rot = freqs.numel(), 2 * freqs.numel()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    a, b = a * c - b * s, a * s + b * c
    turned = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


def _kept(x, group):
    """The values that 4 bits keep of x (64 bits: some lie next to a border between two codes)."""
    x = x.unflatten(-1, (-1, group))
    low = x.amin(-1, keepdim=True).to(torch.float16).double()
    step = ((x.amax(-1, keepdim=True) - low) / 15).to(torch.float16).double()
    codes = torch.where(step > 0, torch.round((x - low) / step), torch.zeros_like(x)).clamp(0, 15)
    return (low + step * codes).flatten(-2)


def _values(codes, steps, lows):
    """The fp32 values of packed codes [..., D / 2]."""
    codes = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).unflatten(-1, (steps.shape[-1], -1)).float()
    return (codes * steps.float().unsqueeze(-1) + lows.float().unsqueeze(-1)).flatten(-2)


def _softmax_product(q, k, v, seen):
    """q [n, Hkv, rows, D], k and v [n, Hkv, keys, D], seen [n, 1, rows, keys]: (out, log of the sum of exponentials). A row that sees nothing gives zeros."""
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(q.shape[-1] ** -0.5).masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_min(torch.finfo(scores.dtype).min)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.clamp_min(torch.finfo(scores.dtype).tiny)
    return out, (torch.log(total) + top).squeeze(-1)


def _padded(x, offsets, longest, heads):
    """Packed [T, H, D] as [seqs, heads, H / heads * longest, D] in fp32."""
    T, H, D = x.shape
    at = (offsets[:-1, None] + torch.arange(longest, device="cuda")).clamp_max(T - 1)
    rows = x[at].float().unflatten(2, (heads, H // heads)).permute(0, 2, 3, 1, 4).contiguous()
    return rows.flatten(2, 3)


def _packed(x, offsets, T, per):
    """[seqs, heads, per * longest, D] back to [T, heads * per, D]."""
    token = torch.arange(T, device="cuda")
    seq = torch.searchsorted(offsets[1:].contiguous(), token.to(torch.int32), right=True)
    rows = x.unflatten(2, (per, -1)).permute(0, 3, 1, 2, 4)
    return rows[seq, token - offsets[seq]].flatten(1, 2)


def _seen(state, queries, keys, lengths_q, lengths_k):
    """[seqs, 1, queries, keys]: which keys a query sees."""
    i, j = torch.arange(queries, device="cuda")[:, None], torch.arange(keys, device="cuda")
    last = (i + (lengths_k - lengths_q)[:, None, None]).unsqueeze(1)
    seen = (j < lengths_k[:, None, None, None]) & (i < lengths_q[:, None, None, None])
    if state.get("causal", True):
        seen = seen & (j <= last)
    if state["window"]:
        seen = seen & (j > last - state["window"])
    return seen


def _attend_packed(state):
    q, offsets, longest = state["q"], state["offsets"], state["longest"]
    Hkv, per = state["k"].shape[1], q.shape[1] // state["k"].shape[1]
    lengths = offsets[1:] - offsets[:-1]
    seen = _seen(state, longest, longest, lengths, lengths).repeat(1, 1, per, 1)
    out, lse = _softmax_product(_padded(q, offsets, longest, Hkv), _padded(state["k"], offsets, longest, Hkv), _padded(state["v"], offsets, longest, Hkv), seen)
    return _packed(out, offsets, q.shape[0], per), _packed(lse.unsqueeze(-1), offsets, q.shape[0], per).squeeze(-1)


def _plain_backward(state):
    q, k, v, offsets, longest = state["q"], state["k"], state["v"], state["offsets"], state["longest"]
    T, Hkv, per, scale = q.shape[0], k.shape[1], q.shape[1] // k.shape[1], q.shape[-1] ** -0.5
    lengths = offsets[1:] - offsets[:-1]
    seen = _seen(state, longest, longest, lengths, lengths).repeat(1, 1, per, 1)
    delta = (state["dout"].float() * state["out"].float()).sum(-1, keepdim=True)
    Q, K, V, dO, lse, delta = (_padded(x, offsets, longest, Hkv) for x in (q, k, v, state["dout"], state["lse"].unsqueeze(-1), delta))
    p = torch.exp(torch.matmul(Q, K.transpose(-1, -2).contiguous()).mul_(scale).sub_(lse)).masked_fill_(~seen, 0)
    dv = torch.matmul(p.transpose(-1, -2).contiguous(), dO)
    ds = torch.matmul(dO, V.transpose(-1, -2).contiguous()).sub_(delta).mul_(p)
    dq, dk = torch.matmul(ds, K).mul_(scale), torch.matmul(ds.transpose(-1, -2).contiguous(), Q).mul_(scale)
    return _packed(dq, offsets, T, per).to(q.dtype), _packed(dk, offsets, T, 1).to(q.dtype), _packed(dv, offsets, T, 1).to(q.dtype)


def _plain(state):
    op = state["op"]
    if op == "rotate":
        return _rotated(state["x"].float(), state["positions"], state["freqs"], state["interleaved"], state["inverse"]).to(state["x"].dtype)
    if op == "append":
        T, offsets = state["q"].shape[0], state["offsets"]
        token = torch.arange(T, device="cuda")
        seq = torch.searchsorted(offsets[1:].contiguous(), token.to(torch.int32), right=True)
        positions = state["lengths"][seq] - (offsets[1:][seq] - token)
        turn = (positions, state["freqs"], state["interleaved"])
        group = state["group"]
        return (_rotated(state["q"].float(), *turn).to(state["q"].dtype), _kept(_rotated(state["k"].double(), *turn), group).bfloat16(), _kept(state["v"].double(), group).bfloat16())
    if op == "cached":
        q, offsets, lengths, new = state["q"], state["offsets"], state["lengths"], state["new"]
        keys, values = (_values(*(part[state["table"]] for part in state[name])).flatten(1, 2).transpose(1, 2).contiguous() for name in ("keys", "values"))
        Hkv, per = keys.shape[1], q.shape[1] // keys.shape[1]
        seen = _seen(state, new, keys.shape[2], offsets[1:] - offsets[:-1], lengths).repeat(1, 1, per, 1)
        out, _ = _softmax_product(_padded(q, offsets, new, Hkv), keys, values, seen)
        return _packed(out, offsets, q.shape[0], per).to(q.dtype)
    if op == "attention":
        out, lse = _attend_packed(state)
        return out.to(state["q"].dtype), lse
    return _plain_backward(state)


def run(state):
    if not own:
        return _plain(state)
    from routed_expert_execution_amd import moe

    ctx, op = state["ctx"], state["op"]
    if op == "rotate":
        moe.moe_rotate(ctx, state["x"], state["positions"], state["rotary"], state["y"], inverse=state["inverse"])
        return state["y"]
    if op == "append":
        moe.moe_kv_append(ctx, state["cache"], state["batch"], state["k"], state["v"], rotary=state["rotary"], q=state["q"], q_out=state["q_out"])
        moe.moe_kv_read(ctx, state["cache"], state["batch"], state["k_held"], state["v_held"])
        return state["q_out"], state["k_held"], state["v_held"]
    if op == "cached":
        moe.moe_attention_cached(ctx, state["cache"], state["batch"], state["q"], state["out"], window=state["window"], workspace=state["workspace"])
        return state["out"]
    if op == "attention":
        moe.moe_attention(ctx, state["q"], state["k"], state["v"], state["offsets"], state["out"], lse=state["lse"], causal=state["causal"], window=state["window"])
        return state["out"], state["lse"]
    moe.moe_attention_backward(ctx, state["dout"], state["q"], state["k"], state["v"], state["out"], state["lse"], state["offsets"], dq=state["dq"], dk=state["dk"], dv=state["dv"],
                               causal=state["causal"], window=state["window"], workspace=state["workspace"])
    return state["dq"], state["dk"], state["dv"]


def _turn(x, positions, freqs, interleaved, sign):
    """Each pair as a complex number, turned by its angle."""
    x, half = x.double().clone(), freqs.numel()
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    angle = sign * torch.outer(positions.double(), freqs.double())
    turned = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle).unsqueeze(1)
    x[..., first], x[..., second] = turned.real, turned.imag
    return x


def _nearest(x, group):
    """The value on a group's grid that each value is nearest to."""
    parts = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    low = parts.min(-1)[0].half().double()
    step = ((parts.max(-1)[0] - low) / 15).half().double()
    grid = low.unsqueeze(-1) + step.unsqueeze(-1) * torch.arange(16, device=x.device, dtype=torch.float64)
    above = torch.where(step.unsqueeze(-1) > 0, (parts - low.unsqueeze(-1)) / step.unsqueeze(-1), torch.zeros_like(parts))
    return torch.gather(grid, -1, above.round().long().clamp(0, 15)).reshape(x.shape)


def _masked(case, queries, keys):
    """[queries, keys], 64 bits: 0 where a query sees a key, minus infinity elsewhere."""
    last = torch.arange(keys - queries, keys, device="cuda").unsqueeze(1)
    j = torch.arange(keys, device="cuda").unsqueeze(0)
    hidden = (j > last) if case.get("causal", True) else torch.zeros(queries, keys, dtype=torch.bool, device="cuda")
    if case["window"]:
        hidden = hidden | (j <= last - case["window"])
    return torch.zeros(queries, keys, dtype=torch.float64, device="cuda").masked_fill(hidden, -math.inf)


def exact(case, seed):
    given = _inputs(case, seed)
    op = case["op"]
    if op == "rotate":
        return _turn(given["x"], given["positions"], given["freqs"], case["interleaved"], -1 if case["inverse"] else 1)
    per = case["H"] // case["Hkv"]
    if op == "append":
        positions = torch.cat([torch.arange(case["before"], case["before"] + n, device="cuda") for n in _new_lengths(case)])
        q, k = (_turn(given[name], positions, given["freqs"], case["interleaved"], 1) for name in ("q", "k"))
        return q, _nearest(k, case["group"]), _nearest(given["v"].double(), case["group"])
    if op == "cached":
        out = torch.empty(given["q"].shape, dtype=torch.float64, device="cuda")
        for s, n in enumerate(_lengths(case["seqs"], case["longest"], case["new"])):
            pages, rows = given["table"][s, : -(-n // case["page"])].long(), slice(s * case["new"], (s + 1) * case["new"])
            mask = _masked(case, case["new"], n)
            for h in range(case["Hkv"]):
                k, v = (_grid(*(part[pages, :, h] for part in given[name]))[:n] for name in ("keys", "values"))
                q = given["q"][rows, h * per: (h + 1) * per].double().transpose(0, 1)
                out[rows, h * per: (h + 1) * per] = torch.matmul(torch.softmax(torch.matmul(q, k.t()) / math.sqrt(case["D"]) + mask, -1), v).transpose(0, 1)
        return out
    q, k, v = (given[name].double() for name in ("q", "k", "v"))
    if op == "attention":
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    else:
        dout, o, dq, dk, dv = given["dout"].double(), given["out"].double(), torch.empty_like(q), torch.zeros_like(k), torch.zeros_like(v)
    at = 0
    for n in _lengths(case["seqs"], case["longest"]):
        mask, rows = _masked(case, n, n), slice(at, at + n)
        at += n
        for h in range(case["H"]):
            scores = torch.matmul(q[rows, h], k[rows, h // per].t()) / math.sqrt(case["D"]) + mask
            if op == "attention":
                lse[rows, h] = torch.logsumexp(scores, -1)
                out[rows, h] = torch.matmul(torch.softmax(scores, -1), v[rows, h // per])
                continue
            p = torch.exp(scores - given["lse"][rows, h, None].double())
            dv[rows, h // per] += torch.matmul(p.t(), dout[rows, h])
            ds = p * (torch.matmul(dout[rows, h], v[rows, h // per].t()) - (dout[rows, h] * o[rows, h]).sum(-1, keepdim=True)) / math.sqrt(case["D"])
            dq[rows, h] = torch.matmul(ds, k[rows, h // per])
            dk[rows, h // per] += torch.matmul(ds.t(), q[rows, h])
    return (out, lse) if op == "attention" else (dq, dk, dv)


def _grid(codes, steps, lows):
    """The 64-bit values of packed codes [pages, tokens, D / 2] of one head, [pages * tokens, D]."""
    q = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    q[..., 0::2], q[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    group = q.shape[-1] // steps.shape[-1]
    q = q * steps.double().repeat_interleave(group, -1) + lows.double().repeat_interleave(group, -1)
    return q.flatten(0, 1)
