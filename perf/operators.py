"""The dense operators of the library in their plain form and as its users call them, with the sizes that they are timed at.

Four operators: a product with 4-bit weights and group scales ("linear"), the gated feed-forward block with such
weights ("linear_gated"), and that block with bf16 or fp32 weights, forwards ("gated") and backwards
("gated_backward").
"""
import math

import torch

own = False

GROUPS = (32, 64, 128)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token through a projection of the decode layer's width: latency
        {"name": "linear_t1", "op": "linear", "T": 1, "K": 2048, "N": 2048, "group": 32, "affine": False, "x": "bf16", "y": "bf16", "pad": 0},
        # one token's logits over a vocabulary of odd size, kept in fp32 for the sampler: bandwidth
        {"name": "linear_t1_vocab", "op": "linear", "T": 1, "K": 4096, "N": 100003, "group": 128, "affine": True, "x": "bf16", "y": "f32", "pad": 0},
        # a few speculative tokens of several requests, fp32 activations that are columns of a wider buffer
        {"name": "linear_t13_f32", "op": "linear", "T": 13, "K": 5184, "N": 6007, "group": 64, "affine": True, "x": "f32", "y": "f32", "pad": 24},
        # a prefill chunk through a square projection: matrix cores
        {"name": "linear_t2048", "op": "linear", "T": 2048, "K": 4096, "N": 4096, "group": 128, "affine": True, "x": "bf16", "y": "bf16", "pad": 0},
        # one token through a dense block: bandwidth and latency
        {"name": "linear_gated_t1", "op": "linear_gated", "T": 1, "K": 2048, "N": 8192, "group": 32, "affine": False, "x": "bf16", "y": "bf16", "pad": 0},
        # a batch of decoding requests, ragged
        {"name": "linear_gated_t37", "op": "linear_gated", "T": 37, "K": 4096, "N": 10240, "group": 64, "affine": True, "x": "bf16", "y": "bf16", "pad": 8},
        # a ragged prefill chunk
        {"name": "linear_gated_t1000", "op": "linear_gated", "T": 1000, "K": 2048, "N": 5504, "group": 128, "affine": True, "x": "bf16", "y": "bf16", "pad": 0},
        # four tokens through the repository's expert shape in bf16
        {"name": "gated_t4", "op": "gated", "T": 4, "d": 2048, "F": 512, "dtype": "bf16", "save": False},
        # a tuning step's forward pass
        {"name": "gated_t4096", "op": "gated", "T": 4096, "d": 2048, "F": 8192, "dtype": "bf16", "save": True},
        # its backward pass
        {"name": "gated_backward_t4096", "op": "gated_backward", "T": 4096, "d": 2048, "F": 8192, "dtype": "bf16"},
        # a short sequence through a block whose widths are whole numbers of nothing
        {"name": "gated_backward_t333", "op": "gated_backward", "T": 333, "d": 1000, "F": 1411, "dtype": "bf16"},
        # a block kept in fp32
        {"name": "gated_backward_f32", "op": "gated_backward", "T": 512, "d": 1024, "F": 2752, "dtype": "f32"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("linear", "linear_gated", "gated", "gated_backward"))
    tokens = _log(rng, 1, 4096)
    if op in ("linear", "linear_gated"):
        group = rng.choice(GROUPS)
        k = group * _log(rng, 128 / group, 8192 / group)
        n = _log(rng, 64, 32768)
        x = rng.choice(("bf16", "bf16", "f32"))
        y = x if op == "linear_gated" else rng.choice((x, "f32"))
        return {"op": op, "T": max(1, min(tokens, 2 ** 34 // (k * n))), "K": k, "N": n, "group": group, "affine": rng.random() < 0.5, "x": x, "y": y,
                "pad": rng.choice((0, 0, 8, 5))}
    d, f = _log(rng, 64, 4096), _log(rng, 64, 8192)
    if rng.random() < 0.6:
        d, f = (d + 7) // 8 * 8, (f + 7) // 8 * 8
    dtype = rng.choice(("bf16", "bf16", "f32"))
    case = {"op": op, "T": max(1, min(tokens, 2 ** (36 if dtype == "bf16" else 33) // (d * f))), "d": d, "F": f, "dtype": dtype}
    if op == "gated":
        case["save"] = rng.random() < 0.5
    return case


def work(case):
    T = case["T"]
    if case["op"] in ("linear", "linear_gated"):
        K, N = case["K"], case["N"]
        weights = N * K // 2 + N * (K // case["group"]) * (3 if case["affine"] else 2)
        two = 2 if case["op"] == "linear_gated" else 1
        e = {"bf16": 2, "f32": 4}
        return {"bytes": two * weights + T * K * e[case["x"]] + T * N * e[case["y"]], "flops": 2 * two * T * N * K}
    d, F, e = case["d"], case["F"], 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "gated":
        return {"bytes": (2 * F * d + T * d + T * F * (3 if case["save"] else 1)) * e, "flops": 4 * T * F * d}
    return {"bytes": (4 * F * d + 2 * T * d + 3 * T * F) * e, "flops": 8 * T * F * d}


def _normal(gen, rows, cols, dtype, scale=1.0, pad=0):
    """[rows, cols] normal values; with pad, the first columns of a wider buffer."""
    return (torch.randn(rows, cols + pad, generator=gen, device="cuda") * scale).to(dtype)[:, :cols]


def _quantised(gen, N, K, group, affine):
    """Two 4-bit codes a byte (the even column in the low half), fp16 scales and, affine, zero points by group."""
    codes = torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(N, K // group, generator=gen, device="cuda") * 0.009 + 0.001).to(torch.float16)
    zeros = torch.randint(4, 12, (N, K // group), generator=gen, device="cuda", dtype=torch.uint8) if affine else None
    return codes, scales, zeros


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] in ("linear", "linear_gated"):
        K, N = case["K"], case["N"]
        inputs = {"x": _normal(gen, case["T"], K, DTYPES[case["x"]], pad=case["pad"])}
        inputs["w"] = _quantised(gen, N, K, case["group"], case["affine"])
        if case["op"] == "linear_gated":
            inputs["w_up"] = _quantised(gen, N, K, case["group"], case["affine"])
        return inputs
    T, d, F, dtype = case["T"], case["d"], case["F"], DTYPES[case["dtype"]]
    inputs = {"x": _normal(gen, T, d, dtype), "w_gate": _normal(gen, F, d, dtype, d ** -0.5), "w_up": _normal(gen, F, d, dtype, d ** -0.5)}
    if case["op"] == "gated_backward":
        # what the forward pass has kept: the two projections in the operands' type
        x = inputs["x"].float()
        inputs["gate"] = (x @ inputs["w_gate"].float().t()).to(dtype)
        inputs["up"] = (x @ inputs["w_up"].float().t()).to(dtype)
        inputs["dh"] = _normal(gen, T, F, dtype)
    return inputs


def prepare(case, seed):
    state = {"op": case["op"], **_inputs(case, seed)}
    if case["op"] in ("linear", "linear_gated"):
        state["y_dtype"] = DTYPES[case["y"]]
    else:
        state["save"] = case.get("save", False)
    if own:
        _handles(case, state)
    return state


def _handles(case, state):
    """What a program of the library keeps between calls: its context, the packed weights, buffers for the results."""
    from routed_expert_execution_amd import moe

    cfg = moe.make_config(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)
    pool = torch.zeros(moe.moe_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    ctx = state["ctx"] = moe.Context(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=pool.device.index, slot_pool=pool)
    empty = lambda rows, cols, dtype: torch.empty(rows, cols, dtype=dtype, device="cuda")  # noqa: E731
    T = case["T"]
    if case["op"] in ("linear", "linear_gated"):
        for name in ("w", "w_up")[: 2 if case["op"] == "linear_gated" else 1]:
            state["q_" + name] = moe.QuantMatrix(ctx, *state[name])
        state["y"] = empty(T, case["N"], state["y_dtype"])
        return
    d, F, dtype = case["d"], case["F"], DTYPES[case["dtype"]]
    if case["op"] == "gated":
        state["h"] = empty(T, F, dtype)
        state["gate"], state["up"] = (empty(T, F, dtype), empty(T, F, dtype)) if case["save"] else (None, None)
        return
    state["dx"], state["dw_gate"], state["dw_up"] = empty(T, d, dtype), empty(F, d, dtype), empty(F, d, dtype)
    state["workspace"] = torch.empty(moe.moe_gated_workspace(ctx, T, d, F, dtype), dtype=torch.uint8, device="cuda")


def _weights(quantised):
    """The fp32 values of a 4-bit matrix."""
    codes, scales, zeros = quantised
    q = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(scales.shape[0], scales.shape[1], -1).float()
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scales.float().unsqueeze(-1)).reshape(scales.shape[0], -1)


def _plain(state):
    op, x = state["op"], state["x"].float()
    if op == "linear":
        return (x @ _weights(state["w"]).t()).to(state["y_dtype"])
    if op == "linear_gated":
        g, u = x @ _weights(state["w"]).t(), x @ _weights(state["w_up"]).t()
        return (g / (1 + torch.exp(-g)) * u).to(state["y_dtype"])
    dtype, w_gate, w_up = state["x"].dtype, state["w_gate"].float(), state["w_up"].float()
    if op == "gated":
        g, u = x @ w_gate.t(), x @ w_up.t()
        h = (g / (1 + torch.exp(-g)) * u).to(dtype)
        return (h, g.to(dtype), u.to(dtype)) if state["save"] else h
    g, u, dh = state["gate"].float(), state["up"].float(), state["dh"].float()
    s = 1 / (1 + torch.exp(-g))
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    return (dg @ w_gate + du @ w_up).to(dtype), (dg.t() @ x).to(dtype), (du.t() @ x).to(dtype)


def run(state):
    if not own:
        return _plain(state)
    from routed_expert_execution_amd import moe

    ctx = state["ctx"]
    if state["op"] == "linear":
        moe.moe_linear(ctx, state["x"], state["q_w"], state["y"])
        return state["y"]
    if state["op"] == "linear_gated":
        moe.moe_linear_gated(ctx, state["x"], state["q_w"], state["q_w_up"], state["y"])
        return state["y"]
    if state["op"] == "gated":
        moe.moe_gated(ctx, state["x"], state["w_gate"], state["w_up"], state["h"], gate_out=state["gate"], up_out=state["up"])
        return (state["h"], state["gate"], state["up"]) if state["save"] else state["h"]
    moe.moe_gated_backward(ctx, state["dh"], state["x"], state["w_gate"], state["w_up"], state["gate"], state["up"], dx=state["dx"],
                           dw_gate=state["dw_gate"], dw_up=state["dw_up"], workspace=state["workspace"])
    return state["dx"], state["dw_gate"], state["dw_up"]


def _dense(quantised, group):
    """The 64-bit values of a 4-bit matrix, column by column parity: even columns are the low halves."""
    codes, scales, zeros = quantised
    w = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    w[:, 0::2] = (codes % 16).double()
    w[:, 1::2] = (codes // 16).double()
    w -= 8.0 if zeros is None else zeros.double().repeat_interleave(group, dim=1)
    return w.mul_(scales.double().repeat_interleave(group, dim=1))


def exact(case, seed):
    given = _inputs(case, seed)
    x = given["x"].double()
    if case["op"] == "linear":
        return torch.matmul(_dense(given["w"], case["group"]), x.t()).t().contiguous()
    if case["op"] == "linear_gated":
        gate = torch.matmul(_dense(given["w"], case["group"]), x.t())
        up = torch.matmul(_dense(given["w_up"], case["group"]), x.t())
        return (gate * up * torch.sigmoid(gate)).t().contiguous()
    w_gate, w_up = given["w_gate"].double(), given["w_up"].double()
    if case["op"] == "gated":
        gate, up = torch.matmul(w_gate, x.t()).t(), torch.matmul(w_up, x.t()).t()
        h = torch.sigmoid(gate) * gate * up
        return (h, gate.contiguous(), up.contiguous()) if case["save"] else h
    gate, up, dh = (given[name].double() for name in ("gate", "up", "dh"))
    sig = torch.sigmoid(gate)
    d_up = dh * (gate * sig)
    d_gate = dh * up * (sig + gate * sig * (1 - sig))
    dx = torch.matmul(torch.cat((d_gate, d_up), dim=1), torch.cat((w_gate, w_up), dim=0))
    return dx, torch.matmul(d_gate.t().contiguous(), x), torch.matmul(d_up.t().contiguous(), x)
