"""What the attention layer's GPU tests share: inputs, and references in 64 bits."""
import math

import torch

from routed_expert_execution_amd import moe

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}  # half a step of a value, relative
U = 2.0 ** -24


def context():
    cfg = moe.make_config(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=-1)
    pool = torch.zeros(moe.moe_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    return moe.Context(1, 1, 1, 128, 128, moe.MOE_Q8_0, 1, 1, device=0, slot_pool=pool)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, T, heads, D, dtype, pad=0):
    """[T, heads, D]; with pad, the first columns of a wider buffer."""
    return torch.randn(T, heads * D + pad, generator=g, device="cuda").to(dtype)[:, : heads * D].unflatten(1, (heads, D))


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return ints(at)


def frequencies(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float()


def rotated(x, positions, freqs, interleaved, inverse=False, scale=1.0):
    """64 bits."""
    x, half = x.double(), freqs.numel()
    angle = positions.double().unsqueeze(1) * freqs.double()
    c, s = scale * torch.cos(angle).unsqueeze(1), scale * torch.sin(angle).unsqueeze(1)
    s = -s if inverse else s
    y = x.clone()
    one = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    two = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., one] * s + x[..., two] * c
    return y


def close(got, ref, tol):
    assert got.shape == ref.shape
    off = (got.double() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((off / tol).nan_to_num(9e9).max()):.3g} of the tolerance"


def page_table(g, lengths, page, spare=2):
    """(table, pages of the pool): the sequences' pages in random order."""
    each = [-(-n // page) for n in lengths]
    total = sum(each) + spare
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lengths), max(1, max(each))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(each):
        table[i, :n] = order[at: at + n]
        at += n
    return table, total


class Held:
    """A cache of known codes: every group has a code 0 and a code 15, so that
    appending the values keeps just these codes, steps and lowest values."""

    def __init__(self, ctx, g, pages, page, heads, D, group, offset=0.3):
        self.cache = moe.KvCache(ctx, pages, page, heads, D, group)
        self.cache.data.fill_(0xA5)
        self.parts = []
        for _ in range(2):
            codes = torch.randint(0, 16, (pages * page, heads, D // group, group), generator=g, device="cuda")
            codes[..., 3], codes[..., group - 2] = 0, 15
            step = (torch.rand(pages * page, heads, D // group, generator=g, device="cuda") * 0.3 + 0.15).half()
            low = (-7.5 * step.float() + offset * torch.randn(step.shape, generator=g, device="cuda")).half()
            self.parts.append((codes, step, low))
        batch = moe.KvBatch(ctx, torch.arange(0, pages * page + 1, page, dtype=torch.int32, device="cuda"), ints([page] * pages),
                            torch.arange(pages, dtype=torch.int32, device="cuda").unsqueeze(1), tokens=pages * page, most_new=page)
        moe.moe_kv_append(ctx, self.cache, batch, *(self.values(i).float() for i in range(2)))
        self.page = page

    def values(self, i):
        codes, step, low = self.parts[i]
        return (codes.double() * step.double().unsqueeze(-1) + low.double().unsqueeze(-1)).flatten(-2)

    def steps(self, i):
        codes, step, _ = self.parts[i]
        return step.double().unsqueeze(-1).expand(codes.shape).flatten(-2)

    def tokens(self, table_row, length):
        """Rows of the pool that a sequence's places lie in."""
        place = torch.arange(length, device="cuda")
        return table_row[place // self.page].long() * self.page + place % self.page


def attend(q, k, v, scale, seen):
    """64 bits: q [n, D], k, v [m, D], seen [n, m] -> (out, p, scores); a row that sees nothing is 0."""
    s = (q @ k.t().contiguous()) * scale
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True).clamp_min(-1e300)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total.clamp_min(1e-300), torch.zeros_like(p))
    return torch.where(p > 0, p, torch.zeros_like(p)) @ v, p, s


def visible(n, m, causal=True, window=0):
    i, j = torch.arange(n, device="cuda")[:, None] + (m - n), torch.arange(m, device="cuda")[None]
    seen = (j <= i) if causal else torch.ones(n, m, dtype=torch.bool, device="cuda")
    return seen & (j > i - window) if window else seen
