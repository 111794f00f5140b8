"""Plain 64-bit forms of the prompt attention, the 4-bit rows and eviction, for the tests (torch, any device)."""
import math

import torch

D, GROUP, LIMIT = 128, 32, 1680.0
HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative
U32 = 2.0 ** -24        # half a step of float32, relative


def starts(lens, dev="cuda"):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(list(lens), dtype=torch.int32).cumsum(0)
    return t.to(dev)


def attend_rows(q, k, v, lse_only=False):
    """One sequence and head: q [lq, d], k, v [lk, d] in 64 bits; the last lq of lk tokens, causal.
    Returns (o, lse, sum p |v|, the largest sum |q_c k_c| of a row's visible keys)."""
    lq, lk = q.shape[0], k.shape[0]
    seen = torch.arange(lk, device=q.device)[None] <= torch.arange(lq, device=q.device)[:, None] + (lk - lq)
    s = (q @ k.T / math.sqrt(D)).masked_fill(~seen, -math.inf)
    if lk == 0:
        z = torch.zeros(lq, D, dtype=torch.float64, device=q.device)
        return z, torch.full((lq,), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros(lq, device=q.device)
    lse = torch.logsumexp(s, -1)
    some = seen.any(-1, keepdim=True)
    p = torch.where(seen & some, torch.exp(s - torch.where(some, lse[:, None], torch.zeros_like(lse[:, None]))),
                    torch.zeros_like(s))
    size = (q.abs() @ k.abs().T).masked_fill(~seen, 0.0).amax(-1)
    return p @ v, lse, p @ v.abs(), size


def score_error(size, n):
    """How far a float32 score (128 products, any order, then the base-2 scale and exponential) and a sum of n
    float32 terms can put a softmax weight off, relative: twice 128 roundings of the products' sizes (the score's
    and the maximum's), the sum's n roundings, and a few for the scale and exp2 (2 ulp plus its argument's rounding,
    at most 2^-16 for arguments to 2^7)."""
    return 2 * 128 * U32 * size / math.sqrt(D) + n * U32 + 2.0 ** -16


# ------------------------------------------------------------- 4-bit rows
def scale_of(amax):
    """S of a group, in 64 bits: amax / 7 up to four significant bits, no finer than 2^-17."""
    want = amax / 7.0
    e = torch.frexp(want).exponent.long() - 1
    quantum = (1 << ((e - 3).clamp_min(-17) + 17)).double() * 2.0 ** -17
    return torch.ceil(want / quantum) * quantum


def quantise(x):
    """x [..., 128] (bf16 or float32 values) -> codes uint8 [..., 64], scale bytes uint8 [..., 4]."""
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=LIMIT, neginf=-LIMIT).clamp(-LIMIT, LIMIT)
    g = x.unflatten(-1, (D // GROUP, GROUP))
    s = scale_of(g.abs().amax(-1, keepdim=True))
    c = torch.where(s > 0, torch.round(g / s.clamp_min(2.0 ** -40)), torch.zeros_like(g)).clamp(-7, 7)
    u = (c + 8).to(torch.uint8).flatten(-2)
    byte = (s.squeeze(-1).to(torch.float16).view(torch.int16) >> 7).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), byte


def values(codes, scales):
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).double() - 8
    s = (scales.to(torch.int16) << 7).view(torch.float16).double()
    return x * s.repeat_interleave(GROUP, -1)


def evict_plan(weights, positions, n, next_pos, keep, sink, recent):
    """(dropped rows below keep, kept rows at keep and above) of one head, both ascending: lists."""
    if n <= keep:
        return [], []
    w, p = weights.tolist(), positions.tolist()

    def order(i):
        held = p[i] < sink or p[i] >= next_pos - recent
        return (0, 0.0, i) if held else (1, math.inf if w[i] != w[i] else -w[i], i)

    kept = set(sorted(range(n), key=order)[:keep])
    return [i for i in range(keep) if i not in kept], sorted(i for i in kept if i >= keep)
