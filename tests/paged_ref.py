"""Plain forms of the paged cache for the tests: its bookkeeping as lists, one sequence after the other, and its 8-bit
rows and attention in 64 bits."""
import math

import torch

from tests.kv4_ref import D, U32, score_error  # noqa: F401

HALF_BF16 = 2.0 ** -8  # half a step of bf16, relative


def quantise(x):
    """x [..., 128] -> e4m3 values in 64 bits, scale bytes: S the smallest 2^e with max|x| <= 448 S, -60 <= e <= 52."""
    lim = 2.0 ** 60
    x = torch.nan_to_num(x.double(), nan=0.0, posinf=lim, neginf=-lim).clamp(-lim, lim)
    amax = x.abs().amax(-1)
    e = torch.full_like(amax, -60.0)
    for i in range(-60, 52):
        e = torch.where(amax > 448.0 * 2.0 ** i, torch.full_like(e, i + 1.0), e)
    s = powers(x.device)[(e + 127).long()][..., None]
    y = x / s
    quantum = torch.full_like(y, 2.0 ** -9)
    for i in range(-5, 9):
        quantum = torch.where(y.abs() >= 2.0 ** i, 2.0 ** (i - 3), quantum)
    return torch.round(y / quantum) * quantum, (e + 127).to(torch.uint8)


def powers(dev):
    return torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=dev)


def values(codes, scales):
    """64-bit values of 8-bit rows (codes: float8_e4m3fn)."""
    return codes.double() * powers(codes.device)[scales.long()][..., None]


def rows_of(c, name, layer, s, n=None):
    """A sequence's first n rows of one layer in 64 bits: [Hkv, n, 128]."""
    n = int(c.lens[s]) if n is None else n
    at = torch.arange(n, device=c.table.device)
    page, r = c.table[s].long()[at // c.page_rows], at % c.page_rows
    x = getattr(c, name + "_pages")[layer]
    if c.k_pages.dtype is torch.bfloat16:
        return x[page, :, r].double().transpose(0, 1)
    codes = x.view(torch.uint8)[page, :, r].view(torch.float8_e4m3fn)
    return values(codes, getattr(c, name + "_scales")[layer][page, :, r]).transpose(0, 1)


class Book:
    """Table, lengths, starts and counts of a cache, and the pools' rows with them."""

    def __init__(self, c):
        self.c, self.P, self.W = c, c.page_rows, c.max_pages
        self.table, self.lens, self.starts = c.table.tolist(), c.lens.tolist(), c.starts.tolist()
        self.refs, self.short, self.wrong = c.refs.tolist(), False, False
        names = ["k_pages", "v_pages"] + (["k_scales", "v_scales"] if c.k_pages.dtype is not torch.bfloat16 else [])
        self.pools = {n: raw(getattr(c, n)).clone() for n in names}

    def pages(self, n):
        return -(-n // self.P)

    def free_pages(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def grow(self, tokens):
        for s, n in enumerate(tokens):
            n, a = max(n, 0), self.lens[s]
            self.starts[s] = a
            for _ in range(n):
                if self.lens[s] == self.W * self.P:
                    self.short = True
                    break
                if self.lens[s] % self.P == 0:
                    free = self.free_pages()
                    if not free:
                        self.short = True
                        break
                    self.table[s][self.lens[s] // self.P] = free[0]
                    self.refs[free[0]] = 1
                self.lens[s] += 1

    def fork(self, src, dst, rows=None):
        n_seqs, old, lens, free = len(self.lens), [list(t) for t in self.table], list(self.lens), self.free_pages()
        before, seen, plan = list(self.refs), set(), []
        for i, (a, b) in enumerate(zip(src, dst)):
            if not (0 <= a < n_seqs and 0 <= b < n_seqs):
                self.wrong = True
            elif b not in seen:
                seen.add(b)
                plan.append((a, b, min(lens[a], max(rows[i], 0)) if rows is not None else lens[a]))
        # another sequence that takes a page as a full one shares it as well
        for a, b, n in plan:
            for p in old[a][:n // self.P] if a != b else []:
                self.refs[p] += 1
        shared, copies = list(self.refs), []
        for a, b, n in plan:
            full, last = n // self.P, None
            if n % self.P:
                last = old[a][full]
                if a == b and shared[last] == 1:
                    pass
                elif free:
                    copies.append((last, free[0], n % self.P))
                    last = free.pop(0)
                    self.refs[last] += 1
                else:
                    self.short, last, n = True, None, full * self.P
            for j, p in enumerate(old[b][:self.pages(lens[b])]):
                if not (a == b and (j < full or p == last)):
                    self.refs[p] -= 1
            for j in range(full):
                self.table[b][j] = old[a][j]
            if last is not None:
                self.table[b][full] = last
            self.lens[b] = self.starts[b] = n
        assert before is not self.refs
        for t in self.pools.values():
            for p, q, n in copies:
                t[:, q, :, :n] = t[:, p, :, :n]

    def free(self, seqs, rows=None):
        self.fork(seqs, seqs, [0] * len(seqs) if rows is None else rows)

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        move = dict(zip([p for p in range(n, len(self.refs)) if self.refs[p]], [p for p in range(n) if not self.refs[p]]))
        for p, q in move.items():
            self.refs[q], self.refs[p] = self.refs[p], 0
            for t in self.pools.values():
                t[:, q] = t[:, p]
        for s, m in enumerate(self.lens):
            for j in range(self.pages(m)):
                self.table[s][j] = move.get(self.table[s][j], self.table[s][j])

    def check(self, pools=True):
        c = self.c
        assert c.lens.tolist() == self.lens and c.starts.tolist() == self.starts
        assert c.refs.tolist() == self.refs
        for s, n in enumerate(self.lens):
            k = self.pages(n)
            assert c.table[s, :k].tolist() == self.table[s][:k], s
        bits = c.free_bits.tolist()
        assert [bits[p // 32] >> p % 32 & 1 for p in range(len(self.refs))] == [int(r == 0) for r in self.refs]
        assert c.n_used.tolist() == [sum(r > 0 for r in self.refs)]
        held = {}
        for s, n in enumerate(self.lens):
            for j in range(self.pages(n)):
                p = self.table[s][j]
                held[p] = held.get(p, 0) + 1
                if j == n // self.P:
                    assert self.refs[p] == 1  # a page that is not full has one holder
        assert [held.get(p, 0) for p in range(len(self.refs))] == self.refs
        if pools:
            for name, t in self.pools.items():
                assert torch.equal(raw(getattr(c, name)), t), name


def raw(t):
    """Comparable bits of a tensor."""
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t.view(torch.int16) if t.dtype == torch.bfloat16 else t
