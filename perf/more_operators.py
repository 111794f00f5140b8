"""What the paged cache is measured on.

The cases follow a server whose sequences come and go: prompts enter a cache
of pages, decode steps attend over it, beams share their prefix, sequences
end, and the pool is closed up.  ``run`` computes each pass in elementary
torch operations, or (``own``) with the library's calls.

A pool holds pages of ``P`` rows (one row: the key or value of one token and
KV head).  Sequence s has ``lens[s]`` rows in the pages ``table[s][0..]``;
``refs`` counts the sequences that hold a page, a page that is not full has one
holder, and a page without holders has its bit set in ``free_bits``.  New pages
are always the free ones of the lowest numbers, in the order of the sequences.

The 8-bit form of a row of 128 values: a power of two S, the smallest with
max|x| <= 448 S (exponent in [-60, 52], stored plus 127), and e4m3 codes of x / S.
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)


# ---------------------------------------------------------------- the cases


def listed():
    batch = ("12288,511,16000,4097,8192,15000,64,7777,13000,2048,16383,10240,6000,1,9001,333,"
             "14000,5000,700,11111,2500,8191,95,4000")
    ragged = "1531,64,777,2048,1,3001"
    return [
        # a few short sequences: all latency
        dict(name="attend_short", kind="attend", type="bf16", hq=16, hkv=2, page=16, lens="1,17,300,77", window=0),
        # one sequence with 128K tokens: all bandwidth
        dict(name="attend_long", kind="attend", type="bf16", hq=32, hkv=8, page=16, lens="131072", window=0),
        # an ordinary ragged batch
        dict(name="attend_batch", kind="attend", type="bf16", hq=32, hkv=8, page=32, lens=batch, window=0),
        # a ragged batch in 8 bits, eight query heads for each KV head
        dict(name="attend_batch_8bit", kind="attend", type="e4m3", hq=32, hkv=4, page=16, lens=batch, window=0),
        # a layer with a sliding window over long sequences, 16 query heads for each KV head
        dict(name="attend_window_8bit", kind="attend", type="e4m3", hq=64, hkv=4, page=64,
             lens="60000,32768,5000,41,20001,65536,30000,4096", window=4096),
        # a decode step of a batch whose new tokens are then rejected: grow, append, attend, roll back
        dict(name="step_batch", kind="step", type="bf16", hq=32, hkv=8, page=16,
             lens=",".join([ragged, "4095,2000,500,8000"] * 3)),
        # an ordinary batch of prompts takes the place of the sequences that have ended, and is read back
        dict(name="admit_packed", kind="admit", type="bf16", hkv=8, page=16, lens=ragged),
        # one long prompt in 8 bits
        dict(name="admit_long_8bit", kind="admit", type="e4m3", hkv=8, page=64, lens="32768"),
        # one request becomes four samples: all latency
        dict(name="fork_samples", kind="fork", hkv=8, page=16, layers=1, lens="1003", beams=4),
        # every step of a beam search: each beam continues one of its request's
        dict(name="fork_beams", kind="fork", hkv=4, page=16, layers=2, lens="6001,2040,3999,513,4500,1777,128,5000", beams=8),
        # a small pool is closed up after some sequences have ended
        dict(name="compact_small", kind="compact", hkv=2, page=16, layers=1, lens="100,200,300,50"),
        # a pool of two thousand pages, half of whose sequences have ended
        dict(name="compact_large", kind="compact", hkv=8, page=16, layers=2, lens="4000,2000,6000,1000,3000,500,7000,8000"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "step", "admit", "fork", "compact"])
    hq, hkv = rng.choice([(8, 8), (32, 8), (16, 2), (12, 4), (10, 2), (32, 4), (32, 2), (24, 1), (7, 7)])
    page = rng.choice([16, 32, 64, 128])
    text = lambda v: ",".join(map(str, v))  # noqa: E731
    if kind in ("attend", "step"):
        n = _log_int(rng, 1, 40 if kind == "attend" else 24)
        top = _log_int(rng, 16, max(64, (800000 if kind == "attend" else 200000) // (n * hkv)))
        lens = text([_log_int(rng, 1, top) for _ in range(n)])
        if kind == "step":
            return dict(kind=kind, type="bf16", hq=hq, hkv=hkv, page=page, lens=lens)
        return dict(kind=kind, type=rng.choice(["bf16", "e4m3"]), hq=hq, hkv=hkv, page=page, lens=lens,
                    window=rng.choice([0, 0, _log_int(rng, 1, 5000)]))
    if kind == "admit":
        lens = [_log_int(rng, 1, 8000) for _ in range(rng.randint(1, 4))]
        return dict(kind=kind, type=rng.choice(["bf16", "e4m3"]), hkv=hkv, page=page, lens=text(lens))
    lens = text([_log_int(rng, 1, 4000) for _ in range(rng.randint(1, 6))])
    hkv = min(hkv, 4)
    if kind == "fork":
        return dict(kind=kind, hkv=hkv, page=page, layers=rng.randint(1, 2), lens=lens, beams=rng.randint(2, 6))
    return dict(kind=kind, hkv=hkv, page=page, layers=rng.randint(1, 2), lens=lens)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _pages(n, page):
    return -(-n // page)


def work(case):
    kind, hkv, page = case["kind"], case["hkv"], case["page"]
    lens = _ints(case["lens"])
    row = 2 * 2 * D if case.get("type", "bf16") == "bf16" else 2 * (D + 1)  # a key and a value row
    if kind in ("attend", "step"):
        new, hq, w = (1 if kind == "step" else 0), case["hq"], case.get("window") or max(lens) + 1
        rows = sum(min(n + new, w) for n in lens)
        # rows, table entries, queries, results and their sums; of a step also the new rows and their pages
        b = rows * hkv * row + 4 * sum(_pages(min(n + new, w), page) for n in lens) + len(lens) * (hq * (4 * D + 4) + 4)
        b += new * len(lens) * (hkv * 2 * row + 16)
        return {"bytes": b, "flops": 4 * D * hq * rows}
    if kind == "admit":
        total, p = sum(lens) * hkv, sum(_pages(n, page) for n in lens)
        # the prompt read, rows written and read again, the values written; a page's entry and count, twice
        return {"bytes": total * (2 * 4 * D + 2 * row) + 32 * p + 16 * len(lens), "flops": 0 if row == 4 * D else 6 * D * total}
    layers = case["layers"]
    if kind == "fork":
        n = [x for x in lens for _ in range(case["beams"])]
        full = sum(x // page for x in n)
        # entries read and written, counts raised and lowered, the rows of the last pages copied
        return {"bytes": 24 * full + 48 * len(n) + 2 * layers * hkv * 4 * D * sum(x % page for x in n), "flops": 0}
    p = sum(_pages(x, page) for x in lens)
    # both rounds move as many pages as the groups hold; entries and counts with them, and both groups end and start again
    return {"bytes": 2 * p * (2 * layers * hkv * page * 4 * D + 24 + 32), "flops": 0}


# --------------------------------------------------------------- the inputs


def _starts(lens, dev):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(dev)


def prepare(case, seed):
    dev, bf = "cuda", torch.bfloat16
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    kind, hkv, page = case["kind"], case["hkv"], case["page"]
    want = _ints(case["lens"])
    s = dict(case, want=want, layers=case.get("layers", 1))
    if kind == "fork":      # beams of one request share what they had before it was forked
        lens = [n for n in want for _ in range(case["beams"])]
    elif kind == "compact":  # two groups
        lens = want + want
    elif kind == "admit":   # sequences that have ended, of the new ones' lengths in another order
        lens = want[1:] + want[:1]
    else:
        lens = want
    n = len(lens)
    held = [_pages(x, page) for x in lens]
    wide = max(held) + 1
    spare = sum(_pages(x, page) for x in want) + n if kind == "admit" else 2 * n
    n_pages = -(-(sum(held) + spare + 7) // 32) * 32
    # a pool that has been in use: pages are handed out in no order
    order = torch.rand(n_pages, generator=gen, device=dev).argsort().to(torch.int32)
    table = torch.zeros(n, wide, dtype=torch.int32, device=dev)
    refs = torch.zeros(n_pages, dtype=torch.int32, device=dev)
    j = torch.arange(wide, device=dev)
    at = torch.tensor([0] + held[:-1], device=dev).cumsum(0)
    pages = torch.tensor(held, device=dev)
    rank = at[:, None] + j[None]
    if kind == "fork":
        # full pages are the first beam's, the last one is each beam's own
        first = torch.arange(n, device=dev) // case["beams"] * case["beams"]
        full = torch.tensor([x // page for x in lens], device=dev)
        rank = torch.where(j[None] < full[:, None], at[first][:, None] + j[None], rank)
    live = j[None] < pages[:, None]
    table = torch.where(live, order[rank.clamp(max=n_pages - 1)], table)
    refs.scatter_add_(0, table.flatten().long(), live.flatten().to(torch.int32))
    size = (s["layers"], n_pages, hkv, page)
    c = s["cache"] = dict(table=table, lens=i32(lens), starts=i32(lens), refs=refs, free_bits=_bits(refs == 0),
                          n_used=(refs > 0).sum(0, keepdim=True).to(torch.int32))
    for name in ("k", "v"):
        x = torch.empty(*size, D, dtype=bf, device=dev)
        for layer in x:  # a layer at a time: the numbers are made in 32 bits
            layer.copy_(normal(*size[1:], D))
        if case.get("type") == "e4m3":
            codes = torch.empty(*size, D, dtype=torch.float8_e4m3fn, device=dev)
            scales = torch.empty(*size, dtype=torch.uint8, device=dev)
            for i in range(s["layers"]):
                for a in range(0, n_pages, 4096):
                    y, e = _quantise(x[i, a:a + 4096])
                    codes[i, a:a + 4096].view(torch.uint8).copy_(y.view(torch.uint8))
                    scales[i, a:a + 4096] = e
            c[name + "_pages"], c[name + "_scales"] = codes, scales
        else:
            c[name + "_pages"] = x
    if kind in ("attend", "step"):
        s["q"] = (2.0 * normal(n, case["hq"], D)).to(bf)
        s["out"] = torch.zeros(n, case["hq"], D, dtype=bf, device=dev)
        s["lse"] = torch.zeros(n, case["hq"], device=dev)
    s["all"] = torch.arange(n, dtype=torch.int32, device=dev)
    if kind == "step":
        s.update(k=normal(n, hkv, D).to(bf), v=normal(n, hkv, D).to(bf), new=torch.ones(n, dtype=torch.int32, device=dev),
                 before=i32(lens), longest=max(lens) + 1)
    elif kind == "attend":
        s["longest"] = max(lens)
    elif kind == "admit":
        s.update(k=normal(sum(want), hkv, D).to(bf), v=normal(sum(want), hkv, D).to(bf), new=i32(want), cu=_starts(want, dev))
        s["k_out"], s["v_out"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
    elif kind == "fork":
        b = case["beams"]
        pick = torch.randint(0, b, (n,), generator=gen, device=dev, dtype=torch.int32)
        if b > 2 and len(want) == 1:  # one request's first sequence becomes all of them
            pick.zero_()
        s["src"] = (s["all"] // b * b + pick).to(torch.int32)
    elif kind == "compact":
        m = len(want)
        group = [s["all"][:m].contiguous(), s["all"][m:].contiguous()]
        s["groups"] = [(g, (c["lens"] * ((s["all"] < m) == (i == 0))).to(torch.int32)) for i, g in enumerate(group)]
    if own:
        from long_context_kv_gb300 import paris

        s["handle"] = paris.PagedCache(**c)
    return s


# ----------------------------------------------------------- the plain forms


def _bits(flags):
    """32 truth values to an int32 word, the first one lowest."""
    w = (flags.reshape(-1, 32).long() << torch.arange(32, device=flags.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _quantise(x):
    """Rows [..., 128] as e4m3 codes and scale bytes."""
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=2.0 ** 60, neginf=-2.0 ** 60).clamp_(-2.0 ** 60, 2.0 ** 60)
    m, e = torch.frexp(x.abs().amax(-1))            # m in [0.5, 1); 448 is 0.875 2^9
    e = (torch.where(m > 0.875, e + 1, e) - 9).clamp_(-60, 52)
    e = torch.where(m == 0, torch.full_like(e, -60), e)
    return (x * _power(-e)[..., None]).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _power(e):
    """2^e as float32, by its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _values(codes, scales):
    """float32 values of 8-bit rows."""
    return codes.float() * _power(scales.to(torch.int32) - 127)[..., None]


def _cached(c, name, layer, at, rows):
    """Rows [n, Hkv, rows, 128] of sequences whose pages are at [n, ...]."""
    x = c[name + "_pages"][layer]
    scales = c.get(name + "_scales")
    x = x[at].float() if scales is None else _values(x.view(torch.uint8)[at].view(x.dtype), scales[layer][at])
    return x.transpose(1, 2).flatten(2, 3)[:, :, :rows]


def _plain_attend(c, q, window, longest):
    n, hq, _ = q.shape
    _, _, hkv, page, _ = c["k_pages"].shape
    at = c["table"][:, :_pages(longest, page)].long()
    k, v = _cached(c, "k", 0, at, longest), _cached(c, "v", 0, at, longest)
    s = (q.float().reshape(n, hkv, hq // hkv, D) * SCALE) @ k.transpose(2, 3)
    j, lens = torch.arange(longest, device=q.device)[None], c["lens"][:, None]
    seen = j < lens
    if window:
        seen &= j >= lens - window
    s.masked_fill_(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, (p @ v) / total, torch.zeros(1, device=q.device))
    return o.reshape(n, hq, D).to(torch.bfloat16), (top + torch.log(total)).reshape(n, hq)


def _free_list(refs):
    """The free pages in ascending order (then zeros), and their number."""
    free = refs == 0
    where = torch.where(free, free.cumsum(0) - 1, torch.full_like(refs, refs.numel(), dtype=torch.int64))
    pages = torch.arange(refs.numel(), device=refs.device)
    return torch.zeros(refs.numel() + 1, dtype=torch.int64, device=refs.device).scatter_(0, where, pages * free)[:-1], free.sum()


def _counted(c):
    c["free_bits"].copy_(_bits(c["refs"] == 0))
    c["n_used"].copy_((c["refs"] > 0).sum(0, keepdim=True))


def _plain_grow(c, new):
    page, wide = c["k_pages"].shape[3], c["table"].shape[1]
    lens, dev = c["lens"].long(), new.device
    new = torch.minimum(new.long().clamp(min=0), wide * page - lens)
    have, need = (lens + page - 1) // page, (lens + new + page - 1) // page
    need = need - have
    first = need.cumsum(0) - need
    pages, n_free = _free_list(c["refs"])
    got = torch.minimum((n_free - first).clamp(min=0), need)
    j = torch.arange(wide, device=dev)[None] - have[:, None]
    fresh = (j >= 0) & (j < got[:, None])
    entry = pages[(first[:, None] + j).clamp(0, pages.numel() - 1)]
    c["table"].copy_(torch.where(fresh, entry.to(torch.int32), c["table"]))
    c["refs"].scatter_add_(0, torch.where(fresh, entry, 0).flatten(), fresh.flatten().to(torch.int32))
    c["starts"].copy_(lens)
    c["lens"].copy_(torch.minimum(lens + new, (have + got) * page))
    _counted(c)


def _places(c, cu, total):
    """Sequence, place and page row of each packed row."""
    r = torch.arange(total, device=cu.device)
    seq = torch.searchsorted(cu[1:].contiguous(), r, right=True)
    return seq, r - cu[seq]


def _plain_store(c, k, v, cu):
    page = c["k_pages"].shape[3]
    seq, at = _places(c, cu, k.shape[0])
    at = c["starts"][seq] + at
    to = c["table"][seq, at // page].long()
    for name, x in (("k", k), ("v", v)):
        if name + "_scales" in c:
            x, e = _quantise(x)
            c[name + "_pages"].view(torch.uint8)[0, to, :, at % page] = x.view(torch.uint8)
            c[name + "_scales"][0, to, :, at % page] = e
        else:
            c[name + "_pages"][0, to, :, at % page] = x


def _plain_read(c, cu, total):
    page = c["k_pages"].shape[3]
    seq, at = _places(c, cu, total)
    to, at = c["table"][seq, at // page].long(), at % page
    out = []
    for name in ("k", "v"):
        x, e = c[name + "_pages"], c.get(name + "_scales")
        x = x[0, to, :, at] if e is None else _values(x.view(torch.uint8)[0, to, :, at].view(x.dtype), e[0, to, :, at])
        out.append(x.to(torch.bfloat16))
    return out


def _plain_fork(c, src, dst, rows=None):
    """Sequence dst[i] becomes the first rows[i] rows (default: all) of sequence src[i] as it was before the call."""
    page, wide = c["k_pages"].shape[3], c["table"].shape[1]
    src, dst, lens, refs = src.long(), dst.long(), c["lens"].long(), c["refs"]
    n = lens[src] if rows is None else torch.minimum(lens[src], rows.long().clamp(min=0))
    j = torch.arange(wide, device=src.device)[None]
    full, part = n // page, n % page > 0
    theirs, old = c["table"][src].long(), c["table"][dst].long()
    shared = j < full[:, None]
    refs.scatter_add_(0, theirs.flatten(), shared.flatten().to(torch.int32))
    last = theirs.gather(1, full.clamp(max=wide - 1)[:, None])[:, 0]
    stay = part & (src == dst) & (refs[last] == 1)
    pages, n_free = _free_list(refs)
    copy = part & ~stay
    rank = copy.cumsum(0) - 1
    copy, full_only = copy & (rank < n_free), copy & (rank >= n_free)
    n = torch.where(full_only, full * page, n)
    fresh = torch.where(copy, pages[rank.clamp(min=0)], last)
    refs.scatter_add_(0, fresh, (copy | stay).to(torch.int32))
    gone = j < ((lens[dst] + page - 1) // page)[:, None]
    refs.scatter_add_(0, old.flatten(), -gone.flatten().to(torch.int32))
    last_one = (j == full[:, None]) & (copy | stay)[:, None]
    c["table"][dst] = torch.where(shared, theirs, torch.where(last_one, fresh[:, None], old)).to(torch.int32)
    # items that copy nothing do what the first one that does is doing, so that no page is written in two ways
    first = copy.to(torch.int32).argmax(0, keepdim=True)
    fresh, last, rows = (torch.where(copy, x, x[first]) for x in (fresh, last, n % page))
    live = (torch.arange(page, device=src.device)[None] < rows[:, None]) & copy.any()
    for name in ("k_pages", "v_pages"):
        x = c[name]
        x[:, fresh] = torch.where(live[None, :, None, :, None], x[:, last], x[:, fresh])
    c["lens"][dst] = n.to(torch.int32)
    c["starts"][dst] = n.to(torch.int32)
    _counted(c)


def _plain_compact(c):
    """The used pages past their number move, in ascending order, to the free ones below it."""
    refs, page = c["refs"], c["k_pages"].shape[3]
    n = refs.numel()
    at, used = torch.arange(n, device=refs.device), refs > 0
    high, low = used & (at >= used.sum()), ~used & (at < used.sum())
    targets = torch.zeros(n + 1, dtype=torch.int64, device=refs.device).scatter_(0, torch.where(low, low.cumsum(0) - 1, n), at)
    to = torch.where(high, targets[(high.cumsum(0) - 1).clamp(min=0)], at)
    source = torch.cat([at, at[:1]]).scatter_(0, torch.where(high, to, n), at)[:n]
    mine = torch.arange(c["table"].shape[1], device=refs.device)[None] < ((c["lens"] + page - 1) // page)[:, None]
    c["table"].copy_(torch.where(mine, to[c["table"].long()], c["table"]))
    refs.copy_(torch.where(high, 0, refs[source]))
    for name in ("k_pages", "v_pages"):
        c[name].copy_(c[name][:, source])
    _counted(c)


# ------------------------------------------------------------------- a pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(s):
    kind, c = s["kind"], s["cache"]
    if kind == "attend":
        out, lse = _plain_attend(c, s["q"], s["window"], s["longest"])
        return {"out": out, "lse": lse}
    if kind == "step":
        _plain_grow(c, s["new"])
        _plain_store(c, s["k"], s["v"], torch.arange(len(s["want"]) + 1, dtype=torch.int32, device=s["k"].device))
        out, lse = _plain_attend(c, s["q"], 0, s["longest"])
        _plain_fork(c, s["all"], s["all"], s["before"])
        return dict(c, out=out, lse=lse)
    if kind == "admit":
        _plain_fork(c, s["all"], s["all"], torch.zeros_like(s["all"]))
        _plain_grow(c, s["new"])
        _plain_store(c, s["k"], s["v"], s["cu"])
        k, v = _plain_read(c, s["cu"], s["k"].shape[0])
        return _held(c, k_out=k, v_out=v)
    if kind == "fork":
        _plain_fork(c, s["src"], s["all"])
        return dict(c)
    for group, new in s["groups"]:
        _plain_fork(c, group, group, torch.zeros_like(group))
        _plain_compact(c)
        _plain_grow(c, new)
    return dict(c)


def _run_own(s):
    kind, c, h = s["kind"], s["cache"], s["handle"]
    if kind == "attend":
        h.paris_paged_attend(s["q"], s["out"], window=s["window"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "step":
        h.paris_paged_grow(s["new"])
        h.paris_paged_append(s["k"], s["v"])
        h.paris_paged_attend(s["q"], s["out"], lse=s["lse"])
        h.paris_paged_free(s["all"], rows=s["before"])
        return dict(c, out=s["out"], lse=s["lse"])
    if kind == "admit":
        h.paris_paged_free(s["all"])
        h.paris_paged_grow(s["new"])
        h.paris_paged_store(s["k"], s["v"], cu=s["cu"], max_new=max(s["want"]))
        h.paris_paged_read(s["k_out"], s["v_out"], cu=s["cu"], max_rows=max(s["want"]))
        return _held(c, k_out=s["k_out"], v_out=s["v_out"])
    if kind == "fork":
        h.paris_paged_fork(s["src"], s["all"])
        return dict(c)
    for group, new in s["groups"]:
        h.paris_paged_free(group)
        h.paris_paged_compact()
        h.paris_paged_grow(new)
    return dict(c)


def _held(c, **more):
    """The cache without its pages' bytes, whose values stand beside it."""
    return dict({name: t for name, t in c.items() if not name.startswith(("k_", "v_"))}, **more)


# ---------------------------------------------------- the same in 64 bits


def _exact_rows(x):
    """The values that 8-bit rows of x stand for, from the definition, in 64 bits."""
    x = x.double()
    s = torch.full_like(x[..., :1], 2.0 ** -60)
    for i in range(-60, 52):
        s = torch.where(x.abs().amax(-1, keepdim=True) > 448.0 * 2.0 ** i, 2.0 ** (i + 1), s)
    y = x / s
    quantum = torch.full_like(y, 2.0 ** -9)  # four significant bits, none below 2^-9
    for i in range(-5, 9):
        quantum = torch.where(y.abs() >= 2.0 ** i, 2.0 ** (i - 3), quantum)
    return torch.round(y / quantum) * quantum * s


class _Sim:
    """The table and the pages' counts of a cache, one sequence after the other."""

    def __init__(self, s):
        c = s["cache"]
        self.page, self.lens, self.starts = s["page"], c["lens"].tolist(), c["lens"].tolist()
        self.table, self.refs = c["table"].tolist(), c["refs"].tolist()
        self.pools = [c["k_pages"], c["v_pages"]]

    def take(self):
        p = self.refs.index(0)
        self.refs[p] = 1
        return p

    def drop(self, s):
        for p in self.table[s][:_pages(self.lens[s], self.page)]:
            self.refs[p] -= 1

    def grow(self, s, n):
        self.starts[s] = self.lens[s]
        for j in range(_pages(self.lens[s], self.page), _pages(self.lens[s] + n, self.page)):
            self.table[s][j] = self.take()
        self.lens[s] += n

    def free(self, s):
        self.drop(s)
        self.lens[s] = self.starts[s] = 0

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        low = [p for p in range(n) if self.refs[p] == 0]
        move = dict(zip([p for p in range(n, len(self.refs)) if self.refs[p]], low))
        for p, t in move.items():
            self.refs[t], self.refs[p] = self.refs[p], 0
        for x in self.pools:
            if move:
                x[:, list(move.values())] = x[:, list(move)]
        for s, n in enumerate(self.lens):
            for j in range(_pages(n, self.page)):
                self.table[s][j] = move.get(self.table[s][j], self.table[s][j])

    def result(self, pools=True, **more):
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        refs = t(self.refs)
        r = dict(table=t(self.table), lens=t(self.lens), starts=t(self.starts), refs=refs, free_bits=_bits(refs == 0),
                 n_used=t([sum(x > 0 for x in self.refs)]))
        if pools:
            r.update(k_pages=self.pools[0].double(), v_pages=self.pools[1].double())
        return dict(r, **more)


def _exact_attend(s, lens, window):
    c, hq, hkv, page = s["cache"], s["hq"], s["hkv"], s["page"]
    powers = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")
    out = torch.zeros(len(lens), hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens), hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        at = torch.arange(first, n, device="cuda")
        entry = c["table"][b].long()[at // page]
        rows = {}
        for name in ("k", "v"):
            x = c[name + "_pages"][0]
            if name + "_scales" in c:
                x = x.view(torch.uint8)[entry, :, at % page].view(x.dtype).double()
                x = x * powers[c[name + "_scales"][0][entry, :, at % page].long()][..., None]
            else:
                x = x[entry, :, at % page].double()
            rows[name] = x.transpose(0, 1)
        g = hq // hkv
        for h in range(hkv):
            sc = s["q"][b, h * g:(h + 1) * g].double() @ rows["k"][h].T / math.sqrt(D)
            lse[b, h * g:(h + 1) * g] = torch.logsumexp(sc, -1)
            out[b, h * g:(h + 1) * g] = torch.softmax(sc, -1) @ rows["v"][h]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    kind, page, sim = s["kind"], s["page"], _Sim(s)
    if kind == "attend":
        out, lse = _exact_attend(s, s["want"], s["window"])
        return {"out": out, "lse": lse}
    every = range(len(sim.lens))
    if kind == "step":
        c = s["cache"]
        for b in every:
            at = sim.lens[b]
            sim.grow(b, 1)
            p = sim.table[b][at // page]
            c["k_pages"][0, p, :, at % page], c["v_pages"][0, p, :, at % page] = s["k"][b], s["v"][b]
            c["table"][b, at // page] = p
        out, lse = _exact_attend(s, sim.lens, 0)
        for b in every:
            if sim.lens[b] % page == 1 or page == 1:
                sim.refs[sim.table[b][sim.lens[b] // page]] -= 1
            sim.lens[b] = sim.starts[b] = sim.lens[b] - 1
        return sim.result(out=out, lse=lse)
    if kind == "admit":
        for b in every:
            sim.free(b)
        for b, n in enumerate(s["want"]):
            sim.grow(b, n)
        k, v = (_exact_rows(x) if case["type"] == "e4m3" else x.double() for x in (s["k"], s["v"]))
        return sim.result(pools=False, k_out=k, v_out=v)
    if kind == "fork":
        src, old = s["src"].tolist(), [list(t) for t in sim.table]
        copies = []
        for b in every:
            for p in old[src[b]][:sim.lens[src[b]] // page]:
                sim.refs[p] += 1
        for b in every:
            n, a = sim.lens[src[b]], src[b]
            full = n // page
            sim.table[b] = old[a][:full] + old[b][full:]
            if n % page:
                if a == b and sim.refs[old[a][full]] == 1:
                    sim.refs[old[a][full]] += 1
                    sim.table[b][full] = old[a][full]
                else:
                    sim.table[b][full] = sim.take()
                    copies.append((old[a][full], sim.table[b][full], n % page))
        for b in every:
            for p in old[b][:_pages(sim.lens[b], page)]:
                sim.refs[p] -= 1
        for x in sim.pools:
            for p, t, n in copies:
                x[:, t, :, :n] = x[:, p, :, :n]
        sim.lens = [sim.lens[a] for a in src]
        sim.starts = list(sim.lens)
        return sim.result()
    for group, new in s["groups"]:
        for b in group.tolist():
            sim.free(b)
        sim.compact()
        sim.starts = list(sim.lens)
        for b in group.tolist():
            sim.grow(b, new[b].item())
    return sim.result()
