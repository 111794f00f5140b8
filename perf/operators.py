"""What the prompt attention and the 4-bit cache are measured on.

The cases follow one layer of a served model from its prompt to its decode
steps: causal attention over packed prompts, the attention weights that the
prompt's last queries give to every key, the cache in 4 bits, attention over
it, and eviction from it by accumulated weight.  ``run`` computes each pass in
elementary torch operations, or (``own``) with the library's calls.

The 4-bit form of a row of 128 values: four groups of 32; a group's scale is
max|x| / 7 rounded up to four significant bits (a positive half-precision
number whose lower seven bits are zero, stored as its upper byte), and a value
is rint(x / scale) in [-7, 7], stored as that number plus 8, two to a byte.
"""
import math

import torch

own = False

D = 128                      # head dimension
GROUP = 32                   # values that share a scale
SCALE = 1.0 / math.sqrt(D)
LIMIT = 1680.0               # 7 times the largest scale (240)


# ---------------------------------------------------------------- the cases


def listed():
    ragged = "1531,64,777,2048,1,3001"
    batch = "16384,1,9001,12288,511,16000,4097,8192,15000,64,7777,13000,2048,16383,10240,6000"
    return [
        # a few short requests that arrive together: all latency
        dict(name="prompt_short", kind="prompt", hq=8, hkv=2, lens_q="1,5,33", lens_k="1,5,33"),
        # an ordinary batch of prompts of very different lengths, packed
        dict(name="prompt_packed", kind="prompt", hq=32, hkv=8, lens_q=ragged, lens_k=ragged),
        # one chunk of a long prompt that is read piece by piece: 512 queries after 32256 tokens
        dict(name="prompt_chunk", kind="prompt", hq=32, hkv=8, lens_q="512", lens_k="32768"),
        # a long prompt, with the share of the heads that one of four GPUs holds
        dict(name="prompt_long", kind="prompt", hq=8, hkv=2, lens_q="32768", lens_k="32768"),
        # the weights that choose what an ordinary batch keeps
        dict(name="weights_packed", kind="weights", hq=32, hkv=8, lens=ragged, window=32),
        # the same for one long prompt
        dict(name="weights_long", kind="weights", hq=32, hkv=8, lens="32768", window=64),
        # one sequence with 128K tokens in the cache: all bandwidth
        dict(name="attend_long", kind="attend", hq=32, hkv=8, rows=131072, lens="131072", accumulate=False),
        # a ragged batch whose decode steps also accumulate the weights
        dict(name="attend_batch", kind="attend", hq=32, hkv=4, rows=16384, lens=batch, accumulate=True),
        # a long prompt's keys and values go into the cache and are read back as what it holds
        dict(name="store_prompt", kind="store", hkv=8, lens="32768", type="bf16"),
        # four sequences under a budget take 512 tokens each and drop as many
        dict(name="evict_chunk", kind="evict", batch=4, hkv=8, keep=8192, chunk=512, sink=16, recent=512),
        # one decode step of one sequence under a small budget: all latency
        dict(name="step_small", kind="step", batch=1, hq=32, hkv=8, keep=2048, sink=16, recent=256),
        # one decode step of a batch under a budget
        dict(name="step_batch", kind="step", batch=32, hq=32, hkv=8, keep=4096, sink=16, recent=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    hq, hkv = rng.choice([(8, 8), (32, 8), (16, 2), (12, 4), (10, 2), (32, 4), (32, 2)])
    kind = rng.choice(["prompt", "prompt", "weights", "attend", "attend", "store", "evict", "step"])
    text = lambda v: ",".join(map(str, v))  # noqa: E731
    if kind == "prompt":
        n = rng.randint(1, 8)
        top = _log_int(rng, 2, int(math.sqrt(4e9 / (n * hq))))
        lk = [_log_int(rng, 1, top) for _ in range(n)]
        lq = [_log_int(rng, 1, k) for k in lk] if rng.random() < 0.4 else lk
        return dict(kind=kind, hq=hq, hkv=hkv, lens_q=text(lq), lens_k=text(lk))
    if kind == "weights":
        return dict(kind=kind, hq=hq, hkv=hkv, lens=text([_log_int(rng, 1, 8000) for _ in range(rng.randint(1, 6))]),
                    window=_log_int(rng, 1, 64))
    if kind == "attend":
        n = _log_int(rng, 1, 32)
        rows = _log_int(rng, 16, max(64, 1000000 // (n * hkv)))
        return dict(kind=kind, hq=hq, hkv=hkv, rows=rows, lens=text([_log_int(rng, 1, rows) for _ in range(n)]),
                    accumulate=rng.random() < 0.5)
    if kind == "store":
        return dict(kind=kind, hkv=hkv, lens=text([_log_int(rng, 1, 16000) for _ in range(rng.randint(1, 4))]),
                    type=rng.choice(["bf16", "f32"]))
    keep = _log_int(rng, 64, 8000)
    sink, recent = rng.randint(0, 16), rng.randint(1, keep // 2)
    if kind == "evict":
        return dict(kind=kind, batch=rng.randint(1, 4), hkv=hkv, keep=keep, chunk=_log_int(rng, 1, 1000), sink=sink,
                    recent=recent)
    return dict(kind=kind, batch=rng.randint(1, 16), hq=hq, hkv=hkv, keep=keep, sink=sink, recent=recent)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _pairs(lq, lk):
    """Visible (query, key) pairs: query i sees the keys up to i + lk - lq."""
    first = max(0, lq - lk)
    return (lq - first) * (lk - lq) + (lq * (lq + 1) - first * (first + 1)) // 2


def work(case):
    kind, hkv = case["kind"], case["hkv"]
    row4 = 2 * (D // 2 + D // GROUP)  # codes and scales of a key and a value row
    if kind == "prompt":
        lq, lk, hq = _ints(case["lens_q"]), _ints(case["lens_k"]), case["hq"]
        pairs = sum(_pairs(a, b) for a, b in zip(lq, lk))
        return {"bytes": 2 * D * (2 * hq * sum(lq) + 2 * hkv * sum(lk)) + 4 * hq * sum(lq), "flops": 4 * D * hq * pairs}
    if kind == "weights":
        lens, hq, w = _ints(case["lens"]), case["hq"], case["window"]
        pairs = sum(_pairs(min(w, n), n) for n in lens)
        seen = sum(min(w, n) for n in lens)
        return {"bytes": sum(lens) * hkv * (2 * D + 4) + seen * hq * (2 * D + 4), "flops": 2 * D * hq * pairs}
    if kind == "attend":
        lens, hq = _ints(case["lens"]), case["hq"]
        rows = sum(lens) * hkv
        return {"bytes": rows * (row4 + (8 if case["accumulate"] else 0)) + len(lens) * hq * 4 * D,
                "flops": 4 * D * hq * sum(lens)}
    if kind == "store":
        rows = sum(_ints(case["lens"])) * hkv
        size = 2 if case["type"] == "bf16" else 4
        return {"bytes": rows * (2 * D * size + 2 * row4 + 8 + 4 * D), "flops": 8 * D * rows}
    heads, keep = case["batch"] * hkv, case["keep"]
    if kind == "evict":
        c = case["chunk"]
        return {"bytes": heads * (c * (4 * D + row4 + 12) + 8 * (keep + c) + 2 * c * (row4 + 8) + keep * (row4 + 4 * D)),
                "flops": heads * c * 16 * D}
    return {"bytes": heads * (keep + 1) * (row4 + 16) + case["batch"] * case["hq"] * 4 * D,
            "flops": 4 * D * case["batch"] * case["hq"] * (keep + 1)}


# --------------------------------------------------------------- the inputs


def _starts(lens, dev):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(dev)


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    bf = torch.bfloat16
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=dev)  # noqa: E731
    kind, hkv = case["kind"], case["hkv"]
    s = dict(case)
    if kind in ("prompt", "weights"):
        hq = case["hq"]
        lq = _ints(case["lens_q"] if kind == "prompt" else case["lens"])
        lk = _ints(case["lens_k"]) if kind == "prompt" else lq
        s.update(cu_q=_starts(lq, dev), cu_k=_starts(lk, dev), max_q=max(lq), max_k=max(lk))
        # keys share a direction, as a layer's keys do; queries are peaked
        s["q"] = (2.0 * normal(sum(lq), hq, D)).to(bf)
        s["k"] = (normal(sum(lk), hkv, D) + 0.5 * normal(1, hkv, D)).to(bf)
        if kind == "prompt":
            s["v"] = normal(sum(lk), hkv, D).to(bf)
            s["out"] = torch.zeros(sum(lq), hq, D, dtype=bf, device=dev)
            s["lse"] = torch.zeros(hq, sum(lq), device=dev)
        else:
            s["lse"] = _window_lse(s["q"], s["k"], lq, case["window"])
            s["weights"] = torch.zeros(hkv, sum(lk), device=dev)
        return s
    if kind == "attend":
        lens, rows, new = _ints(case["lens"]), case["rows"], 0
    elif kind == "store":
        lens = _ints(case["lens"])
        new, rows = lens, max(lens)
    else:
        lens = [case["keep"]] * case["batch"]
        new = case["chunk"] if kind == "evict" else 1
        rows = case["keep"] + new + (63 if kind == "step" else 0)
    n = len(lens)
    c = s["cache"] = dict(
        k_codes=torch.zeros(n, hkv, rows, D // 2, dtype=torch.uint8, device=dev),
        k_scales=torch.zeros(n, hkv, rows, D // GROUP, dtype=torch.uint8, device=dev),
        v_codes=torch.zeros(n, hkv, rows, D // 2, dtype=torch.uint8, device=dev),
        v_scales=torch.zeros(n, hkv, rows, D // GROUP, dtype=torch.uint8, device=dev),
        weights=torch.zeros(n, hkv, rows, device=dev),
        positions=torch.zeros(n, hkv, rows, dtype=torch.int32, device=dev),
        lens=torch.zeros(n, dtype=torch.int32, device=dev),
        next_pos=torch.zeros(n, dtype=torch.int32, device=dev))
    if kind == "store":
        dt = bf if case["type"] == "bf16" else torch.float32
        s.update(cu=_starts(lens, dev), max_new=max(lens), k=normal(sum(lens), hkv, D).to(dt), v=normal(sum(lens), hkv, D).to(dt))
        s["token_weights"] = torch.rand(hkv, sum(lens), generator=gen, device=dev)
        s["k_out"] = torch.zeros(n, hkv, rows, D, dtype=bf, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    else:
        live = (torch.arange(rows, device=dev) < torch.tensor(lens, device=dev)[:, None])[:, None, :]
        for name in ("k", "v"):
            codes, scales = _quantise(normal(n, hkv, rows, D).to(bf))
            c[name + "_codes"].copy_(codes * live[..., None])
            c[name + "_scales"].copy_(scales * live[..., None])
        c["lens"].copy_(torch.tensor(lens))
        c["weights"].copy_(torch.empty(n, hkv, rows, device=dev).exponential_(generator=gen) * live)
        c["positions"].copy_(torch.arange(rows, device=dev).expand(n, hkv, rows) * live)
        c["next_pos"].copy_(c["lens"])
    if kind in ("attend", "step"):
        s["q"] = (2.0 * normal(n, case["hq"], D)).to(bf)
        s["out"] = torch.zeros(n, case["hq"], D, dtype=bf, device=dev)
    if kind in ("evict", "step"):
        # rows of a cache that has been under its budget for a while: the sink, every fourth token, the latest ones
        keep, sink, recent = case["keep"], case["sink"], case["recent"]
        mid = max(0, keep - sink - recent)
        at = torch.cat([torch.arange(sink), sink + 4 * torch.arange(mid), sink + 4 * mid + torch.arange(recent)])[:keep]
        order = torch.rand(n, hkv, keep, generator=gen, device=dev).argsort(-1)
        c["positions"][:, :, :keep] = at.to(dev, torch.int32)[order]
        c["next_pos"].fill_(sink + 4 * mid + recent)
        s["k"] = normal(n * new, hkv, D).to(bf)
        s["v"] = normal(n * new, hkv, D).to(bf)
    if kind == "evict":
        s.update(cu=_starts([new] * n, dev), max_new=new)
        s["token_weights"] = torch.empty(hkv, n * new, device=dev).exponential_(generator=gen)
        s["k_out"] = torch.zeros(n, hkv, keep, D, dtype=bf, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
    if own:
        from long_context_kv_gb300 import paris

        s["handle"] = paris.KV4Cache(**c)
    return s


def _window_lse(q, k, lens, window):
    """log sum exp of the last queries of each sequence; the other queries' are not used."""
    lse = torch.zeros(q.shape[1], q.shape[0], device=q.device)
    g, at = q.shape[1] // k.shape[1], 0
    for n in lens:
        w = min(window, n)
        qs = q[at + n - w: at + n].double().transpose(0, 1)
        ks = k[at: at + n].double().transpose(0, 1).repeat_interleave(g, 0)
        sc = (qs @ ks.transpose(1, 2)) * SCALE
        later = torch.arange(n, device=q.device)[None, :] > torch.arange(n - w, n, device=q.device)[:, None]
        lse[:, at + n - w: at + n] = sc.masked_fill_(later, -math.inf).logsumexp(-1).float()
        at += n
    return lse


# ----------------------------------------------------------- the plain forms


def _quantise(x):
    x = torch.nan_to_num(x.float(), nan=0.0, posinf=LIMIT, neginf=-LIMIT).clamp_(-LIMIT, LIMIT)
    x = x.reshape(*x.shape[:-1], D // GROUP, GROUP)
    t = x.abs().amax(-1)
    t = t / torch.full_like(t, 7.0)  # a division by a number would be a product with its rounded inverse
    up = (t.view(torch.int32) + 0xFFFFF) & ~0xFFFFF
    small = torch.ceil(t * 2.0 ** 17)
    is_small = t < 2.0 ** -14
    scale = torch.where(is_small, small * 2.0 ** -17, up.view(torch.float32))
    byte = torch.where(is_small, small.to(torch.int32), (up >> 20) - 896).to(torch.uint8)
    u = torch.where(scale[..., None] > 0, torch.round(x / scale[..., None]), torch.zeros_like(x)).clamp_(-7, 7) + 8
    u = u.to(torch.uint8).reshape(*x.shape[:-2], D)
    return u[..., 0::2] | (u[..., 1::2] << 4), byte


def _values(codes, scales):
    """The float32 values that codes and scale bytes stand for."""
    u = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], D // GROUP, GROUP)
    scale = (scales.to(torch.int16) << 7).view(torch.float16).float()
    return ((u.float() - 8.0) * scale[..., None]).reshape(*codes.shape[:-1], D)


def _padded(x, starts, longest):
    """Packed rows [total, H, D] as [sequences, H, longest, D]; rows past a sequence's end repeat some row."""
    at = (starts[:-1, None] + torch.arange(longest, device=x.device)[None]).clamp_(max=x.shape[0] - 1)
    return x.float()[at.long()].transpose(1, 2)


def _hidden(lq, lk, max_q, max_k, dev):
    """[sequences, max_q, max_k]: true where query i does not see key j."""
    i = torch.arange(max_q, device=dev)[None, :, None]
    j = torch.arange(max_k, device=dev)[None, None, :]
    return (j > i + (lk - lq)[:, None, None]) | (j >= lk[:, None, None]) | (i >= lq[:, None, None])


def _unpad(starts, total, dev):
    """(sequence, place in it) of each packed row."""
    r = torch.arange(total, device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), r, right=True)
    return seq, r - starts[seq]


def _plain_prompt(s):
    hq, hkv = s["hq"], s["hkv"]
    g, dev = hq // hkv, s["q"].device
    lq, lk = s["cu_q"].diff(), s["cu_k"].diff()
    q = _padded(s["q"], s["cu_q"], s["max_q"])
    k = _padded(s["k"], s["cu_k"], s["max_k"])
    v = _padded(s["v"], s["cu_k"], s["max_k"])
    n, _, mq, _ = q.shape
    p = (q.reshape(n, hkv, g * mq, D) * SCALE) @ k.transpose(2, 3)
    p = p.reshape(n, hkv, g, mq, -1)
    p.masked_fill_(_hidden(lq, lk, s["max_q"], s["max_k"], dev)[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p.sub_(safe).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(n, hkv, g * mq, -1) @ v).reshape(n, hkv, g, mq, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).reshape(n, hq, mq, D)
    lse = (safe + torch.log(total)).reshape(n, hq, mq)
    seq, at = _unpad(s["cu_q"], s["q"].shape[0], dev)
    return {"out": o[seq, :, at].to(torch.bfloat16), "lse": lse[seq, :, at].transpose(0, 1).contiguous()}


def _plain_weights(s):
    hq, hkv, w = s["hq"], s["hkv"], s["window"]
    g, dev = hq // hkv, s["q"].device
    lens = s["cu_k"].diff()
    k = _padded(s["k"], s["cu_k"], s["max_k"])
    n = k.shape[0]
    i = lens[:, None] - w + torch.arange(w, device=dev)[None]           # a window's queries; below 0 there is none
    row = (s["cu_q"][:-1, None] + i.clamp(min=0)).long()
    q = s["q"].float()[row].transpose(1, 2).reshape(n, hkv, g * w, D)
    lse = s["lse"][:, row].transpose(0, 1)                              # [n, hq, w]
    p = ((q * SCALE) @ k.transpose(2, 3)).reshape(n, hkv, g, w, -1)
    p = torch.exp(p - lse.reshape(n, hkv, g, w, 1))
    j = torch.arange(s["max_k"], device=dev)
    seen = (j[None, None, :] <= i[:, :, None]) & (i[:, :, None] >= 0)
    p = torch.where(seen[:, None, None], p, torch.zeros_like(p)).sum((2, 3))
    seq, at = _unpad(s["cu_k"], s["k"].shape[0], dev)
    return {"weights": p[seq, :, at].transpose(0, 1).contiguous()}


def _plain_attend(c, q, accumulate):
    n, hkv, rows, _ = c["k_codes"].shape
    hq = q.shape[1]
    k, v = _values(c["k_codes"], c["k_scales"]), _values(c["v_codes"], c["v_scales"])
    p = (q.float().reshape(n, hkv, hq // hkv, D) * SCALE) @ k.transpose(2, 3)
    beyond = torch.arange(rows, device=q.device)[None] >= c["lens"][:, None]
    p.masked_fill_(beyond[:, None, None], -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    if accumulate:
        c["weights"] += p.sum(2)
    return (p @ v).reshape(n, hq, D).to(torch.bfloat16)


def _plain_store(c, k, v, starts, weights):
    """Packed rows [total, hkv, D] join their sequences at the end."""
    seq, at = _unpad(starts, k.shape[0], k.device)
    row = (c["lens"][seq] + at).long()
    for name, x in (("k", k), ("v", v)):
        codes, scales = _quantise(x)
        c[name + "_codes"][seq, :, row] = codes
        c[name + "_scales"][seq, :, row] = scales
    c["weights"][seq, :, row] = torch.zeros(k.shape[:2], device=k.device) if weights is None else weights.transpose(0, 1)
    c["positions"][seq, :, row] = (c["next_pos"][seq] + at).to(torch.int32)[:, None].expand(-1, k.shape[1])
    c["lens"] += starts.diff()
    c["next_pos"] += starts.diff()


def _plain_evict(c, keep, sink, recent):
    n, hkv, rows = c["weights"].shape
    dev = c["weights"].device
    row = torch.arange(rows, device=dev).expand(n, hkv, rows)
    lens = c["lens"][:, None, None]
    pos = c["positions"]
    held = (pos < sink) | (pos >= (c["next_pos"] - recent)[:, None, None])
    key = torch.where(held, torch.full_like(c["weights"], math.inf), c["weights"])
    key = torch.where(row < lens, key, torch.full_like(key, -math.inf))
    order = key.sort(dim=-1, descending=True, stable=True).indices
    kept = torch.zeros(n, hkv, rows, dtype=torch.bool, device=dev).scatter_(2, order[..., :keep], True)
    full = lens > keep
    hole, tail = ~kept & (row < keep) & full, kept & (row >= keep) & full
    # the i-th kept row past the budget goes to the i-th dropped row within it
    list_at = torch.where(tail, tail.cumsum(-1) - 1, torch.full_like(row, rows))
    tails = torch.zeros(n, hkv, rows + 1, dtype=torch.int64, device=dev).scatter_(2, list_at, row)
    source = torch.where(hole, tails.gather(2, (hole.cumsum(-1) - 1).clamp_(min=0)), row)
    for name in ("k_codes", "k_scales", "v_codes", "v_scales"):
        c[name].copy_(c[name].gather(2, source[..., None].expand_as(c[name])))
    for name in ("weights", "positions"):
        c[name].copy_(c[name].gather(2, source))
    c["lens"].clamp_(max=keep)


# ------------------------------------------------------------------- a pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(s):
    kind = s["kind"]
    if kind == "prompt":
        return _plain_prompt(s)
    if kind == "weights":
        return _plain_weights(s)
    c = s["cache"]
    if kind == "attend":
        out = _plain_attend(c, s["q"], s["accumulate"])
        return {"out": out, "weights": c["weights"]} if s["accumulate"] else {"out": out}
    if kind == "step":
        n = s["batch"]
        _plain_store(c, s["k"], s["v"], torch.arange(n + 1, dtype=torch.int32, device=s["k"].device), None)
        out = _plain_attend(c, s["q"], True)
        _plain_evict(c, s["keep"], s["sink"], s["recent"])
        return dict(c, out=out)
    if kind == "store":
        c["lens"].zero_()
        c["next_pos"].zero_()
    _plain_store(c, s["k"], s["v"], s["cu"], s["token_weights"])
    if kind == "evict":
        _plain_evict(c, s["keep"], s["sink"], s["recent"])
    rows = s["k_out"].shape[2]
    live = (torch.arange(rows, device=s["k"].device)[None] < c["lens"][:, None])[:, None, :, None]
    for name in ("k", "v"):
        x = _values(c[name + "_codes"][:, :, :rows], c[name + "_scales"][:, :, :rows]).to(torch.bfloat16)
        s[name + "_out"] = torch.where(live, x, s[name + "_out"])
    return _held(s)


def _run_own(s):
    from long_context_kv_gb300 import paris

    kind = s["kind"]
    if kind == "prompt":
        paris.paris_prompt_attend(s["q"], s["k"], s["v"], s["out"], cu_q=s["cu_q"], cu_k=s["cu_k"], max_q=s["max_q"],
                                  max_k=s["max_k"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if kind == "weights":
        paris.paris_prompt_weights(s["q"], s["k"], s["lse"], s["weights"], window=s["window"], cu_q=s["cu_q"],
                                   cu_k=s["cu_k"], max_k=s["max_k"])
        return {"weights": s["weights"]}
    c, h = s["cache"], s["handle"]
    if kind == "attend":
        h.paris_kv4_attend(s["q"], s["out"], accumulate=s["accumulate"])
        return {"out": s["out"], "weights": c["weights"]} if s["accumulate"] else {"out": s["out"]}
    if kind == "step":
        h.paris_kv4_append(s["k"], s["v"])
        h.paris_kv4_attend(s["q"], s["out"], accumulate=True)
        h.paris_kv4_evict(s["keep"], s["sink"], s["recent"])
        return dict(c, out=s["out"])
    if kind == "store":
        c["lens"].zero_()
        c["next_pos"].zero_()
    h.paris_kv4_store(s["k"], s["v"], cu=s["cu"], max_new=s["max_new"], weights=s["token_weights"])
    if kind == "evict":
        h.paris_kv4_evict(s["keep"], s["sink"], s["recent"])
    h.paris_kv4_read(s["k_out"], s["v_out"])
    return _held(s)


def _held(s):
    """What the cache holds after a store or an eviction: values, weights, places."""
    c = s["cache"]
    return {"k": s["k_out"], "v": s["v_out"], "weights": c["weights"], "positions": c["positions"], "lens": c["lens"]}


# ---------------------------------------------------- the same in 64 bits


def _exact_rows(x):
    """The value a 4-bit row stands for, from the definition: x [..., D] in 64 bits."""
    x = torch.clamp(x.double(), -LIMIT, LIMIT).unflatten(-1, (D // GROUP, GROUP))
    want = x.abs().amax(-1, keepdim=True) / 7.0
    # four significant bits upwards, and no finer than 2^-17
    exponent = torch.frexp(want).exponent.long() - 1
    quantum = (1 << (exponent - 3).clamp_min(-17) + 17).double() * 2.0 ** -17
    scale = torch.ceil(want / quantum) * quantum
    c = torch.where(scale > 0, torch.round(x / scale.clamp_min(2.0 ** -30)), torch.zeros_like(x))
    return (c * scale).flatten(-2)


def _exact_held(codes, scales):
    low, high = (codes % 16).double() - 8, torch.div(codes, 16, rounding_mode="floor").double() - 8
    x = torch.empty(*codes.shape[:-1], D, dtype=torch.float64, device=codes.device)
    x[..., 0::2], x[..., 1::2] = low, high
    e, m = torch.div(scales, 8, rounding_mode="floor").double(), (scales % 8).double()
    scale = torch.where(e > 0, (8 + m) * (1 << e.long()).double() * 2.0 ** -18, m * 2.0 ** -17)
    return x * scale.repeat_interleave(GROUP, -1)


def exact(case, seed):
    s = prepare(case, seed)
    kind, hkv, dev = case["kind"], case["hkv"], "cuda"
    if kind == "prompt":
        hq, g = case["hq"], case["hq"] // hkv
        out = torch.zeros(s["q"].shape[0], hq, D, dtype=torch.float64, device=dev)
        lse = torch.zeros(hq, s["q"].shape[0], dtype=torch.float64, device=dev)
        a = b = 0
        for lq, lk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
            for h in range(hq):
                k, v = s["k"][b:b + lk, h // g].double(), s["v"][b:b + lk, h // g].double()
                for r in range(0, lq, 2048):
                    e = min(lq, r + 2048)
                    n = min(lk, e + lk - lq)
                    if n <= 0:
                        lse[h, a + r:a + e] = -math.inf
                        continue
                    sc = s["q"][a + r:a + e, h].double() @ k[:n].T / math.sqrt(D)
                    i = torch.arange(r, e, device=dev)[:, None] + (lk - lq)
                    sc[torch.arange(n, device=dev)[None] > i] = -math.inf
                    l = torch.logsumexp(sc, -1)
                    lse[h, a + r:a + e] = l
                    out[a + r:a + e, h] = torch.exp(sc - l.nan_to_num(neginf=0.0)[:, None]) @ v[:n]
            a, b = a + lq, b + lk
        return {"out": out, "lse": lse}
    if kind == "weights":
        hq, g, w = case["hq"], case["hq"] // hkv, case["window"]
        got = torch.zeros(hkv, s["k"].shape[0], dtype=torch.float64, device=dev)
        at = 0
        for n in _ints(case["lens"]):
            for h in range(hq):
                first = max(0, n - w)
                q, k = s["q"][at + first:at + n, h].double(), s["k"][at:at + n, h // g].double()
                p = torch.exp(q @ k.T / math.sqrt(D) - s["lse"][h, at + first:at + n].double()[:, None])
                got[h // g, at:at + n] += torch.tril(p, diagonal=first).sum(0)
            at += n
        return {"weights": got}
    c = s["cache"]
    k, v = (_exact_held(c[x + "_codes"].int(), c[x + "_scales"].int()) for x in ("k", "v"))
    weights, lens = c["weights"].double(), c["lens"].tolist()
    places, nxt = c["positions"].long(), c["next_pos"].tolist()
    if kind in ("store", "evict", "step"):
        sizes = _ints(case["lens"]) if kind == "store" else [case["chunk"] if kind == "evict" else 1] * case["batch"]
        lens = [0] * len(lens) if kind == "store" else lens
        at = 0
        for b, n in enumerate(sizes):
            a, e = lens[b], lens[b] + n
            k[b, :, a:e] = _exact_rows(s["k"][at:at + n]).transpose(0, 1)
            v[b, :, a:e] = _exact_rows(s["v"][at:at + n]).transpose(0, 1)
            weights[b, :, a:e] = s["token_weights"][:, at:at + n].double() if "token_weights" in s else 0.0
            places[b, :, a:e] = nxt[b] + torch.arange(n, device=dev)
            lens[b], nxt[b], at = e, nxt[b] + n, at + n
    out = None
    if kind in ("attend", "step"):
        g = case["hq"] // hkv
        out = torch.zeros(len(lens), case["hq"], D, dtype=torch.float64, device=dev)
        add = kind == "step" or case["accumulate"]
        for b, n in enumerate(lens):
            for h in range(hkv):
                p = torch.softmax(s["q"][b, h * g:(h + 1) * g].double() @ k[b, h, :n].T / math.sqrt(D), -1)
                out[b, h * g:(h + 1) * g] = p @ v[b, h, :n]
                if add:
                    weights[b, h, :n] += p.sum(0)
    if kind in ("evict", "step"):
        keep = case["keep"]
        for b, n in enumerate(lens):
            for h in range(hkv):
                p, w = places[b, h, :n].tolist(), weights[b, h, :n].tolist()
                safe = lambda i: p[i] < case["sink"] or p[i] >= nxt[b] - case["recent"]  # noqa: E731, B023
                kept = set(sorted(range(n), key=lambda i: (not safe(i), -w[i], i))[:keep])  # noqa: B023
                to = [i for i in range(keep) if i not in kept]
                of = sorted(i for i in kept if i >= keep)
                for x in (k, v, weights):
                    x[b, h, to] = x[b, h, of]
    if kind == "attend":
        return {"out": out, "weights": weights} if case["accumulate"] else {"out": out}
    if kind == "step":
        return {"out": out, "weights": weights}
    rows = s["k_out"].shape[2]
    return {"k": k[:, :, :rows], "v": v[:, :, :rows], "weights": weights}
