"""The paged cache's calls in the ways in which programs make them: captured, on threads, with limits, with arrays that
do not agree, with values that are not finite.  Against the direct call, lists, or the definition in 64 bits."""
import math
import os
import subprocess
import sys
import threading

import pytest
import torch

from long_context_kv_gb300 import paris as P
from tests import kv4_ref as K4
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
BF, E4 = torch.bfloat16, torch.float8_e4m3fn
i32 = lambda v: torch.tensor(list(v), dtype=torch.int32, device="cuda")  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_kv_gb300 import build
    build.build()
    P.load()


def rand(*s, seed=0):
    return torch.randn(*s, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def filled(lens, hkv, page=16, dtype=BF, seed=0, spare=4, kv=None, max_pages=None):
    """A cache with rows; kv: packed rows (k, v)."""
    held = [-(-n // page) for n in lens]
    c = P.PagedCache.create(len(lens), hkv, sum(held) + spare, max_pages or max(max(held), 1), page_rows=page, dtype=dtype)
    k, v = kv or (rand(sum(lens), hkv, R.D, seed=seed).to(BF), rand(sum(lens), hkv, R.D, seed=seed + 1).to(BF))
    c.paris_paged_grow(i32(lens))
    c.paris_paged_store(k, v, cu=K4.starts(lens), max_new=max(lens))
    c.paris_paged_check()
    return c


# Heads, sequences and rooms whose workspace is at most a megabyte although sequences are split into several units.
SMALL = [(8, 8, [3000]), (8, 8, [3000, 17, 2999, 1, 1024, 500, 2048, 1777]), (8, 2, [2048]), (32, 8, [512]), (4, 1, [4096])]


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("hq,hkv,lens", SMALL)
def test_captured_attention_is_the_direct_call_s(hq, hkv, lens, dtype):
    c = filled(lens, hkv, dtype=dtype, seed=1)
    q = (2 * rand(2, len(lens), hq, R.D, seed=2)).to(BF)
    want = torch.zeros_like(q), torch.zeros(2, len(lens), hq, device="cuda")
    outs, lses = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    for i in range(2):
        c.paris_paged_attend(q[i], want[0][i], lse=want[1][i])
    assert 0 < c._ws[hq][0] <= 1 << 20
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for i in range(2):
            c.paris_paged_attend(q[i], outs[i], lse=lses[i])
    for _ in range(3):
        outs.fill_(9.0)
        lses.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs, want[0]) and torch.equal(lses, want[1])
    c.paris_paged_check()


@pytest.mark.parametrize("dtype", [BF, E4])
def test_threads_that_attend_on_one_stream(dtype):
    c = filled([5000, 1, 900], 2, dtype=dtype, seed=3)
    q = (2 * rand(4, 3, 8, R.D, seed=4)).to(BF)
    want, outs = torch.zeros_like(q), torch.zeros(4, 50, 3, 8, R.D, dtype=BF, device="cuda")
    for i in range(4):
        c.paris_paged_attend(q[i], want[i])
    c = P.PagedCache(c.k_pages, c.v_pages, c.table, c.lens, c.starts, c.refs, c.free_bits, c.n_used,
                     *((c.k_scales, c.v_scales) if dtype is E4 else ()))  # without what calls keep
    errors, start = [], threading.Barrier(4)

    def work(i):
        try:
            start.wait()
            for n in range(50):
                c.paris_paged_attend(q[i], outs[i, n])
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(4):
        assert torch.all(outs[i] == want[i])
    c.paris_paged_check()


def state(c):
    return {n: getattr(c, n).tolist() for n in ("table", "lens", "starts", "refs", "n_used")}


# The pages that are free (by free_bits), and what n_used claims: as many as are wanted.
@pytest.mark.parametrize("free", [0, 1, 2])
@pytest.mark.parametrize("stray", [False, True])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_a_fork_with_fewer_free_pages_than_n_used_says(dtype, stray, free):
    """Entries that get no page keep their full ones, in the small fork and the large one, and no row is written
    outside of the pages that were found."""
    made = []
    for max_pages in (4, 4096):  # one block; a kernel a step
        lens = [20, 33, 5, 0, 0]
        c = filled(lens, 2, dtype=dtype, seed=5, spare=free, max_pages=max_pages)
        guard = [torch.cat([R.raw(t)[:, :1], R.raw(t), R.raw(t)[:, :1]], 1).fill_(77) for t in (c.k_pages, c.v_pages)]
        pools = [g[:, 1:-1].view(t.dtype) for g, t in zip(guard, (c.k_pages, c.v_pages))]
        for pool, t in zip(pools, (c.k_pages, c.v_pages)):
            R.raw(pool).copy_(R.raw(t))
        if stray:
            c.free_bits[-1] |= -1 << (c.n_pages % 32)
        n_used = int(c.n_used)
        c = P.PagedCache(*pools, c.table, c.lens, c.starts, c.refs, c.free_bits, c.n_used - 4,
                         *((c.k_scales, c.v_scales) if dtype is E4 else ()))
        bytes_before = [g.clone() for g in guard]
        c.paris_paged_fork(i32([0, 1, 2]), i32([3, 4, 0]))
        got = [3, 4, 0][:free]
        with pytest.raises(P.ParisError, match="no room"):
            c.paris_paged_check()
        want = {3: 20, 4: 33, 0: 5}
        assert c.lens.tolist() == [want[s] if s in got else want[s] // 16 * 16 if s in want else lens[s] for s in range(5)]
        assert c.starts.tolist() == [c.lens[s].item() if s in want else 0 for s in range(5)]
        # what the first sequence held of its own is given back
        assert int(c.n_used) == n_used - 4 + len(got) - 1
        held = [p for s, n in enumerate(c.lens.tolist()) for p in c.table[s, :-(-n // 16)].tolist()]
        assert c.refs.tolist() == [held.count(p) for p in range(c.n_pages)]
        new = [int(c.table[s, want[s] // 16]) for s in got]
        for g, b in zip(guard, bytes_before):
            same = torch.ones(g.shape[1], dtype=torch.bool, device="cuda")
            same[[p + 1 for p in new]] = False
            assert torch.equal(g[:, same], b[:, same])
        made.append({n: [x[:4] for x in v] if n == "table" else v for n, v in state(c).items()})
    assert made[0] == made[1]


def test_growing_with_fewer_free_pages_than_n_used_says():
    for stray in (False, True):
        c = filled([20, 33, 5], 1, seed=6, spare=3, max_pages=40)
        if stray:
            c.free_bits[-1] |= -1 << (c.n_pages % 32)
        c.n_used -= 5
        c.paris_paged_grow(i32([13, 100, 1]))  # one page, six pages, none
        with pytest.raises(P.ParisError, match="no room"):
            c.paris_paged_check()
        assert c.lens.tolist() == [33, 80, 6] and c.starts.tolist() == [20, 33, 5]
        assert int(c.n_used) == c.n_pages - 5 and not torch.any(pages_free(c))
        assert sorted(p for s, n in enumerate((3, 5, 1)) for p in c.table[s, :n].tolist()) == list(range(c.n_pages))


@pytest.mark.parametrize("off", [-6, -1, 0, 2, 1000])
@pytest.mark.parametrize("lens", [[20, 33, 5, 64, 0, 100], [500, 20000, 9000, 20000]])
def test_closing_up_goes_by_free_bits(lens, off):
    """A wrong n_used costs no sequence a page; the right one is there afterwards."""
    c = filled(lens, 1, seed=9, spare=40)
    c.paris_paged_free(i32([0, 2]))
    b = R.Book(c)
    if c.n_pages % 32:
        c.free_bits[-1] |= -1 << c.n_pages % 32
    c.n_used += off
    c.paris_paged_compact()
    b.compact()
    b.check()
    c.paris_paged_check()


def pages_free(c):
    at = torch.arange(c.n_pages, device="cuda")
    return c.free_bits[at // 32] >> at % 32 & 1


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("limit", [0, 1, 7, 16, 37, 1000, 1 << 40])
def test_limits_hold_for_batches_as_for_packed_rows(limit, dtype):
    T, grown = 37, [37, 5, 0]
    k, v = (rand(3, 2, T, R.D, seed=7 + i).to(BF) for i in range(2))
    fresh = lambda: P.PagedCache.create(3, 2, 12, 4, dtype=dtype)  # noqa: E731
    c, want = fresh(), fresh()
    for x in (c, want):
        x.paris_paged_grow(i32(grown))
    c.paris_paged_store(k, v, max_new=limit)
    rows = [x.transpose(1, 2).reshape(3 * T, 2, R.D) for x in (k, v)]
    want.paris_paged_store(*rows, cu=i32([0, T, 2 * T, 3 * T]), max_new=limit)
    for name in ("k_pages", "v_pages"):
        assert torch.equal(R.raw(getattr(c, name)), R.raw(getattr(want, name)))
    for s, n in enumerate(grown):
        assert torch.all(R.rows_of(c, "k", 0, s)[:, min(n, limit):] == 0)
        if dtype is BF:
            assert torch.equal(R.rows_of(c, "k", 0, s)[:, :min(n, limit)], k[s, :, :min(n, limit)].double())
    c.paris_paged_store(k, v)
    out = torch.full((2, 3, 2, T, R.D), 6.0, dtype=BF, device="cuda")
    c.paris_paged_read(*out, max_rows=limit)
    for i, name in enumerate(("k", "v")):
        for s, n in enumerate(grown):
            n = min(n, limit)
            assert torch.all(out[i, s, :, n:] == 6.0)
            assert torch.equal(out[i, s, :, :n].double(), R.rows_of(c, name, 0, s)[:, :n])


@pytest.mark.parametrize("dtype", [BF, E4])
def test_packed_rows_of_many_sequences_without_a_better_limit(dtype):
    """The most rows that a call can name, for 4096 sequences: what it does goes by the starts."""
    n, hkv, page = 4096, 2, 256
    c = P.PagedCache.create(n, hkv, 200, 1 << 15, page_rows=page, dtype=dtype)
    lens = [0] * n
    lens[0], lens[70], lens[4000], lens[4095] = 20000, 3, 9000, 8193
    c.paris_paged_grow(i32(lens))
    total = sum(lens)
    k, v = (rand(total, hkv, R.D, seed=8 + i).to(BF) for i in range(2))
    cu, st, ref = K4.starts(lens), P._STRIDES.pack(hkv * R.D, R.D, 0), c._ref
    out = torch.full((2, total, hkv, R.D), 6.0, dtype=BF, device="cuda")
    most, lib, stream = (1 << 31) - 1, P.load(), torch.cuda.current_stream().cuda_stream
    for limit in (most, 1 << 40):
        P._check(lib.paris_paged_store(ref, 0, k.data_ptr(), v.data_ptr(), P.PARIS_BF16, st, st, most, cu.data_ptr(), limit, stream))
        P._check(lib.paris_paged_read(ref, 0, out[0].data_ptr(), out[1].data_ptr(), st, st, most, cu.data_ptr(), limit, stream))
    c.paris_paged_check()
    at = 0
    for s in (0, 70, 4000, 4095):
        for i, (name, x) in enumerate((("k", k), ("v", v))):
            rows = x[at:at + lens[s]]
            if dtype is E4:
                codes, byte = R.quantise(rows)
                rows = codes * R.powers("cuda")[byte.long()][..., None]
            assert torch.equal(R.rows_of(c, name, 0, s).transpose(0, 1), rows.double())
            assert torch.equal(out[i, at:at + lens[s]].double(), rows.double())
        at += lens[s]


# Query heads, KV heads and lengths: sequences of one unit; split ones of few heads (joined by parts of the channels, an
# eighth and a quarter each), and of many, with others of one unit beside them.
PATHS = [(1, 1, [40]), (8, 2, [200, 1, 64]), (16, 1, [333]), (40, 2, [130, 90]), (4, 1, [3000]), (8, 1, [5000, 45, 0, 90]),
         (128, 1, [2000]), (64, 2, [3000, 100, 2500]), (48, 16, [1500, 0, 1800, 60, 41]), (6, 3, [50 + i for i in range(60)])]


def definition(c, q, b, window, at=None):
    """Results of sequence b in 64 bits, what its terms add up to without their signs, and its bound of a score's error."""
    n, hkv = int(c.lens[b]), c.n_kv_heads
    first = max(0, n - window) if window else 0
    g = q.shape[1] // hkv
    ks, vs = (R.rows_of(c, name, 0, b)[:, first:] for name in ("k", "v"))
    if at is not None:
        ks, vs = ks[:, at], vs[:, at]
    qs = q[b].double().reshape(hkv, g, R.D)
    p = torch.softmax(qs @ ks.transpose(1, 2) / math.sqrt(R.D), -1)
    size = (qs.abs() @ ks.abs().transpose(1, 2)).amax(-1)
    return [x.reshape(-1, R.D) for x in (p @ vs, p @ vs.abs())], R.score_error(size, n).reshape(-1, 1)


def close(got, want, mass, e):
    """Infinities and NaN are the definition's; the rest as close as weights of two bf16 parts, scores and the
    rounding of the result make it."""
    got, fin = got.double(), torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[torch.isinf(want)], want[torch.isinf(want)])
    tol = R.HALF_BF16 * want.abs() + (1 + R.HALF_BF16) * (e + 2.0 ** -16) * mass
    assert torch.all((got - want).abs()[fin] <= tol[fin])


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("hq,hkv,lens", PATHS)
def test_values_that_are_not_finite(hq, hkv, lens, window):
    k, v = (rand(sum(lens), hkv, R.D, seed=20 + i).to(BF) for i in range(2))
    at = 0
    for n in lens:
        if n >= 40:  # within the window, but for one
            v[at + n - 3, 0, 5] = math.inf
            v[at + n - 33, -1, 6] = -math.inf
            v[at + n - 20, :, 9], v[at + n - 10, :, 9] = math.inf, -math.inf
            v[at + n - 39, 0, 127] = math.nan
        if n >= 90:
            v[at + n - 80, :, 40:44] = math.inf
        at += n
    c = filled(lens, hkv, seed=0, kv=(k, v))
    q = (2 * rand(len(lens), hq, R.D, seed=22)).to(BF)
    out, lse = torch.full_like(q, 9.0), torch.full((len(lens), hq), 9.0, device="cuda")
    c.paris_paged_attend(q, out, window=window, lse=lse)
    clean = filled(lens, hkv, kv=(k, v.nan_to_num(0.0, 0.0, 0.0)))
    out2, lse2 = torch.full_like(q, 9.0), torch.full_like(lse, 9.0)
    clean.paris_paged_attend(q, out2, window=window, lse=lse2)
    assert torch.equal(lse, lse2)
    for b, n in enumerate(lens):
        if n == 0:
            assert torch.all(out[b] == 0)
            continue
        (want, mass), e = definition(c, q, b, window)
        close(out[b], want, mass, e)
        if n >= 40:
            assert torch.isinf(want).any() and torch.isnan(want).any()
    again = torch.full_like(q, 9.0)
    c.paris_paged_attend(q, again, window=window)
    assert torch.equal(again.nan_to_num(7.0), out.nan_to_num(7.0))
    queue, _, rows, blocks = next(iter(c._spaces.values()))[:16].view(torch.int32).tolist()
    assert queue == rows == blocks == 0  # kept for the next call
    c.paris_paged_check()


@pytest.mark.parametrize("hq,hkv,lens", PATHS)
def test_large_values_leave_their_mean(hq, hkv, lens):
    """Sums past float32's range on the way to means within it."""
    v = (3e38 * (1 + 0.1 * rand(sum(lens), hkv, R.D, seed=30).clamp(-1, 1))).to(BF)
    v[:, :, 64:] = -v[:, :, 64:]
    v[:, :, ::7] = rand(sum(lens), hkv, 19, seed=31).to(BF)
    c = filled(lens, hkv, kv=(rand(sum(lens), hkv, R.D, seed=32).to(BF), v))
    q = (2 * rand(len(lens), hq, R.D, seed=33)).to(BF)
    out = torch.full_like(q, 9.0)
    c.paris_paged_attend(q, out)
    for b, n in enumerate(lens):
        if n > 0:
            (want, mass), e = definition(c, q, b, 0)
            assert torch.isfinite(out[b]).all()
            close(out[b], want, mass, e)


@pytest.mark.parametrize("hq,hkv,lens", PATHS)
def test_rows_without_weight_add_nothing_whatever_they_hold(hq, hkv, lens):
    """Scores 256 below the others are weights of 2^-369: none, in float32."""
    k, v = (rand(sum(lens), hkv, R.D, seed=40 + i) for i in range(2))
    k[:, :, 0] = 0
    q = rand(len(lens), hq, R.D, seed=42)
    q[:, :, 0] = 256.0
    light = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
    light[::3] = True
    light[torch.tensor([sum(lens[:i]) for i, n in enumerate(lens) if n > 0], device="cuda")] = False
    k[light, :, 0] = -256 * math.sqrt(R.D) / 256.0 - 4.0
    v[light, :, ::2] = math.inf
    v[light, :, 1::4] = math.nan
    c = filled(lens, hkv, kv=(k.to(BF), v.to(BF)))
    out = torch.full((len(lens), hq, R.D), 9.0, dtype=BF, device="cuda")
    c.paris_paged_attend(q.to(BF), out)
    at = 0
    for b, n in enumerate(lens):
        if n > 0:
            (want, mass), e = definition(c, q.to(BF), b, 0, at=(~light[at:at + n]).nonzero()[:, 0])
            close(out[b], want, mass, e)
        at += n


@pytest.mark.parametrize("max_pages", [4, 4096])
@pytest.mark.parametrize("spare", [0, 1, 5])
def test_a_fork_takes_no_page_that_it_gives_back(spare, max_pages):
    """New pages are those that were free before the call, though it frees pages of lower numbers."""
    lens = [20, 40, 30, 10, 50]
    c = filled(lens, 1, seed=50, spare=spare, max_pages=max_pages)
    refs, own = c.refs.tolist(), [c.table[s, :-(-n // 16)].tolist() for s, n in enumerate(lens)]
    c.paris_paged_fork(i32([4, 4, 4]), i32([0, 1, 2]))  # pages 0 to 6 are given back, three pages are asked for
    got = min(spare, 3)
    assert c.lens.tolist() == [50 if s < got else 48 for s in range(3)] + lens[3:]
    new = [int(c.table[s, 3]) for s in range(got)]
    assert all(refs[p] == 0 for p in new) and new == sorted(p for p, r in enumerate(refs) if r == 0)[:got]
    assert all(int(c.refs[p]) == 0 for s in range(3) for p in own[s])
    for s in range(3):
        assert c.table[s, :3].tolist() == own[4][:3]
        n = int(c.lens[s])
        assert torch.equal(R.rows_of(c, "v", 0, s, n), R.rows_of(c, "v", 0, 4, n))
    c.paris_paged_grow(i32([0, 0, 0, 32, 0]))  # and now they are free
    assert c.table[3, 1:3].tolist() == [0, 1]


@pytest.mark.parametrize("dtype", [BF, E4])
def test_two_branches_of_one_graph_attend_at_once(dtype):
    """Layers' attention side by side: each branch's calls have workspaces of its own."""
    c = filled([3000, 700], 8, dtype=dtype, seed=60)
    q = (2 * rand(2, 4, 2, 8, R.D, seed=61)).to(BF)
    want, outs = torch.zeros_like(q), torch.zeros_like(q)
    for i in range(2):
        for n in range(4):
            c.paris_paged_attend(q[i, n], want[i, n])
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        for n in range(4):
            c.paris_paged_attend(q[0, n], outs[0, n])
            c.paris_paged_attend(q[1, n], outs[1, n], stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for _ in range(20):
        outs.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs, want)
    c.paris_paged_check()


@pytest.mark.parametrize("hq,hkv,lens", PATHS)
def test_captured_attention_over_values_that_are_not_finite(hq, hkv, lens):
    """What is computed again is found anew by each replay, and forgotten."""
    k, v = (rand(sum(lens), hkv, R.D, seed=70 + i).to(BF) for i in range(2))
    c = filled(lens, hkv, kv=(k, v))
    q = (2 * rand(len(lens), hq, R.D, seed=72)).to(BF)
    out, graph = torch.zeros_like(q), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.paris_paged_attend(q, out)
    for bad in (False, True, False, True):
        x = v.clone()
        if bad:
            for at in (sum(lens[:i]) for i, n in enumerate(lens) if n > 0):
                x[at, :, 3], x[at, :, 100] = math.inf, -math.inf
        c.starts.zero_()
        c.paris_paged_store(k, x, cu=K4.starts(lens), max_new=max(lens))
        want = torch.zeros_like(q)
        c.paris_paged_attend(q, want)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        used = [b for b, n in enumerate(lens) if n > 0]
        for channel, value in ((3, math.inf), (100, -math.inf)):
            assert torch.all((out[used][..., channel] == value) == bad)
        assert torch.isfinite(out[..., 4:100]).all()
    c.paris_paged_check()


FIRST = """
import torch
from long_context_kv_gb300 import paris as P
P.load()
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
for dtype in (torch.bfloat16, torch.float8_e4m3fn):
    for n in (100, 4000):  # one unit a sequence, several
        c = P.PagedCache.create(2, 2, 300, n // 16 + 2, dtype=dtype)
        k = torch.randn(2, 2, n, 128, device="cuda").to(torch.bfloat16)
        q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
        ko, vo, out, tokens, src, dst = torch.zeros_like(k), torch.zeros_like(k), torch.zeros_like(q), i32(n, 3), i32(0), i32(1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.paris_paged_grow(tokens)
            c.paris_paged_store(k, k)
            c.paris_paged_attend(q, out)
            c.paris_paged_read(ko, vo)
            c.paris_paged_fork(src, dst)
            c.paris_paged_free(src)
            c.paris_paged_compact()
        graph.replay()
        c.paris_paged_check()
        assert c.lens.tolist() == [0, n] and (dtype is not torch.bfloat16 or torch.equal(ko[0], k[0]))
        s = ko[0].repeat_interleave(4, 0).double() @ q[0].double()[:, :, None] / 128 ** 0.5
        o = (torch.softmax(s, 1) * vo[0].repeat_interleave(4, 0).double()).sum(1)
        assert (o - out[0].double()).abs().max() < 2.0 ** -6
"""


def test_first_calls_of_a_process_may_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
