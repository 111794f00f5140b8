"""The paged cache (paris_paged_*): its bookkeeping entry for entry against lists, stored rows bit for bit against the
64-bit definition, attention against 64-bit forms over the rows' exact values, and all of them together."""
import math
import random

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


def rand(*s, seed=0, amp=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return amp * torch.randn(*s, generator=gen, device="cuda")


def empty(n_seqs, hkv, n_pages, max_pages, page=16, layers=1, dtype=BF, order="hrd", garbage=True):
    """An empty cache; order "rhd": a page's rows outside its heads; garbage: NaN in rows and scales not in use."""
    c = P.PagedCache.create(n_seqs, hkv, n_pages, max_pages, page_rows=page, n_layers=layers, dtype=dtype)
    kw = {n: getattr(c, n) for n in ("table", "lens", "starts", "refs", "free_bits", "n_used")}
    if dtype is E4:
        kw.update(k_scales=c.k_scales, v_scales=c.v_scales)
    pages = {}
    for name in ("k_pages", "v_pages"):
        t = getattr(c, name)
        if order == "rhd":
            t = t.view(torch.uint8) if dtype is E4 else t
            t = t.transpose(2, 3).contiguous().transpose(2, 3)
            t = t.view(E4) if dtype is E4 else t
        pages[name] = t
    if garbage:
        for t in pages.values():
            R.raw(t).fill_(255 if dtype is E4 else 0x7FFF)
        if dtype is E4:
            c.k_scales.fill_(255)
            c.v_scales.fill_(255)
        c.table.fill_(-7)
    return P.PagedCache(**pages, **kw)


def filled(lens, hkv, page=16, dtype=BF, seed=0, layers=1, order="hrd", spare=8, kv=None, extra=0):
    """A cache whose sequences have rows, in pages of no order; kv: packed rows (k, v)."""
    need = sum(-(-n // page) for n in lens)
    c = empty(len(lens), hkv, need + spare, max(max(-(-n // page) for n in lens), 1) + extra, page, layers, dtype, order)
    total = sum(lens)
    k, v = kv if kv is not None else (rand(total, hkv, R.D, seed=seed).to(BF), rand(total, hkv, R.D, seed=seed + 1).to(BF))
    parts = [max(1, n // 2) if n > 1 else n for n in lens]
    at = 0
    for sizes in (parts, [n - p for n, p in zip(lens, parts)]):  # in two growths, so that the pages are mixed up
        c.paris_paged_grow(i32(sizes))
        rows = []
        at = 0
        for n, p in zip(lens, parts):
            rows.append(range(at, at + p) if sizes is parts else range(at + p, at + n))
            at += n
        pick = torch.tensor([r for x in rows for r in x], device="cuda", dtype=torch.long)
        if len(pick):
            for layer in range(layers):
                c.paris_paged_store(k[pick], v[pick], cu=K4.starts(sizes), max_new=max(sizes), layer=layer)
    c.paris_paged_check()
    return c, k, v


# ------------------------------------------------------------------ rows
def edge_rows(dtype):
    x = rand(60, 2, R.D, seed=1)
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 1e-4
    x[3] *= 1e5
    x[4] *= 1e17
    x[5, :, 3] = math.nan
    x[6, :, 40] = math.inf
    x[7, :, 41] = -math.inf
    x[8] = 448.0 * torch.sign(x[8])
    x[9] = 449.0 * torch.sign(x[9])
    x[10, :, 0] = 448.0
    x[10, :, 1:] = torch.arange(127, device="cuda") * 2.0 ** -10  # ties, subnormal codes among them
    x[11, :, 0] = 3.0e38
    x[12] = 2.0 ** -130
    x[13, :, 0] = 1.75
    x[14, :, 0] = 1.7578125
    x[15] = torch.round(x[15] * 16) / 16
    return x.to(dtype)


@pytest.mark.parametrize("order", ["hrd", "rhd"])
@pytest.mark.parametrize("src", [BF, torch.float32])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_stored_rows_are_the_definition_bit_for_bit(dtype, src, order):
    x, y = edge_rows(src), rand(60, 2, R.D, seed=2).to(src)
    c = empty(3, 2, 9, 5, dtype=dtype, order=order)
    lens = [33, 0, 27]
    c.paris_paged_grow(i32(lens))
    c.paris_paged_store(x, y, cu=K4.starts(lens))
    ko, vo = (torch.full((60, 2, R.D), 5.0, dtype=BF, device="cuda") for _ in range(2))
    c.paris_paged_read(ko, vo, cu=K4.starts(lens))
    at = 0
    for s, n in enumerate(lens):
        for name, src_rows, out in (("k", x, ko), ("v", y, vo)):
            rows = src_rows[at:at + n]
            if dtype is BF:
                want = rows.to(BF).double()
            else:
                codes, byte = R.quantise(rows)
                want = codes * R.powers("cuda")[byte.long()][..., None]
            got = R.rows_of(c, name, 0, s).transpose(0, 1)
            assert torch.equal(got.nan_to_num(nan=7.5), want.nan_to_num(nan=7.5))
            assert torch.equal(out[at:at + n].double().nan_to_num(nan=7.5), want.nan_to_num(nan=7.5))
        at += n
    c.paris_paged_check()
    # what no sequence holds is as it was
    held = torch.zeros(9, 16, dtype=torch.bool, device="cuda")
    for s, n in enumerate(lens):
        for r in range(n):
            held[c.table[s, r // 16], r % 16] = True
    for t in (c.k_pages, c.v_pages):
        rest = R.raw(t)[0].transpose(1, 2)[~held]
        assert torch.all(rest == (255 if dtype is E4 else 0x7FFF))


@pytest.mark.parametrize("dtype", [BF, E4])
def test_rows_of_strided_tensors_and_batches(dtype):
    n, hkv, T = 3, 3, 37
    big = rand(n, T, hkv + 2, 3, R.D, seed=3).to(BF)
    k, v = big[:, :, 1:1 + hkv, 0].transpose(1, 2), big[:, :, 2:2 + hkv, 2].transpose(1, 2)  # [n, H, T, d]
    c = empty(n, hkv, 12, 4, dtype=dtype)
    c.paris_paged_grow(i32([T, 5, 0]))
    c.paris_paged_store(k, v)
    back = torch.full((n, T, 2 * hkv, R.D), 3.0, dtype=BF, device="cuda")
    ko, vo = back[:, :, :hkv].transpose(1, 2), back[:, :, hkv:].transpose(1, 2)
    c.paris_paged_read(ko, vo)
    for s, m in enumerate((T, 5, 0)):
        for src, out, name in ((k, ko, "k"), (v, vo, "v")):
            want = src[s, :, :m].double()
            if dtype is E4:
                codes, byte = R.quantise(want)
                want = codes * R.powers("cuda")[byte.long()][..., None]
            assert torch.equal(out[s, :, :m].double(), want) and torch.equal(R.rows_of(c, name, 0, s), want)
            assert torch.all(out[s, :, m:] == 3.0)


def test_starts_that_leave_rows_out_or_lie_outside():
    c = empty(3, 2, 12, 4)
    x = rand(50, 2, R.D, seed=5).to(BF)
    c.paris_paged_grow(i32([20, 7, 16]))
    cu = i32([3, 23, 30, 46])  # three rows in front and four behind are nobody's
    c.paris_paged_store(x, x, cu=cu, max_new=20)
    out = torch.full((50, 2, R.D), 4.0, dtype=BF, device="cuda")
    c.paris_paged_read(out, out.clone(), cu=cu)
    assert torch.all(out[:3] == 4.0) and torch.all(out[46:] == 4.0) and torch.equal(out[3:46], x[3:46])
    # a start past the rows counts as their end, one before the start in front as that
    before = R.raw(c.k_pages).clone()
    c.paris_paged_store(x, x, cu=i32([60, 70, 10, -5]))
    assert torch.equal(R.raw(c.k_pages), before)
    c.paris_paged_store(-x, -x, cu=i32([-9, 4, 2, 1000]), max_new=50)
    assert torch.equal(R.rows_of(c, "k", 0, 0)[:, :4].transpose(0, 1), -x[:4].double())
    assert torch.equal(R.rows_of(c, "k", 0, 0)[:, 4:].transpose(0, 1), x[7:23].double())
    assert torch.equal(R.rows_of(c, "k", 0, 1).transpose(0, 1), x[23:30].double())
    assert torch.equal(R.rows_of(c, "v", 0, 2).transpose(0, 1), -x[2:18].double())


def test_a_store_writes_the_last_growth_only():
    c = empty(2, 1, 8, 4)
    x = rand(40, 1, R.D, seed=4).to(BF)
    c.paris_paged_grow(i32([20, 3]))
    c.paris_paged_store(x[:23], x[:23], cu=K4.starts([20, 3]))
    c.paris_paged_grow(i32([0, 30]))
    c.paris_paged_store(x[:10], x[:10], cu=K4.starts([5, 5]))  # the first has not grown, the second by more
    assert torch.equal(R.rows_of(c, "k", 0, 0)[0], x[:20, 0].double())
    assert torch.equal(R.rows_of(c, "k", 0, 1)[0, :8], torch.cat([x[20:23, 0], x[5:10, 0]]).double())
    assert torch.isnan(R.rows_of(c, "k", 0, 1)[0, 8:]).all()
    c.paris_paged_store(x[:9], x[:9], cu=K4.starts([0, 9]), max_new=7)
    assert torch.equal(R.rows_of(c, "v", 0, 1)[0, 3:10], x[:7, 0].double())
    assert torch.isnan(R.rows_of(c, "v", 0, 1)[0, 10:]).all()


# ----------------------------------------------------------- bookkeeping
def test_growing_takes_the_lowest_free_pages_in_order():
    c = empty(5, 1, 70, 6)
    b = R.Book(c)
    for tokens in ([1, 0, 17, -4, 40], [15, 16, 0, 1, 8], [1, 1, 1, 1, 1], [96, 0, 0, 0, 0], [0, 0, 0, 0, 500]):
        c.paris_paged_grow(i32(tokens))
        b.grow(tokens)
        b.check()
    assert b.short
    with pytest.raises(P.ParisError, match="no room"):
        c.paris_paged_check()
    c.paris_paged_check()  # cleared


@pytest.mark.parametrize("n_pages", [1, 31, 33, 40000])
def test_growing_past_the_pool(n_pages):
    c = empty(3, 1, n_pages, 20000)
    b = R.Book(c)
    for tokens in ([5, 3, 2], [16 * n_pages // 2, 16 * n_pages // 2, 100], [1 << 30, 1, 1 << 30]):
        c.paris_paged_grow(i32(tokens))
        if n_pages < 100:
            b.grow(tokens)
            b.check()
    assert int(c.n_used) == n_pages and int((c.refs == 1).sum()) == n_pages and not c.free_bits.any()
    held = torch.cat([c.table[s, :-(-int(c.lens[s]) // 16)] for s in range(3)])
    assert torch.equal(held.sort().values, torch.arange(n_pages, dtype=torch.int32, device="cuda"))
    with pytest.raises(P.ParisError):
        c.paris_paged_check()


@pytest.mark.parametrize("n", [1500, 4096])
def test_many_sequences(n):
    c = empty(n, 1, n + 500, 3)
    b = R.Book(c)
    gen = random.Random(5)
    for step in range(2):
        tokens = [gen.choice([0, 0, 1, 3, 16]) for _ in range(n)]
        c.paris_paged_grow(i32(tokens))
        free = b.free_pages()  # the lists' own walk is quadratic
        for s, t in enumerate(tokens):
            b.starts[s] = b.lens[s]
            for j in range(b.pages(b.lens[s]), b.pages(b.lens[s] + t)):
                b.table[s][j] = free.pop(0)
                b.refs[b.table[s][j]] = 1
            b.lens[s] += t
        b.check(pools=False)
    src = [gen.randrange(n) for _ in range(n)]
    dst = [gen.randrange(n) for _ in range(n)]
    c.paris_paged_fork(i32(src), i32(dst))
    b.fork(src, dst)
    b.check()
    c.paris_paged_free(i32(range(0, n, 2)))
    b.free(list(range(0, n, 2)))
    c.paris_paged_compact()
    b.compact()
    b.check()


FORKS = {
    "samples": ([0, 0, 0], [3, 4, 5], None),
    "rotate": ([1, 2, 3, 0], [0, 1, 2, 3], None),
    "onto itself": ([0, 1, 2, 3, 4, 5], [0, 1, 2, 3, 4, 5], None),
    "prefixes": ([0, 0, 2, 2, 1], [1, 2, 3, 0, 4], [16, 33, 0, 15, 48]),
    "cut": ([0, 1, 2], [0, 1, 2], [20, 1000, 0]),
    "twice the same": ([0, 1, 2, 3], [4, 4, 4, 5], None),
    "out of range": ([-1, 6, 0, 0, 2], [0, 1, 6, -3, 5], None),
    "cut beside a fork": ([1, 1], [1, 3], [20, 48]),
    "negative rows": ([0, 1], [0, 4], [-5, -1]),
}


@pytest.mark.parametrize("dtype,layers,page,order", [(BF, 1, 16, "hrd"), (BF, 3, 32, "rhd"), (E4, 2, 16, "hrd"), (E4, 1, 64, "rhd")])
@pytest.mark.parametrize("name", FORKS)
def test_forks(name, dtype, layers, page, order):
    src, dst, rows = FORKS[name]
    c, _, _ = filled([50, 64, 17, 1, 0, 130], 2, page, dtype, seed=10, layers=layers, order=order, extra=2)
    b = R.Book(c)
    for _ in range(3):
        c.paris_paged_fork(i32(src), i32(dst), None if rows is None else i32(rows))
        b.fork(src, dst, rows)
        b.check()
    assert not b.short
    if b.wrong:
        with pytest.raises(P.ParisError, match="out of range"):
            c.paris_paged_check()
    c.paris_paged_check()


@pytest.mark.parametrize("spare", [0, 1, 2])
def test_forks_without_room_keep_their_full_pages(spare):
    c, _, _ = filled([50, 64, 17, 0, 0, 0], 2, seed=11, spare=spare)
    b = R.Book(c)
    c.paris_paged_fork(i32([0, 2, 1, 0]), i32([3, 4, 5, 2]))
    b.fork([0, 2, 1, 0], [3, 4, 5, 2])
    b.check()
    assert b.short
    with pytest.raises(P.ParisError, match="no room"):
        c.paris_paged_check()


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("seed", range(6))
def test_long_runs_of_forks_growths_ends_and_closings(seed, dtype):
    gen = random.Random(seed)
    page = gen.choice([16, 32, 128])
    n = gen.choice([1, 4, 9])
    c = empty(n, 2, gen.choice([20, 37, 64]), 8, page=page, layers=2, dtype=dtype)
    b = R.Book(c)
    for step in range(40):
        what = gen.choice(["grow", "grow", "grow", "fork", "free", "cut", "compact"])
        some = [gen.randrange(n) for _ in range(gen.randint(1, n))]
        if what == "grow":
            tokens = [gen.choice([0, 1, 1, page - 1, page, 3 * page + 2]) for _ in range(n)]
            c.paris_paged_grow(i32(tokens))
            b.grow(tokens)
            x = rand(n, 2, 3 * page + 2, R.D, seed=1000 * seed + step).to(BF)
            c.paris_paged_store(x, x, layer=step % 2)
            for name in b.pools:  # rows themselves are checked elsewhere
                b.pools[name] = R.raw(getattr(c, name)).clone()
        elif what == "fork":
            src = [gen.randrange(n) for _ in some]
            c.paris_paged_fork(i32(src), i32(some))
            b.fork(src, some)
        elif what == "free":
            c.paris_paged_free(i32(some))
            b.free(some)
        elif what == "cut":
            rows = [gen.randint(0, max(b.lens)) for _ in some]
            c.paris_paged_free(i32(some), rows=i32(rows))
            b.free(some, rows)
        else:
            c.paris_paged_compact()
            b.compact()
        b.check()


@pytest.mark.parametrize("n_pages", [5, 64, 1000, 70000])
def test_a_pool_is_closed_up(n_pages):
    c = empty(8, 1, n_pages, max(1, n_pages // 8))
    cap = 16 * max(1, n_pages // 8)
    c.paris_paged_grow(i32([cap] * 8))
    x = rand(n_pages, 16, 32, seed=12)
    R.raw(c.k_pages)[0, :, 0, :, :32] = x.to(BF).view(torch.int16)
    rows = {s: R.rows_of(c, "k", 0, s).nan_to_num(nan=7.5) for s in (1, 3, 6)}
    c.paris_paged_free(i32([0, 2, 4, 5, 7]))
    used = int(c.n_used)
    c.paris_paged_compact()
    assert int(c.n_used) == used and torch.equal((c.refs > 0), torch.arange(n_pages, device="cuda") < used)
    for s, want in rows.items():
        assert torch.all(c.table[s, :-(-int(c.lens[s]) // 16)] < max(used, 1))
        assert torch.equal(R.rows_of(c, "k", 0, s).nan_to_num(nan=7.5), want)
    if n_pages <= 1000:
        R.Book(c).check()
    c.paris_paged_grow(i32([0, 0, 20, 0, 0, 0, 0, 0]))
    assert c.table[2, 0].item() == used


# ------------------------------------------------------------- attention
def check_attend(c, q, out, lse, window=0, layer=0):
    hkv, g = c.n_kv_heads, q.shape[1] // c.n_kv_heads
    e4m3 = c.k_pages.dtype == E4
    for b in range(c.n_seqs):
        n = int(c.lens[b])
        first = max(0, n - window) if window else 0
        if n == 0:
            assert torch.all(out[b] == 0) and torch.all(lse[b] == -math.inf)
            continue
        ks, vs = (R.rows_of(c, name, layer, b)[:, first:] for name in ("k", "v"))
        for h in range(hkv):
            k, v = ks[h], vs[h]
            qs = q[b, h * g:(h + 1) * g].double()
            s = qs @ k.T / math.sqrt(R.D)
            p = torch.softmax(s, -1)
            o, mass = p @ v, p @ v.abs()
            size = (qs.abs() @ k.abs().T).amax(-1)
            e = R.score_error(size, n)
            # weights enter the product with V as two bf16 parts (2^-16 of each), or as halves (2^-11) whose smallest
            # step, 2^-25 below weights kept 2^7 up, counts against the heaviest row; 8-bit rows take the query in halves
            # too, its smallest step 2^-25 of its largest value
            w = 2.0 ** -11 if e4m3 else 2.0 ** -16
            tol = R.HALF_BF16 * o.abs() + ((1 + R.HALF_BF16) * (e + w))[:, None] * mass
            if e4m3:
                tol += ((p * v.abs().amax(-1)).amax(-1) * (n - first) * 2.0 ** -30)[:, None]
                f = 2.0 * qs.abs().amax(-1) * k.abs().sum(-1).amax() * 2.0 ** -24 / math.sqrt(R.D)
                tol += f[:, None] * mass
                e = e + f
            got = out[b, h * g:(h + 1) * g].double()
            assert torch.all((got - o).abs() <= tol), (b, h, ((got - o).abs() / tol).max())
            want = torch.logsumexp(s, -1)
            d = (lse[b, h * g:(h + 1) * g].double() - want).abs()
            assert torch.all(d <= e + 8 * R.U32 * want.abs()), (b, h, d.max())


def attend(c, q, window=0, layer=0):
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    c.paris_paged_attend(q, out, window=window, lse=lse, layer=layer)
    return out, lse


@pytest.mark.parametrize("dtype,page,order", [(BF, 16, "hrd"), (BF, 64, "rhd"), (E4, 16, "rhd"), (E4, 32, "hrd"), (E4, 256, "hrd")])
@pytest.mark.parametrize("g", [1, 3, 4, 5, 8, 12, 16, 17, 40, 128])
@pytest.mark.parametrize("lens", [[1], [0, 15, 16, 17], [63, 64, 65, 2, 127, 129], [1000, 257]])
def test_attention_over_the_rows_in_use(lens, g, dtype, page, order):
    hkv = 2 if g < 40 else 1
    c, _, _ = filled(lens, hkv, page, dtype, seed=20 + g, order=order)
    q = rand(len(lens), hkv * g, R.D, seed=40, amp=2.0).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)
    out2 = torch.full_like(q, 9.0)
    c.paris_paged_attend(q, out2)  # without lse, and in the same workspace
    assert torch.equal(out, out2)
    c.paris_paged_check()


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 31, 32, 33, 100, 1000, 1 << 40])
def test_attention_in_a_window(window, dtype):
    lens = [1, 0, 16, 33, 100, 517, 1000]
    c, _, _ = filled(lens, 2, 16, dtype, seed=50)
    q = rand(len(lens), 8, R.D, seed=51, amp=2.0).to(BF)
    out, lse = attend(c, q, window)
    check_attend(c, q, out, lse, window)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("n,hq,hkv", [(20000, 8, 2), (33333, 3, 1), (5000, 64, 8)])
def test_attention_over_long_sequences(n, hq, hkv, dtype):
    c, _, _ = filled([n, 40], hkv, 16, dtype, seed=60)
    q = rand(2, hq, R.D, seed=61, amp=2.0).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)
    assert torch.equal(attend(c, q)[0], out)


@pytest.mark.parametrize("lens", [[300 if b in (0, 40, 99) else 0 for b in range(100)],
                                  [3000 if b == 70 else b % 5 for b in range(128)], [b % 300 for b in range(131)],
                                  [1] * 700, [5000] + [0] * 1000 + [7]])
@pytest.mark.parametrize("dtype", [BF, E4])
def test_attention_over_many_sequences(lens, dtype):
    c, _, _ = filled(lens, 1, 16, dtype, seed=62)
    q = rand(len(lens), 4, R.D, seed=63, amp=2.0).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("g", [2, 8, 16])
@pytest.mark.parametrize("amp", [0.0, 1e-30, 1e-4, 60.0])
def test_queries_of_any_size(amp, g, dtype):
    c, _, _ = filled([300], 1, 16, dtype, seed=64)
    q = (rand(1, g, R.D, seed=65) * amp).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("g", [2, 8, 16])
@pytest.mark.parametrize("amp,rows", [(1e7, 300), (1e12, 9000), (1e28, 300), (1e36, 300)])
def test_scores_far_apart_leave_one_row(amp, rows, g, dtype):
    gen = torch.Generator().manual_seed(500 + g)
    k, v = (torch.randn(rows, 1, R.D, generator=gen).to(BF) for _ in range(2))
    q = (torch.randn(1, g, R.D, generator=gen) * amp).to(BF)
    c, _, _ = filled([rows], 1, 16, dtype, kv=(k.cuda(), v.cuda()))
    kd, vd = R.rows_of(c, "k", 0, 0)[0], R.rows_of(c, "v", 0, 0)[0]
    s = q[0].double().cuda() @ kd.T / math.sqrt(R.D)
    top = s.topk(2, dim=-1)
    size = (q[0].double().cuda().abs() @ kd.abs().T).amax(-1) / math.sqrt(R.D)
    assert torch.all(top.values[:, 0] - top.values[:, 1] > 2.0 ** -15 * size + 150 * math.log(2))
    out, lse = attend(c, q.cuda())
    assert torch.equal(out[0].double(), vd[top.indices[:, 0]])
    assert torch.all((lse[0].double() - top.values[:, 0]).abs() <= 2.0 ** -15 * size)


@pytest.mark.parametrize("g", [4, 8])
def test_rows_of_very_different_sizes(g):
    k, v = rand(400, 1, R.D, seed=66), rand(400, 1, R.D, seed=67)
    size = torch.exp2(torch.randint(-40, 40, (400, 1, 1), device="cuda", generator=torch.Generator("cuda").manual_seed(68)).float())
    c, _, _ = filled([400], 1, 16, E4, kv=(k.to(BF), (v * size).to(BF)))
    q = rand(1, g, R.D, seed=69).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)
    c, _, _ = filled([400], 1, 16, E4, kv=((k * torch.exp2(-size.log2().abs() / 8)).to(BF), (v * size).to(BF)))
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_a_heavy_row_of_small_values_beside_large_ones_of_no_weight(dtype):
    k, v = torch.zeros(200, 1, R.D, device="cuda"), rand(200, 1, R.D, seed=70)
    k[:, 0, 0] = -90.0
    k[150, 0, 0] = 90.0  # the only row of weight
    v[:] *= 1e3
    v[150] *= 1e-9
    c, _, _ = filled([200], 1, 16, dtype, kv=(k.to(BF), v.to(BF)))
    q = torch.zeros(1, 4, R.D, device="cuda")
    q[..., 0] = 20.0
    out, lse = attend(c, q.to(BF))
    assert torch.equal(out[0, 0].double(), R.rows_of(c, "v", 0, 0)[0, 150])


@pytest.mark.parametrize("g", [4, 8, 16])
def test_queries_and_rows_that_are_not_finite(g):
    c, k, v = filled([100, 40], 1, 16, BF, seed=71)
    q = rand(2, g, R.D, seed=72).to(BF)
    want, _ = attend(c, q)
    bad = q.clone()
    bad[0, 2, 7] = math.nan
    got, lse = attend(c, bad)
    assert torch.isnan(got[0, 2]).all() and torch.isnan(lse[0, 2])
    keep = [h for h in range(g) if h != 2]
    assert torch.equal(got[0, keep], want[0, keep]) and torch.equal(got[1], want[1])
    # a key with a score of -inf has no weight; where there are no others the result is zeros
    q = q.abs()
    page, r = c.table[0, 33 // 16].item(), 33 % 16
    c.k_pages[0, page, 0, r] = -math.inf
    got, lse = attend(c, q)
    rest = torch.arange(100, device="cuda") != 33
    s = q[0].double() @ R.rows_of(c, "k", 0, 0)[0][rest].T / math.sqrt(R.D)
    o = torch.softmax(s, -1) @ R.rows_of(c, "v", 0, 0)[0][rest]
    assert torch.all((got[0].double() - o).abs() <= 2.0 ** -6)
    assert torch.all((lse[0].double() - torch.logsumexp(s, -1)).abs() <= 2.0 ** -10)
    c.k_pages.fill_(-math.inf)
    got, lse = attend(c, q)
    assert torch.all(got == 0) and torch.all(lse == -math.inf)


def test_lengths_and_entries_outside_the_cache_count_as_the_nearest():
    c, _, _ = filled([64, 64], 1, seed=73, spare=0)
    q = rand(2, 2, R.D, seed=74).to(BF)
    c.lens.copy_(i32([1 << 30, -3]))
    out, lse = attend(c, q)
    c.lens.copy_(i32([64, 0]))
    check_attend(c, q, out, lse)
    order = c.table.clone()
    c.table[0] = i32([-1, 0, 7, 99])
    out, lse = attend(c, q)
    c.table[0] = i32([0, 0, 7, 7])
    check_attend(c, q, out, lse)
    c.table.copy_(order)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_layers_are_apart(dtype):
    c, k, v = filled([70, 20], 2, 32, dtype, seed=75, layers=3, order="rhd")
    c.paris_paged_grow(i32([1, 1]))
    x = rand(3, 2, 2, 2, R.D, seed=76).to(BF)
    for layer in (2, 0, 1):
        c.paris_paged_append(x[layer, 0], x[layer, 1], layer=layer)
    q = rand(2, 4, R.D, seed=77).to(BF)
    outs = []
    for layer in range(3):
        out, lse = attend(c, q, layer=layer)
        check_attend(c, q, out, lse, layer=layer)
        outs.append(out)
    assert not torch.equal(outs[0], outs[1])


def test_appended_rows_of_strided_tensors():
    c = empty(3, 2, 6, 2)
    both = rand(3, 4, 2, 2, R.D, seed=81).to(BF)  # keys and values of several layers side by side
    for layer in range(1, 3):
        c.paris_paged_grow(i32([1, 0, 1]))
        c.paris_paged_append(both[:, layer, 0], both[:, layer, 1])
    f = rand(3, 2, R.D, seed=82)
    c.paris_paged_grow(i32([0, 1, 1]))
    c.paris_paged_append(f, f.to(torch.float32))
    assert c.lens.tolist() == [2, 1, 3]
    for i, name in enumerate(("k", "v")):
        for s, rows in ((0, [both[0, 1, i], both[0, 2, i]]), (1, [f[1]]), (2, [both[2, 1, i], both[2, 2, i], f[2]])):
            assert torch.equal(R.rows_of(c, name, 0, s).transpose(0, 1), torch.stack([x.to(BF) for x in rows]).double())
    with pytest.raises(ValueError, match="contiguous"):
        c.paris_paged_append(both[:, 1, 0].transpose(1, 2).contiguous().transpose(1, 2), both[:, 1, 1])


@pytest.mark.parametrize("dtype", [BF, E4])
def test_a_pool_past_four_gigabytes(dtype):
    n_pages = 140000 if dtype is BF else 280000  # 8 heads of 16 rows: 4.6 GB of keys
    c = empty(1, 8, n_pages, 40, garbage=False, dtype=dtype)
    c.table[0, :40] = torch.arange(n_pages - 40, n_pages, dtype=torch.int32, device="cuda").flip(0)
    c.lens.fill_(600)
    k, v = rand(600, 8, R.D, seed=78).to(BF), rand(600, 8, R.D, seed=79).to(BF)
    c.paris_paged_store(k, v, cu=K4.starts([600]))  # starts is 0
    assert torch.any(R.raw(c.k_pages)[0, n_pages - 1]) and not torch.any(R.raw(c.k_pages)[0, :n_pages - 40][::7])
    q = rand(1, 16, R.D, seed=80).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)
    ko, vo = torch.zeros(600, 8, R.D, dtype=BF, device="cuda"), torch.zeros(600, 8, R.D, dtype=BF, device="cuda")
    c.paris_paged_read(ko, vo, cu=K4.starts([600]))
    assert torch.equal(ko.double().transpose(0, 1), R.rows_of(c, "k", 0, 0))
    # and copied there and back: the last 38 pages move to the front
    c.refs[n_pages - 38:] = 1
    c.free_bits.copy_(pack_bits(c.refs == 0))
    c.n_used.fill_(38)
    c.paris_paged_compact()
    assert c.table[0, :38].max() < 38
    got, _ = attend(c, q)
    assert torch.equal(got, out)


def pack_bits(flags):
    w = torch.zeros(-(-flags.numel() // 32) * 32, dtype=torch.int64, device=flags.device)
    w[:flags.numel()] = flags
    w = (w.reshape(-1, 32) << torch.arange(32, device=flags.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


# --------------------------------------------------------------- together
@pytest.mark.parametrize("dtype", [BF, E4])
def test_prompts_become_beams_and_make_room_for_others(dtype):
    lens, hq, hkv, page, layers = [70, 33, 48], 8, 2, 16, 2
    n = 6
    q, k, v = (rand(sum(lens), h, R.D, seed=90 + i).to(BF) for i, h in enumerate((hq, hkv, hkv)))
    out, cu = torch.empty_like(q), K4.starts(lens)
    c = empty(n, hkv, 40, 16, page, layers, dtype)
    b = R.Book(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu, max_q=max(lens), max_k=max(lens))
        c.paris_paged_grow(i32(lens + [0] * 3))
        for layer in range(layers):
            c.paris_paged_store(k, v, cu=K4.starts(lens + [0] * 3), max_new=max(lens), layer=layer)
        c.paris_paged_fork(i32([0, 0, 2]), i32([3, 4, 5]))
    torch.cuda.synchronize()
    b.grow(lens + [0] * 3)
    for name in b.pools:
        b.pools[name] = R.raw(getattr(c, name)).clone()
    b.fork([0, 0, 2], [3, 4, 5])
    b.check(pools=False)
    for name in ("k", "v"):
        assert torch.equal(R.rows_of(c, name, 1, 3), R.rows_of(c, name, 1, 0))
    for step in range(20):
        x = rand(layers, 2, n, hkv, R.D, seed=100 + step).to(BF)
        qd = rand(n, hq, R.D, seed=200 + step, amp=2.0).to(BF)
        c.paris_paged_grow(i32([1] * n))
        b.grow([1] * n)
        for layer in range(layers):
            c.paris_paged_append(x[layer, 0], x[layer, 1], layer=layer)
            got, lse = attend(c, qd, layer=layer)
            check_attend(c, qd, got, lse, layer=layer)
        for name in b.pools:
            b.pools[name] = R.raw(getattr(c, name)).clone()
        if step % 4 == 1:
            src = [3, 0, 2, 4, 0, 5]
            c.paris_paged_fork(i32(src), i32(range(n)))
            b.fork(src, list(range(n)))
        if step == 9:
            c.paris_paged_free(i32([1]))
            b.free([1])
            c.paris_paged_compact()
            b.compact()
        if step == 14:
            rows = [x - 5 for x in b.lens]
            c.paris_paged_free(i32(range(n)), rows=i32(rows))
            b.free(list(range(n)), rows)
        b.check()
    c.paris_paged_check()
    # what the cache holds is a prompt's past: a chunk of queries reads it back
    m = b.lens[0]
    ko, vo = torch.zeros(m, hkv, R.D, dtype=BF, device="cuda"), torch.zeros(m, hkv, R.D, dtype=BF, device="cuda")
    c.paris_paged_read(ko, vo, cu=K4.starts([m, 0, 0, 0, 0, 0]), layer=0)
    qc, oc, lc = rand(1, hq, R.D, seed=300).to(BF), torch.zeros(1, hq, R.D, dtype=BF, device="cuda"), torch.zeros(hq, 1, device="cuda")
    P.paris_prompt_attend(qc, ko, vo, oc, cu_q=K4.starts([1]), cu_k=K4.starts([m]), lse=lc)
    got, lse = attend(c, torch.cat([qc] * n))
    assert torch.all((lc[:, 0] - lse[0]).abs() < 1e-3)
    assert torch.all((oc[0].double() - got[0].double()).abs() < 2.0 ** -6 * (1 + oc[0].double().abs()))


def test_steps_in_a_replayed_graph_walk_on():
    def mk():
        c, _, _ = filled([30, 15, 0, 1], 2, seed=110, spare=60, extra=12)
        return c

    eager, graphed = mk(), mk()
    k, v, q = (rand(4, h, R.D, seed=111 + h).to(BF) for h in (2, 2, 8))
    outs = [torch.zeros_like(q), torch.zeros_like(q)]
    one, src, dst, back = i32([1, 1, 1, 2]), i32([0, 1]), i32([2, 1]), i32([20])

    def step(c, out):
        c.paris_paged_grow(one)
        c.paris_paged_append(k, v)
        c.paris_paged_attend(q, out)
        c.paris_paged_fork(src, dst)
        c.paris_paged_free(dst[1:], rows=back)
        c.paris_paged_compact()
        c.paris_paged_attend(q, out, window=9)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(graphed, outs[1])
    for i in range(40):
        k.copy_(rand(4, 2, R.D, seed=400 + i))
        q.copy_(rand(4, 8, R.D, seed=500 + i))
        step(eager, outs[0])
        graph.replay()
        torch.cuda.synchronize()
        # bit for bit: the fourth sequence's second row of a step is not written, and its NaN stays
        assert torch.equal(R.raw(outs[0]), R.raw(outs[1]))
        for name in ("table", "lens", "starts", "refs", "free_bits", "n_used", "k_pages", "v_pages"):
            assert torch.equal(R.raw(getattr(eager, name)), R.raw(getattr(graphed, name))), name
    R.Book(graphed).check()
    assert graphed.lens.tolist() == [70, 20, 70, 81]


def test_readers_on_two_streams_at_once():
    c, _, _ = filled([9000, 1, 700], 2, seed=120)
    q = rand(2, 3, 8, R.D, seed=121, amp=2.0).to(BF)
    want = [attend(c, x) for x in q]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = torch.zeros(2, 20, 3, 8, R.D, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    for i in range(20):
        for j, s in enumerate(streams):
            c.paris_paged_attend(q[j], outs[j, i], stream=s)
    torch.cuda.synchronize()
    for j in range(2):
        assert torch.all(outs[j] == want[j][0])


def test_two_graphs_and_a_stream_at_once():
    c, _, _ = filled([7000, 300, 0, 1, 2500], 2, dtype=E4, seed=122)
    q = rand(3, 5, 16, R.D, seed=123, amp=2.0).to(BF)
    want = [attend(c, x)[0] for x in q]
    outs = torch.zeros(3, 5, 16, R.D, dtype=BF, device="cuda")
    graphs, streams = [torch.cuda.CUDAGraph() for _ in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for g, i in zip(graphs, range(2)):
        with torch.cuda.graph(g):
            for _ in range(5):
                c.paris_paged_attend(q[i], outs[i])
    for _ in range(10):
        outs.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        c.paris_paged_attend(q[2], outs[2])
        torch.cuda.synchronize()
        for i in range(3):
            assert torch.equal(outs[i], want[i])
    c.paris_paged_check()


def test_attention_with_different_numbers_of_heads_in_turn():
    c, _, _ = filled([3000, 20], 2, dtype=BF, seed=124)
    for hq in (2, 256, 8, 64, 16, 2):
        q = rand(2, hq, R.D, seed=125 + hq, amp=2.0).to(BF)
        out, lse = attend(c, q)
        check_attend(c, q, out, lse)


def test_many_kv_heads():
    c, _, _ = filled([40, 100], 300, dtype=E4, seed=126)
    q = rand(2, 600, R.D, seed=127).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)


@pytest.mark.parametrize("dtype", [BF, E4])
def test_pages_of_256_rows_and_windows_that_begin_inside(dtype):
    c, _, _ = filled([900, 256, 255, 513], 2, 256, dtype, seed=128, order="rhd")
    q = rand(4, 32, R.D, seed=129, amp=2.0).to(BF)
    for window in (0, 1, 100, 257, 600):
        out, lse = attend(c, q, window)
        check_attend(c, q, out, lse, window)


@pytest.mark.parametrize("dtype", [BF, E4])
@pytest.mark.parametrize("n,hq", [(150000, 4), (400000, 2), (150000, 128)])
def test_one_kv_head_over_hundreds_of_units(n, hq, dtype):
    """Partial sums of up to 680 units a sequence, and (128 query heads) of many sequences' worth of heads."""
    c, _, _ = filled([n, 0, 700], 1, 64, dtype, seed=131)
    q = rand(3, hq, R.D, seed=132, amp=2.0).to(BF)
    out, lse = attend(c, q)
    check_attend(c, q, out, lse)
    again, lse2 = attend(c, q)
    assert torch.equal(again, out) and torch.equal(lse2, lse)
    c.paris_paged_check()


def test_a_dropped_cache_is_kept_for_the_streams_that_use_it():
    x = rand(1, 1, R.D, seed=130).to(BF)
    s = torch.cuda.Stream()
    c = P.PagedCache.create(1, 1, 40, 4)
    own = {t.data_ptr() for t in (*c._tensors, c._status)}
    one = i32([1])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(4 * 10 ** 9)
        c.paris_paged_grow(one)
        c.paris_paged_append(x, x)
    c.record_stream(s)
    del c
    new = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(5000)]
    assert not s.query()
    assert own.isdisjoint(t.data_ptr() for t in new)
    torch.cuda.synchronize()
