"""The 4-bit cache (paris_kv4_*): rows bit for bit against the 64-bit definition, decode attention and accumulated
weights against 64-bit forms over the rows' exact values, eviction row for row, and all of them together from a prompt
to decode steps under a budget."""
import math

import pytest
import torch

from long_context_kv_gb300 import paris as P
from tests import kv4_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_kv_gb300 import build
    build.build()
    P.load()


def rand(*s, seed=0, amp=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return amp * torch.randn(*s, generator=gen, device="cuda")


# ------------------------------------------------------------------ store
def edge_rows(dtype):
    x = rand(40, 2, R.D, seed=1)
    x[0] = 0
    x[1] *= 1e-6
    x[2] *= 1e-4
    x[3] *= 1000.0
    x[4] *= 1e5
    x[5, :, 3] = math.nan
    x[6, :, 40] = math.inf
    x[7, :, 41] = -math.inf
    x[8] = 7.0 * 1.5 * torch.sign(x[8])             # S is exactly 1.5
    x[9] = 1.75 * torch.round(4 * x[9]) / 2         # many ties of x / S
    x[10] = x[10].clamp(-0.9e-4, 0.9e-4)
    x[11, :, ::2] = 1680.0
    x[12] = 2.0 ** -130
    return x.to(dtype)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_stored_rows_are_the_definition_bit_for_bit(dtype):
    x = edge_rows(dtype)
    y = rand(40, 2, R.D, seed=2).to(dtype)
    c = P.KV4Cache.create(1, 2, 64)
    c.paris_kv4_store(x, y, cu=R.starts([40]))
    for codes, scales, src in ((c.k_codes, c.k_scales, x), (c.v_codes, c.v_scales, y)):
        wc, ws = R.quantise(src)
        assert torch.equal(scales[0, :, :40], ws.transpose(0, 1))
        assert torch.equal(codes[0, :, :40], wc.transpose(0, 1))
        assert torch.all(codes[0, :, 40:] == 0) and torch.all(scales[0, :, 40:] == 0)
    assert c.lens.tolist() == [40] and c.next_pos.tolist() == [40]
    assert torch.equal(c.positions[0, :, :40], torch.arange(40, device="cuda", dtype=torch.int32).expand(2, 40))
    ko, vo = (torch.full((1, 2, 50, R.D), 5.0, dtype=BF, device="cuda") for _ in range(2))
    c.paris_kv4_read(ko, vo)
    assert torch.equal(ko[0, :, :40].double(), R.values(c.k_codes, c.k_scales)[0, :, :40])
    assert torch.equal(vo[0, :, :40].double(), R.values(c.v_codes, c.v_scales)[0, :, :40])
    assert torch.all(ko[:, :, 40:] == 5.0) and torch.all(vo[:, :, 40:] == 5.0)
    c.paris_kv4_check()


def test_a_value_is_off_by_at_most_half_a_step():
    x = rand(300, 3, R.D, seed=3, amp=4.0).to(BF)
    v = R.values(*R.quantise(x))
    s = R.scale_of(x.double().unflatten(-1, (4, 32)).abs().amax(-1)).repeat_interleave(32, -1)
    assert torch.all((v - x.double()).abs() <= s / 2)
    c = P.KV4Cache.create(1, 3, 300)
    c.paris_kv4_store(x, x, cu=R.starts([300]))
    assert torch.equal(R.values(c.k_codes, c.k_scales)[0].transpose(0, 1), v)


@pytest.mark.parametrize("lens", [[1], [3, 0, 17], [16, 15, 33, 1], [500, 7]])
def test_ragged_stores_pile_up(lens):
    n, h = len(lens), 3
    c = P.KV4Cache.create(n, h, 1100)
    want = [[] for _ in lens]
    for turn in range(2):
        k, v = rand(sum(lens), h, R.D, seed=turn).to(BF), rand(sum(lens), h, R.D, seed=9 + turn).to(BF)
        w = rand(h, sum(lens), seed=20 + turn) if turn else None
        c.paris_kv4_store(k, v, cu=R.starts(lens), max_new=max(lens), weights=w)
        a = 0
        for i, m in enumerate(lens):
            want[i].append((k[a:a + m], v[a:a + m], torch.zeros(h, m, device="cuda") if w is None else w[:, a:a + m]))
            a += m
    for i, m in enumerate(lens):
        k, v = (torch.cat([t[j] for t in want[i]]) for j in (0, 1))
        assert c.lens[i] == 2 * m and c.next_pos[i] == 2 * m
        assert torch.equal(c.k_codes[i, :, :2 * m], R.quantise(k)[0].transpose(0, 1))
        assert torch.equal(c.v_codes[i, :, :2 * m], R.quantise(v)[0].transpose(0, 1))
        assert torch.equal(c.v_scales[i, :, :2 * m], R.quantise(v)[1].transpose(0, 1))
        assert torch.equal(c.weights[i, :, :2 * m], torch.cat([t[2] for t in want[i]], 1))
        assert torch.equal(c.positions[i, 0, :2 * m].cpu(), torch.arange(2 * m, dtype=torch.int32))


def test_padded_layout_views_and_append():
    b, h, t = 3, 2, 21
    x = rand(b, t, 2 * h, R.D, seed=4).transpose(1, 2)      # float32 views [b, heads, t, d]
    c = P.KV4Cache.create(b, h, 64)
    w = rand(b, h, t, seed=5)
    c.paris_kv4_store(x[:, :h], x[:, h:], weights=w)
    k, v = rand(b, h, R.D, seed=6).to(BF), rand(b, h, R.D, seed=7).to(BF)
    c.paris_kv4_append(k, v)
    assert c.lens.tolist() == [t + 1] * b
    for codes, scales, old, new in ((c.k_codes, c.k_scales, x[:, :h], k), (c.v_codes, c.v_scales, x[:, h:], v)):
        oc, os_ = R.quantise(old)
        nc, ns = R.quantise(new)
        assert torch.equal(codes[:, :, :t], oc) and torch.equal(scales[:, :, :t], os_)
        assert torch.equal(codes[:, :, t], nc) and torch.equal(scales[:, :, t], ns)
    assert torch.equal(c.weights[:, :, :t], w) and torch.all(c.weights[:, :, t] == 0)


def test_a_full_cache_drops_tokens_and_says_so():
    c = P.KV4Cache.create(2, 1, 10)
    k = rand(14, 1, R.D, seed=8).to(BF)
    c.paris_kv4_store(k, k, cu=R.starts([12, 2]))
    assert c.lens.tolist() == [10, 2]
    assert torch.equal(c.k_codes[0, :, :10], R.quantise(k[:10])[0].transpose(0, 1))
    with pytest.raises(P.ParisError) as e:
        c.paris_kv4_check()
    assert e.value.status == P.PARIS_EDEVICE
    c.paris_kv4_check()  # cleared
    before = c.k_codes.clone()
    c.paris_kv4_append(k[:2], k[:2])
    assert c.lens.tolist() == [10, 3] and torch.equal(c.k_codes[0], before[0])
    with pytest.raises(P.ParisError):
        c.paris_kv4_check()


# ----------------------------------------------------------------- attend
def filled(lens, h, rows, seed=0, garbage=True):
    c = P.KV4Cache.create(len(lens), h, rows)
    if garbage:  # rows that are not in use hold anything
        for t in (c.k_codes, c.v_codes, c.k_scales, c.v_scales):
            t.fill_(255)
        c.weights.fill_(math.nan)
    k, v = rand(sum(lens), h, R.D, seed=seed).to(BF), rand(sum(lens), h, R.D, seed=seed + 1).to(BF)
    c.paris_kv4_store(k, v, cu=R.starts(lens))
    return c


def check_attend(c, q, out, weights_before=None):
    hq, g = q.shape[1], q.shape[1] // c.n_kv_heads
    for b in range(c.batch):
        n = int(c.lens[b])
        if n == 0:
            assert torch.all(out[b] == 0)
            continue
        for h in range(c.n_kv_heads):
            k = R.values(c.k_codes[b, h, :n], c.k_scales[b, h, :n])
            v = R.values(c.v_codes[b, h, :n], c.v_scales[b, h, :n])
            qs = q[b, h * g:(h + 1) * g].double()
            p = torch.softmax(qs @ k.T / math.sqrt(R.D), -1)
            o, mass = p @ v, p @ v.abs()
            # two half-precision parts of a query or a weight: 2^-22 of it, and 2^-25 of the largest (1)
            size = (qs.abs() @ k.abs().T).amax(-1)
            floor = (qs.abs().amax(-1) * k.abs().sum(-1).amax()) * 2.0 ** -24
            e = R.score_error(size, n) + 2 * (2.0 ** -22 * size + floor) / math.sqrt(R.D)
            tol = R.HALF_BF16 * o.abs() + ((1 + R.HALF_BF16) * (e + 2.0 ** -21))[:, None] * mass
            tol += 2.0 ** -24 * p.amax(-1, keepdim=True) * v.abs().sum(0)
            got = out[b, h * g:(h + 1) * g].double()
            assert torch.all((got - o).abs() <= tol), ((got - o).abs() / tol).max()
            if weights_before is not None:
                w0 = weights_before[b, h, :n].double()
                want = w0 + p.sum(0)
                d = (c.weights[b, h, :n].double() - want).abs()
                assert torch.all(d <= (p * e[:, None]).sum(0) + (g + 1) * R.U32 * want.abs() + 1e-30), d.max()
    if weights_before is not None:
        rows = torch.arange(c.max_rows, device="cuda")[None] >= c.lens[:, None]
        beyond = rows[:, None].expand_as(c.weights)
        assert torch.equal(torch.isnan(c.weights[beyond]), torch.isnan(weights_before[beyond]))


@pytest.mark.parametrize("g", [1, 3, 4, 8, 12, 16])
@pytest.mark.parametrize("lens", [[1], [0, 31, 32, 33], [127, 128, 129, 2], [1000, 257]])
def test_attention_over_the_rows_in_use(g, lens):
    h = 2
    c = filled(lens, h, 1024, seed=30 + g)
    q = rand(len(lens), h * g, R.D, seed=40, amp=2.0).to(BF)
    out = torch.full_like(q, 9.0)
    c.paris_kv4_attend(q, out)
    check_attend(c, q, out)
    before = c.weights.clone()
    out2 = torch.full_like(q, 9.0)
    c.paris_kv4_attend(q, out2, accumulate=True)
    assert torch.equal(out, out2)
    check_attend(c, q, out2, before)


@pytest.mark.parametrize("lens", [[300 if b in (0, 40, 99) else 0 for b in range(100)],
                                  [3000 if b == 70 else b % 5 for b in range(128)], [b % 300 for b in range(131)]])
def test_attention_over_many_sequences(lens):
    c = filled(lens, 2, max(lens) + 4, seed=33)
    q = rand(len(lens), 6, R.D, seed=34, amp=2.0).to(BF)
    before, out = c.weights.clone(), torch.full_like(q, 9.0)
    c.paris_kv4_attend(q, out, accumulate=True)
    check_attend(c, q, out, before)


@pytest.mark.parametrize("rows", [1, 5, 130, 20000])
def test_attention_with_float32_queries_and_full_caches(rows):
    c = filled([rows], 1, rows, seed=50, garbage=False)
    q = rand(1, 4, R.D, seed=51, amp=3.0)
    out = torch.zeros(1, 4, R.D, dtype=BF, device="cuda")
    before = c.weights.clone()
    c.paris_kv4_attend(q, out, accumulate=True)
    check_attend(c, q, out, before)


@pytest.mark.parametrize("amp", [0.0, 1e-20, 1e-4, 60.0, 1e4])
def test_queries_of_any_size(amp):
    c = filled([300], 1, 512, seed=52)
    q = (rand(1, 2, R.D, seed=53) * amp)
    out = torch.zeros(1, 2, R.D, dtype=BF, device="cuda")
    c.paris_kv4_attend(q, out)
    check_attend(c, q, out)


def one_hot_case(amp, g, rows, seed):
    """Scores so far apart that each head's softmax is one row: (k, v, q) and each head's row, made on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(rows, 1, R.D, generator=gen).to(BF) for _ in range(2))
    q = (torch.randn(1, g, R.D, generator=gen) * amp).to(BF)
    s = q[0].double() @ R.values(*R.quantise(k))[:, 0].T / math.sqrt(R.D)
    top = s.topk(2, dim=-1)
    size = (q[0].double().abs() @ R.values(*R.quantise(k))[:, 0].abs().T).amax(-1) / math.sqrt(R.D)
    # 128 float32 products of any order and two half parts of 2^-22 put a score off by less than 2^-16 of its terms; a
    # weight of 2^-150 is 0
    assert torch.all(top.values[:, 0] - top.values[:, 1] > 2.0 ** -15 * size + 150 * math.log(2))
    return k, v, q, top.indices[:, 0]


def check_one_hot(amp, dtype, g, rows):
    k, v, q, at = (t.cuda() for t in one_hot_case(amp, g, rows, seed=500 + g))
    c = P.KV4Cache.create(1, 1, rows)
    c.paris_kv4_store(k, v, cu=R.starts([rows]))
    out = torch.full((1, g, R.D), 9.0, dtype=BF, device="cuda")
    c.paris_kv4_attend(q.to(dtype), out, accumulate=True)
    assert torch.equal(out[0].double(), R.values(c.v_codes, c.v_scales)[0, 0][at])
    assert torch.equal(c.weights[0, 0], torch.bincount(at, minlength=rows).float())


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("g", [2, 8])
@pytest.mark.parametrize("amp,rows", [(1e7, 300), (1e9, 9000), (1e20, 300), (1e28, 300), (1e28, 9000)])
def test_scores_far_apart_leave_one_row(amp, rows, g, dtype):
    check_one_hot(amp, dtype, g, rows)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("g", [2, 8])
@pytest.mark.parametrize("amp,rows", [(1e32, 300), (1e36, 300), (1e36, 9000), (4e37, 300)])
def test_the_largest_finite_queries(amp, rows, g, dtype):
    check_one_hot(amp, dtype, g, rows)


@pytest.mark.parametrize("amp", [1e-28, 1e-34, 1e-38])
def test_the_smallest_queries(amp):
    c = filled([300], 1, 512, seed=52)
    q = (rand(1, 8, R.D, seed=53) * amp)
    out = torch.zeros(1, 8, R.D, dtype=BF, device="cuda")
    c.paris_kv4_attend(q, out)
    check_attend(c, q, out)


@pytest.mark.parametrize("batch", [2, 33, 128, 129, 300])
def test_batches_of_very_different_lengths(batch):
    gen = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 40, (batch,), generator=gen).tolist()
    lens[batch // 2] = 700
    c = filled(lens, 1, 704, seed=61)
    q = rand(batch, 4, R.D, seed=62, amp=2.0).to(BF)
    out = torch.full_like(q, 9.0)
    before = c.weights.clone()
    c.paris_kv4_attend(q, out, accumulate=True)
    check_attend(c, q, out, before)
    check_evict(c, 20, 1, 4)


def test_many_kv_heads():
    h = 300
    c = P.KV4Cache.create(2, h, 24)
    k, v = rand(30, h, R.D, seed=63).to(BF), rand(30, h, R.D, seed=64).to(BF)
    c.paris_kv4_store(k, v, cu=R.starts([11, 19]))
    assert torch.equal(c.k_codes[0, :, :11], R.quantise(k[:11])[0].transpose(0, 1))
    assert torch.equal(c.v_codes[1, :, :19], R.quantise(v[11:])[0].transpose(0, 1))
    assert torch.equal(c.v_scales[1, :, :19], R.quantise(v[11:])[1].transpose(0, 1))
    q = rand(2, h, R.D, seed=65).to(BF)
    out = torch.zeros_like(q)
    c.paris_kv4_attend(q, out)
    check_attend(c, q, out)


def test_a_query_that_is_not_finite_spoils_only_its_own_head():
    c = filled([100], 1, 128, seed=54)
    q = rand(1, 4, R.D, seed=55).to(BF)
    want, got = (torch.zeros(1, 4, R.D, dtype=BF, device="cuda") for _ in range(2))
    c.paris_kv4_attend(q, want)
    q[0, 2, 7] = math.nan
    c.paris_kv4_attend(q, got)
    assert torch.isnan(got[0, 2]).all()
    assert torch.equal(got[0, [0, 1, 3]], want[0, [0, 1, 3]])


def test_scales_of_very_different_rows():
    k, v = rand(200, 1, R.D, seed=56), rand(200, 1, R.D, seed=57)
    size = torch.exp2(torch.randint(-14, 10, (200, 1, 1), device="cuda").float())
    c = P.KV4Cache.create(1, 1, 256)
    c.paris_kv4_store(k.clamp(-3, 3), (v * size).to(BF).float(), cu=R.starts([200]))
    q = rand(1, 8, R.D, seed=58).to(BF)
    out = torch.zeros_like(q)
    c.paris_kv4_attend(q, out)
    check_attend(c, q, out)


def test_lengths_outside_the_cache_count_as_the_nearest():
    c = filled([64, 64], 1, 64, seed=59, garbage=False)
    q = rand(2, 2, R.D, seed=60).to(BF)
    c.lens.copy_(torch.tensor([1000, -3]))
    out = torch.full_like(q, 9.0)
    c.paris_kv4_attend(q, out)
    c.lens.copy_(torch.tensor([64, 0]))
    check_attend(c, q, out)


# ------------------------------------------------------------------ evict
def snapshot(c):
    return {n: getattr(c, n).clone() for n in ("k_codes", "v_codes", "k_scales", "v_scales", "weights", "positions")}


def snapshot_tensors(c):
    return c.k_codes, c.v_codes, c.k_scales, c.v_scales, c.weights, c.positions, c.lens, c.next_pos


def check_evict(c, keep, sink, recent):
    before, lens = snapshot(c), c.lens.tolist()
    nxt = c.next_pos.tolist()
    c.paris_kv4_evict(keep, sink, recent)
    torch.cuda.synchronize()
    assert c.lens.tolist() == [min(n, keep) for n in lens] and c.next_pos.tolist() == nxt
    for b, n in enumerate(lens):
        for h in range(c.n_kv_heads):
            to, of = R.evict_plan(before["weights"][b, h, :n], before["positions"][b, h, :n], n, nxt[b], keep, sink, recent)
            for name, t in before.items():
                t[b, h, to] = t[b, h, of]
    for name, t in before.items():
        assert torch.equal(getattr(c, name).view(torch.uint8), t.view(torch.uint8)), name
    c.paris_kv4_check()


@pytest.mark.parametrize("rows", [64, 5000, 40000])
@pytest.mark.parametrize("ties", [False, True])
def test_eviction_keeps_the_heaviest_rows(rows, ties):
    lens = [rows, rows // 2 + 3, 1, 0]
    c = filled(lens, 2, rows, seed=70)
    w = torch.rand(4, 2, rows, generator=torch.Generator(device="cuda").manual_seed(71), device="cuda")
    c.weights.copy_(torch.floor(w * 4) if ties else w)
    check_evict(c, rows // 2, min(4, rows // 8), rows // 8)
    check_evict(c, rows // 2, min(4, rows // 8), rows // 8)  # nothing to do
    check_evict(c, max(1, rows // 9), 0, 1)                  # and once more, over rows that have moved
    check_evict(c, 1, 0, 0)


def test_eviction_of_one_row_at_a_time():
    c = filled([41, 41], 2, 48, seed=72)
    c.weights.copy_(torch.rand(2, 2, 48, device="cuda"))
    for step in range(6):
        check_evict(c, 40, 2, 5)
        x = rand(2, 2, R.D, seed=80 + step).to(BF)
        c.paris_kv4_append(x, x)
        c.weights[:, :, 40] = torch.rand(2, 2, device="cuda")


@pytest.mark.parametrize("rows", [2, 33, 1500, 9000, 20000])
def test_eviction_of_one_row_among_equal_ones(rows):
    c = filled([rows, rows], 2, rows, seed=75)
    c.weights.fill_(0.25)
    c.weights[1, 1, rows // 2:] = 0.5
    check_evict(c, rows - 1, 1 if rows > 2 else 0, 0)


@pytest.mark.parametrize("ties", [False, True])
def test_eviction_of_more_rows_than_a_cluster_holds(ties):
    rows = 300001
    c = filled([rows], 1, rows, seed=76)
    w = torch.rand(1, 1, rows, generator=torch.Generator(device="cuda").manual_seed(77), device="cuda")
    c.weights.copy_(torch.floor(w * 3) if ties else w)
    check_evict(c, rows - 1, 16, 100)
    check_evict(c, 270000, 16, 100)
    check_evict(c, 100000, 16, 100)
    check_evict(c, 99999, 0, 0)


def test_eviction_with_odd_weights_and_many_protected_rows():
    c = filled([100], 1, 100, seed=73)
    c.weights.copy_(torch.randn(1, 1, 100, device="cuda"))
    c.weights[0, 0, 5:40:5] = math.nan
    c.weights[0, 0, 50] = math.inf
    c.weights[0, 0, 51] = -math.inf
    c.weights[0, 0, 60:70] = 0.0
    c.weights[0, 0, 62:66] = -0.0
    check_evict(c, 70, 3, 10)
    check_evict(c, 30, 3, 10)
    c.positions.fill_(0)          # every row counts as the sink: the lowest rows stay
    check_evict(c, 9, 4, 5)


def test_a_keep_that_no_sequence_exceeds_changes_nothing():
    c = filled([20, 3], 1, 32, seed=74)
    check_evict(c, 32, 0, 0)
    check_evict(c, 31, 0, 0)
    check_evict(c, 20, 0, 0)


# --------------------------------------------------------------- together
def test_from_a_prompt_to_decode_steps_under_a_budget():
    lens, hq, hkv, keep, sink, recent, window = [700, 90, 333], 8, 2, 128, 4, 32, 16
    g, n = hq // hkv, len(lens)
    q, k, v = (rand(sum(lens), h, R.D, seed=90 + i).to(BF) for i, h in enumerate((hq, hkv, hkv)))
    cu = R.starts(lens)
    out, lse = torch.empty_like(q), torch.empty(hq, sum(lens), device="cuda")
    w = torch.empty(hkv, sum(lens), device="cuda")
    c = P.KV4Cache.create(n, hkv, max(lens))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu, max_q=max(lens), max_k=max(lens), lse=lse)
        P.paris_prompt_weights(q, k, lse, w, window=window, cu_q=cu, cu_k=cu, max_k=max(lens))
        c.paris_kv4_store(k, v, cu=cu, max_new=max(lens), weights=w)
        c.paris_kv4_evict(keep, sink, recent)
    torch.cuda.synchronize()
    a = 0
    for b, m in enumerate(lens):
        for h in range(hkv):
            pos = list(range(m))
            to, of = R.evict_plan(w[h, a:a + m], torch.arange(m), m, m, keep, sink, recent)
            for i, j in zip(to, of):
                pos[i] = j
            assert c.positions[b, h, :min(m, keep)].tolist() == pos[:keep]
        a += m
    assert c.lens.tolist() == [min(m, keep) for m in lens]
    for step in range(5):
        x = rand(3, n, hkv, R.D, seed=100 + step).to(BF)
        qd = rand(n, hq, R.D, seed=200 + step, amp=2.0).to(BF)
        od = torch.empty_like(qd)
        c.paris_kv4_append(x[0], x[1])
        before = c.weights.clone()
        c.paris_kv4_attend(qd, od, accumulate=True)
        check_attend(c, qd, od, before)
        check_evict(c, keep, sink, recent)
    assert c.lens.tolist() == [128, 95, 128] and c.next_pos.tolist() == [m + 5 for m in lens]


def test_a_dropped_cache_is_kept_for_the_streams_that_use_it():
    x = rand(1, 1, R.D, seed=310).to(BF)
    s = torch.cuda.Stream()
    c = P.KV4Cache.create(1, 1, 64)
    own = {t.data_ptr() for t in (*snapshot_tensors(c), c._words)}
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(4 * 10 ** 9)  # two seconds: the append runs after them
        c.paris_kv4_append(x, x)
    c.record_stream(s)
    del c
    new = [torch.empty(2, dtype=torch.int32, device="cuda") for _ in range(5000)]
    assert not s.query()
    assert own.isdisjoint(t.data_ptr() for t in new)
    torch.cuda.synchronize()


def test_steps_of_a_cache_made_for_far_longer_sequences():
    # the capacity asks for clusters in the eviction, the lengths for a few tiles
    lens, hq, hkv, keep = [1000, 37, 4000], 8, 2, 900
    c = filled(lens, hkv, 140000, seed=320)
    gen = torch.Generator(device="cuda").manual_seed(321)
    for b, n in enumerate(lens):
        c.weights[b, :, :n] = torch.rand(hkv, n, generator=gen, device="cuda")
    check_evict(c, keep, 4, 100)
    for step in range(3):
        x = rand(2, len(lens), hkv, R.D, seed=330 + step).to(BF)
        q = rand(len(lens), hq, R.D, seed=340 + step, amp=2.0).to(BF)
        out = torch.full_like(q, 9.0)
        c.paris_kv4_append(x[0], x[1])
        before = c.weights.clone()
        c.paris_kv4_attend(q, out, accumulate=True)
        check_attend(c, q, out, before)
        check_evict(c, keep, 4, 100)
    assert c.lens.tolist() == [900, 40, 900]


def test_a_long_prompt_is_evicted_down_to_its_budget():
    n, hkv = 33000, 2
    c = filled([n, n // 2], hkv, n, seed=350)
    gen = torch.Generator(device="cuda").manual_seed(351)
    c.weights[0] = torch.rand(hkv, n, generator=gen, device="cuda") ** 8  # a prompt's: most of them small
    c.weights[1, :, :n // 2] = torch.rand(hkv, n // 2, generator=gen, device="cuda") ** 8
    check_evict(c, 4096, 16, 512)
    q = rand(2, 8, R.D, seed=352, amp=2.0).to(BF)
    before, out = c.weights.clone(), torch.full_like(q, 9.0)
    c.paris_kv4_attend(q, out, accumulate=True)
    check_attend(c, q, out, before)


def test_steps_in_a_replayed_graph_walk_on():
    lens, hq, hkv, keep = [100, 37], 4, 2, 64
    mk = lambda: filled(lens, hkv, 128, seed=300, garbage=False)  # noqa: E731
    eager, graphed = mk(), mk()
    k, v = rand(2, hkv, R.D, seed=301).to(BF), rand(2, hkv, R.D, seed=302).to(BF)
    q = rand(2, hq, R.D, seed=303).to(BF)
    outs = [torch.zeros_like(q), torch.zeros_like(q)]

    def step(c, out):
        c.paris_kv4_append(k, v)
        c.paris_kv4_attend(q, out, accumulate=True)
        c.paris_kv4_evict(keep, 2, 8)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(graphed, outs[1])
    for i in range(70):
        k.copy_(rand(2, hkv, R.D, seed=400 + i))
        q.copy_(rand(2, hq, R.D, seed=500 + i))
        step(eager, outs[0])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
    assert graphed.lens.tolist() == [64, 64] and graphed.next_pos.tolist() == [170, 107]
    for name, t in snapshot(eager).items():
        assert torch.equal(getattr(graphed, name), t), name
