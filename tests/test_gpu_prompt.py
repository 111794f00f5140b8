"""Causal attention over prompts (paris_prompt_attend) and the window weights (paris_prompt_weights) against 64-bit
forms: packed and padded sequences, chunks, single tokens, empty sequences and rows that see nothing, grouped heads,
strided inputs, infinities and NaN where a query does not see them, other streams and captured graphs."""
import math

import pytest
import torch

from long_context_kv_gb300 import paris as P
from tests import kv4_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HEADS = [(1, 1), (8, 2), (3, 1), (10, 2), (16, 1), (6, 6)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_kv_gb300 import build
    build.build()
    P.load()


def make(lens_q, lens_k, hq, hkv, seed=0, amp=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q = (amp * n(sum(lens_q), hq, R.D)).to(BF)
    k = (n(sum(lens_k), hkv, R.D) + 0.5 * n(1, hkv, R.D)).to(BF)
    return q, k, n(sum(lens_k), hkv, R.D).to(BF)


def check_seq(q, k, v, out, lse, g):
    """One sequence: q, out [lq, Hq, d], k, v [lk, Hkv, d], lse [Hq, lq]."""
    lk = k.shape[0]
    for h in range(q.shape[1]):
        o, want_lse, mass, size = R.attend_rows(q[:, h].double(), k[:, h // g].double(), v[:, h // g].double())
        e = R.score_error(size, lk)
        # the result's rounding, the weights' rounding to bf16, and what the scores are off
        tol = R.HALF_BF16 * o.abs() + ((1 + R.HALF_BF16) * (R.HALF_BF16 + e))[:, None] * mass + 1e-30
        bad = ((out[:, h].double() - o).abs() > tol).nonzero()
        assert not len(bad), (h, bad[0].tolist(), out[bad[0][0], h, bad[0][1]].item(), o[tuple(bad[0])].item())
        if lse is not None:
            none = want_lse == -math.inf
            assert torch.equal(lse[h] == -math.inf, none)
            assert torch.all(out[none, h] == 0)
            d = (lse[h].double() - want_lse)[~none].abs()
            assert torch.all(d <= (e + 2 * R.U32 * want_lse.abs())[~none]), d.max()


def check(lens_q, lens_k, hq, hkv, seed=0, amp=2.0):
    q, k, v = make(lens_q, lens_k, hq, hkv, seed, amp)
    out = torch.full_like(q, 7.0)
    lse = torch.full((hq, q.shape[0]), 7.0, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts(lens_q), cu_k=R.starts(lens_k), max_q=max(lens_q),
                          max_k=max(lens_k), lse=lse)
    torch.cuda.synchronize()
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        check_seq(q[a:a + lq], k[b:b + lk], v[b:b + lk], out[a:a + lq], lse[:, a:a + lq], hq // hkv)
        a, b = a + lq, b + lk


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens", [[1], [1, 5, 33], [127, 128, 129], [0, 7, 0, 300], [64, 257, 1, 511]])
def test_packed_prompts(hq, hkv, lens):
    check(lens, lens, hq, hkv, seed=1)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (5, 1), (2, 2)])
@pytest.mark.parametrize("lens_q,lens_k", [([1], [1]), ([1], [5000]), ([1, 1, 1], [70, 1, 1300]), ([17], [4096]),
                                           ([130, 3], [131, 900]), ([300], [2000])])
def test_the_last_queries_of_longer_sequences(hq, hkv, lens_q, lens_k):
    check(lens_q, lens_k, hq, hkv, seed=2)


@pytest.mark.parametrize("lens_q,lens_k", [([5], [3]), ([300], [100]), ([4, 2], [0, 2]), ([129, 8], [1, 8])])
def test_queries_before_the_first_key_see_nothing(lens_q, lens_k):
    check(lens_q, lens_k, 4, 2, seed=3)


@pytest.mark.parametrize("amp", [0.0, 30.0])
def test_flat_and_very_peaked_scores(amp):
    check([700], [700], 4, 2, seed=4, amp=amp)


def one_hot_prompt(lens_q, lens_k, hq, hkv, amp, seed):
    """Scores so far apart that each row's softmax is one key: q, k, v, each row's key, its score and how far float32
    puts that off, on the CPU."""
    gen = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(sum(n), h, R.D, generator=gen) for n, h in ((lens_q, hq), (lens_k, hkv), (lens_k, hkv)))
    q, k, v = (q * amp).to(BF), (k * amp).to(BF), v.to(BF)
    best = torch.zeros(hq, sum(lens_q), dtype=torch.int64)
    top, off = torch.zeros(2, hq, sum(lens_q), dtype=torch.float64)
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        seen = torch.arange(lk)[None] <= torch.arange(lq)[:, None] + (lk - lq)
        for h in range(hq):
            x, y = q[a:a + lq, h].double(), k[b:b + lk, h * hkv // hq].double()
            s = (x @ y.T / math.sqrt(R.D)).masked_fill(~seen, -math.inf)
            t = s.topk(min(2, lk), dim=-1)
            # 128 float32 products and the scale put a score off by less than 2^-16 of its terms; weights of 2^-150 are 0
            off[h, a:a + lq] = 2.0 ** -16 * (x.abs() @ y.abs().T).amax(-1) / math.sqrt(R.D)
            if lk > 1:
                assert torch.all(t.values[:, 0] - t.values[:, 1] > 2 * off[h, a:a + lq] + 150 * math.log(2))
            best[h, a:a + lq], top[h, a:a + lq] = b + t.indices[:, 0], t.values[:, 0]
        a, b = a + lq, b + lk
    return q, k, v, best, top, off


@pytest.mark.parametrize("amp", [1e3, 3e4, 1e5, 1e15])
@pytest.mark.parametrize("lens_q,lens_k,hq,hkv,seed", [([3, 40, 7], [3, 40, 7], 4, 2, 1), ([4], [3000], 2, 1, 2),
                                                       ([1, 2] * 80, [1, 30] * 80, 2, 1, 2)])
def test_scores_far_apart_leave_one_key(lens_q, lens_k, hq, hkv, seed, amp):
    q, k, v, best, top, off = one_hot_prompt(lens_q, lens_k, hq, hkv, amp, seed)
    out = torch.full_like(q, 7.0, device="cuda")
    lse = torch.full((hq, q.shape[0]), 7.0, device="cuda")
    P.paris_prompt_attend(q.cuda(), k.cuda(), v.cuda(), out, cu_q=R.starts(lens_q), cu_k=R.starts(lens_k), max_q=max(lens_q),
                          max_k=max(lens_k), lse=lse)
    for h in range(hq):
        want = v[best[h], h * hkv // hq].double()
        # the weight's rounding and the result's
        assert torch.all((out[:, h].cpu().double() - want).abs() <= 2.01 * R.HALF_BF16 * want.abs())
    assert torch.all((lse.cpu().double() - top).abs() <= off)


def test_a_longer_prompt_with_a_running_maximum_that_grows():
    lens = [2500]
    q, k, v = make(lens, lens, 4, 1, seed=5)
    k *= torch.linspace(0.1, 6.0, 2500, device="cuda").to(BF)[:, None, None]
    out = torch.empty_like(q)
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts(lens), cu_k=R.starts(lens))
    check_seq(q, k, v, out, None, 4)


@pytest.mark.parametrize("hq,hkv", [(128, 1), (100, 1), (66, 2)])
def test_many_query_heads_share_a_kv_head(hq, hkv):
    check([3, 150], [3, 150], hq, hkv, seed=16)
    check([2], [700], hq, hkv, seed=17)


def test_many_sequences():
    # more than are walked by query block; some empty, one long
    gen = torch.Generator().manual_seed(18)
    lens = torch.randint(0, 50, (150,), generator=gen).tolist()
    lens[70] = 900
    check(lens, lens, 8, 2, seed=18)
    lens_q = [min(n, 3) for n in lens]
    check(lens_q, lens, 4, 4, seed=19)


def test_padded_layout_and_strided_views():
    b, hq, hkv, t = 3, 6, 2, 190
    gen = torch.Generator(device="cuda").manual_seed(6)
    fused = torch.randn(b, t, (hq + 2 * hkv) * R.D, generator=gen, device="cuda").to(BF)
    x = fused.unflatten(-1, (hq + 2 * hkv, R.D)).transpose(1, 2)     # [b, heads, t, d], a view
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    out = torch.zeros(b, t, hq, R.D, dtype=BF, device="cuda").transpose(1, 2)
    lse = torch.zeros(b, hq, t, device="cuda")
    P.paris_prompt_attend(q, k, v, out, lse=lse)
    for i in range(b):
        check_seq(q[i].transpose(0, 1), k[i].transpose(0, 1), v[i].transpose(0, 1), out[i].transpose(0, 1), lse[i], 3)


def test_packed_views_of_a_fused_projection():
    lens, hq, hkv = [200, 61], 4, 2
    fused = torch.randn(261, (hq + 2 * hkv) * R.D, device="cuda").to(BF).unflatten(-1, (-1, R.D))
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    out = torch.zeros(261, hq, R.D, dtype=BF, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts(lens), cu_k=R.starts(lens))
    check_seq(q[:200], k[:200], v[:200], out[:200], None, 2)
    check_seq(q[200:], k[200:], v[200:], out[200:], None, 2)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_a_query_does_not_see_does_not_reach_it(bad):
    # rows between and behind the sequences, and later rows of the own sequence
    hq, hkv, n = 4, 2, 400
    q, k, v = make([n], [n], hq, hkv, seed=7)
    want = torch.empty_like(q)
    cu = torch.tensor([0, 150], dtype=torch.int32, device="cuda")
    P.paris_prompt_attend(q, k, v, want, cu_q=cu, cu_k=cu, max_q=150, max_k=150)
    check_seq(q[:150], k[:150], v[:150], want[:150], None, 2)
    for first in (150, 100, 1):
        k2, v2, q2 = k.clone(), v.clone(), q.clone()
        k2[first:], v2[first:], q2[150:] = bad, bad, bad
        out = torch.full_like(q, 7.0)
        P.paris_prompt_attend(q2, k2, v2, out, cu_q=cu, cu_k=cu, max_q=150, max_k=150)
        check_seq(q[:first], k[:first], v[:first], out[:first], None, 2)
        assert torch.all(out[150:] == 7.0)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_a_chunk_does_not_see_does_not_reach_it(bad):
    # few queries over many keys: the keys are split among blocks
    q, k, v = make([20], [3100], 4, 2, seed=20)
    k[3000:], v[3000:] = bad, bad                       # past the sequence's end
    cq, ck = R.starts([20]), torch.tensor([0, 3000], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    P.paris_prompt_attend(q, k, v, out, cu_q=cq, cu_k=ck, max_q=20, max_k=3100)
    check_seq(q, k[:3000], v[:3000], out, None, 2)
    v[2990:3000] = bad                                  # seen by the last ten queries only
    P.paris_prompt_attend(q, k, v, out, cu_q=cq, cu_k=ck, max_q=20, max_k=3100)
    want, _, mass, size = R.attend_rows(q[:10, 0].double(), k[:2990, 0].double(), v[:2990, 0].double())
    tol = R.HALF_BF16 * want.abs() + ((1 + R.HALF_BF16) * (R.HALF_BF16 + R.score_error(size, 2990)))[:, None] * mass
    assert torch.all((out[:10, 0].double() - want).abs() <= tol)
    assert not torch.isfinite(out[10:]).any()


def test_non_finite_values_that_a_query_sees_reach_it():
    q, k, v = make([200], [200], 2, 1, seed=8)
    v[60, 0, 5] = math.nan
    out = torch.empty_like(q)
    cu = R.starts([200])
    P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu)
    assert torch.all(torch.isnan(out[60:, :, 5])) and not torch.isnan(out[:60]).any()
    assert not torch.isnan(out[:, :, 6:]).any()


@pytest.mark.parametrize("hq,hkv,n", [(4, 2, 90), (8, 1, 30)])
def test_not_finite_values_of_one_sequence_leave_the_others_alone(hq, hkv, n):
    # blocks that walk several sequences, clean ones in front of the others and behind them
    gen = torch.Generator().manual_seed(23)
    lens = torch.randint(1, 200, (n,), generator=gen).tolist()
    bad = n // 2
    lens[bad] = 333
    g = hq // hkv
    q, k, v = make(lens, lens, hq, hkv, seed=23)
    a = sum(lens[:bad])
    v[a + 300, 0, 9] = math.nan
    v[a + 200, hkv - 1, 5] = math.inf
    out = torch.full_like(q, 7.0)
    lse = torch.full((hq, q.shape[0]), 7.0, device="cuda")
    cu = R.starts(lens)
    P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu, max_q=max(lens), max_k=max(lens), lse=lse)
    P.paris_prompt_check()
    at = 0
    for i, m in enumerate(lens):
        s = slice(at, at + m if i != bad else at + 200)
        check_seq(q[s], k[s], v[s], out[s], lse[:, s], g)
        at += m
    rows = out[a:a + 333]
    assert torch.isnan(rows[300:, :g, 9]).all() and not torch.isnan(rows[:300, :g, 9]).any()
    assert torch.all(rows[200:, hq - g:, 5] == math.inf) and torch.isfinite(rows[:200, hq - g:, 5]).all()
    v0 = v[a:a + 333].clone()
    v0[:, :, [5, 9]] = 0
    got = rows.clone()
    got[:, :, [5, 9]] = 0
    check_seq(q[a:a + 333], k[a:a + 333], v0, got, lse[:, a:a + 333], g)


def test_a_not_finite_value_that_long_rows_see_costs_no_other_sequence():
    # 256 rows that see a NaN over 800000 keys take seconds to compute again; the blocks walk other sequences too
    n, others = 800000, 400
    gen = torch.Generator(device="cuda").manual_seed(24)
    rand = lambda rows: torch.randn(rows, 1, R.D, generator=gen, device="cuda").to(BF)  # noqa: E731
    q, k, v = rand(256 + others), rand(n + others), rand(n + others)
    v[3, 0, 7] = math.nan
    out = torch.full_like(q, 7.0)
    lse = torch.full((1, q.shape[0]), 7.0, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts([256] + [1] * others), cu_k=R.starts([n] + [1] * others), max_q=256,
                          max_k=n, lse=lse)
    P.paris_prompt_check()
    assert torch.equal(out[256:], v[n:])  # one key each
    assert torch.isnan(out[:256, 0, 7]).all() and torch.isfinite(out[:256, 0, 8:]).all()
    v[3, 0, 7] = out[252:256, 0, 7] = 0
    check_seq(q[252:256], k[:n], v[:n], out[252:256], lse[:, 252:256], 1)


@pytest.mark.parametrize("lens_q,lens_k", [([200], [200]), ([9], [3000]), ([3, 70] * 80, [3, 90] * 80)])
def test_the_largest_finite_values(lens_q, lens_k):
    # sums of two such values pass float32's range, their mean does not
    hq, hkv = 2, 1
    q, k, v = make(lens_q, lens_k, hq, hkv, seed=26, amp=0.3)
    v = (3e38 * torch.sign(v) - 1e38 * (v > 1)).to(BF)
    v[:, :, ::4] = 3.3e38
    out = torch.full_like(q, 7.0)
    lse = torch.full((hq, q.shape[0]), 7.0, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts(lens_q), cu_k=R.starts(lens_k), max_q=max(lens_q),
                          max_k=max(lens_k), lse=lse)
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        check_seq(q[a:a + lq], k[b:b + lk], v[b:b + lk], out[a:a + lq], lse[:, a:a + lq], hq // hkv)
        a, b = a + lq, b + lk


def walked(lens_q, hq, hkv):
    """Items that the fullest of 152 blocks walks: 256 rows of a KV head each."""
    tokens = 2 * (128 // (hq // hkv))
    return sum(-(-n // tokens) for n in lens_q) * hkv / 152


@pytest.mark.parametrize("n,top,hq,hkv", [(40, 650, 32, 2), (200, 280, 16, 2), (64, 200, 24, 24), (65, 200, 24, 24)])
def test_blocks_that_walk_many_items(n, top, hq, hkv):
    # by query block (up to 64 sequences) and one sequence after the other; some empty, some whose queries see nothing
    gen = torch.Generator().manual_seed(27 + n)
    lens_k = torch.randint(1, top, (n,), generator=gen).tolist()
    lens_q = [m if i % 4 else max(1, m // 3) for i, m in enumerate(lens_k)]
    lens_k[3], lens_q[5], lens_k[7] = 0, 0, max(1, lens_q[7] // 2)
    assert walked(lens_q, hq, hkv) > 8
    check(lens_q, lens_k, hq, hkv, seed=28)


def test_blocks_that_walk_many_items_of_a_padded_batch():
    b, hq, hkv, t = 21, 16, 2, 1200
    gen = torch.Generator(device="cuda").manual_seed(29)
    q, k, v = (torch.randn(b, h, t, R.D, generator=gen, device="cuda").to(BF) for h in (hq, hkv, hkv))
    assert walked([t] * b, hq, hkv) > 10
    out, lse = torch.full_like(q, 7.0), torch.zeros(b, hq, t, device="cuda")
    P.paris_prompt_attend(q, k, v, out, lse=lse)
    for i in range(b):
        check_seq(q[i].transpose(0, 1), k[i].transpose(0, 1), v[i].transpose(0, 1), out[i].transpose(0, 1), lse[i], hq // hkv)
    P.paris_prompt_check()


@pytest.mark.parametrize("lq", [32768, 300])
def test_prompts_of_32768_keys(lq):
    lk, hq, hkv = 32768, 4, 2
    q, k, v = make([lq], [lk], hq, hkv, seed=30)
    out, lse = torch.full_like(q, 7.0), torch.zeros(hq, lq, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts([lq]), cu_k=R.starts([lk]), lse=lse)
    rows = sorted({*range(0, lq, max(1, lq // 40)), 1, 127, 128, 129, 255, 256, lq - 2, lq - 1})
    for i in rows:
        n = i + 1 + lk - lq
        check_seq(q[i:i + 1], k[:n], v[:n], out[i:i + 1], lse[:, i:i + 1], hq // hkv)


@pytest.mark.parametrize("lens_q,lens_k", [([200], [200]), ([9], [3000]), ([3, 70] * 80, [3, 90] * 80)])
def test_scores_of_minus_infinity_have_no_weight(lens_q, lens_k):
    # the first keys of each sequence, and NaN values that the last query alone sees: the rows before it are computed twice
    hq, hkv = 2, 1
    q, k, v = make(lens_q, lens_k, hq, hkv, seed=32)
    q[:, :, 0] = 1.0
    a = b = 0
    for lq, lk in zip(lens_q, lens_k):
        k[b:b + lk // 2, :, 0] = -math.inf
        v[b + lk - 1] = math.nan
        b += lk
    out = torch.full_like(q, 7.0)
    lse = torch.full((hq, q.shape[0]), 7.0, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts(lens_q), cu_k=R.starts(lens_k), max_q=max(lens_q),
                          max_k=max(lens_k), lse=lse)
    b = 0
    for lq, lk in zip(lens_q, lens_k):
        none = lk // 2  # left out: the result is that of the other keys, and 0 for queries that see no other
        see = lk - lq
        if lq > 1:
            first = max(0, none - see)  # the first query that sees a key with a weight
            assert torch.all(out[a:a + first] == 0) and torch.all(lse[:, a:a + first] == -math.inf)
            check_seq(q[a + first:a + lq - 1], k[b + none:b + lk - 1], v[b + none:b + lk - 1], out[a + first:a + lq - 1],
                      lse[:, a + first:a + lq - 1], hq // hkv)
        assert torch.isnan(out[a + lq - 1]).all()
        a, b = a + lq, b + lk


def test_rows_that_no_sequence_owns_are_left_alone():
    q, k, v = make([300], [300], 2, 2, seed=9)
    cu = torch.tensor([20, 90, 90, 250], dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    lse = torch.full((2, 300), 3.0, device="cuda")
    P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu, max_q=160, max_k=160, lse=lse)
    for a, b in ((20, 90), (90, 250)):
        check_seq(q[a:b], k[a:b], v[a:b], out[a:b], lse[:, a:b], 1)
    for a, b in ((0, 20), (250, 300)):
        assert torch.all(out[a:b] == 3.0) and torch.all(lse[:, a:b] == 3.0)


def test_starts_outside_the_axis_are_clamped():
    q, k, v = make([64], [64], 2, 1, seed=10)
    cu = torch.tensor([-5, 40, 30, 1000], dtype=torch.int32, device="cuda")  # rows 0-40, none, 30-64
    out = torch.zeros_like(q)
    P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu)
    check_seq(q[:30], k[:30], v[:30], out[:30], None, 2)


def test_no_sequences_and_no_rows():
    e = torch.empty(0, 4, R.D, dtype=BF, device="cuda")
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.paris_prompt_attend(e, e[:, :2], e[:, :2], e.clone(), cu_q=z, cu_k=z)
    q, k, v = make([9], [0], 4, 2)
    out = torch.full_like(q, 5.0)
    P.paris_prompt_attend(q, k, v, out, cu_q=R.starts([9]), cu_k=R.starts([0]))
    assert torch.all(out == 0)


def test_other_stream_and_a_captured_graph_with_new_starts():
    q, k, v = make([600], [600], 8, 2, seed=11)
    cu = R.starts([600])
    s = torch.cuda.Stream()
    want, got = torch.zeros_like(q), torch.zeros_like(q)
    P.paris_prompt_attend(q, k, v, want, cu_q=cu, cu_k=cu)
    s.wait_stream(torch.cuda.current_stream())
    P.paris_prompt_attend(q, k, v, got, cu_q=cu, cu_k=cu, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(want, got)
    cu2 = torch.tensor([0, 600], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.paris_prompt_attend(q, k, v, got, cu_q=cu2, cu_k=cu2)
    for n in (600, 129, 1):
        cu2.copy_(torch.tensor([0, n]))
        got.fill_(2.0)
        graph.replay()
        torch.cuda.synchronize()
        check_seq(q[:n], k[:n], v[:n], got[:n], None, 4)
        assert torch.all(got[n:] == 2.0)


def test_two_calls_give_the_same_bits():
    q, k, v = make([1, 900], [7000, 900], 8, 2, seed=12)
    cu, ck = R.starts([1, 900]), R.starts([7000, 900])
    outs = []
    for _ in range(3):
        outs.append(torch.zeros_like(q))
        P.paris_prompt_attend(q, k, v, outs[-1], cu_q=cu, cu_k=ck, max_q=900, max_k=7000)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------ window weights
def weights_ref(q, k, lse, g, window):
    """[Hkv, lk] and the bound of each: q [lq, Hq, d], k [lk, Hkv, d], lse [Hq, lq]."""
    lq, lk = q.shape[0], k.shape[0]
    w = min(window, lq)
    out = torch.zeros(k.shape[1], lk, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for h in range(q.shape[1]):
        qs, ks = q[lq - w:, h].double(), k[:, h // g].double()
        i = torch.arange(lq - w, lq, device=q.device)[:, None] + (lk - lq)
        seen = (torch.arange(lk, device=q.device)[None] <= i) & (lse[h, lq - w:, None] != -math.inf)
        ls = lse[h, lq - w:, None].double()
        p = torch.where(seen, torch.exp(qs @ ks.T / math.sqrt(R.D) - ls.nan_to_num(neginf=0.0)), 0.0)
        e = 128 * R.U32 * (qs.abs() @ ks.abs().T) / math.sqrt(R.D) + 2 * R.U32 * ls.nan_to_num(neginf=0.0).abs() + 2.0 ** -16
        out[h // g] += p.sum(0)
        tol[h // g] += (p * e).sum(0)
    return out, tol + out * (w * g * R.U32)


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("lens,window", [([1], 1), ([5, 1, 40], 8), ([0, 200, 129], 32), ([700], 64), ([90], 500),
                                         ([30], 0)])
def test_window_weights(hq, hkv, lens, window):
    q, k, v = make(lens, lens, hq, hkv, seed=13)
    cu = R.starts(lens)
    lse = torch.zeros(hq, q.shape[0], device="cuda")
    P.paris_prompt_attend(q, k, v, torch.empty_like(q), cu_q=cu, cu_k=cu, lse=lse)
    got = torch.full((hkv, k.shape[0]), 9.0, device="cuda")
    P.paris_prompt_weights(q, k, lse, got, window=window, cu_q=cu, cu_k=cu, max_k=max(lens))
    a = 0
    for n in lens:
        want, tol = weights_ref(q[a:a + n], k[a:a + n], lse[:, a:a + n], hq // hkv, window)
        assert torch.all((got[:, a:a + n].double() - want).abs() <= tol + 1e-30)
        if n and window:
            assert abs(got[:, a:a + n].sum().item() - hq * min(n, window)) < 1e-3 * hq * min(n, window)
        a += n


def test_window_weights_of_chunks_padded_layout_and_queries_that_see_nothing():
    q, k, v = make([50, 9], [300, 4], 4, 2, seed=14)
    cq, ck = R.starts([50, 9]), R.starts([300, 4])
    lse = torch.zeros(4, 59, device="cuda")
    P.paris_prompt_attend(q, k, v, torch.empty_like(q), cu_q=cq, cu_k=ck, lse=lse)
    got = torch.full((2, 304), 9.0, device="cuda")
    P.paris_prompt_weights(q, k, lse, got, window=20, cu_q=cq, cu_k=ck)
    for (a, b), (c, d) in (((0, 50), (0, 300)), ((50, 59), (300, 304))):
        want, tol = weights_ref(q[a:b], k[c:d], lse[:, a:b], 2, 20)
        assert torch.all((got[:, c:d].double() - want).abs() <= tol + 1e-30)
    x = torch.randn(2, 5, 77, R.D, device="cuda").to(BF)
    qd, kd = x[:, :4], x[:, 4:]
    lse = torch.zeros(2, 4, 77, device="cuda")
    P.paris_prompt_attend(qd, kd, kd, torch.empty_like(qd), lse=lse)
    got = torch.full((2, 1, 77), 9.0, device="cuda")
    P.paris_prompt_weights(qd, kd, lse, got, window=5)
    for i in range(2):
        want, tol = weights_ref(qd[i].transpose(0, 1), kd[i].transpose(0, 1), lse[i], 4, 5)
        assert torch.all((got[i].double() - want).abs() <= tol + 1e-30)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("hq,hkv,n,window", [(4, 2, 300, 32), (8, 2, 400, 64), (1, 1, 400, 32), (4, 1, 700, 200)])
def test_queries_whose_lse_says_so_add_nothing(hq, hkv, n, window, bad):
    # padding at the end of a batch's prompts: lse = -inf there, and anything in q
    q, k, v = make([n], [n], hq, hkv, seed=25)
    cu = R.starts([n])
    lse = torch.zeros(hq, n, device="cuda")
    P.paris_prompt_attend(q, k, v, torch.empty_like(q), cu_q=cu, cu_k=cu, lse=lse)
    lse[:, n - 5:] = -math.inf
    lse[0, n - window] = -math.inf
    want, tol = weights_ref(q, k, lse, hq // hkv, window)
    q[n - 5:] = bad
    q[n - window, 0] = bad
    got = torch.full((hkv, n), 9.0, device="cuda")
    P.paris_prompt_weights(q, k, lse, got, window=window, cu_q=cu, cu_k=cu)
    assert torch.all((got.double() - want).abs() <= tol + 1e-30)


def test_window_weights_of_many_query_heads_and_sequences():
    for lens, hq, hkv, window in (([40, 300], 128, 1, 7), ([5] * 70 + [400], 6, 2, 4)):
        q, k, v = make(lens, lens, hq, hkv, seed=21)
        cu = R.starts(lens)
        lse = torch.zeros(hq, q.shape[0], device="cuda")
        P.paris_prompt_attend(q, k, v, torch.empty_like(q), cu_q=cu, cu_k=cu, lse=lse)
        got = torch.full((hkv, k.shape[0]), 9.0, device="cuda")
        P.paris_prompt_weights(q, k, lse, got, window=window, cu_q=cu, cu_k=cu, max_k=max(lens))
        a = 0
        for n in lens:
            want, tol = weights_ref(q[a:a + n], k[a:a + n], lse[:, a:a + n], hq // hkv, window)
            assert torch.all((got[:, a:a + n].double() - want).abs() <= tol + 1e-30)
            a += n


@pytest.mark.parametrize("lens,hkv", [([0, 3] * 45 + [200], 2), ([300] + [0] * 60 + [2, 700], 2), ([260, 1], 80)])
def test_window_weights_of_uneven_sequences(lens, hkv):
    q, k, v = make(lens, lens, hkv, hkv, seed=22)
    cu = R.starts(lens)
    lse = torch.zeros(hkv, q.shape[0], device="cuda")
    P.paris_prompt_attend(q, k, v, torch.empty_like(q), cu_q=cu, cu_k=cu, lse=lse)
    got = torch.full((hkv, k.shape[0]), 9.0, device="cuda")
    P.paris_prompt_weights(q, k, lse, got, window=6, cu_q=cu, cu_k=cu, max_k=max(lens))
    a = 0
    for n in lens:
        want, tol = weights_ref(q[a:a + n], k[a:a + n], lse[:, a:a + n], 1, 6)
        assert torch.all((got[:, a:a + n].double() - want).abs() <= tol + 1e-30)
        a += n


def test_window_weights_in_a_captured_graph_with_new_starts():
    hq, hkv, total = 8, 2, 700
    q, k, v = make([total], [total], hq, hkv, seed=31)
    cu = torch.tensor([0, 300, total], dtype=torch.int32, device="cuda")
    lse = torch.zeros(hq, total, device="cuda")
    got = torch.zeros(hkv, total, device="cuda")
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        P.paris_prompt_attend(q, k, v, out, cu_q=cu, cu_k=cu, lse=lse)
        P.paris_prompt_weights(q, k, lse, got, window=40, cu_q=cu, cu_k=cu)
    for ends in ((300, 700), (1, 129), (0, 512)):
        cu.copy_(torch.tensor([0, *ends]))
        got.fill_(9.0)
        graph.replay()
        a = 0
        for e in ends:
            want, tol = weights_ref(q[a:e], k[a:e], lse[:, a:e], hq // hkv, 40)
            assert torch.all((got[:, a:e].double() - want).abs() <= tol + 1e-30)
            a = e
        assert torch.all(got[:, ends[-1]:] == 9.0)


def test_window_weights_do_not_see_other_rows():
    q, k, v = make([100], [100], 4, 2, seed=15)
    cu = torch.tensor([0, 60], dtype=torch.int32, device="cuda")
    lse = torch.zeros(4, 100, device="cuda")
    P.paris_prompt_attend(q, k, v, torch.empty_like(q), cu_q=cu, cu_k=cu, lse=lse)
    k[60:], q[60:], lse[:, 60:] = math.nan, math.nan, math.nan
    got = torch.full((2, 100), 9.0, device="cuda")
    P.paris_prompt_weights(q, k, lse, got, window=16, cu_q=cu, cu_k=cu)
    want, tol = weights_ref(q[:60], k[:60], lse[:, :60], 2, 16)
    assert torch.all((got[:, :60].double() - want).abs() <= tol + 1e-30)
    assert torch.all(got[:, 60:] == 9.0)


def test_two_calls_at_once_on_two_streams():
    q, k, v = make([500, 900], [500, 900], 8, 2, seed=22)
    cu = R.starts([500, 900])
    want, lse = torch.zeros_like(q), torch.zeros(8, 1400, device="cuda")
    P.paris_prompt_attend(q, k, v, want, cu_q=cu, cu_k=cu, lse=lse)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.zeros_like(q) for _ in range(6)]
    ws = [torch.zeros(2, 1400, device="cuda") for _ in range(3)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        P.paris_prompt_attend(q, k, v, o, cu_q=cu, cu_k=cu, stream=streams[i % 3])
        P.paris_prompt_weights(q, k, lse, ws[i % 3], window=16, cu_q=cu, cu_k=cu, stream=streams[i % 3])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(w, ws[0]) for w in ws)
    P.paris_prompt_check()
