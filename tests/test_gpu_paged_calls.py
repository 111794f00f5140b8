"""The paged cache's calls in the ways in which programs make them: captured, on threads, with limits, with arrays that
do not agree, with values that are not finite.  Against the direct call, lists, or the definition in 64 bits."""
import math
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
