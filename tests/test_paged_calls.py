"""How the binding's paged calls hand out what a call needs, without a GPU: memory that lasts as long as its address is
used, the same on threads, limits and devices."""
import contextlib
import ctypes
import threading
import time

import pytest
import torch

from long_context_kv_gb300 import build as B
from long_context_kv_gb300 import paris as P

BF = torch.bfloat16
WORKSPACE, COUNTERS = 5000, 16


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P.load()


class Heap:
    """Memory whose lowest free bytes go first, and that takes back what is dropped: an allocator with small blocks."""

    def __init__(self):
        self.held, self.made, self.written = {}, 0, []

    def take(self, n):
        n, at = max(-(-n // 512) * 512, 512), 1 << 20
        for a, b in sorted(self.held.values()):
            if at + n <= a:
                break
            at = b
        self.made += 1
        self.held[self.made] = (at, at + n)
        return Block(self, self.made, at, n)


class Block:
    def __init__(self, heap, number, at, n):
        self.heap, self.number, self.at, self.n = heap, number, at, n

    def __del__(self):
        if self.number is not None:
            del self.heap.held[self.number]

    def data_ptr(self):
        return self.at

    def numel(self):
        return self.n

    def __getitem__(self, s):
        a, b, _ = s.indices(self.n)
        part = Block(self.heap, None, self.at + a, b - a)
        part.whole = self  # a view keeps its memory
        return part

    def zero_(self):
        self.heap.written.append((self.at, self.at + self.n))
        return self


class Calls:
    """In place of the library: what the attention is handed, and how many calls of it are under way."""

    def __init__(self, heap, pause=0.0):
        self.heap, self.pause, self.now, self.most, self.seen = heap, pause, 0, 0, []

    def paris_paged_attend_workspace(self, cache, hq, n, m):
        time.sleep(self.pause)
        ctypes.cast(n, ctypes.POINTER(ctypes.c_size_t))[0] = WORKSPACE * hq
        ctypes.cast(m, ctypes.POINTER(ctypes.c_size_t))[0] = COUNTERS
        return P.PARIS_OK

    def paris_paged_attend(self, cache, layer, q, hq, window, out, lse, ws, n, counters, m, stream):
        self.now += 1
        self.most = max(self.most, self.now)
        time.sleep(self.pause)
        for a, size in ((ws, n), (counters, m)):
            assert a % 16 == 0 and any(x <= a and a + size <= y for x, y in self.heap.held.values()), "memory given back"
        self.seen.append(((ws, ws + n), (counters, counters + m)))
        self.now -= 1
        return P.PARIS_OK


@pytest.fixture
def cache(monkeypatch):
    c = object.__new__(P.PagedCache)
    c.n_seqs, c.n_kv_heads, c._index, c.device, c._ref = 2, 2, 0, "cuda:0", None
    c._begin()
    heap = Heap()
    c.heap, c.calls, c.capturing = heap, Calls(heap), False

    def scratch(n, device, stream):
        time.sleep(c.calls.pause)
        return heap.take(n)

    monkeypatch.setattr(P, "_torch", torch)
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: None)
    monkeypatch.setattr(P, "_scratch", scratch)
    monkeypatch.setattr(P, "_on", lambda *a: None)
    monkeypatch.setattr(P, "_raw_stream", lambda index, stream: 7)
    monkeypatch.setattr(P.PagedCache, "_capturing", staticmethod(lambda stream: c.capturing))
    monkeypatch.setattr(P, "_lib", c.calls)
    return c


def attend(c, hq=4):
    q = torch.zeros(2, hq, 128, dtype=BF)
    c.paris_paged_attend(q, q)


def apart(x, y):
    return x[1] <= y[0] or y[1] <= x[0]


@pytest.mark.parametrize("capturing", [False, True])
def test_workspace_and_counters_do_not_meet(cache, capturing):
    cache.capturing = capturing
    for hq in (4, 8, 4, 2):
        before = len(cache.heap.written)
        attend(cache, hq)
        ws, counters = cache.calls.seen[-1]
        assert apart(ws, counters)
        assert ws[1] - ws[0] == WORKSPACE * hq
        zeroed = cache.heap.written[before:]
        assert all(apart(z, ws) for z in zeroed)  # nothing that a call under way may use
        if capturing:
            assert counters in zeroed  # a graph's counters are its own, zero before each replay's first use
    if capturing:
        assert not cache.heap.held  # nothing of a graph is kept, and outside of one
        cache.capturing = False
        attend(cache)
        assert cache.calls.seen[-1][1] in cache.heap.written


def test_counters_are_zeros_once_and_stay_the_stream_s_own(cache):
    for hq in (2, 4, 2, 4):
        attend(cache, hq)
    used = [counters for _, counters in cache.calls.seen]
    assert cache.heap.written == list(dict.fromkeys(used)) and used[1:] == [used[1]] * 3


def test_two_threads_take_turns_on_a_stream(cache):
    """A call is two launches with one workspace: they stay together, and first calls make one workspace."""
    cache.calls.pause, errors = 0.01, []
    start = threading.Barrier(4)

    def work():
        try:
            start.wait()
            for _ in range(5):
                attend(cache)
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    assert len(cache.calls.seen) == 20 and cache.calls.most == 1 and cache.heap.made == 1


def test_a_call_that_fails_leaves_the_others_their_turn(cache):
    q = torch.zeros(2, 4, 128, dtype=BF)
    for kw in (dict(layer=1 << 40), dict(window=1 << 70)):
        with pytest.raises(ValueError, match="out of range"):
            cache.paris_paged_attend(q, q, **kw)
    attend(cache)
    assert len(cache.calls.seen) == 1


@pytest.mark.parametrize("packed", [False, True])
def test_a_limit_of_no_rows_leaves_nothing_to_do(lib, packed):
    """Also without starts: nothing is launched, nothing refused."""
    arrays = ("k_pages", "v_pages", "k_scales", "v_scales", "table", "lens", "starts", "refs", "free_bits", "n_used", "status")
    st = P.paris_page_strides(1 << 20, 4096, 2048, 128)
    c = ctypes.byref(P.paris_paged(n_seqs=2, n_layers=2, n_kv_heads=2, head_dim=128, page_rows=16, dtype=P.PARIS_BF16, n_pages=40,
                                   max_pages=8, k=st, v=st, **{n: 4096 for n in arrays}))
    s, cu = ctypes.byref(P.paris_strides(256, 128, 1024)), ctypes.c_void_p(4096) if packed else None
    assert lib.paris_paged_store(c, 0, None, None, P.PARIS_BF16, s, s, 4, cu, 0, None) == P.PARIS_OK
    assert lib.paris_paged_read(c, 0, None, None, s, s, 4, cu, 0, None) == P.PARIS_OK
    assert lib.paris_paged_store(c, 0, None, None, P.PARIS_BF16, s, s, 4, cu, 1, None) == P.PARIS_EINVAL
    assert lib.paris_paged_read(c, 0, None, None, s, s, 4, cu, 1, None) == P.PARIS_EINVAL


class OtherDevice:
    """torch with cuda:0 as the current device."""

    class _C:
        _cuda_getDevice = staticmethod(lambda: 0)


@pytest.mark.parametrize("cls,call", [(P.PagedCache, "paris_paged_check"), (P.KV4Cache, "paris_kv4_check")])
def test_a_check_is_made_on_the_cache_s_device(monkeypatch, cls, call):
    asked = []
    monkeypatch.setattr(P, "_torch", OtherDevice)
    monkeypatch.setattr(P, "load", lambda: type("Lib", (), {call: lambda self, c: asked.append(c) or P.PARIS_OK})())
    c = object.__new__(cls)
    c._index, c._ref = 1, "the cache"
    with pytest.raises(ValueError, match="cuda:1, the current device is cuda:0"):
        getattr(c, call)()
    assert not asked
    c._index = 0
    getattr(c, call)()
    assert asked == ["the cache"]
