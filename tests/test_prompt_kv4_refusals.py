"""What the prompt calls and the 4-bit cache refuse, before any device work: in the C ABI (sizes, strides, alignment,
missing pointers) and in the Python binding (shapes, types, devices)."""
import ctypes
import re

import pytest
import torch

from long_context_kv_gb300 import build as B
from long_context_kv_gb300 import paris as P

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P.load()


def prompt(**kw):
    s = P.paris_strides(1024, 128, 1 << 20)
    p = P.paris_prompt(n_seqs=2, n_q_heads=8, n_kv_heads=2, head_dim=128, rows_q=64, rows_k=64, cu_q=4096, cu_k=4096,
                       max_q=64, max_k=64, q=s, k=s, v=s, out=s)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("bad,text", [
    (dict(head_dim=64), "head_dim"), (dict(n_seqs=-1), "n_seqs"), (dict(n_seqs=65536), "n_seqs"),
    (dict(n_kv_heads=0), "n_q_heads"), (dict(n_q_heads=7), "n_q_heads"), (dict(n_q_heads=258), "128 per KV head"),
    (dict(cu_q=None), "both"), (dict(rows_q=-1), "rows_q"), (dict(rows_k=1 << 31), "rows_k"), (dict(max_q=-1), "max_q"),
    (dict(q=P.paris_strides(1023, 128, 0)), "q: the token stride"),
    (dict(k=P.paris_strides(1024, 64, 0)), "k: the head stride"),
    (dict(v=P.paris_strides(0, 128, 0)), "v: the token stride"),
    (dict(out=P.paris_strides(-1024, 128, 0)), "out: the token stride"),
    (dict(cu_q=None, cu_k=None, q=P.paris_strides(1024, 128, 4)), "q: the seq stride"),
    (dict(k=P.paris_strides(1 << 31, 128, 0)), "k: the token stride"),
])
def test_prompt_descriptions(lib, bad, text):
    n = ctypes.c_size_t(5)
    assert lib.paris_prompt_workspace(ctypes.byref(prompt(**bad)), ctypes.byref(n)) == P.PARIS_EINVAL
    assert text in lib.paris_last_error(None).decode()
    a = ctypes.c_void_p(4096)
    assert lib.paris_prompt_attend(ctypes.byref(prompt(**bad)), a, a, a, P.PARIS_BF16, a, None, None, 0,
                                   None) == P.PARIS_EINVAL


def test_prompt_pointers_types_and_workspace(lib):
    a, odd = ctypes.c_void_p(4096), ctypes.c_void_p(4100)
    call = lambda p, q, k, v, t, o, ws=None, n=0: lib.paris_prompt_attend(  # noqa: E731
        ctypes.byref(p), q, k, v, t, o, None, ws, n, None)
    assert call(prompt(), a, a, a, P.PARIS_F32, a) == P.PARIS_EINVAL
    for args in ((None, a, a, a), (a, None, a, a), (a, a, None, a), (a, a, a, None)):
        assert call(prompt(), *args[:3], P.PARIS_BF16, args[3]) == P.PARIS_EINVAL
        assert "NULL" in lib.paris_last_error(None).decode()
    for i in range(4):
        args = [a] * 4
        args[i] = odd
        assert call(prompt(), *args[:3], P.PARIS_BF16, args[3]) == P.PARIS_EINVAL
        assert "aligned" in lib.paris_last_error(None).decode()
    assert lib.paris_prompt_workspace(ctypes.byref(prompt()), None) == P.PARIS_EINVAL
    assert call(prompt(n_seqs=0), None, None, None, P.PARIS_BF16, None) == P.PARIS_OK  # nothing to do
    w = lambda p, window: lib.paris_prompt_weights(ctypes.byref(p), a, a, P.PARIS_BF16, a, window, a, None)  # noqa: E731
    assert w(prompt(), -1) == P.PARIS_EINVAL
    assert w(prompt(), (1 << 24) + 1) == P.PARIS_EINVAL
    assert w(prompt(n_seqs=0), 4) == P.PARIS_OK
    assert lib.paris_prompt_weights(ctypes.byref(prompt()), a, a, P.PARIS_F32, a, 1, a, None) == P.PARIS_EINVAL
    assert lib.paris_prompt_weights(ctypes.byref(prompt()), a, a, P.PARIS_BF16, None, 1, a, None) == P.PARIS_EINVAL


def cache(**kw):
    arrays = ("k_codes", "v_codes", "k_scales", "v_scales", "weights", "positions", "lens", "next_pos", "counters", "status")
    c = P.paris_kv4(batch=2, n_kv_heads=2, head_dim=128, max_rows=256, **{n: 4096 for n in arrays})
    for k, v in kw.items():
        setattr(c, k, v)
    return c


@pytest.mark.parametrize("bad,text", [
    (dict(head_dim=64), "head_dim"), (dict(batch=0), "batch"), (dict(n_kv_heads=0), "n_kv_heads"),
    (dict(batch=40000), "65535"), (dict(max_rows=0), "max_rows"), (dict(max_rows=1 << 31), "max_rows"),
    (dict(lens=None), "NULL"), (dict(k_codes=None), "NULL"), (dict(status=None), "NULL"), (dict(v_scales=4104), "aligned"),
    (dict(weights=4104), "aligned"),
])
def test_cache_descriptions(lib, bad, text):
    c, n, a = ctypes.byref(cache(**bad)), ctypes.c_size_t(), ctypes.c_void_p(4096)
    s = ctypes.byref(P.paris_strides(256, 128, 256))
    for st in (lib.paris_kv4_workspace(c, 4, 0, ctypes.byref(n)), lib.paris_kv4_evict_workspace(c, ctypes.byref(n)),
               lib.paris_kv4_append(c, a, a, P.PARIS_BF16, None), lib.paris_kv4_read(c, a, a, 4, None),
               lib.paris_kv4_store(c, a, a, P.PARIS_BF16, s, s, 4, a, 4, None, None),
               lib.paris_kv4_attend(c, a, P.PARIS_BF16, 4, 0, a, a, 1 << 30, None),
               lib.paris_kv4_evict(c, 8, 0, 0, a, 1 << 30, None), lib.paris_kv4_check(c)):
        assert st == P.PARIS_EINVAL
        assert text in lib.paris_last_error(None).decode()


def test_cache_calls(lib):
    c, n, a, odd = ctypes.byref(cache()), ctypes.c_size_t(), ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    s, thin = ctypes.byref(P.paris_strides(256, 128, 1024)), ctypes.byref(P.paris_strides(8, 128, 1024))
    E = P.PARIS_EINVAL
    assert lib.paris_kv4_store(c, a, a, 7, s, s, 4, a, 4, None, None) == E
    assert lib.paris_kv4_store(c, a, a, P.PARIS_BF16, None, s, 4, a, 4, None, None) == E
    assert lib.paris_kv4_store(c, a, a, P.PARIS_BF16, s, thin, 4, a, 4, None, None) == E
    assert lib.paris_kv4_store(c, a, a, P.PARIS_BF16, s, s, -1, a, 4, None, None) == E
    assert lib.paris_kv4_store(c, a, a, P.PARIS_BF16, s, s, 4, a, -1, None, None) == E
    assert lib.paris_kv4_store(c, None, a, P.PARIS_BF16, s, s, 4, a, 4, None, None) == E
    assert lib.paris_kv4_store(c, a, odd, P.PARIS_BF16, s, s, 4, a, 4, None, None) == E
    assert lib.paris_kv4_store(c, None, None, P.PARIS_BF16, s, s, 0, a, 4, None, None) == P.PARIS_OK
    for hq in (0, 1, 3, 34):
        assert lib.paris_kv4_workspace(c, hq, 0, ctypes.byref(n)) == E
    assert lib.paris_kv4_workspace(c, 8, 0, ctypes.byref(n)) == P.PARIS_OK and n.value > 0
    plain = n.value
    assert lib.paris_kv4_workspace(c, 8, 1, ctypes.byref(n)) == P.PARIS_OK and n.value == plain + 2 * 8 * 256 * 4
    assert lib.paris_kv4_attend(c, a, P.PARIS_BF16, 8, 0, a, a, plain - 1, None) == E
    assert "workspace" in lib.paris_last_error(None).decode()
    assert lib.paris_kv4_attend(c, a, P.PARIS_BF16, 8, 0, a, None, plain, None) == E
    assert lib.paris_kv4_attend(c, None, P.PARIS_BF16, 8, 0, a, a, plain, None) == E
    assert lib.paris_kv4_attend(c, odd, P.PARIS_BF16, 8, 0, a, a, plain, None) == E
    assert lib.paris_kv4_attend(c, a, 9, 8, 0, a, a, plain, None) == E
    assert lib.paris_kv4_evict_workspace(c, ctypes.byref(n)) == P.PARIS_OK
    for keep, sink, recent in ((0, 0, 0), (8, -1, 0), (8, 0, -1), (8, 9, 0), (8, 4, 5), (8, 0, 1 << 62)):
        assert lib.paris_kv4_evict(c, keep, sink, recent, a, n.value, None) == E
    assert lib.paris_kv4_evict(c, 8, 0, 0, a, n.value - 1, None) == E
    assert lib.paris_kv4_evict(c, 256, 0, 0, a, n.value, None) == P.PARIS_OK  # no sequence can have more
    assert lib.paris_kv4_read(c, a, a, 257, None) == E and lib.paris_kv4_read(c, a, None, 4, None) == E
    assert lib.paris_kv4_read(c, a, a, 0, None) == P.PARIS_OK
    assert lib.paris_kv4_check(None) == E


def test_struct_fields_match_the_header():
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "paris.h")).read(), flags=re.S)
    for cls in (P.paris_strides, P.paris_prompt, P.paris_kv4):
        body = re.search(r"typedef struct \{([^{}]*)\} " + cls.__name__ + ";", src).group(1)
        names = re.findall(r"([a-z_]+)\s*[,;]", body)
        assert names == [f[0] for f in cls._fields_], cls.__name__


def test_binding_checks_shapes_types_and_devices(lib):
    q, k = torch.zeros(10, 4, 128, dtype=BF), torch.zeros(10, 2, 128, dtype=BF)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        P.paris_prompt_attend(q, k, k, q.clone(), cu_q=cu, cu_k=cu)
    with pytest.raises(ValueError, match="both"):
        P.paris_prompt_attend(q, k, k, q.clone(), cu_q=cu)
    with pytest.raises(TypeError, match="bfloat16"):
        P.paris_prompt_attend(q.float(), k, k, q.clone(), cu_q=cu, cu_k=cu)
    with pytest.raises(ValueError, match="CUDA"):
        P.KV4Cache.create(1, 2, 16, device="cpu")
    z = torch.zeros(1, 2, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="k_codes"):
        P.KV4Cache(z[..., :32], z, z, z, z, z, z, z)
    with pytest.raises((ValueError, TypeError)):
        P.KV4Cache(z, z, z, z, z, z, z, z)


def test_numbers_that_a_c_argument_does_not_hold(lib):
    # ctypes would take 2^32 + 4 for 4, and 2^64 + 1 for 1
    q, k = torch.zeros(10, 4, 128, dtype=BF), torch.zeros(10, 2, 128, dtype=BF)
    c = object.__new__(P.KV4Cache)
    for window in (1 << 31, (1 << 32) + 4, -(1 << 32) + 4):
        with pytest.raises(ValueError, match="window.*out of range"):
            P.paris_prompt_weights(q, k, None, None, window=window)
    for big in ((1 << 64) + 1, 1 << 63, -(1 << 64) + 1):
        with pytest.raises(ValueError, match="max_new.*out of range"):
            c.paris_kv4_store(k, k, cu=k, max_new=big)
        for args, name in (((big, 0, 0), "keep"), ((4, big, 0), "sink"), ((4, 0, big), "recent")):
            with pytest.raises(ValueError, match=name + ".*out of range"):
                c.paris_kv4_evict(*args)


def test_packed_descriptions_are_the_structures():
    assert P._PROMPT.size == ctypes.sizeof(P.paris_prompt)
    assert P._STRIDES.size == ctypes.sizeof(P.paris_strides)
    p = P.paris_prompt.from_buffer_copy(P._PROMPT.pack(*range(1, 23)))
    got = [p.n_seqs, p.n_q_heads, p.n_kv_heads, p.head_dim, p.rows_q, p.rows_k, p.cu_q, p.cu_k, p.max_q, p.max_k]
    for x in (p.q, p.k, p.v, p.out):
        got += [x.token, x.head, x.seq]
    assert got == list(range(1, 23))
