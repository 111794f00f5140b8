"""What the paged cache refuses, before any device work: in the C ABI (sizes, strides, alignment, missing pointers) and
in the Python binding (shapes, types, devices)."""
import ctypes
import os
import re

import pytest
import torch

from long_context_kv_gb300 import build as B
from long_context_kv_gb300 import paris as P

BF = torch.bfloat16
E = P.PARIS_EINVAL


@pytest.fixture(scope="module")
def lib():
    B.build()
    return P.load()


def cache(**kw):
    arrays = ("k_pages", "v_pages", "k_scales", "v_scales", "table", "lens", "starts", "refs", "free_bits", "n_used", "status")
    s = P.paris_page_strides(1 << 20, 4096, 2048, 128)
    c = P.paris_paged(n_seqs=2, n_layers=2, n_kv_heads=2, head_dim=128, page_rows=16, dtype=P.PARIS_BF16, n_pages=40,
                      max_pages=8, k=s, v=s, **{n: 4096 for n in arrays})
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD = [
    (dict(head_dim=64), "head_dim"), (dict(n_seqs=0), "n_seqs"), (dict(n_seqs=4097), "n_seqs"),
    (dict(n_kv_heads=0), "n_kv_heads"), (dict(n_seqs=4096, n_kv_heads=16), "65535"), (dict(n_layers=0), "n_layers"),
    (dict(page_rows=8), "page_rows"), (dict(page_rows=48), "page_rows"), (dict(page_rows=512), "page_rows"),
    (dict(dtype=P.PARIS_F32), "dtype"), (dict(n_pages=0), "n_pages"), (dict(n_pages=(1 << 21) + 1), "n_pages"),
    (dict(n_seqs=4096, n_kv_heads=1, max_pages=(1 << 21) + 1), "2^37"), (dict(max_pages=0), "max_pages"), (dict(max_pages=(1 << 26) + 1), "max_pages"), (dict(lens=None), "NULL"),
    (dict(k_pages=None), "NULL"), (dict(status=None), "NULL"), (dict(dtype=P.PARIS_E4M3, k_scales=None), "NULL"),
    (dict(v_pages=4104), "aligned"), (dict(dtype=P.PARIS_E4M3, v_scales=4104), "aligned"),
    (dict(k=P.paris_page_strides(0, 4096, 2048, 128)), "k_pages: the layer stride"),
    (dict(k=P.paris_page_strides(1 << 20, 4100, 2048, 128)), "k_pages: the page stride"),
    (dict(v=P.paris_page_strides(1 << 20, 4096, -2048, 128)), "v_pages: the head stride"),
    (dict(v=P.paris_page_strides(1 << 20, 4096, 2048, 64)), "v_pages: the row stride"),
    (dict(v=P.paris_page_strides(1 << 38, 4096, 2048, 128)), "v_pages: the layer stride"),
    (dict(dtype=P.PARIS_E4M3, k=P.paris_page_strides(1 << 20, 4096, 2048, 136)), "k_pages: the row stride"),
]


@pytest.mark.parametrize("bad,text", BAD)
def test_cache_descriptions(lib, bad, text):
    c, n, m, a = ctypes.byref(cache(**bad)), ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_void_p(4096)
    s, big = ctypes.byref(P.paris_strides(256, 128, 256)), 1 << 40
    for st in (lib.paris_paged_grow(c, a, None), lib.paris_paged_store(c, 0, a, a, P.PARIS_BF16, s, s, 4, a, 4, None),
               lib.paris_paged_read(c, 0, a, a, s, s, 4, a, 4, None),
               lib.paris_paged_attend_workspace(c, 4, ctypes.byref(n), ctypes.byref(m)),
               lib.paris_paged_attend(c, 0, a, 4, 0, a, None, a, big, a, big, None),
               lib.paris_paged_fork_workspace(c, 1, ctypes.byref(n)), lib.paris_paged_fork(c, a, a, None, 1, a, big, None),
               lib.paris_paged_free(c, a, None, 1, a, big, None), lib.paris_paged_compact_workspace(c, ctypes.byref(n)),
               lib.paris_paged_compact(c, a, big, None), lib.paris_paged_check(c)):
        assert st == E
        assert text in lib.paris_last_error(None).decode()


def test_cache_calls(lib):
    c, a, odd = ctypes.byref(cache()), ctypes.c_void_p(4096), ctypes.c_void_p(4104)
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    s, thin = ctypes.byref(P.paris_strides(256, 128, 1024)), ctypes.byref(P.paris_strides(8, 128, 1024))
    bf = P.PARIS_BF16
    assert lib.paris_paged_grow(c, None, None) == E
    for layer in (-1, 2):
        assert lib.paris_paged_store(c, layer, a, a, bf, s, s, 4, a, 4, None) == E
        assert "layer" in lib.paris_last_error(None).decode()
        assert lib.paris_paged_read(c, layer, a, a, s, s, 4, a, 4, None) == E
        assert lib.paris_paged_attend(c, layer, a, 4, 0, a, None, a, 1 << 30, a, 1 << 30, None) == E
    for dtype in (7, P.PARIS_E4M3):
        assert lib.paris_paged_store(c, 0, a, a, dtype, s, s, 4, a, 4, None) == E
    assert lib.paris_paged_store(c, 0, a, a, bf, None, s, 4, a, 4, None) == E
    assert lib.paris_paged_store(c, 0, a, a, bf, s, thin, 4, a, 4, None) == E
    assert lib.paris_paged_store(c, 0, a, a, bf, s, s, -1, a, 4, None) == E
    assert lib.paris_paged_store(c, 0, a, a, bf, s, s, 4, a, -1, None) == E
    assert lib.paris_paged_store(c, 0, None, a, bf, s, s, 4, a, 4, None) == E
    assert lib.paris_paged_store(c, 0, a, odd, bf, s, s, 4, a, 4, None) == E
    assert lib.paris_paged_read(c, 0, a, odd, s, s, 4, a, 4, None) == E
    for call in (lib.paris_paged_store(c, 0, None, None, bf, s, s, 0, a, 4, None),
                 lib.paris_paged_read(c, 0, None, None, s, s, 4, a, 0, None),
                 lib.paris_paged_fork(c, None, None, None, 0, None, 0, None),
                 lib.paris_paged_free(c, None, None, 0, None, 0, None)):
        assert call == P.PARIS_OK  # nothing to do
    for hq in (0, 1, 3, 258):
        assert lib.paris_paged_attend_workspace(c, hq, ctypes.byref(n), ctypes.byref(m)) == E
    assert lib.paris_paged_attend_workspace(c, 8, ctypes.byref(n), ctypes.byref(m)) == P.PARIS_OK and n.value and m.value
    call = lambda q=a, hq=8, w=0, o=a, ws=a, nb=n.value, cn=a, mb=m.value: lib.paris_paged_attend(  # noqa: E731
        c, 0, q, hq, w, o, None, ws, nb, cn, mb, None)
    for kw in (dict(q=None), dict(o=None), dict(q=odd), dict(o=odd), dict(hq=7), dict(w=-1), dict(ws=None), dict(ws=odd),
               dict(nb=n.value - 1), dict(cn=None), dict(cn=odd), dict(mb=m.value - 1)):
        assert call(**kw) == E, kw
    for k in (-1, 3):
        assert lib.paris_paged_fork_workspace(c, k, ctypes.byref(n)) == E
        assert lib.paris_paged_fork(c, a, a, None, k, a, 1 << 30, None) == E
        assert lib.paris_paged_free(c, a, None, k, a, 1 << 30, None) == E
    assert lib.paris_paged_fork_workspace(c, 2, ctypes.byref(n)) == P.PARIS_OK
    for args in ((None, a, None, 2, a, n.value), (a, None, None, 2, a, n.value), (a, a, None, 2, None, n.value),
                 (a, a, None, 2, odd, n.value), (a, a, None, 2, a, n.value - 1)):
        assert lib.paris_paged_fork(c, *args, None) == E
    assert lib.paris_paged_free(c, None, None, 2, a, n.value, None) == E
    assert lib.paris_paged_free(c, a, a, 2, a, n.value - 1, None) == E
    assert lib.paris_paged_free(c, a, a, 2, None, n.value, None) == E
    assert lib.paris_paged_compact_workspace(c, ctypes.byref(n)) == P.PARIS_OK
    assert lib.paris_paged_compact(c, a, n.value - 1, None) == E
    assert lib.paris_paged_compact(c, None, n.value, None) == E
    assert lib.paris_paged_check(None) == E
    for f, args in ((lib.paris_paged_attend_workspace, (8, None, None)), (lib.paris_paged_fork_workspace, (1, None)),
                    (lib.paris_paged_compact_workspace, (None,))):
        assert f(c, *args) == E


def test_struct_fields_match_the_header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "paris.h")).read(), flags=re.S)
    for cls in (P.paris_page_strides, P.paris_paged):
        body = re.search(r"typedef struct \{([^{}]*)\} " + cls.__name__ + ";", src).group(1)
        names = re.findall(r"([a-z_]+)\s*[,;]", body)
        assert names == [f[0] for f in cls._fields_], cls.__name__


def test_binding_checks_shapes_types_and_devices(lib):
    kw = dict(n_seqs=2, n_kv_heads=2, n_pages=33, max_pages=4)
    with pytest.raises(ValueError, match="CUDA"):
        P.PagedCache.create(device="cpu", **kw)
    with pytest.raises(TypeError, match="dtype"):
        P.PagedCache.create(device="cpu", dtype=torch.float16, **kw)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(1, 33, 2, 16, 128, dtype=BF)
    good = dict(k_pages=k, v_pages=k, table=i(2, 4), lens=i(2), starts=i(2), refs=i(33), free_bits=i(2), n_used=i(1))
    for bad, err in ((dict(k_pages=k[0]), "k_pages"), (dict(k_pages=k[..., :64]), "k_pages"), (dict(v_pages=k[:, :32]), "v_pages"),
                     (dict(table=i(8)), "table"), (dict(lens=i(3)), "lens"), (dict(refs=i(32)), "refs"),
                     (dict(free_bits=i(1)), "free_bits"), (dict(lens=i(2).long()), "lens"),
                     (dict(k_scales=k), "scales"), (dict(n_used=i(2)), "n_used")):
        with pytest.raises((ValueError, TypeError), match=err):
            P.PagedCache(**dict(good, **bad))
    f8 = k.view(torch.uint8)[..., :128].contiguous().view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="scales"):
        P.PagedCache(**dict(good, k_pages=f8, v_pages=f8))
    c = object.__new__(P.PagedCache)
    c.n_seqs, c.n_kv_heads, c._index, c._token_shape = 2, 2, 0, (2, 2, 128)
    q, t = torch.zeros(2, 4, 128, dtype=BF), torch.zeros(5, 2, 128, dtype=BF)
    cu = i(3)
    for call in (lambda: c.paris_paged_attend(q, q), lambda: c.paris_paged_grow(i(2)), lambda: c.paris_paged_fork(i(1), i(1)),
                 lambda: c.paris_paged_free(i(1)), lambda: c.paris_paged_store(t, t, cu=cu),
                 lambda: c.paris_paged_read(t, t, cu=cu)):
        with pytest.raises(ValueError, match="device"):
            call()
    for call in (lambda: c.paris_paged_attend(q.float(), q), lambda: c.paris_paged_attend(q, q.float()),
                 lambda: c.paris_paged_attend(q[:1], q), lambda: c.paris_paged_attend(q, q, lse=torch.zeros(2, 3)),
                 lambda: c.paris_paged_grow(i(3)), lambda: c.paris_paged_grow(i(2).long()), lambda: c.paris_paged_fork(i(2), i(1)),
                 lambda: c.paris_paged_fork(i(2), i(2), rows=i(1)), lambda: c.paris_paged_free(i(4)[::2]),
                 lambda: c.paris_paged_free(i(2, 2)), lambda: c.paris_paged_store(t, t[:4], cu=cu),
                 lambda: c.paris_paged_store(t[:, :1], t[:, :1], cu=cu), lambda: c.paris_paged_append(t, t)):
        with pytest.raises((ValueError, TypeError)):
            call()


def test_numbers_that_a_c_argument_does_not_hold(lib):
    c = object.__new__(P.PagedCache)
    t = torch.zeros(5, 2, 128, dtype=BF)
    for big in ((1 << 64) + 1, 1 << 63):
        with pytest.raises(ValueError, match="max_new.*out of range"):
            c.paris_paged_store(t, t, cu=t, max_new=big)
        with pytest.raises(ValueError, match="max_rows.*out of range"):
            c.paris_paged_read(t, t, cu=t, max_rows=big)
