"""Thin ctypes binding of the ParisKV C ABI (include/paris.h).

Argument marshalling only: tensors are passed as raw pointers
(``tensor.data_ptr()``) with the current torch CUDA stream; every step of the
retrieval path runs in the CUDA library.  There is no CPU fallback: if the
library is missing or fails to load, every entry point raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libparis.so")

PARIS_OK, PARIS_EINVAL, PARIS_ENOMEM, PARIS_ECUDA, PARIS_ESTATE, PARIS_ECAPACITY, PARIS_EDEVICE = 0, -1, -2, -3, -4, -6, -7
PARIS_F32, PARIS_BF16 = 0, 1
PARIS_VOTE_RANK, PARIS_VOTE_FLAT = 0, 1
PARIS_TOPK_BY_SCORE, PARIS_TOPK_BY_POSITION = 0, 1
(DUMP_IDS, DUMP_CODES, DUMP_W, DUMP_VOTES, DUMP_CANDS, DUMP_CAND_EST, DUMP_QT, DUMP_QNORM, DUMP_HOT,
 DUMP_LEVELS, DUMP_KV, DUMP_TRACE) = range(12)

# Every function the header declares, with its ctypes signature.
_SIGNATURES = {
    "paris_create": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p)]),
    "paris_destroy": (None, [ctypes.c_void_p]),
    "paris_encode_prefill": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                            ctypes.c_int64, ctypes.c_void_p]),
    "paris_append_decode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                           ctypes.c_void_p]),
    "paris_retrieve": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p]),
    "paris_sparse_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_void_p]),
    "paris_get_state": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "paris_check_device": (ctypes.c_int, [ctypes.c_void_p]),
    "paris_debug_dump": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_size_t]),
    "paris_last_error": (ctypes.c_char_p, [ctypes.c_void_p]),
    "paris_rsq_levels": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_sparse_attend_gqa": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_void_p]),
    "paris_set_centroids": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_dense_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_void_p]),
    "paris_sparse_attend_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                                   ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_decode_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p]),
    "paris_launch_counts": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "paris_profile_begin": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "paris_profile_end": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_prompt_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
    "paris_prompt_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p]),
    "paris_prompt_check": (ctypes.c_int, []),
    "paris_prompt_weights": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                            ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_kv4_store": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_kv4_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_void_p]),
    "paris_kv4_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                           ctypes.POINTER(ctypes.c_size_t)]),
    "paris_kv4_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "paris_kv4_evict_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
    "paris_kv4_evict": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "paris_kv4_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                      ctypes.c_void_p]),
    "paris_kv4_check": (ctypes.c_int, [ctypes.c_void_p]),
}

KERNELS = ["place_kv", "encode", "build_index", "append", "decode", "attend", "fill", "dense", "union"]


class paris_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "n_kv_heads", "n_q_heads", "head_dim", "n_sub", "rho", "sink", "local", "update_buf",
        "topk", "cand_bp", "max_ctx", "retrieval_on_host", "vote_weighting", "topk_order")]


class paris_state(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("T", "N", "n_local", "n_buf", "C", "k_eff", "n_flushes")]


class paris_strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("token", "head", "seq")]


class paris_prompt(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("n_seqs", "n_q_heads", "n_kv_heads", "head_dim")]
                + [(n, ctypes.c_int64) for n in ("rows_q", "rows_k")]
                + [(n, ctypes.c_void_p) for n in ("cu_q", "cu_k")]
                + [(n, ctypes.c_int64) for n in ("max_q", "max_k")]
                + [(n, paris_strides) for n in ("q", "k", "v", "out")])


class paris_kv4(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("batch", "n_kv_heads", "head_dim")] + [("max_rows", ctypes.c_int64)]
                + [(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales", "weights", "positions",
                                                  "lens", "next_pos", "counters", "status")])


_lib = None


def load(path: str = LIB_PATH):
    """Load libparis.so (built by long_context_kv_gb300.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"ParisKV CUDA library not built: {path} is missing "
                           "(run long_context_kv_gb300.build.build())")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class ParisError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{msg} (status {status})")
        self.status = status


def _check(st, ctx=None):
    if st != PARIS_OK:
        raise ParisError(st, load().paris_last_error(ctx).decode())


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return PARIS_F32
    if t.dtype == torch.bfloat16:
        return PARIS_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.data_ptr() % 16:
        raise ValueError("tensor data must be 16-byte aligned")
    return ctypes.c_void_p(t.data_ptr())


def paris_rsq_levels(m: int):
    """The library's float64 Lloyd-Max levels (host computation, no GPU)."""
    lev = (ctypes.c_double * 8)()
    thr = (ctypes.c_double * 7)()
    _check(load().paris_rsq_levels(m, lev, thr))
    return np.array(lev[:]), np.array(thr[:])


def make_config(**kw) -> paris_config:
    cfg = paris_config()
    defaults = dict(batch=1, n_kv_heads=1, n_q_heads=1, head_dim=128, n_sub=16, rho=4, sink=0, local=0,
                    update_buf=128, topk=64, cand_bp=1000, max_ctx=4096, retrieval_on_host=0,
                    vote_weighting=PARIS_VOTE_RANK, topk_order=PARIS_TOPK_BY_SCORE)
    defaults.update(kw)
    for k, v in defaults.items():
        setattr(cfg, k, int(v))
    return cfg


class Context:
    """One layer's ParisKV cache (wraps paris_create / paris_destroy)."""

    def __init__(self, cfg: paris_config, srht_signs: np.ndarray):
        lib = load()
        self.cfg = cfg
        signs = np.ascontiguousarray(srht_signs, dtype=np.int8)
        h = ctypes.c_void_p()
        _check(lib.paris_create(ctypes.byref(cfg), signs.ctypes.data_as(ctypes.c_void_p), ctypes.byref(h)))
        self._h = h

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            load().paris_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def handle(self):
        return self._h

    # -- the ABI calls, same names --------------------------------------------
    def paris_encode_prefill(self, K, V, T=None, stream=None):
        T = K.shape[2] if T is None else T
        _check(load().paris_encode_prefill(self._h, _ptr(K), _ptr(V), _dtype_code(K), T, _stream(stream)), self._h)

    def paris_append_decode(self, k, v, stream=None):
        _check(load().paris_append_decode(self._h, _ptr(k), _ptr(v), _dtype_code(k), _stream(stream)), self._h)

    def paris_retrieve(self, q, topk_idx, topk_score=None, stream=None) -> int:
        k_eff = ctypes.c_int64()
        _check(load().paris_retrieve(self._h, _ptr(q), _dtype_code(q), _ptr(topk_idx), _ptr(topk_score),
                                     ctypes.byref(k_eff), _stream(stream)), self._h)
        return k_eff.value

    def paris_sparse_attend(self, q, topk_idx, out, stream=None):
        _check(load().paris_sparse_attend(self._h, _ptr(q), _dtype_code(q), _ptr(topk_idx), _ptr(out),
                                          _stream(stream)), self._h)

    def paris_sparse_attend_gqa(self, q, topk_idx, out, stream=None):
        """Sparse attention over the window and the union of the KV head's query heads' top-k."""
        _check(load().paris_sparse_attend_gqa(self._h, _ptr(q), _dtype_code(q), _ptr(topk_idx), _ptr(out),
                                              _stream(stream)), self._h)

    def paris_set_centroids(self, centroids=None, stream=None):
        """Learned centroids, device float32 [Hkv][16][256][8] (None: the analytic sign patterns)."""
        _check(load().paris_set_centroids(self._h, _ptr(centroids) if centroids is not None else None,
                                          _stream(stream)), self._h)

    def paris_dense_attend(self, q, out, stream=None):
        """Dense attention over every cached token (the full-attention comparator)."""
        _check(load().paris_dense_attend(self._h, _ptr(q), _dtype_code(q), _ptr(out), _stream(stream)), self._h)

    def paris_sparse_attend_noalloc(self, q, topk_idx, out, stream=None):
        """paris_sparse_attend with its scratch in the library's fixed area (no allocation)."""
        _check(load().paris_sparse_attend_noalloc(self._h, _ptr(q), _dtype_code(q), _ptr(topk_idx), _ptr(out),
                                                  _stream(stream)), self._h)

    def paris_decode_step(self, k, v, q, topk_idx, topk_score, out, stream=None) -> int:
        k_eff = ctypes.c_int64()
        _check(load().paris_decode_step(self._h, _ptr(k), _ptr(v), _dtype_code(k), _ptr(q), _dtype_code(q),
                                        _ptr(topk_idx), _ptr(topk_score), _ptr(out), ctypes.byref(k_eff),
                                        _stream(stream)), self._h)
        return k_eff.value

    def paris_get_state(self) -> dict:
        st = paris_state()
        _check(load().paris_get_state(self._h, ctypes.byref(st)), self._h)
        return {n: getattr(st, n) for n, _ in paris_state._fields_}

    def paris_launch_counts(self) -> dict:
        arr = (ctypes.c_int64 * len(KERNELS))()
        _check(load().paris_launch_counts(self._h, arr), self._h)
        return dict(zip(KERNELS, arr[:]))

    def paris_profile_begin(self, max_launches: int):
        _check(load().paris_profile_begin(self._h, int(max_launches)), self._h)

    def paris_profile_end(self):
        """Returns {kernel: (total_ms, launches)} for the profiled window."""
        ms = (ctypes.c_double * len(KERNELS))()
        n = (ctypes.c_int64 * len(KERNELS))()
        _check(load().paris_profile_end(self._h, ms, n), self._h)
        return {k: (ms[i], n[i]) for i, k in enumerate(KERNELS)}

    def paris_check_device(self):
        _check(load().paris_check_device(self._h), self._h)

    def paris_debug_dump(self, what: int, seq: int = 0, head: int = 0):
        st = self.paris_get_state()
        N, C, T = st["N"], st["C"], st["T"]
        d, B, rho = self.cfg.head_dim, self.cfg.n_sub, self.cfg.rho
        shapes = {
            DUMP_IDS: ((N, B), np.uint8), DUMP_CODES: ((N, d // 2), np.uint8), DUMP_W: ((N, B), np.float32),
            DUMP_VOTES: ((N,), np.uint8), DUMP_CANDS: ((C,), np.int32), DUMP_CAND_EST: ((C,), np.float32),
            DUMP_QT: ((d,), np.float32), DUMP_QNORM: ((1,), np.float32), DUMP_HOT: ((B, rho), np.uint32),
            DUMP_LEVELS: ((15,), np.float32), DUMP_KV: ((2, T, d), np.uint16),
            DUMP_TRACE: ((64 + 8 * 4096 * 4,), np.uint64),
        }
        shape, dt = shapes[what]
        out = np.zeros(shape, dtype=dt)
        _check(load().paris_debug_dump(self._h, what, seq, head, out.ctypes.data_as(ctypes.c_void_p),
                                       out.nbytes), self._h)
        return out


# -- the prompt's own attention, and the 4-bit cache ---------------------------
# These calls are made once or more for every token: what they check is
# checked with as few calls into torch as it takes, and pointers go to the
# library as plain integers.
HEAD_DIM = 128
_torch = None  # torch, from the first call that needs it on
_codes = {}    # its dtypes' codes
# paris_prompt and paris_strides: packing is quicker than filling a ctypes structure
_PROMPT, _STRIDES = struct.Struct("4i2q2P2q12q"), struct.Struct("3q")


def _with_torch():
    global _torch
    if _torch is None:
        import torch
        _codes.update({torch.float32: PARIS_F32, torch.bfloat16: PARIS_BF16})
        _torch = torch
    return _torch


def _code(t):
    """The code of a tensor's dtype, when torch is there already."""
    c = _codes.get(t.dtype)
    return _dtype_code(t) if c is None else c


def _on(index, *tensors):
    """Every tensor on CUDA device `index`, and that the current one."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors on different devices: {t.device} and cuda:{index}")
    if index < 0:
        raise ValueError("tensors must be on a CUDA device")
    now = (_torch or _with_torch())._C._cuda_getDevice()
    if now != index:
        raise ValueError(f"the tensors are on cuda:{index}, the current device is cuda:{now}")


def _number(x, name, bits=64):
    """An integer for a C argument of so many bits: ctypes would keep only the lower ones of a larger one."""
    x = int(x)
    if x.bit_length() >= bits:
        raise ValueError(f"{name}: {x} is out of range")
    return x


def _raw_stream(index, stream):
    """The stream's handle: the one given, or the device's current one."""
    if stream is not None:
        return stream.cuda_stream
    return (_torch or _with_torch())._C._cuda_getCurrentRawStream(index)


def _flat(t):
    """Address of a contiguous, 16-byte aligned tensor (None: no address)."""
    if t is None:
        return None
    p = t.data_ptr()
    if p % 16 or not t.is_contiguous():
        raise ValueError("tensors must be contiguous, their data 16-byte aligned")
    return p or None


def _shaped(t, name, shape, dtype):
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")


def _heads(t, name, packed):
    """A tensor of heads as (rows, heads, sequence axis, strides): [rows, H, d] packed, [batch, H, T, d] otherwise."""
    shape = t.shape
    if len(shape) != (3 if packed else 4) or shape[-1] != HEAD_DIM:
        want = "[rows, heads, 128]" if packed else "[batch, heads, T, 128]"
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {want}")
    if packed:
        return shape[0], shape[1], 1, _strides(t, name, packed)
    return shape[2], shape[1], shape[0], _strides(t, name, packed)


def _strides(t, name, packed):
    st = t.stride()
    if st[-1] != 1 and t.numel():
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return (st[0], st[1], 0) if packed else (st[2], st[1], st[0])


def _scratch(nbytes, device, stream):
    """Scratch of one call, from the caching allocator of the call's stream."""
    torch = _torch or _with_torch()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _prompt(q, k, cu_q, cu_k, max_q, max_k, v=None, out=None):
    """A checked paris_prompt, its query heads, query rows, KV heads and key rows, and whether it is packed."""
    torch = _torch or _with_torch()
    bf16 = torch.bfloat16
    if (cu_q is None) != (cu_k is None):
        raise ValueError("cu_q and cu_k must both be given or both be None")
    packed = cu_q is not None
    for t in (q, k, v, out):
        if t is not None and t.dtype is not bf16:
            raise TypeError(f"the prompt calls take bfloat16 tensors (got {t.dtype})")
    _on(q.get_device(), q, k, v, out, cu_q, cu_k)
    rows_q, hq, seqs, qs = _heads(q, "q", packed)
    rows_k, hkv, k_seqs, ks = _heads(k, "k", packed)
    if k_seqs != seqs:
        raise ValueError(f"q and k: batches of {seqs} and {k_seqs}")
    starts_q = starts_k = 0
    if packed:
        n = cu_q.shape
        for c, name in ((cu_q, "cu_q"), (cu_k, "cu_k")):
            if c.dtype is not torch.int32 or not c.is_contiguous() or c.shape != n or len(n) != 1 or n[0] == 0:
                raise ValueError(f"{name}: a contiguous int32 tensor of n + 1 starts, as many for q as for k")
        seqs, starts_q, starts_k = n[0] - 1, cu_q.data_ptr(), cu_k.data_ptr()
    vs = os_ = (0, 0, 0)
    if v is not None:
        if v.shape != k.shape:
            raise ValueError(f"v: shape {tuple(v.shape)}, expected {tuple(k.shape)}")
        vs = _strides(v, "v", packed)
    if out is not None:
        if out.shape != q.shape:
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {tuple(q.shape)}")
        os_ = _strides(out, "out", packed)
    return _PROMPT.pack(seqs, hq, hkv, HEAD_DIM, rows_q, rows_k, starts_q, starts_k, rows_q if max_q is None else max_q,
                        rows_k if max_k is None else max_k, *qs, *ks, *vs, *os_), hq, rows_q, hkv, rows_k, packed


def _raw(t):
    return t.data_ptr() or None if t is not None else None


def paris_prompt_attend(q, k, v, out, cu_q=None, cu_k=None, max_q=None, max_k=None, lse=None, stream=None):
    """Causal attention over whole prompts, or over the last queries of each sequence.

    Packed: q, out [rows_q, Hq, 128], k, v [rows_k, Hkv, 128] and the int32 starts cu_q, cu_k [n + 1] on the device
    (max_q, max_k: at least the longest sequence's rows, default all rows).  Otherwise [batch, heads, T, 128].
    Any strides with a contiguous last dimension and 16-byte aligned rows.  lse: float32 [Hq, rows_q] or
    [batch, Hq, T], or None.
    """
    p, hq, rows_q, _, _, packed = _prompt(q, k, cu_q, cu_k, max_q, max_k, v, out)
    index = q.get_device()
    if lse is not None:
        if lse.get_device() != index:
            _on(index, lse)
        _shaped(lse, "lse", (hq, rows_q) if packed else q.shape[:3], _torch.float32)
    lib = _lib or load()
    n = ctypes.c_size_t()
    _check(lib.paris_prompt_workspace(p, ctypes.byref(n)))
    need = n.value
    ws = _scratch(need, q.device, stream) if need else None
    _check(lib.paris_prompt_attend(p, _raw(q), _raw(k), _raw(v), PARIS_BF16, _raw(out), _flat(lse), _raw(ws), need,
                                   _raw_stream(index, stream)))


def paris_prompt_check():
    """Synchronise; raise if a prompt call gave up a wait."""
    _check(load().paris_prompt_check())


def paris_prompt_weights(q, k, lse, weights, window, cu_q=None, cu_k=None, max_k=None, stream=None):
    """weights[h, j]: the softmax weights that each sequence's last `window` queries give to its key j, added up over
    them and over the query heads of KV head h.  lse as paris_prompt_attend gives it; weights: float32 [Hkv, rows_k]
    (packed) or [batch, Hkv, T]."""
    window = _number(window, "window", 32)
    p, hq, rows_q, hkv, rows_k, packed = _prompt(q, k, cu_q, cu_k, None, max_k)
    index = q.get_device()
    _on(index, lse, weights)
    _shaped(lse, "lse", (hq, rows_q) if packed else q.shape[:3], _torch.float32)
    _shaped(weights, "weights", (hkv, rows_k) if packed else k.shape[:3], _torch.float32)
    _check((_lib or load()).paris_prompt_weights(p, _raw(q), _raw(k), PARIS_BF16, _flat(lse), window,
                                                 _flat(weights), _raw_stream(index, stream)))


class KV4Cache:
    """A cache in 4 bits (paris_kv4): its arrays are torch tensors, given by the caller or made by `create`.

    k_codes, v_codes uint8 [batch, Hkv, max_rows, 64]; k_scales, v_scales uint8 [batch, Hkv, max_rows, 4];
    weights float32 and positions int32 [batch, Hkv, max_rows]; lens and next_pos int32 [batch].  As with any tensor, a
    cache that another stream than its own still uses is dropped only after `record_stream`.
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales, weights, positions, lens, next_pos):
        torch = _with_torch()
        if k_codes.dim() != 4 or k_codes.shape[3] != HEAD_DIM // 2:
            raise ValueError(f"k_codes: shape {tuple(k_codes.shape)}, expected [batch, heads, max_rows, 64]")
        b, h, r = k_codes.shape[:3]
        want = dict(k_codes=((b, h, r, 64), torch.uint8), v_codes=((b, h, r, 64), torch.uint8),
                    k_scales=((b, h, r, 4), torch.uint8), v_scales=((b, h, r, 4), torch.uint8),
                    weights=((b, h, r), torch.float32), positions=((b, h, r), torch.int32),
                    lens=((b,), torch.int32), next_pos=((b,), torch.int32))
        given = dict(k_codes=k_codes, k_scales=k_scales, v_codes=v_codes, v_scales=v_scales, weights=weights,
                     positions=positions, lens=lens, next_pos=next_pos)
        for name, (shape, dtype) in want.items():
            _shaped(given[name], name, shape, dtype)
            if given[name].device != k_codes.device or k_codes.device.type != "cuda":
                raise ValueError(f"{name}: on {given[name].device}; a cache is on one CUDA device")
            if not given[name].is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            setattr(self, name, given[name])
        self.batch, self.n_kv_heads, self.max_rows, self.device = b, h, r, k_codes.device
        self._index, self._token_shape = k_codes.get_device(), (b, h, HEAD_DIM)
        # counters and the status word, made here and zero between calls
        self._words = torch.zeros(b + 1, dtype=torch.int32, device=k_codes.device)
        self._c = paris_kv4(batch=b, n_kv_heads=h, head_dim=HEAD_DIM, max_rows=r,
                            counters=self._words.data_ptr(), status=self._words.data_ptr() + 4 * b,
                            **{n: t.data_ptr() for n, t in given.items()})
        self._ref = ctypes.byref(self._c)
        self._ws, self._spaces = {}, {}

    @classmethod
    def create(cls, batch, n_kv_heads, max_rows, device="cuda"):
        """An empty cache."""
        import torch
        z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
        n = (batch, n_kv_heads, max_rows)
        return cls(k_codes=z(*n, 64, dtype=torch.uint8), k_scales=z(*n, 4, dtype=torch.uint8),
                   v_codes=z(*n, 64, dtype=torch.uint8), v_scales=z(*n, 4, dtype=torch.uint8),
                   weights=z(*n, dtype=torch.float32), positions=z(*n, dtype=torch.int32),
                   lens=z(batch, dtype=torch.int32), next_pos=z(batch, dtype=torch.int32))

    def record_stream(self, stream):
        """torch.Tensor.record_stream for all of the cache's memory, also for what only the cache knows of: once it is
        dropped, none of it is given away before what `stream` has been given until then is done."""
        for t in (self.k_codes, self.k_scales, self.v_codes, self.v_scales, self.weights, self.positions, self.lens,
                  self.next_pos, self._words):
            t.record_stream(stream)

    def _bytes(self, key, call):
        """Workspace bytes of a call, asked once per kind of call."""
        n = ctypes.c_size_t()
        _check(call(ctypes.byref(n)))
        self._ws[key] = n.value
        return n.value

    def _space(self, nbytes, stream, handle):
        """Address of the workspace of a call: kept for each stream, whose calls take turns with it; during a capture
        one of the graph's own."""
        if stream is None:
            capturing = _torch._C._cuda_isCurrentStreamCapturing()
        else:
            with _torch.cuda.stream(stream):
                capturing = _torch._C._cuda_isCurrentStreamCapturing()
        if capturing:
            return _scratch(nbytes, self.device, stream).data_ptr()
        t = self._spaces.get(handle)
        if t is None or t.numel() < nbytes:
            t = self._spaces[handle] = _scratch(nbytes, self.device, stream)
        return t.data_ptr()

    def paris_kv4_store(self, k, v, cu=None, max_new=None, weights=None, stream=None):
        """Add tokens: packed [rows, Hkv, 128] with int32 starts cu [batch + 1] (max_new: at least the most tokens of
        a sequence, default all rows), or [batch, Hkv, T, 128].  weights: float32 [Hkv, rows] or [batch, Hkv, T]."""
        packed = cu is not None
        if max_new is not None:
            max_new = _number(max_new, "max_new")
        rows, heads, seqs, ks = _heads(k, "k", packed)
        if v.shape != k.shape or v.dtype is not k.dtype:
            raise ValueError("k and v must have the same shape and dtype")
        vs = _strides(v, "v", packed)
        if heads != self.n_kv_heads or (not packed and seqs != self.batch):
            raise ValueError(f"k: shape {tuple(k.shape)} for a cache of {self.batch} sequences, {self.n_kv_heads} heads")
        _on(self._index, k, v, cu, weights)
        if packed and (cu.dtype is not _torch.int32 or cu.shape != (self.batch + 1,) or not cu.is_contiguous()):
            raise ValueError("cu: a contiguous int32 tensor of batch + 1 starts")
        if weights is not None:
            _shaped(weights, "weights", (heads, rows) if packed else k.shape[:3], _torch.float32)
        _check((_lib or load()).paris_kv4_store(
            self._ref, _raw(k), _raw(v), _code(k), _STRIDES.pack(*ks), _STRIDES.pack(*vs),
            rows, _raw(cu), rows if max_new is None else max_new, _flat(weights), _raw_stream(self._index, stream)))

    def paris_kv4_append(self, k, v, stream=None):
        """Add one token to every sequence: k, v [batch, Hkv, 128]."""
        _shaped(k, "k", self._token_shape, k.dtype)
        _shaped(v, "v", self._token_shape, k.dtype)
        _on(self._index, k, v)
        _check((_lib or load()).paris_kv4_append(self._ref, _flat(k), _flat(v), _code(k),
                                                 _raw_stream(self._index, stream)))

    def paris_kv4_attend(self, q, out, accumulate=False, stream=None):
        """out = softmax(K q / sqrt(d)) V over the rows in use: q, out [batch, Hq, 128]; accumulate: add each row's
        softmax weights, over its query heads, to `weights`."""
        shape = q.shape
        if len(shape) != 3 or shape[0] != self.batch or shape[2] != HEAD_DIM:
            raise ValueError(f"q: shape {tuple(shape)}, expected [{self.batch}, heads, 128]")
        _shaped(out, "out", shape, _torch.bfloat16)
        _on(self._index, q, out)
        lib, hq, acc = _lib or load(), shape[1], 1 if accumulate else 0
        n = self._ws.get((hq, acc)) or self._bytes((hq, acc), lambda b: lib.paris_kv4_workspace(self._ref, hq, acc, b))
        handle = _raw_stream(self._index, stream)
        _check(lib.paris_kv4_attend(self._ref, _flat(q), _code(q), hq, acc, _flat(out),
                                    self._space(n, stream, handle), n, handle))

    def paris_kv4_evict(self, keep, sink=0, recent=0, stream=None):
        """At most `keep` rows for each sequence: protected ones and the heaviest others."""
        keep, sink, recent = _number(keep, "keep"), _number(sink, "sink"), _number(recent, "recent")
        _on(self._index)
        lib = _lib or load()
        n = self._ws.get("evict") or self._bytes("evict", lambda b: lib.paris_kv4_evict_workspace(self._ref, b))
        handle = _raw_stream(self._index, stream)
        _check(lib.paris_kv4_evict(self._ref, keep, sink, recent, self._space(n, stream, handle), n, handle))

    def paris_kv4_read(self, k_out, v_out, stream=None):
        """The values of the first rows: k_out, v_out bfloat16 [batch, Hkv, rows, 128]."""
        if k_out.dim() != 4:
            raise ValueError(f"k_out: shape {tuple(k_out.shape)}, expected [batch, heads, rows, 128]")
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            _shaped(t, name, (self.batch, self.n_kv_heads, k_out.shape[2], HEAD_DIM), _torch.bfloat16)
        _on(self._index, k_out, v_out)
        _check((_lib or load()).paris_kv4_read(self._ref, _flat(k_out), _flat(v_out), k_out.shape[2],
                                               _raw_stream(self._index, stream)))

    def paris_kv4_check(self):
        """Synchronise; raise if a store found no room."""
        _check(load().paris_kv4_check(self._ref))
