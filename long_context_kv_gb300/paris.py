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
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libparis.so")

PARIS_OK, PARIS_EINVAL, PARIS_ENOMEM, PARIS_ECUDA, PARIS_ESTATE, PARIS_ECAPACITY, PARIS_EDEVICE = 0, -1, -2, -3, -4, -6, -7
PARIS_F32, PARIS_BF16, PARIS_E4M3 = 0, 1, 2
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
    "paris_paged_grow": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "paris_paged_store": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_void_p]),
    "paris_paged_attend_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t),
                                                    ctypes.POINTER(ctypes.c_size_t)]),
    "paris_paged_attend": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                          ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "paris_paged_read": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p]),
    "paris_paged_fork_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]),
    "paris_paged_fork": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "paris_paged_free": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "paris_paged_compact_workspace": (ctypes.c_int, [ctypes.c_void_p, ctypes.POINTER(ctypes.c_size_t)]),
    "paris_paged_compact": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "paris_paged_check": (ctypes.c_int, [ctypes.c_void_p]),
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


class paris_page_strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("layer", "page", "head", "row")]


class paris_paged(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("n_seqs", "n_layers", "n_kv_heads", "head_dim", "page_rows", "dtype")]
                + [(n, ctypes.c_int64) for n in ("n_pages", "max_pages")]
                + [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages")] + [(n, paris_page_strides) for n in ("k", "v")]
                + [(n, ctypes.c_void_p) for n in ("k_scales", "v_scales", "table", "lens", "starts", "refs", "free_bits",
                                                  "n_used", "status")])


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
        _on(self._index)  # the library waits for the current device
        _check(load().paris_kv4_check(self._ref))


class PagedCache:
    """A cache of pages that sequences share (paris_paged): its arrays are torch tensors, given by the caller or made by
    `create`.

    k_pages, v_pages bfloat16 or float8_e4m3fn [layers, n_pages, Hkv, page_rows, 128], in any order of the first four
    dimensions in memory; with float8_e4m3fn k_scales, v_scales uint8 [layers, n_pages, Hkv, page_rows]; table int32
    [sequences, max_pages]; lens and starts int32 [sequences]; refs int32 [n_pages]; free_bits int32
    [(n_pages + 31) // 32]; n_used int32 [1].  paris_paged_attend and paris_paged_read may be called from several threads
    at once; calls that change the cache are ordered by the caller against all others.  As with any tensor, a cache that
    another stream than its own still uses is dropped only after `record_stream`.
    """

    def __init__(self, k_pages, v_pages, table, lens, starts, refs, free_bits, n_used, k_scales=None, v_scales=None):
        torch = _with_torch()
        if k_pages.dim() != 5 or k_pages.shape[4] != HEAD_DIM:
            raise ValueError(f"k_pages: shape {tuple(k_pages.shape)}, expected [layers, n_pages, heads, page_rows, 128]")
        if k_pages.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError(f"k_pages: dtype {k_pages.dtype}, expected bfloat16 or float8_e4m3fn")
        if table.dim() != 2:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected [sequences, max_pages]")
        layers, n_pages, hkv, rows = k_pages.shape[:4]
        n, width = table.shape
        i32, e4m3 = torch.int32, k_pages.dtype is torch.float8_e4m3fn
        if (k_scales is None) == e4m3 or (v_scales is None) == e4m3:
            raise ValueError("k_scales and v_scales belong to float8_e4m3fn pages")
        want = dict(k_pages=(k_pages.shape, k_pages.dtype), v_pages=(k_pages.shape, k_pages.dtype),
                    table=((n, width), i32), lens=((n,), i32), starts=((n,), i32), refs=((n_pages,), i32),
                    free_bits=(((n_pages + 31) // 32,), i32), n_used=((1,), i32))
        given = dict(k_pages=k_pages, v_pages=v_pages, table=table, lens=lens, starts=starts, refs=refs, free_bits=free_bits,
                     n_used=n_used)
        if e4m3:
            want.update(k_scales=(k_pages.shape[:4], torch.uint8), v_scales=(k_pages.shape[:4], torch.uint8))
            given.update(k_scales=k_scales, v_scales=v_scales)
        for name, (shape, dtype) in want.items():
            _shaped(given[name], name, shape, dtype)
        for name, t in given.items():
            if t.device != k_pages.device or k_pages.device.type != "cuda":
                raise ValueError(f"{name}: on {t.device}; a cache is on one CUDA device")
            if name in ("k_pages", "v_pages"):
                if t.numel() and t.stride(4) != 1:
                    raise ValueError(f"{name}: the last dimension must be contiguous")
            elif not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        self.__dict__.update(given)
        self.n_seqs, self.n_layers, self.n_pages, self.n_kv_heads, self.page_rows = n, layers, n_pages, hkv, rows
        self.max_pages, self.device, self._index = width, k_pages.device, k_pages.get_device()
        self._tensors = tuple(given.values())
        self._status = torch.zeros(1, dtype=i32, device=self.device)
        strides = lambda t: paris_page_strides(*t.stride()[:4])  # noqa: E731
        self._c = paris_paged(n_seqs=n, n_layers=layers, n_kv_heads=hkv, head_dim=HEAD_DIM, page_rows=rows,
                              dtype=PARIS_E4M3 if e4m3 else PARIS_BF16, n_pages=n_pages, max_pages=width,
                              k=strides(k_pages), v=strides(v_pages), status=self._status.data_ptr(),
                              **{name: t.data_ptr() for name, t in given.items()})
        self._ref = ctypes.byref(self._c)
        self._token_shape = (n, hkv, HEAD_DIM)
        self._begin()

    def _begin(self):
        """What calls keep for the ones after them: sizes, workspaces and, of attention, a stream's arguments."""
        self._ws, self._spaces, self._ready, self._lock = {}, {}, {}, threading.Lock()

    @classmethod
    def create(cls, n_seqs, n_kv_heads, n_pages, max_pages, page_rows=16, n_layers=1, dtype=None, device="cuda"):
        """An empty cache; dtype: bfloat16 (the default) or float8_e4m3fn."""
        torch = _with_torch()
        dtype = torch.bfloat16 if dtype is None else dtype
        z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device=device)  # noqa: E731
        size = (n_layers, n_pages, n_kv_heads, page_rows)
        bits = torch.full(((n_pages + 31) // 32,), -1, dtype=torch.int32)
        if n_pages % 32:
            bits[-1] = (1 << n_pages % 32) - 1
        more = {}
        if dtype is torch.float8_e4m3fn:
            more = dict(k_scales=z(*size, dtype=torch.uint8), v_scales=z(*size, dtype=torch.uint8))
        pages = lambda: z(*size, HEAD_DIM, dtype=torch.uint8 if more else dtype).view(dtype)  # noqa: E731
        return cls(pages(), pages(), table=z(n_seqs, max_pages), lens=z(n_seqs), starts=z(n_seqs), refs=z(n_pages),
                   free_bits=bits.to(device), n_used=z(1), **more)

    def record_stream(self, stream):
        """torch.Tensor.record_stream for all of the cache's memory, also for what only the cache knows of: once it is
        dropped, none of it is given away before what `stream` has been given until then is done."""
        for t in (*self._tensors, self._status):
            t.record_stream(stream)

    @staticmethod
    def _capturing(stream):
        if stream is None:
            return _torch._C._cuda_isCurrentStreamCapturing()
        with _torch.cuda.stream(stream):
            return _torch._C._cuda_isCurrentStreamCapturing()

    def _space(self, nbytes, stream, handle, counters=0):
        """The workspace of a call, behind `counters` bytes that are zeros at first (both 16-byte aligned): one tensor,
        which the caller holds until its call is made, since both are taken from what is free.  It is kept for each
        stream, whose calls take turns with it; during a capture it is the graph's own."""
        capturing = self._capturing(stream)
        front = -(-counters // 16) * 16
        t = None if capturing else self._spaces.get((handle, front))
        if t is None or t.numel() < front + nbytes:
            t = _scratch(front + nbytes, self.device, stream)
            if front and stream is None:
                t[:front].zero_()
            elif front:
                with _torch.cuda.stream(stream):
                    t[:front].zero_()
            if not capturing:
                self._spaces[handle, front] = t
                self._ready.clear()
        return t, t.data_ptr() + front

    def _sizes(self, key, call, count):
        """Workspace bytes of a call, asked once per kind of call."""
        ns = [ctypes.c_size_t() for _ in range(count)]
        _check(call(*[ctypes.byref(n) for n in ns]))
        self._ws[key] = [n.value for n in ns]
        return self._ws[key]

    def _list(self, t, name, n=None):
        if t.dtype is not _torch.int32 or t.dim() != 1 or not t.is_contiguous() or (n is not None and len(t) != n):
            raise ValueError(f"{name}: a contiguous int32 tensor of {'one dimension' if n is None else n}")
        return t.data_ptr() or None

    def _rows(self, k, v, cu, longest, name):
        """The checked tensors of a store or read call: rows, strides, the most rows of a sequence."""
        packed = cu is not None
        if longest is not None:
            longest = _number(longest, name)
        rows, heads, seqs, ks = _heads(k, "k", packed)
        if v.dtype is not k.dtype or v.shape != k.shape:
            raise ValueError("k and v must have the same shape and dtype")
        vs = _strides(v, "v", packed)
        if heads != self.n_kv_heads or (not packed and seqs != self.n_seqs):
            raise ValueError(f"k: shape {tuple(k.shape)} for a cache of {self.n_seqs} sequences, {self.n_kv_heads} heads")
        _on(self._index, k, v, cu)
        if packed and (cu.dtype is not _torch.int32 or cu.shape != (self.n_seqs + 1,) or not cu.is_contiguous()):
            raise ValueError("cu: a contiguous int32 tensor of n_seqs + 1 starts")
        return rows, _STRIDES.pack(*ks), _STRIDES.pack(*vs), rows if longest is None else longest

    def paris_paged_grow(self, tokens, stream=None):
        """Room for tokens[s] more rows of every sequence: tokens int32 [n_seqs]."""
        p = self._list(tokens, "tokens", self.n_seqs)
        _on(self._index, tokens)
        _check((_lib or load()).paris_paged_grow(self._ref, p, _raw_stream(self._index, stream)))

    def paris_paged_store(self, k, v, cu=None, max_new=None, layer=0, stream=None):
        """Write a layer's rows that the last growth added: packed [rows, Hkv, 128] with int32 starts cu [n_seqs + 1]
        (max_new: at least the most tokens of a sequence, default all rows), or [n_seqs, Hkv, T, 128]."""
        rows, ks, vs, longest = self._rows(k, v, cu, max_new, "max_new")
        _check((_lib or load()).paris_paged_store(self._ref, _number(layer, "layer", 32), _raw(k), _raw(v), _code(k), ks, vs,
                                                  rows, _raw(cu), longest, _raw_stream(self._index, stream)))

    def paris_paged_append(self, k, v, layer=0, stream=None):
        """Write a layer's row of the one token that the last growth added to every sequence: k, v [n_seqs, Hkv, 128]
        with any strides that paris_paged_store takes.  Sequences that have not grown are left as they are."""
        _shaped(k, "k", self._token_shape, k.dtype)
        _shaped(v, "v", self._token_shape, k.dtype)
        _on(self._index, k, v)
        strides = []
        for t, name in ((k, "k"), (v, "v")):
            seq, head, channel = t.stride()
            if channel != 1 and t.numel():
                raise ValueError(f"{name}: the last dimension must be contiguous")
            strides.append(_STRIDES.pack(HEAD_DIM, head, seq))
        _check((_lib or load()).paris_paged_store(self._ref, _number(layer, "layer", 32), _raw(k), _raw(v), _code(k), *strides,
                                                  1, None, 1, _raw_stream(self._index, stream)))

    def _attend_space(self, lib, hq, stream, handle):
        """The tensor of both workspaces of an attention call, and its arguments."""
        n, m = self._ws.get(hq) or self._sizes(hq, lambda a, b: lib.paris_paged_attend_workspace(self._ref, hq, a, b), 2)
        space, ws = self._space(n, stream, handle, m)
        ready = ws, n, space.data_ptr(), m
        if not self._capturing(stream):
            self._ready[handle, hq] = ready
        return space, ready

    def paris_paged_attend(self, q, out, window=0, lse=None, layer=0, stream=None):
        """out = softmax(K q / sqrt(d)) V over a layer's rows in use, or the last `window` of them: q, out bfloat16
        [n_seqs, Hq, 128]; lse: float32 [n_seqs, Hq], or None."""
        shape, bf16 = q.shape, _torch.bfloat16
        if len(shape) != 3 or shape[0] != self.n_seqs or shape[2] != HEAD_DIM:
            raise ValueError(f"q: shape {tuple(shape)}, expected [{self.n_seqs}, heads, 128]")
        if q.dtype is not bf16 or out.dtype is not bf16 or out.shape != shape:
            _shaped(q, "q", shape, bf16)
            _shaped(out, "out", shape, bf16)
        if lse is not None:
            _shaped(lse, "lse", shape[:2], _torch.float32)
        _on(self._index, q, out, lse)
        lib, hq, handle = _lib or load(), shape[1], _raw_stream(self._index, stream)
        with self._lock:  # a call is several launches with its stream's workspace: threads take turns
            # those of a stream that has been here before (never one that is being captured)
            ready = self._ready.get((handle, hq))
            if ready is None or self._capturing(stream):
                space, ready = self._attend_space(lib, hq, stream, handle)
            _check(lib.paris_paged_attend(self._ref, _number(layer, "layer", 32), _flat(q), hq, _number(window, "window"),
                                          _flat(out), _flat(lse), *ready, handle))

    def paris_paged_read(self, k_out, v_out, cu=None, max_rows=None, layer=0, stream=None):
        """A layer's values of the first rows: bfloat16 [rows, Hkv, 128] with int32 starts cu [n_seqs + 1] (max_rows: at
        least the most rows of a sequence), or [n_seqs, Hkv, T, 128].  Rows past a sequence's end stay as they were."""
        rows, ks, vs, longest = self._rows(k_out, v_out, cu, max_rows, "max_rows")
        if k_out.dtype is not _torch.bfloat16:
            raise TypeError(f"k_out: dtype {k_out.dtype}, expected {_torch.bfloat16}")
        _check((_lib or load()).paris_paged_read(self._ref, _number(layer, "layer", 32), _raw(k_out), _raw(v_out), ks, vs, rows,
                                                 _raw(cu), longest, _raw_stream(self._index, stream)))

    def _fork_space(self, n, stream, handle):
        key = ("fork", n)
        lib = _lib or load()
        sizes = self._ws.get(key) or self._sizes(key, lambda b: lib.paris_paged_fork_workspace(self._ref, n, b), 1)
        return *self._space(sizes[0], stream, handle), sizes[0]

    def paris_paged_fork(self, src, dst, rows=None, stream=None):
        """Sequence dst[i] becomes the first rows[i] rows (None: all) of sequence src[i] as it was before the call: full
        pages are shared, the last one is copied.  src, dst, rows: int32 [n]."""
        n = src.shape[0] if src.dim() else 0
        a, b = self._list(src, "src"), self._list(dst, "dst", n)
        r = None if rows is None else self._list(rows, "rows", n)
        _on(self._index, src, dst, rows)
        handle = _raw_stream(self._index, stream)
        space, ws, size = self._fork_space(n, stream, handle)
        _check((_lib or load()).paris_paged_fork(self._ref, a, b, r, n, ws, size, handle))

    def paris_paged_free(self, seqs, rows=None, stream=None):
        """End the listed sequences (rows None), or cut them to rows[i] rows: int32 [n]."""
        n = seqs.shape[0] if seqs.dim() else 0
        a = self._list(seqs, "seqs")
        r = None if rows is None else self._list(rows, "rows", n)
        _on(self._index, seqs, rows)
        handle = _raw_stream(self._index, stream)
        space, ws, size = (None, None, 0) if rows is None else self._fork_space(n, stream, handle)
        _check((_lib or load()).paris_paged_free(self._ref, a, r, n, ws, size, handle))

    def paris_paged_compact(self, stream=None):
        """Move the pages in use to the front of the pool."""
        _on(self._index)
        lib, handle = _lib or load(), _raw_stream(self._index, stream)
        sizes = self._ws.get("compact") or self._sizes("compact",
                                                       lambda b: lib.paris_paged_compact_workspace(self._ref, b), 1)
        space, ws = self._space(sizes[0], stream, handle)
        _check(lib.paris_paged_compact(self._ref, ws, sizes[0], handle))

    def paris_paged_check(self):
        """Synchronise; raise if a call found no room or a sequence out of range, or if attention gave up a wait."""
        _on(self._index)  # the library waits for the current device, and asks that one
        _check(load().paris_paged_check(self._ref))
