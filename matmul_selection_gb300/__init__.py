"""Python binding of the GB300 autotuned matmul C ABI (include/mm.h).

Argument marshalling only: every entry point forwards to the shared library
built from ``csrc/`` (``_build/libmm_gb300.so``); nothing here computes.  The
names are the C names.  Data arguments accept raw device addresses (int) or
objects with ``data_ptr()`` (torch tensors); ``stream`` accepts an int
handle, a ``torch.cuda.Stream`` or None (legacy default stream).

Importing the package loads the library and fails loudly when it has not
been built (``python matmul_selection_gb300/build.py``).  The operators that a
model calls once a layer and token go through a small extension module
(``csrc/binding/fastcall.cpp``): the same C functions, the arguments converted
in C.  Where it was not built for this Python they go through ctypes as well,
which costs 2-3 us more a call.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import operator
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libmm_gb300.so")

# status codes
MM_OK = 0
MM_ERR_INVALID_ARG = 1
MM_ERR_UNSUPPORTED = 2
MM_ERR_CUDA = 3
MM_ERR_NO_VALID_CANDIDATE = 4
MM_ERR_CACHE_VALIDATION = 5
MM_ERR_IO = 6
MM_ERR_TIMEOUT = 7
MM_ERR_NOT_FOUND = 8

MM_BF16, MM_F16, MM_F32 = 0, 1, 2
MM_E4M3 = 3  # only where an operator names it
MM_I32, MM_I64 = 4, 5  # likewise
MM_NN, MM_NT, MM_TN, MM_TT = 0, 1, 2, 3
LAYOUTS = {"NN": MM_NN, "NT": MM_NT, "TN": MM_TN, "TT": MM_TT}


class mm_dtypes(ctypes.Structure):
    _fields_ = [("a", ctypes.c_int32), ("b", ctypes.c_int32), ("c", ctypes.c_int32)]


class mm_batch(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("stride_a", ctypes.c_int64),
                ("stride_b", ctypes.c_int64), ("stride_c", ctypes.c_int64)]


class mm_key(ctypes.Structure):
    _fields_ = [("bytes", ctypes.c_uint8 * 64)]


class mm_stats(ctypes.Structure):
    _fields_ = [("calls", ctypes.c_uint64), ("hits", ctypes.c_uint64),
                ("misses", ctypes.c_uint64), ("tunes", ctypes.c_uint64),
                ("launches", ctypes.c_uint64), ("bench_launches", ctypes.c_uint64),
                ("last_tune_ms", ctypes.c_double), ("total_tune_ms", ctypes.c_double)]


class MMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"mm status {status}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with "
                      "`python matmul_selection_gb300/build.py` (needs nvcc)")
_lib = ctypes.CDLL(LIB_PATH)


def _load_fastcall():
    path = os.path.join(_HERE, "_build", "mm_fastcall" + importlib.machinery.EXTENSION_SUFFIXES[0])
    if not os.path.exists(path):
        return None
    loader = importlib.machinery.ExtensionFileLoader("mm_fastcall", path)
    module = importlib.util.module_from_spec(
        importlib.util.spec_from_file_location("mm_fastcall", path, loader=loader))
    loader.exec_module(module)
    return module


_i64, _i32, _vp, _cp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_char_p
_P32 = ctypes.POINTER(ctypes.c_int32)
_sig = {
    "mm_tune_key": (_i32, [_i64, _i64, _i64, _i64, _i64, _i64, mm_dtypes, ctypes.c_int,
                           ctypes.POINTER(mm_batch), ctypes.POINTER(mm_key), ctypes.c_char_p,
                           ctypes.c_size_t]),
    "mm_autotune_execute": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, mm_dtypes,
                                   ctypes.c_int, ctypes.POINTER(mm_batch), _vp]),
    "mm_autotune_execute_host": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64,
                                        mm_dtypes, ctypes.c_int, ctypes.POINTER(mm_batch), _vp]),
    "mm_cache_load": (_i32, [_cp]),
    "mm_cache_save": (_i32, [_cp]),
    "mm_tune_file": (_i32, [_cp, ctypes.POINTER(ctypes.c_int)]),
    "mm_cache_clear": (_i32, []),
    "mm_cache_size": (_i64, []),
    "mm_candidate_count": (_i32, []),
    "mm_candidate_name": (_cp, [_i32]),
    "mm_candidate_launches": (ctypes.c_uint64, [_i32]),
    "mm_candidate_checksum": (ctypes.c_uint64, []),
    "mm_execute_candidate": (_i32, [_i32, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64,
                                    mm_dtypes, ctypes.c_int, ctypes.POINTER(mm_batch), _vp]),
    "mm_lookup": (_i32, [ctypes.POINTER(mm_key), _P32]),
    "mm_plan": (_i32, [_i64, _i64, _i64, _i64, _i64, _i64, mm_dtypes, ctypes.c_int,
                       ctypes.POINTER(mm_batch), _i32, _P32, _P32, _P32, _P32, _P32, _P32]),
    "mm_group_name": (_cp, [_i32]),
    "mm_default_candidate": (_i32, [_i64, _i64, _i64, _i64, _i64, _i64, mm_dtypes, ctypes.c_int,
                                    ctypes.POINTER(mm_batch)]),
    "mm_roofline_limit_ns": (ctypes.c_double, [ctypes.c_double] * 6),
    "mm_device_peaks": (_i32, [ctypes.POINTER(ctypes.c_double)] * 3),
    "mm_set_option": (_i32, [_cp, _cp]),
    "mm_get_option": (_i32, [_cp, ctypes.c_char_p, ctypes.c_size_t]),
    "mm_get_stats": (_i32, [ctypes.POINTER(mm_stats)]),
    "mm_reset_stats": (None, []),
    "mm_last_error": (_cp, []),
    "mm_version": (_cp, []),
    "mm_shutdown": (None, []),
    "mm_splitk_gemm_noalloc": (_i32, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64,
                                      mm_dtypes, ctypes.c_int, _vp]),
    "mm_splitk_gemm_noalloc_status": (_i32, [_vp]),
    "mm_rmsnorm": (_i32, [_vp] * 7 + [_i64] * 6 + [mm_dtypes, ctypes.c_float, _vp]),
    "mm_rmsnorm_backward": (_i32, [_vp] * 7 + [_i64] * 6 + [mm_dtypes, ctypes.c_float, _vp]),
    "mm_gemm_w4": (_i32, [_vp] * 5 + [_i64] * 7 + [_i32, mm_dtypes, _vp]),
    "mm_gemm_q8": (_i32, [_vp] * 5 + [_i64] * 6 + [mm_dtypes, _vp]),
    "mm_embedding": (_i32, [_vp] * 3 + [_i64] * 5 + [mm_dtypes, ctypes.c_float, _vp]),
    "mm_embedding_backward": (_i32, [_vp] * 4 + [_i64] * 6 + [mm_dtypes, ctypes.c_float, _vp]),
    "mm_cross_entropy": (_i32, [_vp] * 5 + [_i64] * 5 + [mm_dtypes, _vp]),
    "mm_cross_entropy_backward": (_i32, [_vp] * 7 + [_i64] * 7 + [mm_dtypes, _vp]),
    "mm_operator_status": (_i32, [_vp]),
}
for _name, (_res, _args) in _sig.items():
    _f = getattr(_lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_sig)


def _ptr(x):
    if x is None or isinstance(x, int):
        return x
    try:  # a torch tensor, the common case
        return x.data_ptr()
    except AttributeError:
        pass
    if hasattr(x, "ctypes"):  # numpy array (host entry point)
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream  # torch.cuda.Stream


_dtypes_of = {}  # (a, b, c) -> the struct, passed by value


def _dt(dt):
    if isinstance(dt, mm_dtypes):
        return dt
    dt = tuple(dt)
    got = _dtypes_of.get(dt)
    if got is None:
        # a number past 32 bits is no type: refused by the call
        a, b, c = (t if -1 << 31 <= t < 1 << 31 else -1 for t in dt)
        got = _dtypes_of[dt] = mm_dtypes(a, b, c)
    return got


def _layout(layout):
    return LAYOUTS[layout] if isinstance(layout, str) else int(layout)


def _batch(batch):
    if batch is None:
        return None
    if isinstance(batch, mm_batch):
        return ctypes.byref(batch)
    return ctypes.byref(mm_batch(*batch))


def mm_last_error() -> str:
    return _lib.mm_last_error().decode()


def mm_version() -> str:
    return _lib.mm_version().decode()


def check(status: int) -> int:
    """Raise MMError for a non-OK status (with the library's message)."""
    if status != MM_OK:
        raise MMError(status, mm_last_error())
    return status


def mm_tune_key(M, N, K, lda, ldb, ldc, dtypes, layout, batch=None):
    """Returns (status, key bytes, canonical text)."""
    k = mm_key()
    buf = ctypes.create_string_buffer(512)
    st = _lib.mm_tune_key(M, N, K, lda, ldb, ldc, _dt(dtypes), _layout(layout), _batch(batch),
                          ctypes.byref(k), buf, 512)
    return st, bytes(k.bytes), buf.value.decode()


def mm_autotune_execute(lhs, rhs, out, M, N, K, lda, ldb, ldc, dtypes, layout, batch=None,
                        stream=None):
    return _lib.mm_autotune_execute(_ptr(lhs), _ptr(rhs), _ptr(out), M, N, K, lda, ldb, ldc,
                                    _dt(dtypes), _layout(layout), _batch(batch), _stream(stream))


def mm_autotune_execute_host(lhs, rhs, out, M, N, K, lda, ldb, ldc, dtypes, layout, batch=None,
                             stream=None):
    return _lib.mm_autotune_execute_host(_ptr(lhs), _ptr(rhs), _ptr(out), M, N, K, lda, ldb, ldc,
                                         _dt(dtypes), _layout(layout), _batch(batch),
                                         _stream(stream))


def mm_execute_candidate(index, lhs, rhs, out, M, N, K, lda, ldb, ldc, dtypes, layout,
                         batch=None, stream=None):
    return _lib.mm_execute_candidate(index, _ptr(lhs), _ptr(rhs), _ptr(out), M, N, K, lda, ldb,
                                     ldc, _dt(dtypes), _layout(layout), _batch(batch),
                                     _stream(stream))


def mm_cache_load(path=None):
    return _lib.mm_cache_load(path.encode() if path else None)


def mm_tune_file(path):
    """Tune every problem recorded in `path` by the record_untuned option;
    returns (status, number tuned)."""
    n = ctypes.c_int(0)
    st = _lib.mm_tune_file(path.encode(), ctypes.byref(n))
    return st, n.value


def mm_cache_save(path=None):
    return _lib.mm_cache_save(path.encode() if path else None)


def mm_cache_clear():
    return _lib.mm_cache_clear()


def mm_cache_size():
    return _lib.mm_cache_size()


def mm_candidate_count():
    return _lib.mm_candidate_count()


def mm_candidate_name(i):
    r = _lib.mm_candidate_name(i)
    return r.decode() if r is not None else None


def mm_candidate_launches(i):
    return _lib.mm_candidate_launches(i)


def mm_candidate_checksum():
    return _lib.mm_candidate_checksum()


def candidate_names():
    return [mm_candidate_name(i) for i in range(mm_candidate_count())]


def mm_lookup(key: bytes):
    k = mm_key()
    ctypes.memmove(k.bytes, key, 64)
    idx = ctypes.c_int32(-1)
    st = _lib.mm_lookup(ctypes.byref(k), ctypes.byref(idx))
    return st, idx.value


def mm_plan(M, N, K, lda, ldb, ldc, dtypes, layout, batch=None, cap=256):
    """Returns a list of dicts {cand, group, tier, supported, group_prio, prio}."""
    arrs = [(ctypes.c_int32 * cap)() for _ in range(6)]
    n = _lib.mm_plan(M, N, K, lda, ldb, ldc, _dt(dtypes), _layout(layout), _batch(batch), cap,
                     *arrs)
    if n < 0:
        raise MMError(MM_ERR_INVALID_ARG, mm_last_error())
    keys = ("cand", "group", "tier", "supported", "group_prio", "prio")
    return [{k: arrs[j][i] for j, k in enumerate(keys)} for i in range(n)]


def mm_default_candidate(M, N, K, lda, ldb, ldc, dtypes, layout, batch=None):
    return _lib.mm_default_candidate(M, N, K, lda, ldb, ldc, _dt(dtypes), _layout(layout),
                                     _batch(batch))


def mm_group_name(g):
    r = _lib.mm_group_name(g)
    return r.decode() if r is not None else None


def mm_device_peaks():
    """(status, bf16 ops/s, bytes/s, launch ns) of the current device."""
    v = [ctypes.c_double(0) for _ in range(3)]
    st = _lib.mm_device_peaks(*[ctypes.byref(x) for x in v])
    return (st,) + tuple(x.value for x in v)


def mm_roofline_limit_ns(ops, peak_ops_per_s, nbytes, peak_bytes_per_s, threshold, launch_ns):
    return _lib.mm_roofline_limit_ns(ops, peak_ops_per_s, nbytes, peak_bytes_per_s, threshold,
                                     launch_ns)


def mm_set_option(name, value):
    return _lib.mm_set_option(name.encode(), str(value).encode())


def mm_get_option(name):
    buf = ctypes.create_string_buffer(1024)
    st = _lib.mm_get_option(name.encode(), buf, 1024)
    return st, buf.value.decode()


def mm_get_stats():
    s = mm_stats()
    _lib.mm_get_stats(ctypes.byref(s))
    return {f: getattr(s, f) for f, _ in mm_stats._fields_}


def mm_reset_stats():
    _lib.mm_reset_stats()


def mm_shutdown():
    _lib.mm_shutdown()


def mm_splitk_gemm_noalloc(lhs, rhs, out, M, N, K, lda, ldb, ldc, dtypes, layout, stream=None):
    """Split-K GEMM into the library's fixed workspace: no device allocation."""
    return _lib.mm_splitk_gemm_noalloc(_ptr(lhs), _ptr(rhs), _ptr(out), M, N, K, lda, ldb, ldc,
                                       _dt(dtypes), _layout(layout), _stream(stream))


def mm_splitk_gemm_noalloc_status(stream=None):
    """Synchronise `stream` and report (and clear) a bounded wait that gave up
    in a no-allocation call since the previous query."""
    return _lib.mm_splitk_gemm_noalloc_status(_stream(stream))


def _int64(v):
    v = operator.index(v)
    if not -1 << 63 <= v < 1 << 63:
        raise OverflowError("int too large for a 64-bit argument")
    return v


def _real(v):
    if isinstance(v, (str, bytes)):
        raise TypeError("a number expected")
    return float(v)


class _Ctypes:
    """The extension module's functions through ctypes."""

    @staticmethod
    def rmsnorm(*args):
        return _Ctypes._call(_lib.mm_rmsnorm, 7, 6, args)

    @staticmethod
    def rmsnorm_backward(*args):
        return _Ctypes._call(_lib.mm_rmsnorm_backward, 7, 6, args)

    @staticmethod
    def gemm_w4(*args):
        if not -1 << 31 <= _int64(args[12]) < 1 << 31:
            args = (*args[:12], 0, *args[13:])  # no group: refused by the call
        return _Ctypes._call(_lib.mm_gemm_w4, 5, 8, args)

    @staticmethod
    def gemm_q8(*args):
        return _Ctypes._call(_lib.mm_gemm_q8, 5, 6, args)

    @staticmethod
    def embedding(*args):
        return _Ctypes._call(_lib.mm_embedding, 3, 5, args)

    @staticmethod
    def embedding_backward(*args):
        return _Ctypes._call(_lib.mm_embedding_backward, 4, 6, args)

    @staticmethod
    def cross_entropy(*args):
        return _Ctypes._call(_lib.mm_cross_entropy, 5, 5, args)

    @staticmethod
    def cross_entropy_backward(*args):
        return _Ctypes._call(_lib.mm_cross_entropy_backward, 7, 7, args)

    @staticmethod
    def _call(f, pointers, integers, args):
        dt, *reals = args[pointers + integers:-1]
        if len(dt) != 3:
            raise TypeError("types: a tuple of three")
        return f(*map(_ptr, args[:pointers]), *map(_int64, args[pointers:pointers + integers]),
                 _dt(tuple(map(_int64, dt))), *map(_real, reals), _stream(args[-1]))


_fast = _load_fastcall() or _Ctypes


def _types(dt):
    return (dt.a, dt.b, dt.c) if isinstance(dt, mm_dtypes) else tuple(dt)


def mm_rmsnorm(x, residual, weight, h, y, scale, rstd, rows, cols, ldx, ldr, ldh, ldy, dtypes, eps,
               stream=None):
    """h = x + residual, y = h / rms(h) * weight; y in 8 bits takes `scale`."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.rmsnorm(x, residual, weight, h, y, scale, rstd, rows, cols, ldx, ldr, ldh, ldy,
                         dtypes, eps, stream)


def mm_rmsnorm_backward(dy, dh, h, weight, rstd, dx, dweight, rows, cols, lddy, lddh, ldh, lddx,
                        dtypes, eps, stream=None):
    """The gradients of mm_rmsnorm to its input and its weight."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.rmsnorm_backward(dy, dh, h, weight, rstd, dx, dweight, rows, cols, lddy, lddh, ldh,
                                  lddx, dtypes, eps, stream)


def mm_gemm_w4(A, codes, scales, zeros, out, M, N, K, lda, ldw, lds, ldc, group, dtypes,
               stream=None):
    """out = A . W^T, W in 4-bit codes with group scales and zero points."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.gemm_w4(A, codes, scales, zeros, out, M, N, K, lda, ldw, lds, ldc, group, dtypes,
                         stream)


def mm_gemm_q8(A, B, scale_a, scale_b, out, M, N, K, lda, ldb, ldc, dtypes, stream=None):
    """out = A . B^T of e4m3 operands with row scales of A and of B."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.gemm_q8(A, B, scale_a, scale_b, out, M, N, K, lda, ldb, ldc, dtypes, stream)


def mm_embedding(weight, tokens, out, rows, cols, vocab, ldw, ldo, dtypes, scale=1.0, stream=None):
    """out[t] = scale * weight[tokens[t]]; zeros where there is no such token."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.embedding(weight, tokens, out, rows, cols, vocab, ldw, ldo, dtypes, scale, stream)


def mm_embedding_backward(dout, tokens, base, dweight, rows, cols, vocab, lddo, ldb, lddw, dtypes,
                          scale=1.0, stream=None):
    """dweight[v] = base[v] + scale * the sum of dout over the places of token v."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.embedding_backward(dout, tokens, base, dweight, rows, cols, vocab, lddo, ldb, lddw,
                                    dtypes, scale, stream)


def mm_cross_entropy(x, weight, targets, loss, lse, rows, cols, vocab, ldx, ldw, dtypes, stream=None):
    """Softmax cross entropy of x . weight^T; the logits are not kept."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.cross_entropy(x, weight, targets, loss, lse, rows, cols, vocab, ldx, ldw, dtypes, stream)


def mm_cross_entropy_backward(x, weight, targets, lse, dloss, dx, dweight, rows, cols, vocab, ldx, ldw,
                              lddx, lddw, dtypes, stream=None):
    """The gradients of mm_cross_entropy to x and to its matrix."""
    if type(dtypes) is not tuple:
        dtypes = _types(dtypes)
    return _fast.cross_entropy_backward(x, weight, targets, lse, dloss, dx, dweight, rows, cols, vocab,
                                        ldx, ldw, lddx, lddw, dtypes, stream)


def mm_operator_status(stream=None):
    """Synchronise `stream`; report (and clear) a bounded wait that gave up in
    an operator's kernel since the previous query."""
    return _lib.mm_operator_status(_stream(stream))


def library_handle():
    return _lib
