"""Thin ctypes binding of ``libh2o_gb300.so`` with the C ABI's names.

Argument marshalling only: every device-memory argument is a raw pointer
(an ``int``) or any object with ``data_ptr()`` (a torch tensor), every host
buffer of the state calls is a numpy array, and streams are ``cudaStream_t``
values (``int``) or objects with a ``cuda_stream`` attribute.  All compute
runs in the library; a failing call raises ``H2OError`` with the library's
message.  Importing this module does not load the library; the first call
does, and raises if the library was not built (there is no fallback).

The binding remembers each handle's shape (units, budget, head_dim, element
type, query heads per unit, last prompt length) from the calls that made it,
and checks the type and size of every host array, and of every tensor it
is given, before the library writes into or reads from it; a raw integer
pointer is passed through unchecked.

The paged-cache calls (``h2o_page_*``, ``h2o_prefix_*``) have no handle: they
take torch tensors only, read every size from the tensors' shapes and check
them against one another; without a `stream` they run on torch's current one.
"""
import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libh2o_gb300.so")

H2O_OK = 0
H2O_ERR_ARG = -1
H2O_ERR_STATE = -2
H2O_ERR_ALLOC = -3
H2O_ERR_CUDA = -4
H2O_ERR_DEVICE_TIMEOUT = -5
H2O_ERR_UNSUPPORTED = -6
H2O_F32 = 0
H2O_BF16 = 1
H2O_KV8 = 2
H2O_KV4 = 4

# every symbol include/h2o.h declares, with (restype, argtypes)
_vp = ctypes.c_void_p
_i = ctypes.c_int
_d = ctypes.c_double
_ll = ctypes.c_longlong
SIGNATURES = {
    "h2o_init": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _i, _i, _d, _vp]),
    "h2o_init_gqa": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _i, _i, _i, _d, _vp]),
    "sh_init": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _i, _i, _d, _vp]),
    "sh_prefill": (_i, [_vp, _vp, _vp, _vp, _i]),
    "sh_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "h2o_prefill": (_i, [_vp, _vp, _vp, _vp, _i]),
    "h2o_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "lsh_init": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _i, _i, _d, _vp, _vp]),
    "lsh_prefill": (_i, [_vp, _vp, _vp, _vp, _i]),
    "lsh_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "h2o_get_state": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "h2o_set_state": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "h2o_get_prefill_stats": (_i, [_vp, _vp, _vp, _vp]),
    "h2o_get_kv_scales": (_i, [_vp, _vp, _vp]),
    "h2o_set_kv_scales": (_i, [_vp, _vp, _vp]),
    "h2o_set_stream": (_i, [_vp, _vp]),
    "h2o_set_decode_split": (_i, [_vp, _i]),
    "h2o_sync": (_i, [_vp]),
    "h2o_destroy": (None, [_vp]),
    "h2o_last_error": (ctypes.c_char_p, []),
    "h2o_prompt_scores_noalloc": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _d, _vp, _vp]),
    "h2o_selftest_wait_timeout": (_i, [_vp]),
    "fg_init": (_i, [ctypes.POINTER(_vp), _i, _i, _i, _i, _d, _i, _i, _i, _i, _d, _vp]),
    "fg_prefill": (_i, [_vp, _vp, _vp, _vp, _i]),
    "fg_decode_step": (_i, [_vp, _vp, _vp, _vp, _vp, _vp]),
    "fg_get_policy": (_i, [_vp, _vp, _vp, _vp]),
    "h2o_page_tables": (_i, [_vp, _vp, _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp]),
    "h2o_page_write": (_i, [_vp, _vp, _ll, _ll, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]),
    "h2o_page_attend": (_i, [_vp, _ll, _vp, _vp, _i, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _i, _i, _i, _d,
                             _vp, _ll, _vp, _vp]),
    "h2o_prefix_attend": (_i, [_vp, _ll, _vp, _vp, _i, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp, _i, _vp, _i, _i, _d,
                               _vp, _ll, _vp, _ll, _vp]),
    "h2o_prefix_work_bytes": (_ll, [_i, _i, _i, _i, _i, _i]),
}

H2O_NOALLOC_MAX_TOKENS = 1 << 20

_lib = None


class H2OError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__("h2o status %d: %s" % (code, msg))
        self.code = code


def lib():
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libh2o_gb300.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if isinstance(x, np.ndarray):
        if not x.flags["C_CONTIGUOUS"]:
            raise ValueError("host array must be C-contiguous")
        return x.ctypes.data
    if hasattr(x, "data_ptr"):
        if hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise ValueError("tensor must be contiguous")
        return x.data_ptr()
    raise TypeError("cannot take a pointer of %r" % type(x))


def _stream(s):
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc):
    if rc != H2O_OK:
        raise H2OError(rc, h2o_last_error())


# handle -> its shape, recorded by the init calls
_meta = {}


def _remember(h, kind, U, B, d, dtype, G=1):
    kv8, kv4 = bool(dtype & H2O_KV8), bool(dtype & H2O_KV4)
    elem = np.int8 if kv8 else np.uint8 if kv4 else (np.uint16 if (dtype & H2O_BF16) else np.float32)
    # elements of one stored row: a 4-bit row packs two codes per byte
    _meta[h] = dict(kind=kind, U=U, B=B, d=d, G=G, elem=np.dtype(elem), row=d // 2 if kv4 else d,
                    kv8=kv8, kv4=kv4, T=0, in_size=2 if dtype & H2O_BF16 else 4)
    return h


def _info(h):
    m = _meta.get(h)
    if m is None:
        raise ValueError("unknown handle %r (not created by this binding, or destroyed)" % (h,))
    return m


def _host(x, dtype, n, what):
    """x is None or a C-contiguous numpy array of `dtype` with n elements."""
    if x is None:
        return None
    if not isinstance(x, np.ndarray):
        raise TypeError("%s must be a numpy array (host memory)" % what)
    if x.dtype != np.dtype(dtype):
        raise TypeError("%s must have dtype %s (got %s)" % (what, np.dtype(dtype), x.dtype))
    if x.size != n:
        raise ValueError("%s must have %d elements (got %d)" % (what, n, x.size))
    if not x.flags["C_CONTIGUOUS"]:
        raise ValueError("%s must be C-contiguous" % what)
    return x


def _dev(x, nbytes, what, dtypes=None):
    """Check a device tensor's size (and dtype) when it is one; raw integer
    pointers pass unchecked."""
    if x is None or isinstance(x, int) or not hasattr(x, "numel"):
        return x
    if getattr(x, "device", None) is not None and getattr(x.device, "type", "cuda") != "cuda":
        raise ValueError("%s must be on the GPU" % what)
    got = x.numel() * x.element_size()
    if got < nbytes:
        raise ValueError("%s holds %d bytes, needs %d" % (what, got, nbytes))
    if dtypes is not None and str(x.dtype).replace("torch.", "") not in dtypes:
        raise TypeError("%s must be of dtype %s (got %s)" % (what, "/".join(dtypes), x.dtype))
    return x


def h2o_last_error():
    return lib().h2o_last_error().decode()


def h2o_init(budget, heavy, recent, batch, heads, head_dim, dtype, scale, stream=None):
    h = _vp()
    _check(lib().h2o_init(ctypes.byref(h), budget, heavy, recent, batch, heads, head_dim, dtype,
                          float(scale), _stream(stream)))
    return _remember(h.value, "h2o", batch * heads, budget, head_dim, dtype)


def h2o_init_gqa(budget, heavy, recent, batch, kv_heads, groups, head_dim, dtype, scale, stream=None):
    h = _vp()
    _check(lib().h2o_init_gqa(ctypes.byref(h), budget, heavy, recent, batch, kv_heads, groups, head_dim,
                              dtype, float(scale), _stream(stream)))
    return _remember(h.value, "h2o", batch * kv_heads, budget, head_dim, dtype, groups)


def lsh_init(budget, recent, batch, heads, head_dim, dtype, scale, W, stream=None):
    h = _vp()
    _dev(W, head_dim * 32 * 4, "W", ("float32",))
    _check(lib().lsh_init(ctypes.byref(h), budget, recent, batch, heads, head_dim, dtype, float(scale),
                          _ptr(W), _stream(stream)))
    return _remember(h.value, "lsh", batch * heads, budget, head_dim, dtype)


def h2o_prefill(h, Q, K, V, T):
    _prompt_args(h, Q, K, V, T)
    _check(lib().h2o_prefill(h, _ptr(Q), _ptr(K), _ptr(V), int(T)))
    _info(h)["T"] = int(T)


def lsh_prefill(h, Q, K, V, T):
    _prompt_args(h, Q, K, V, T)
    _check(lib().lsh_prefill(h, _ptr(Q), _ptr(K), _ptr(V), int(T)))
    _info(h)["T"] = int(T)


def h2o_decode_step(h, q, k, v, out, victim_out=None):
    _step_args(h, q, k, v, out, victim_out)
    _check(lib().h2o_decode_step(h, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(victim_out)))


def lsh_decode_step(h, q, k, v, out, victim_out=None):
    _step_args(h, q, k, v, out, victim_out)
    _check(lib().lsh_decode_step(h, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(victim_out)))


def sh_init(budget, heavy, recent, batch, heads, head_dim, dtype, scale, stream=None):
    h = _vp()
    _check(lib().sh_init(ctypes.byref(h), budget, heavy, recent, batch, heads, head_dim, dtype,
                         float(scale), _stream(stream)))
    return _remember(h.value, "sh", batch * heads, budget, head_dim, dtype)


def sh_prefill(h, Q, K, V, T):
    _prompt_args(h, Q, K, V, T)
    _check(lib().sh_prefill(h, _ptr(Q), _ptr(K), _ptr(V), int(T)))
    _info(h)["T"] = int(T)


def sh_decode_step(h, q, k, v, out, victim_out=None):
    _step_args(h, q, k, v, out, victim_out)
    _check(lib().sh_decode_step(h, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(victim_out)))


def _prompt_args(h, Q, K, V, T):
    m = _info(h)
    row = m["d"] * m["in_size"]
    _dev(Q, m["U"] * m["G"] * int(T) * row, "Q")
    _dev(K, m["U"] * int(T) * row, "K")
    _dev(V, m["U"] * int(T) * row, "V")


def _step_args(h, q, k, v, out, victim_out):
    m = _info(h)
    row = m["d"] * m["in_size"]
    _dev(q, m["U"] * m["G"] * row, "q")
    _dev(k, m["U"] * row, "k")
    _dev(v, m["U"] * row, "v")
    _dev(out, m["U"] * m["G"] * m["d"] * 4, "out", ("float32",))
    _dev(victim_out, m["U"] * 4, "victim_out", ("int32",))


def _state_args(h, K, V, score, pos, code, occupancy, next_pos):
    m = _info(h)
    UB = m["U"] * m["B"]
    _host(K, m["elem"], UB * m["row"], "K")
    _host(V, m["elem"], UB * m["row"], "V")
    _host(score, np.float64, UB, "score")
    _host(pos, np.int32, UB, "pos")
    _host(code, np.uint32, UB, "code")
    _host(occupancy, np.int32, m["U"], "occupancy")
    _host(next_pos, np.int32, m["U"], "next_pos")


def fg_init(budget, heavy, recent, full_budget, tau, batch, heads, head_dim, dtype, scale, stream=None):
    h = _vp()
    _check(lib().fg_init(ctypes.byref(h), budget, heavy, recent, full_budget, float(tau), batch, heads, head_dim,
                         dtype, float(scale), _stream(stream)))
    return _remember(h.value, "fg", batch * heads, max(budget, full_budget), head_dim, dtype)


def fg_prefill(h, Q, K, V, T):
    _prompt_args(h, Q, K, V, T)
    _check(lib().fg_prefill(h, _ptr(Q), _ptr(K), _ptr(V), int(T)))
    _info(h)["T"] = int(T)


def fg_decode_step(h, q, k, v, out, victim_out=None):
    _step_args(h, q, k, v, out, victim_out)
    _check(lib().fg_decode_step(h, _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(victim_out)))


def fg_get_policy(h, policy=None, rec_local=None, rec_freq=None):
    U = _info(h)["U"]
    _host(policy, np.int32, U, "policy")
    _host(rec_local, np.float64, U, "rec_local")
    _host(rec_freq, np.float64, U, "rec_freq")
    _check(lib().fg_get_policy(h, _ptr(policy), _ptr(rec_local), _ptr(rec_freq)))


def h2o_get_state(h, K=None, V=None, score=None, pos=None, code=None, occupancy=None, next_pos=None):
    _state_args(h, K, V, score, pos, code, occupancy, next_pos)
    _check(lib().h2o_get_state(h, _ptr(K), _ptr(V), _ptr(score), _ptr(pos), _ptr(code), _ptr(occupancy),
                               _ptr(next_pos)))


def h2o_set_state(h, K=None, V=None, score=None, pos=None, code=None, occupancy=None, next_pos=None):
    _state_args(h, K, V, score, pos, code, occupancy, next_pos)
    _check(lib().h2o_set_state(h, _ptr(K), _ptr(V), _ptr(score), _ptr(pos), _ptr(code), _ptr(occupancy),
                               _ptr(next_pos)))


def h2o_get_prefill_stats(h, m=None, l=None, c=None):
    i = _info(h)
    n = i["U"] * i["T"]
    _host(m, np.float32, n * i["G"], "m")
    _host(l, np.float32, n * i["G"], "l")
    _host(c, np.float64, n, "c")
    _check(lib().h2o_get_prefill_stats(h, _ptr(m), _ptr(l), _ptr(c)))


def h2o_get_kv_scales(h, kscale=None, vscale=None):
    i = _info(h)
    _host(kscale, np.float32, i["U"] * i["B"], "kscale")
    _host(vscale, np.float32, i["U"] * i["B"], "vscale")
    _check(lib().h2o_get_kv_scales(h, _ptr(kscale), _ptr(vscale)))


def h2o_set_kv_scales(h, kscale, vscale):
    i = _info(h)
    _host(kscale, np.float32, i["U"] * i["B"], "kscale")
    _host(vscale, np.float32, i["U"] * i["B"], "vscale")
    _check(lib().h2o_set_kv_scales(h, _ptr(kscale), _ptr(vscale)))


def h2o_set_stream(h, stream):
    _check(lib().h2o_set_stream(h, _stream(stream)))


def h2o_set_decode_split(h, ctas_per_unit):
    _check(lib().h2o_set_decode_split(h, int(ctas_per_unit)))


def h2o_sync(h):
    _check(lib().h2o_sync(h))


def h2o_destroy(h):
    lib().h2o_destroy(h)
    _meta.pop(h, None)


def h2o_selftest_wait_timeout(h):
    _check(lib().h2o_selftest_wait_timeout(h))


def h2o_prompt_scores_noalloc(Q, K, batch, heads, T, head_dim, dtype, scale, c, stream=None):
    """Prompt column sums into ``c`` without any device allocation (scratch
    is a fixed array inside the library); see include/h2o.h."""
    esz = 2 if dtype & H2O_BF16 else 4
    _dev(Q, batch * heads * int(T) * head_dim * esz, "Q")
    _dev(K, batch * heads * int(T) * head_dim * esz, "K")
    _dev(c, batch * heads * int(T) * 8, "c", ("float64",))
    _check(lib().h2o_prompt_scores_noalloc(_ptr(Q), _ptr(K), batch, heads, int(T), head_dim, dtype,
                                           float(scale), _ptr(c), _stream(stream)))


# ------------------------------------------------------------- paged caches
#
# A decode step's kernels take a few microseconds, so the checks are made of
# the cheapest comparisons there are; what is wrong is found out afterwards.

_CODES = {"torch.bfloat16": H2O_BF16, "torch.float32": H2O_F32}
_types = None          # (int32, uint8, {element type: its code}, the current device's index, its current stream)


def _torch_types():
    global _types
    if _types is None:
        import torch
        _types = (torch.int32, torch.uint8, {getattr(torch, k[6:]): v for k, v in _CODES.items()}, torch.cuda.current_device,
                  torch.cuda.current_stream)
    return _types


def _wrong(x, what, dtype, shape, device):
    """Raise for a tensor that is not a contiguous one of `dtype` and `shape` on `device`."""
    if not hasattr(x, "data_ptr"):
        raise TypeError("%s must be a tensor" % what)
    if x.dtype is not dtype:
        raise TypeError("%s must be of dtype %s (got %s)" % (what, dtype, x.dtype))
    if x.get_device() != device:
        raise ValueError("%s must be on %s (got %s)" % (what, "cuda:%d" % device if device >= 0 else "the CPU", x.device))
    if x.shape != shape and not (len(shape) == 1 and x.numel() == shape[0]):
        raise ValueError("%s must have shape %s (got %s)" % (what, list(shape), list(x.shape)))
    raise ValueError("%s must be contiguous" % what)


def _tensor(x, what, dtype, shape, device):
    """The pointer of a contiguous tensor of `dtype` and `shape` on device `device`."""
    try:
        if x.dtype is dtype and x.shape == shape and x.get_device() == device and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    _wrong(x, what, dtype, shape, device)


def _array(x, what, dtype, n, device):
    """The pointer of a contiguous tensor of n elements of `dtype` on device `device`."""
    try:
        if x.dtype is dtype and x.numel() == n and x.get_device() == device and x.is_contiguous():
            return x.data_ptr()
    except AttributeError:
        pass
    _wrong(x, what, dtype, (n,), device)


def _head_rows(x, what, dtype, shape, device):
    """Pointer and row stride of [rows][heads][channels] whose rows may lie apart."""
    try:
        if x.dtype is dtype and x.shape == shape and x.get_device() == device:
            rows, heads, d = shape
            s = x.stride()
            if s[2] != 1 or (heads > 1 and s[1] != d):
                raise ValueError("%s must have contiguous heads and channels" % what)
            return x.data_ptr(), s[0] if rows > 1 else heads * d
    except AttributeError:
        pass
    _wrong(x, what, dtype, shape, device)


def _dim(x, what, rank):
    """x's shape, which has `rank` dimensions."""
    shape = getattr(x, "shape", None)
    if shape is None or not hasattr(x, "data_ptr"):
        raise TypeError("%s must be a tensor" % what)
    if len(shape) != rank:
        raise ValueError("%s must have %d dimensions (got %s)" % (what, rank, list(shape)))
    return shape


def _count(x, what):
    if not hasattr(x, "data_ptr"):
        raise TypeError("%s must be a tensor" % what)
    return x.numel()


def _on_current(x, current):
    """The index of the GPU that x is on, which is the current device."""
    device = x.get_device()
    if device < 0:
        raise ValueError("tensors must be on the GPU (got %s)" % x.device)
    if device != current():
        raise ValueError("tensors are on cuda:%d, which is not the current device" % device)
    return device


def _on_stream(stream):
    """The stream's handle; None: torch's current one, as for any other work on tensors."""
    return _stream(_types[4]() if stream is None else stream)


def _pool(K, V):
    """(device, element type, its code, K's and V's pointers, K's shape) of a page pool."""
    types = _torch_types()
    shape = getattr(K, "shape", None)
    code = types[2].get(getattr(K, "dtype", None))
    if code is None:
        raise TypeError("K must be a tensor of dtype float32 or bfloat16 (got %s)" % getattr(K, "dtype", type(K)))
    if len(shape) != 4:
        raise ValueError("K must be [pages][kv_heads][page_size][head_dim] (got %s)" % list(shape))
    device = _on_current(K, types[3])
    dt = K.dtype
    return device, dt, code, _tensor(K, "K", dt, shape, device), _tensor(V, "V", dt, shape, device), shape


def h2o_page_tables(len_before, n_new, free_pages, page_size, table, len_after, row_start, row_seq, row_pos, slot, status,
                    stream=None):
    """Pages and slots of a step's new tokens; see include/h2o.h.  All int32:
    len_before, n_new, len_after [requests], free_pages [any], table
    [requests][width], row_start [requests + 1], row_seq, row_pos, slot
    [rows_cap], status [4]."""
    types = _torch_types()
    i32, current = types[0], types[3]
    n, width = _dim(table, "table", 2)
    dev = _on_current(table, current)
    free, cap = _count(free_pages, "free_pages"), _count(slot, "slot")
    rc = lib().h2o_page_tables(
        _array(len_before, "len_before", i32, n, dev), _array(n_new, "n_new", i32, n, dev), n,
        _array(free_pages, "free_pages", i32, free, dev), free, page_size, _array(table, "table", i32, n * width, dev), width,
        _array(len_after, "len_after", i32, n, dev), _array(row_start, "row_start", i32, n + 1, dev),
        _array(row_seq, "row_seq", i32, cap, dev), _array(row_pos, "row_pos", i32, cap, dev), _array(slot, "slot", i32, cap, dev),
        cap, _array(status, "status", i32, 4, dev), _on_stream(stream))
    if rc:
        _check(rc)


def h2o_page_write(k, v, slot, K, V, bounds, stream=None):
    """Key and value rows [rows][kv_heads][head_dim] into their slots; see include/h2o.h."""
    dev, dt, code, Kp, Vp, (pages, heads, ps, d) = _pool(K, V)
    rows = _count(slot, "slot")
    shape = (rows, heads, d)
    kp, ks = _head_rows(k, "k", dt, shape, dev)
    vp, vs = _head_rows(v, "v", dt, shape, dev)
    rc = lib().h2o_page_write(kp, vp, ks, vs, _array(slot, "slot", _types[0], rows, dev), rows, Kp, Vp,
                              _tensor(bounds, "bounds", dt, (pages, heads, 2, d), dev), pages, heads, ps, d, code,
                              _on_stream(stream))
    if rc:
        _check(rc)


def _query_rows(q, row_seq, row_pos, table, out, dev, dt, heads, d):
    i32 = _types[0]
    n, width = _dim(table, "table", 2)
    rows, hq, _ = _dim(q, "q", 3)
    if hq < 1 or heads < 1 or hq % heads:
        raise ValueError("q must be [rows][kv_heads * groups][head_dim] (got %s for %d cache heads)" % (list(q.shape), heads))
    shape = (rows, hq, d)
    qp, qs = _head_rows(q, "q", dt, shape, dev)
    op, os_ = _head_rows(out, "out", dt, shape, dev)
    return (qp, qs, _array(row_seq, "row_seq", i32, rows, dev), _array(row_pos, "row_pos", i32, rows, dev), rows,
            hq // heads, _array(table, "table", i32, n * width, dev), n, width, op, os_)


def h2o_page_attend(q, row_seq, row_pos, K, V, bounds, table, budget, recent, scale, out, picked=None, stream=None):
    """Attention over the `recent` newest pages and the best-scoring others;
    see include/h2o.h."""
    dev, dt, code, Kp, Vp, (pages, heads, ps, d) = _pool(K, V)
    qp, qs, sp, pp, rows, groups, tp, n, width, op, os_ = _query_rows(q, row_seq, row_pos, table, out, dev, dt, heads, d)
    bp = None if bounds is None else _tensor(bounds, "bounds", dt, (pages, heads, 2, d), dev)
    kp = None if picked is None else _tensor(picked, "picked", _types[0], (rows, heads, budget), dev)
    rc = lib().h2o_page_attend(qp, qs, sp, pp, rows, Kp, Vp, bp, pages, heads, groups, ps, d, code, tp, n, width, budget,
                               recent, scale, op, os_, kp, _on_stream(stream))
    if rc:
        _check(rc)


def h2o_prefix_work_bytes(rows, kv_heads, groups, head_dim, prefix_len, dtype):
    n = lib().h2o_prefix_work_bytes(rows, kv_heads, groups, head_dim, prefix_len, dtype)
    if n < 0:
        raise H2OError(int(n), h2o_last_error())
    return n


def h2o_prefix_attend(q, row_seq, row_pos, K, V, prefix_table, prefix_len, table, scale, out, work, stream=None):
    """Attention over a prefix that all rows share and each request's own
    pages; work: a uint8 tensor of h2o_prefix_work_bytes.  See include/h2o.h."""
    dev, dt, code, Kp, Vp, (pages, heads, ps, d) = _pool(K, V)
    qp, qs, sp, pp, rows, groups, tp, n, width, op, os_ = _query_rows(q, row_seq, row_pos, table, out, dev, dt, heads, d)
    xp = None
    if prefix_table is not None:
        listed = _count(prefix_table, "prefix_table")
        xp = _array(prefix_table, "prefix_table", _types[0], listed, dev)
        if listed * ps < prefix_len:
            raise ValueError("prefix_table lists %d pages of %d tokens, prefix_len is %d" % (listed, ps, prefix_len))
    size = _count(work, "work")
    rc = lib().h2o_prefix_attend(qp, qs, sp, pp, rows, Kp, Vp, pages, heads, groups, ps, d, code, xp, prefix_len, tp, n,
                                 width, scale, op, os_, _array(work, "work", _types[1], size, dev), size, _on_stream(stream))
    if rc:
        _check(rc)
