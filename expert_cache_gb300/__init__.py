"""Python binding of libft, the GB300 routed-expert cache (argument marshalling only).

Every function below forwards to the C function of the same name declared in
``include/ft.h``; tensors are passed as raw pointers (``tensor.data_ptr()``) and
streams as ``torch.cuda.Stream.cuda_stream`` handles.  No step of the hot path
runs in Python.  Importing this module fails loudly when ``libft.so`` has not
been built (``python -m expert_cache_gb300.build`` or ``__graft_entry__.build()``).
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libft.so")

FT_OK, FT_ERR_ARG, FT_ERR_CUDA, FT_ERR_CAPACITY, FT_ERR_STATE, FT_ERR_TIMEOUT, FT_ERR_UNPINNED = range(7)
FT_DEV_BAD_ID, FT_DEV_TIMEOUT, FT_DEV_SCALE_RANGE = 0x1, 0x2, 0x4
FT_FORMAT_NVFP4, FT_FORMAT_MXFP4 = 0, 1
FORMATS = {"nvfp4": FT_FORMAT_NVFP4, "mxfp4": FT_FORMAT_MXFP4}
FT_SPLIT_FULL_OFFLOAD, FT_SPLIT_QSTAR = 0, 1
FT_PREFILL_DOUBLE_BUFFER = 1
FT_PREFILL_DEBUG_X = 2
FT_PREFILL_ON_DEMAND = 4
FT_BACKEND_OFFLOAD, FT_BACKEND_HYBRID = 0, 1
FT_KV_NVFP4, FT_KV_FP8 = 0, 1
KV_FORMATS = {"nvfp4": FT_KV_NVFP4, "fp8": FT_KV_FP8}
FT_PROF_KINDS = 5
PROF_NAMES = ("decode", "prefill_gemm1", "prefill_gemm2", "prefill_other", "prefill_copy")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")

_lib = ctypes.CDLL(LIB_PATH)

c_void_p, c_int32, c_uint32, c_int64, c_size_t, c_double, c_float = (
    ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_size_t,
    ctypes.c_double, ctypes.c_float)


class FtSplit(ctypes.Structure):
    _fields_ = [("mode", c_int32), ("f_q16", c_uint32)]


class FtCacheDesc(ctypes.Structure):
    _fields_ = [("L", c_int32), ("E", c_int32), ("H", c_int32), ("I", c_int32),
                ("k_max", c_int32), ("B_max", c_int32), ("capacity", c_int32),
                ("capacity_max", c_int32), ("T_max", c_int32),
                ("host_pool", c_void_p), ("slot_buf", c_void_p), ("workspace", c_void_p),
                ("shared_experts", c_void_p), ("split", FtSplit), ("format", c_int32)]


class FtHostDesc(ctypes.Structure):
    _fields_ = [("L", c_int32), ("E", c_int32), ("H", c_int32), ("I", c_int32),
                ("k_max", c_int32), ("B_max", c_int32), ("format", c_int32),
                ("host_pool", c_void_p), ("n_threads", c_int32), ("cpus", c_void_p),
                ("mailbox", c_void_p)]


class FtBwProfile(ctypes.Structure):
    _fields_ = [("pcie_gbs", c_double), ("cpu_gbs", c_double), ("pcie_ov_gbs", c_double),
                ("cpu_ov_gbs", c_double), ("recommend", c_int32), ("f_q16", c_uint32),
                ("n_records", c_int32)]


class FtKvDesc(ctypes.Structure):
    _fields_ = [("L", c_int32), ("n_pages", c_int32), ("page_size", c_int32), ("n_kv_heads", c_int32),
                ("head_dim", c_int32), ("n_q_heads", c_int32), ("max_seqs", c_int32),
                ("format", c_int32), ("k_scale", c_float), ("v_scale", c_float),
                ("pool", c_void_p), ("workspace", c_void_p)]


def _sig(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_P = ctypes.POINTER
_f = {
    "ft_record_bytes": _sig("ft_record_bytes", c_int32, c_int32, c_int32, _P(c_size_t)),
    "ft_record_bytes_format": _sig("ft_record_bytes_format", c_int32, c_int32, c_int32, c_int32,
                                   _P(c_size_t)),
    "ft_quantize_experts_mx": _sig("ft_quantize_experts_mx", c_int32, c_void_p, c_void_p, c_int32,
                                   c_int32, c_int32, c_void_p, c_void_p),
    "ft_cache_required_sizes": _sig("ft_cache_required_sizes", c_int32, _P(FtCacheDesc),
                                    _P(c_size_t), _P(c_size_t)),
    "ft_cache_create": _sig("ft_cache_create", c_int32, _P(FtCacheDesc), _P(c_void_p)),
    "ft_cache_destroy": _sig("ft_cache_destroy", None, c_void_p),
    "ft_cache_resize": _sig("ft_cache_resize", c_int32, c_void_p, c_int32, c_void_p, c_void_p),
    "ft_set_split": _sig("ft_set_split", c_int32, c_void_p, FtSplit),
    "ft_split_from_bandwidth": _sig("ft_split_from_bandwidth", c_uint32, c_double, c_double),
    "ft_split_from_overlap": _sig("ft_split_from_overlap", c_uint32, c_double, c_double),
    "ft_moe_decode": _sig("ft_moe_decode", c_int32, c_void_p, c_int32, c_void_p, c_void_p,
                          c_void_p, c_int32, c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                          c_void_p),
    "ft_moe_decode_static": _sig("ft_moe_decode_static", c_int32, c_void_p, c_int32, c_void_p,
                                 c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_void_p,
                                 c_void_p, c_void_p, c_void_p),
    "ft_moe_prefill_layer": _sig("ft_moe_prefill_layer", c_int32, c_void_p, c_int32, c_void_p,
                                 c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_int32,
                                 c_void_p, c_void_p),
    "ft_cache_snapshot": _sig("ft_cache_snapshot", c_int32, c_void_p, c_void_p, c_void_p,
                              c_void_p, c_void_p),
    "ft_cache_restore": _sig("ft_cache_restore", c_int32, c_void_p, c_void_p, c_void_p, c_void_p,
                             c_int64, c_void_p),
    "ft_cache_set_trace": _sig("ft_cache_set_trace", c_int32, c_void_p, c_void_p, c_int32),
    "ft_cache_capacity": _sig("ft_cache_capacity", c_int32, c_void_p, _P(c_int32)),
    "ft_cache_status": _sig("ft_cache_status", c_int32, c_void_p, _P(c_int32)),
    "ft_check_bounded_waits": _sig("ft_check_bounded_waits", c_int32, _P(c_uint32)),
    "ft_quantize_experts": _sig("ft_quantize_experts", c_int32, c_void_p, c_void_p, c_int32,
                                c_int32, c_int32, c_void_p, c_void_p),
    "ft_pinned_alloc": _sig("ft_pinned_alloc", c_int32, c_size_t, _P(c_void_p)),
    "ft_pinned_free": _sig("ft_pinned_free", c_int32, c_void_p),
    "ft_measure_h2d": _sig("ft_measure_h2d", c_int32, c_void_p, c_void_p, c_size_t, c_int32,
                           _P(c_double)),
    "ft_profile_enable": _sig("ft_profile_enable", c_int32, c_void_p, c_int32),
    "ft_profile_read": _sig("ft_profile_read", c_int32, c_void_p, _P(c_double), _P(c_int64)),
    "ft_host_mailbox_bytes": _sig("ft_host_mailbox_bytes", c_int32, c_int32, c_int32, c_int32,
                                  _P(c_size_t)),
    "ft_host_branch_create": _sig("ft_host_branch_create", c_int32, _P(FtHostDesc), _P(c_void_p)),
    "ft_host_branch_destroy": _sig("ft_host_branch_destroy", None, c_void_p),
    "ft_host_moe": _sig("ft_host_moe", c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32,
                        c_int32, c_void_p),
    "ft_host_branch_stats": _sig("ft_host_branch_stats", c_int32, c_void_p, _P(c_int64), _P(c_int64)),
    "ft_cache_set_host_branch": _sig("ft_cache_set_host_branch", c_int32, c_void_p, c_void_p),
    "ft_profile_bandwidth": _sig("ft_profile_bandwidth", c_int32, c_void_p, c_void_p, c_int32,
                                 c_void_p, _P(FtBwProfile)),
    "ft_recommend_backend": _sig("ft_recommend_backend", c_int32, c_double, c_double),
    "ft_kv_required_sizes": _sig("ft_kv_required_sizes", c_int32, _P(FtKvDesc), _P(c_size_t),
                                 _P(c_size_t)),
    "ft_kv_create": _sig("ft_kv_create", c_int32, _P(FtKvDesc), _P(c_void_p)),
    "ft_kv_destroy": _sig("ft_kv_destroy", None, c_void_p),
    "ft_kv_append": _sig("ft_kv_append", c_int32, c_void_p, c_int32, c_void_p, c_void_p, c_int64,
                         c_int64, c_void_p, c_int32, c_void_p),
    "ft_kv_read": _sig("ft_kv_read", c_int32, c_void_p, c_int32, c_void_p, c_int32, c_void_p,
                       c_void_p, c_void_p),
    "ft_kv_attention": _sig("ft_kv_attention", c_int32, c_void_p, c_void_p, c_void_p),
    "ft_kv_status": _sig("ft_kv_status", c_int32, c_void_p, _P(c_int32)),
    "ft_kv_check_bounded_waits": _sig("ft_kv_check_bounded_waits", c_int32, _P(c_uint32)),
    "ft_kv_last_error": _sig("ft_kv_last_error", ctypes.c_char_p, c_void_p),
    "ft_status_string": _sig("ft_status_string", ctypes.c_char_p, c_int32),
    "ft_last_error": _sig("ft_last_error", ctypes.c_char_p, c_void_p),
}

EXPORTED = tuple(_f)


class FtError(RuntimeError):
    def __init__(self, status, msg=""):
        super().__init__(f"{_f['ft_status_string'](status).decode()} ({status}) {msg}".strip())
        self.status = status


def _ptr(t):
    """Raw address of a tensor / ndarray / int / None."""
    try:
        return t.data_ptr()
    except AttributeError:
        pass
    if t is None or isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    raise TypeError(f"cannot take the address of {type(t)}")


_raw_stream = None


def _stream(s):
    """cudaStream_t of a stream; None: torch's current one (asked for without building a
    Stream object, which costs 3 us a call)."""
    global _raw_stream
    if s is None:
        if _raw_stream is None:
            import torch
            raw, device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
            torch.cuda.init()
            _raw_stream = raw, getattr(torch._C, "_cuda_getDevice", device)
        raw, device = _raw_stream
        return raw(device())
    return s if isinstance(s, int) else s.cuda_stream


def _check(status, handle=None):
    if status != FT_OK:
        msg = _f["ft_last_error"](handle).decode() if handle else ""
        raise FtError(status, msg)


# ----------------------------------------------------------------- thin wrappers

def ft_record_bytes(H, I, fmt="nvfp4"):
    out = c_size_t()
    if fmt == "nvfp4":
        _check(_f["ft_record_bytes"](H, I, ctypes.byref(out)))
    else:
        _check(_f["ft_record_bytes_format"](FORMATS[fmt], H, I, ctypes.byref(out)))
    return out.value


def ft_cache_required_sizes(desc: FtCacheDesc):
    rb, wb = c_size_t(), c_size_t()
    _check(_f["ft_cache_required_sizes"](ctypes.byref(desc), ctypes.byref(rb), ctypes.byref(wb)))
    return rb.value, wb.value


def ft_cache_create(desc: FtCacheDesc):
    h = c_void_p()
    _check(_f["ft_cache_create"](ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def ft_cache_destroy(handle):
    _f["ft_cache_destroy"](handle)


def ft_cache_resize(handle, new_capacity, new_slot_buf, stream=None):
    _check(_f["ft_cache_resize"](handle, new_capacity, _ptr(new_slot_buf), _stream(stream)), handle)


def ft_set_split(handle, mode, f_q16=65536):
    _check(_f["ft_set_split"](handle, FtSplit(mode, f_q16)), handle)


def ft_split_from_bandwidth(b_p, b_h):
    return int(_f["ft_split_from_bandwidth"](b_p, b_h))


def ft_split_from_overlap(p_ov, c_ov):
    return int(_f["ft_split_from_overlap"](p_ov, c_ov))


def ft_moe_decode(handle, layer, x, topk_ids, topk_w, B, k, y, deferred, route_slot=None,
                  counters=None, stream=None):
    _check(_f["ft_moe_decode"](handle, layer, _ptr(x), _ptr(topk_ids), _ptr(topk_w), B, k,
                               _ptr(y), _ptr(deferred), _ptr(route_slot), _ptr(counters),
                               _stream(stream)), handle)


def ft_moe_decode_static(handle, layer, x, topk_ids, topk_w, B, k, y, deferred, route_slot=None,
                         counters=None, stream=None):
    _check(_f["ft_moe_decode_static"](handle, layer, _ptr(x), _ptr(topk_ids), _ptr(topk_w), B, k,
                                      _ptr(y), _ptr(deferred), _ptr(route_slot), _ptr(counters),
                                      _stream(stream)), handle)


def ft_moe_prefill_layer(handle, layer, x, topk_ids, topk_w, T, k, y, flags=FT_PREFILL_DOUBLE_BUFFER,
                         debug_h=None, stream=None):
    _check(_f["ft_moe_prefill_layer"](handle, layer, _ptr(x), _ptr(topk_ids), _ptr(topk_w), T, k,
                                      _ptr(y), flags, _ptr(debug_h), _stream(stream)), handle)


def ft_cache_capacity(handle):
    c = c_int32()
    _check(_f["ft_cache_capacity"](handle, ctypes.byref(c)), handle)
    return c.value


def ft_cache_snapshot(handle, L, E):
    """(slot_for_id [L*E], id_of_slot [C], usage [C], tick) as numpy arrays / int."""
    C = ft_cache_capacity(handle)
    sfi = np.empty(L * E, np.int32)
    ios = np.empty(C, np.int32)
    usage = np.empty(C, np.int64)
    tick = np.empty(1, np.int64)
    _check(_f["ft_cache_snapshot"](handle, sfi.ctypes.data, ios.ctypes.data, usage.ctypes.data,
                                   tick.ctypes.data), handle)
    return sfi, ios, usage, int(tick[0])


def ft_cache_restore(handle, slot_for_id, id_of_slot, usage, tick, stream=None):
    sfi = np.ascontiguousarray(slot_for_id, np.int32)
    ios = np.ascontiguousarray(id_of_slot, np.int32)
    us = np.ascontiguousarray(usage, np.int64)
    _check(_f["ft_cache_restore"](handle, sfi.ctypes.data, ios.ctypes.data, us.ctypes.data,
                                  int(tick), _stream(stream)), handle)


# one stats-ring record: tick, layer, n_hit, m, q, n_def_routes, n_units, t_commit_ns
TRACE_DTYPE = np.dtype([("tick", np.int64), ("layer", np.int32), ("n_hit", np.int32),
                        ("m", np.int32), ("q", np.int32), ("n_def_routes", np.int32),
                        ("n_units", np.int32), ("t_commit_ns", np.int64)])
TRACE_HEADER_BYTES = 16


def ft_cache_set_trace(handle, ring, capacity):
    _check(_f["ft_cache_set_trace"](handle, _ptr(ring), int(capacity)), handle)


def trace_records(ring_bytes: np.ndarray, capacity: int):
    """(count, records in write order) of a stats ring copied to the host."""
    count = int(ring_bytes[:8].view(np.uint64)[0])
    recs = ring_bytes[TRACE_HEADER_BYTES:TRACE_HEADER_BYTES + capacity * TRACE_DTYPE.itemsize]
    recs = recs.view(TRACE_DTYPE)
    n = min(count, capacity)
    start = count % capacity if count > capacity else 0
    order = [(start + i) % capacity for i in range(n)]
    return count, recs[order]


def ft_cache_status(handle):
    s = c_int32()
    _check(_f["ft_cache_status"](handle, ctypes.byref(s)), handle)
    return s.value


def ft_check_bounded_waits():
    bits = c_uint32()
    _check(_f["ft_check_bounded_waits"](ctypes.byref(bits)))
    return bits.value


def ft_quantize_experts(w_gu, w_d, n, H, I, records, stream=None, fmt="nvfp4"):
    name = "ft_quantize_experts" if fmt == "nvfp4" else "ft_quantize_experts_mx"
    _check(_f[name](_ptr(w_gu), _ptr(w_d), n, H, I, _ptr(records), _stream(stream)))


def ft_pinned_alloc(nbytes):
    p = c_void_p()
    _check(_f["ft_pinned_alloc"](nbytes, ctypes.byref(p)))
    return p.value


def ft_pinned_free(ptr):
    _check(_f["ft_pinned_free"](ptr))


def ft_measure_h2d(pinned, dev, nbytes, reps=5):
    g = c_double()
    _check(_f["ft_measure_h2d"](_ptr(pinned), _ptr(dev), nbytes, reps, ctypes.byref(g)))
    return g.value


FT_PROF_ALL = (1 << FT_PROF_KINDS) - 1


def ft_profile_enable(handle, kinds=True):
    """kinds: True (all kinds), False (off) or a bit mask of kinds (bit i: kind i)."""
    mask = FT_PROF_ALL if kinds is True else (0 if kinds is False else int(kinds))
    _check(_f["ft_profile_enable"](handle, mask), handle)


def ft_profile_read(handle):
    ms = (c_double * FT_PROF_KINDS)()
    n = (c_int64 * FT_PROF_KINDS)()
    _check(_f["ft_profile_read"](handle, ms, n), handle)
    return {PROF_NAMES[i]: (ms[i], n[i]) for i in range(FT_PROF_KINDS)}


def ft_host_mailbox_bytes(H, k_max, B_max):
    n = c_size_t()
    _check(_f["ft_host_mailbox_bytes"](H, k_max, B_max, ctypes.byref(n)))
    return n.value


def ft_host_branch_create(desc: FtHostDesc):
    h = c_void_p()
    _check(_f["ft_host_branch_create"](ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def ft_host_branch_destroy(hb):
    _f["ft_host_branch_destroy"](hb)


def ft_host_moe(hb, x, deferred, w, B, k, y):
    _check(_f["ft_host_moe"](hb, _ptr(x), _ptr(deferred), _ptr(w), B, k, _ptr(y)))


def ft_host_branch_stats(hb):
    jobs, mb = c_int64(), c_int64()
    _check(_f["ft_host_branch_stats"](hb, ctypes.byref(jobs), ctypes.byref(mb)))
    return jobs.value, mb.value


def ft_cache_set_host_branch(handle, hb):
    _check(_f["ft_cache_set_host_branch"](handle, hb), handle)


def ft_profile_bandwidth(handle, hb, n_records, stream=None):
    out = FtBwProfile()
    _check(_f["ft_profile_bandwidth"](handle, hb, n_records, _stream(stream), ctypes.byref(out)), handle)
    return {k: getattr(out, k) for k, _ in FtBwProfile._fields_}


def ft_recommend_backend(cpu_gbs, pcie_gbs):
    return _f["ft_recommend_backend"](cpu_gbs, pcie_gbs)


def _check_kv(status, handle=None):
    if status != FT_OK:
        raise FtError(status, _f["ft_kv_last_error"](handle).decode() if handle else "")


def ft_kv_required_sizes(desc: FtKvDesc):
    """(pool bytes, workspace bytes)"""
    pb, wb = c_size_t(), c_size_t()
    _check_kv(_f["ft_kv_required_sizes"](ctypes.byref(desc), ctypes.byref(pb), ctypes.byref(wb)))
    return pb.value, wb.value


def ft_kv_create(desc: FtKvDesc):
    if _bf16 is None:
        _load_types()
    h = c_void_p()
    _check_kv(_f["ft_kv_create"](ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def ft_kv_destroy(handle):
    _f["ft_kv_destroy"](handle)


_bf16 = _i32 = _f32 = _i64 = _u64 = None                    # torch's types, known from the first handle on


def _load_types():
    global _bf16, _i32, _f32, _i64, _u64
    try:
        import torch
    except ImportError:                                     # raw addresses only
        return
    _bf16, _i32, _f32, _i64, _u64 = torch.bfloat16, torch.int32, torch.float32, torch.int64, torch.uint64


def _refuse(t, what, needs):
    raise FtError(FT_ERR_ARG, f"{what}: {t.dtype}, sizes {tuple(t.shape)}, strides {t.stride()}; needs {needs}")


def _address(t, dtype, what, dense=True):
    """Address of an array.  A raw one stands for itself; a tensor has to be of the type, and dense."""
    try:
        p = t.data_ptr()
    except AttributeError:
        return _ptr(t) or 0
    if t.dtype is not dtype or (dense and not t.is_contiguous()):
        _refuse(t, what, f"dense {dtype}" if dense else dtype)
    return p


def _inner_dense(t, s):
    at = 1
    for n, x in zip(t.shape[:0:-1], s[:0:-1]):
        if x != at and n != 1:
            return False
        at *= n
    return True


def _token_stride(t, what):
    """Token stride in elements of a tensor whose tokens are dense.  That of a single token means nothing: its
    elements, rounded to what the calls ask for."""
    try:
        s = t.stride()
    except AttributeError:
        raise TypeError(f"{what}: a raw address needs its token stride") from None
    if not ((len(s) == 2 and s[1] == 1) or t.is_contiguous() or _inner_dense(t, s)):
        _refuse(t, what, "dense rows, or a token stride")
    return s[0] if t.shape[0] != 1 else t.numel() + 7 & ~7


# The calls below look at the tensors' types and strides themselves where that takes one test per tensor (a call's host
# time is a step's), and leave raw addresses and refusals to _address.  A token stride that is given says how the
# tensor's memory is meant; one that is not is the tensor's.
_kv_append, _kv_read, _kv_attention = _f["ft_kv_append"], _f["ft_kv_read"], _f["ft_kv_attention"]


def ft_kv_append(handle, layer, k, v, slots, n, k_stride=None, v_stride=None, stream=None):
    try:
        pk, pv, ps = k.data_ptr(), v.data_ptr(), slots.data_ptr()
        plain = k.dtype is _bf16 and v.dtype is _bf16 and slots.dtype is _i32 and slots.is_contiguous()
    except AttributeError:
        plain = False
    if not plain:
        pk, pv = _address(k, _bf16, "append: k", False), _address(v, _bf16, "append: v", False)
        ps = _address(slots, _i32, "append: slots")
    if k_stride is None:
        k_stride = _token_stride(k, "append: k")
    if v_stride is None:
        v_stride = _token_stride(v, "append: v")
    status = _kv_append(handle, layer, pk, pv, k_stride, v_stride, ps, n, _stream(stream))
    if status:
        _check_kv(status, handle)


def ft_kv_read(handle, layer, slots, n, k_out, v_out, stream=None):
    try:
        ps, pk, pv = slots.data_ptr(), k_out.data_ptr(), v_out.data_ptr()
        plain = (slots.dtype is _i32 and k_out.dtype is _bf16 and v_out.dtype is _bf16 and slots.is_contiguous()
                 and k_out.is_contiguous() and v_out.is_contiguous())
    except AttributeError:
        plain = False
    if not plain:
        ps = _address(slots, _i32, "read: slots")
        pk, pv = _address(k_out, _bf16, "read: k_out"), _address(v_out, _bf16, "read: v_out")
    status = _kv_read(handle, layer, ps, n, pk, pv, _stream(stream))
    if status:
        _check_kv(status, handle)


# ft_kv_attn, packed at once (one conversion per field would cost more than the launch)
_KV_ATTN = struct.Struct("@3P2q4P7if")


def ft_kv_attention(handle, layer, q, q_start, kv_len, block_table, table_stride, n_seqs, n_tokens,
                    max_q, o, tree_mask=None, window=0, n_sink=0, sm_scale=1.0, lse=None,
                    q_stride=None, o_stride=None, stream=None):
    try:
        pq, po, pt = q.data_ptr(), o.data_ptr(), block_table.data_ptr()
        ps, pl = q_start.data_ptr(), kv_len.data_ptr()
        plain = (q.dtype is _bf16 and o.dtype is _bf16 and block_table.dtype is _i32 and q_start.dtype is _i32
                 and kv_len.dtype is _i32 and block_table.is_contiguous() and q_start.is_contiguous()
                 and kv_len.is_contiguous())
        pe = pm = 0
        if lse is not None:
            pe = lse.data_ptr()
            plain = plain and lse.dtype is _f32 and lse.is_contiguous()
        if tree_mask is not None:
            pm = tree_mask.data_ptr()
            plain = plain and tree_mask.dtype is _i64 and tree_mask.is_contiguous()
    except AttributeError:
        plain = False
    if not plain:
        pq, po = _address(q, _bf16, "attention: q", False), _address(o, _bf16, "attention: o", False)
        pt = _address(block_table, _i32, "attention: block_table", False)        # its rows may be parts of longer ones
        if pt and not isinstance(block_table, int) and not (block_table.is_contiguous() or block_table.stride(-1) == 1):
            _refuse(block_table, "attention: block_table", "dense rows")
        ps, pl = _address(q_start, _i32, "attention: q_start"), _address(kv_len, _i32, "attention: kv_len")
        pe = _address(lse, _f32, "attention: lse")
        pm = _address(tree_mask, _u64 if getattr(tree_mask, "dtype", None) is _u64 else _i64, "attention: tree_mask")
    if q_stride is None:
        q_stride = _token_stride(q, "attention: q")
    if o_stride is None:
        o_stride = _token_stride(o, "attention: o")
    status = _kv_attention(handle, _KV_ATTN.pack(pq, po, pe, q_stride, o_stride, ps, pl, pt, pm, layer, table_stride,
                                                 n_seqs, n_tokens, max_q, window, n_sink, sm_scale), _stream(stream))
    if status:
        _check_kv(status, handle)


def ft_kv_status(handle):
    s = c_int32()
    _check_kv(_f["ft_kv_status"](handle, ctypes.byref(s)), handle)
    return s.value


def ft_kv_check_bounded_waits():
    bits = c_uint32()
    _check_kv(_f["ft_kv_check_bounded_waits"](ctypes.byref(bits)))
    return bits.value


# ----------------------------------------------------------------- memory plumbing

class PinnedBuffer:
    """Page-locked, device-mapped host bytes from ft_pinned_alloc, viewed as a
    uint8 numpy array and a CPU torch tensor sharing the same memory."""

    def __init__(self, nbytes: int):
        self.nbytes = int(nbytes)
        self.ptr = ft_pinned_alloc(self.nbytes)
        self.array = np.ctypeslib.as_array((ctypes.c_uint8 * self.nbytes).from_address(self.ptr))

    def tensor(self):
        import torch
        return torch.from_numpy(self.array)

    def free(self):
        if self.ptr:
            ft_pinned_free(self.ptr)
            self.ptr = None
            self.array = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class ExpertCache:
    """Owns the device memory of one cache (slot buffer, workspace; torch allocations)
    and the ft_cache handle over a caller-provided pinned host pool."""

    def __init__(self, L, E, H, I, k_max, B_max, capacity, host_pool_ptr, shared=None,
                 split=(FT_SPLIT_FULL_OFFLOAD, 65536), capacity_max=0, T_max=0, device="cuda",
                 fmt="nvfp4"):
        import torch
        self.L, self.E, self.H, self.I = L, E, H, I
        self.desc = FtCacheDesc(L, E, H, I, k_max, B_max, capacity, capacity_max, T_max,
                                None, None, None, None, FtSplit(*split), FORMATS[fmt])
        self.rec_bytes, ws_bytes = ft_cache_required_sizes(self.desc)
        cmax = capacity_max or capacity
        self.slot_buf = torch.empty(cmax * self.rec_bytes, dtype=torch.uint8, device=device)
        self.workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=device)
        self.shared = shared
        self.desc.host_pool = host_pool_ptr
        self.desc.slot_buf = self.slot_buf.data_ptr()
        self.desc.workspace = self.workspace.data_ptr()
        self.desc.shared_experts = _ptr(shared)
        self.handle = ft_cache_create(self.desc)

    def close(self):
        if self.handle:
            ft_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class KVCache:
    """Owns the device memory (torch allocations) and the ft_kv handle of a quantised
    key/value cache; `pool` may be given (a uint8 tensor of ft_kv_required_sizes bytes, its
    tokens are kept)."""

    def __init__(self, L, n_pages, page_size, n_kv_heads, head_dim, n_q_heads, max_seqs,
                 fmt="nvfp4", k_scale=1.0, v_scale=1.0, pool=None, device="cuda"):
        import torch
        self.handle = None
        self.desc = FtKvDesc(L, n_pages, page_size, n_kv_heads, head_dim, n_q_heads, max_seqs,
                             KV_FORMATS[fmt], k_scale, v_scale, None, None)
        self.pool_bytes, ws_bytes = ft_kv_required_sizes(self.desc)
        if pool is None:
            pool = torch.empty(self.pool_bytes, dtype=torch.uint8, device=device)
        elif pool.numel() * pool.element_size() < self.pool_bytes or not pool.is_contiguous():
            raise ValueError(f"pool must be contiguous and hold {self.pool_bytes} bytes")
        self.pool = pool
        self.workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=pool.device)
        self.desc.pool = pool.data_ptr()
        self.desc.workspace = self.workspace.data_ptr()
        self.handle = ft_kv_create(self.desc)

    def close(self):
        if self.handle:
            ft_kv_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HostBranch:
    """Owns one host branch (ft_host_branch_create) and its pinned mailbox."""

    def __init__(self, L, E, H, I, k_max, B_max, host_pool_ptr, n_threads, cpus=None, fmt="nvfp4",
                 mailbox=True):
        self.H = H
        self.mailbox = PinnedBuffer(ft_host_mailbox_bytes(H, k_max, B_max)) if mailbox else None
        self._cpus = (ctypes.c_int32 * n_threads)(*cpus) if cpus is not None else None
        self.desc = FtHostDesc(L, E, H, I, k_max, B_max, FORMATS[fmt], host_pool_ptr, n_threads,
                               ctypes.addressof(self._cpus) if self._cpus is not None else None,
                               self.mailbox.ptr if self.mailbox else None)
        self.handle = ft_host_branch_create(self.desc)

    def close(self):
        if self.handle:
            ft_host_branch_destroy(self.handle)
            self.handle = None
        if self.mailbox is not None:
            self.mailbox.free()
            self.mailbox = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
