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
FT_DEV_BAD_ID, FT_DEV_TIMEOUT, FT_DEV_SCALE_RANGE, FT_DEV_NO_PAGES = 0x1, 0x2, 0x4, 0x8
FT_FORMAT_NVFP4, FT_FORMAT_MXFP4 = 0, 1
FORMATS = {"nvfp4": FT_FORMAT_NVFP4, "mxfp4": FT_FORMAT_MXFP4}
FT_SPLIT_FULL_OFFLOAD, FT_SPLIT_QSTAR = 0, 1
FT_PREFILL_DOUBLE_BUFFER = 1
FT_PREFILL_DEBUG_X = 2
FT_PREFILL_ON_DEMAND = 4
FT_BACKEND_OFFLOAD, FT_BACKEND_HYBRID = 0, 1
FT_KV_NVFP4, FT_KV_FP8 = 0, 1
KV_FORMATS = {"nvfp4": FT_KV_NVFP4, "fp8": FT_KV_FP8}
FT_DTYPE_BF16, FT_DTYPE_F32 = 0, 1
FT_ROUTE_SOFTMAX, FT_ROUTE_SIGMOID = 0, 1
ROUTE_SCORES = {"softmax": FT_ROUTE_SOFTMAX, "sigmoid": FT_ROUTE_SIGMOID}
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
    "ft_kv_plan": _sig("ft_kv_plan", c_int32, c_void_p, c_void_p, c_void_p),
    "ft_rope_table": _sig("ft_rope_table", c_int32, c_void_p, c_int32, c_int32, c_double, c_void_p, c_void_p),
    "ft_kv_append_rotated": _sig("ft_kv_append_rotated", c_int32, c_void_p, c_void_p, c_void_p),
    "ft_moe_route": _sig("ft_moe_route", c_int32, c_void_p, c_void_p),
    "ft_logprobs": _sig("ft_logprobs", c_int32, c_void_p, c_void_p),
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


_bf16 = _i32 = _f32 = _f64 = _i64 = _u64 = None             # torch's types, known from the first handle on
_DTYPES = {}                                                # types of logits


def _load_types():
    global _bf16, _i32, _f32, _f64, _i64, _u64
    try:
        import torch
    except ImportError:                                     # raw addresses only
        return
    _bf16, _i32, _f32, _f64, _i64, _u64 = torch.bfloat16, torch.int32, torch.float32, torch.float64, torch.int64, torch.uint64
    _DTYPES.update({_bf16: FT_DTYPE_BF16, _f32: FT_DTYPE_F32})


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


def _token_stride(t, what, n):
    """Token stride in elements of a tensor of n or more tokens, one per row, that are dense.  That of a single token means
    nothing: its elements, rounded to what the calls ask for.  (Fewer rows are not tokens: n tokens at the stride of a
    batch of them would lie behind the tensor.)"""
    try:
        s = t.stride()
    except AttributeError:
        raise TypeError(f"{what}: a raw address needs its token stride") from None
    if not ((len(s) == 2 and s[1] == 1) or t.is_contiguous() or _inner_dense(t, s)):
        _refuse(t, what, "dense rows, or a token stride")
    rows = t.shape[0] if s else -1
    if rows < n or rows < 0:
        _refuse(t, what, f"a row for each of {n} tokens, or a token stride")
    return s[0] if rows != 1 else t.numel() + 7 & ~7


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
        k_stride = _token_stride(k, "append: k", n)
    if v_stride is None:
        v_stride = _token_stride(v, "append: v", n)
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
        q_stride = _token_stride(q, "attention: q", n_tokens)
    if o_stride is None:
        o_stride = _token_stride(o, "attention: o", n_tokens)
    status = _kv_attention(handle, _KV_ATTN.pack(pq, po, pe, q_stride, o_stride, ps, pl, pt, pm, layer, table_stride,
                                                 n_seqs, n_tokens, max_q, window, n_sink, sm_scale), _stream(stream))
    if status:
        _check_kv(status, handle)

# ft_kv_step, ft_kv_qkv, ft_route and ft_logprob, packed at once
_KV_STEP = struct.Struct("@14P3i4x")
_KV_QKV = struct.Struct("@5P5q5P5if")
_ONE = 1 << 40                                              # token stride of a single token, which means nothing
_ROUTE = struct.Struct("@4Pq9if")
_LOGPROB = struct.Struct("@6Pq4if4x")
_kv_plan, _kv_append_rotated, _moe_route, _logprobs = (
    _f["ft_kv_plan"], _f["ft_kv_append_rotated"], _f["ft_moe_route"], _f["ft_logprobs"])


def ft_kv_plan(handle, n_new, len, held, block_table, table_stride, free_pages, n_free, n_seqs, n_tokens, q_start, kv_len, slots,
               len_out, held_out, n_free_out, positions=None, tree_mask=None, stream=None):
    i32 = _i32
    pp = pm = 0
    try:
        p = (n_new.data_ptr(), len.data_ptr(), held.data_ptr(), n_free.data_ptr(), free_pages.data_ptr(), q_start.data_ptr(),
             kv_len.data_ptr(), slots.data_ptr(), len_out.data_ptr(), held_out.data_ptr(), n_free_out.data_ptr())
        pt = block_table.data_ptr()
        plain = (n_new.dtype is i32 and len.dtype is i32 and held.dtype is i32 and n_free.dtype is i32 and free_pages.dtype is i32
                 and q_start.dtype is i32 and kv_len.dtype is i32 and slots.dtype is i32 and len_out.dtype is i32
                 and held_out.dtype is i32 and n_free_out.dtype is i32 and block_table.dtype is i32
                 and n_new.is_contiguous() and len.is_contiguous() and held.is_contiguous() and n_free.is_contiguous()
                 and free_pages.is_contiguous() and q_start.is_contiguous() and kv_len.is_contiguous() and slots.is_contiguous()
                 and len_out.is_contiguous() and held_out.is_contiguous() and n_free_out.is_contiguous() and block_table.is_contiguous())
        if positions is not None:
            pp = positions.data_ptr()
            plain = plain and positions.dtype is i32 and positions.is_contiguous()
        if tree_mask is not None:
            pm = tree_mask.data_ptr()
            plain = plain and tree_mask.dtype is _i64 and tree_mask.is_contiguous()
    except AttributeError:
        plain = False
    if not plain:
        p = [_address(t, _i32, f"plan: {name}") for t, name in (
            (n_new, "n_new"), (len, "len"), (held, "held"), (n_free, "n_free"), (free_pages, "free_pages"), (q_start, "q_start"),
            (kv_len, "kv_len"), (slots, "slots"), (len_out, "len_out"), (held_out, "held_out"), (n_free_out, "n_free_out"))]
        pt = _address(block_table, _i32, "plan: block_table", False)             # its rows may be parts of longer ones
        if pt and not isinstance(block_table, int) and not (block_table.is_contiguous() or block_table.stride(-1) == 1):
            _refuse(block_table, "plan: block_table", "dense rows")
        pp = _address(positions, _i32, "plan: positions")
        pm = _address(tree_mask, _u64 if getattr(tree_mask, "dtype", None) is _u64 else _i64, "plan: tree_mask")
    status = _kv_plan(handle, _KV_STEP.pack(p[0], p[1], p[2], p[3], pt, p[4], pm, p[5], p[6], p[7], pp, p[8], p[9], p[10],
                                            n_seqs, table_stride, n_tokens), _stream(stream))
    if status:
        _check_kv(status, handle)


def ft_rope_table(inv_freq, rope_dim, n_positions, table, mscale=1.0, stream=None):
    if _bf16 is None:
        _load_types()
    pi, pt = _address(inv_freq, _f64, "rope_table: inv_freq"), _address(table, _f32, "rope_table: table")
    _check(_f["ft_rope_table"](pi, rope_dim, n_positions, mscale, pt, _stream(stream)))


def ft_kv_append_rotated(handle, layer, q, k, v, slots, n, q_out, positions, rope, rope_dim, n_positions, k_out=None, q_norm=None,
                         k_norm=None, eps=1e-6, interleaved=False, q_stride=None, k_stride=None, v_stride=None, q_out_stride=None,
                         k_out_stride=None, stream=None):
    pko = pqn = pkn = pr = pp = 0
    try:
        pq, pk, pv, po, ps = q.data_ptr(), k.data_ptr(), v.data_ptr(), q_out.data_ptr(), slots.data_ptr()
        plain = (q.dtype is _bf16 and k.dtype is _bf16 and v.dtype is _bf16 and q_out.dtype is _bf16 and slots.dtype is _i32
                 and slots.is_contiguous())
        if rope is not None:
            pr, pp = rope.data_ptr(), positions.data_ptr()
            plain = plain and rope.dtype is _f32 and positions.dtype is _i32 and rope.is_contiguous() and positions.is_contiguous()
        if k_out is not None:
            pko = k_out.data_ptr()
            plain = plain and k_out.dtype is _bf16
        if q_norm is not None:
            pqn = q_norm.data_ptr()
            plain = plain and q_norm.dtype is _f32 and q_norm.is_contiguous()
        if k_norm is not None:
            pkn = k_norm.data_ptr()
            plain = plain and k_norm.dtype is _f32 and k_norm.is_contiguous()
    except AttributeError:
        plain = False
    if not plain:
        pq, pk, pv, po, pko = (_address(t, _bf16, f"append_rotated: {name}", False)
                               for t, name in ((q, "q"), (k, "k"), (v, "v"), (q_out, "q_out"), (k_out, "k_out")))
        ps, pp = _address(slots, _i32, "append_rotated: slots"), _address(positions, _i32, "append_rotated: positions")
        pr, pqn, pkn = (_address(t, _f32, f"append_rotated: {name}") for t, name in ((rope, "rope"), (q_norm, "q_norm"), (k_norm, "k_norm")))
    try:
        if q_stride is None:
            q_stride = (_ONE if n == 1 else s if n * (s := q.stride()[0]) <= q.numel() else _token_stride(
                q, "append_rotated: q", n)) if q.is_contiguous() else _token_stride(q, "append_rotated: q", n)
        if k_stride is None:
            k_stride = (_ONE if n == 1 else s if n * (s := k.stride()[0]) <= k.numel() else _token_stride(
                k, "append_rotated: k", n)) if k.is_contiguous() else _token_stride(k, "append_rotated: k", n)
        if v_stride is None:
            v_stride = (_ONE if n == 1 else s if n * (s := v.stride()[0]) <= v.numel() else _token_stride(
                v, "append_rotated: v", n)) if v.is_contiguous() else _token_stride(v, "append_rotated: v", n)
        if q_out_stride is None:
            q_out_stride = (_ONE if n == 1 else s if n * (s := q_out.stride()[0]) <= q_out.numel() else _token_stride(
                q_out, "append_rotated: q_out", n)) if q_out.is_contiguous() else _token_stride(q_out, "append_rotated: q_out", n)
        if k_out_stride is None:
            k_out_stride = 0 if not pko else (_ONE if n == 1 else s if n * (s := k_out.stride()[0]) <= k_out.numel() else _token_stride(
                k_out, "append_rotated: k_out", n)) if k_out.is_contiguous() else _token_stride(k_out, "append_rotated: k_out", n)
    except AttributeError:
        raise TypeError("append_rotated: a raw address needs its token stride") from None
    status = _kv_append_rotated(handle, _KV_QKV.pack(pq, pk, pv, po, pko, q_stride, k_stride, v_stride, q_out_stride, k_out_stride,
                                                     pqn, pkn, pr, pp, ps, layer, n, rope_dim, n_positions, interleaved, eps), _stream(stream))
    if status:
        _check_kv(status, handle)


def _logits(t, width, what, stride, dtype):
    """(address, type, row stride) of rows of logits."""
    if _bf16 is None:
        _load_types()
    try:
        p, d = t.data_ptr(), t.dtype
    except AttributeError:
        if stride is None:
            raise TypeError(f"{what}: a raw address needs its row stride") from None
        return _ptr(t) or 0, FT_DTYPE_F32 if dtype == "fp32" else FT_DTYPE_BF16, stride
    if d is not _bf16 and d is not _f32:
        _refuse(t, what, "torch.bfloat16 or torch.float32")
    if stride is None:
        s = t.stride()
        if t.dim() != 2 or (s[1] != 1 and t.shape[1] != 1):
            _refuse(t, what, "dense rows, or a row stride")
        stride = s[0] if t.shape[0] != 1 else width
    return p, FT_DTYPE_BF16 if d is _bf16 else FT_DTYPE_F32, stride


def ft_moe_route(logits, T, E, k, topk_ids, topk_w, score="softmax", bias=None, n_group=1, topk_group=1, group_best=1, renormalise=True,
                 scale=1.0, stride=None, dtype="bf16", stream=None):
    """dtype ("bf16" or "fp32") names the type of logits that are given as a raw address."""
    pb = 0
    try:
        pl, pi, pw, dt = logits.data_ptr(), topk_ids.data_ptr(), topk_w.data_ptr(), _DTYPES.get(logits.dtype)
        plain = dt is not None and topk_ids.dtype is _i32 and topk_w.dtype is _f32 and topk_ids.is_contiguous() and topk_w.is_contiguous()
        if bias is not None:
            pb = bias.data_ptr()
            plain = plain and bias.dtype is _f32 and bias.is_contiguous()
        step = stride
        if step is None:
            step = logits.stride(0)
            plain = plain and logits.is_contiguous() and step >= E and logits.dim() == 2
    except (AttributeError, IndexError):
        plain = False
    if not plain:
        pl, dt, step = _logits(logits, E, "route: logits", stride, dtype)
        pi, pw, pb = _address(topk_ids, _i32, "route: topk_ids"), _address(topk_w, _f32, "route: topk_w"), _address(bias, _f32, "route: bias")
    status = _moe_route(_ROUTE.pack(pl, pb, pi, pw, step, T, E, k, dt, ROUTE_SCORES[score], n_group, topk_group, group_best,
                                    bool(renormalise), scale), _stream(stream))
    if status:
        _check(status)


def ft_logprobs(logits, n, V, tokens=None, logp=None, entropy=None, top_ids=None, top_logp=None, k=0, scale=1.0, stride=None, dtype="bf16",
                stream=None):
    """dtype ("bf16" or "fp32") names the type of logits that are given as a raw address."""
    pt = pp = pe = pi = px = 0
    try:
        pl, dt = logits.data_ptr(), _DTYPES.get(logits.dtype)
        plain = dt is not None
        if logp is not None:
            pt, pp = tokens.data_ptr(), logp.data_ptr()
            plain = plain and tokens.dtype is _i32 and logp.dtype is _f32 and tokens.is_contiguous() and logp.is_contiguous()
        if entropy is not None:
            pe = entropy.data_ptr()
            plain = plain and entropy.dtype is _f32 and entropy.is_contiguous()
        if top_ids is not None:
            pi, px = top_ids.data_ptr(), top_logp.data_ptr()
            plain = plain and top_ids.dtype is _i32 and top_logp.dtype is _f32 and top_ids.is_contiguous() and top_logp.is_contiguous()
        step = stride
        if step is None:
            step = logits.stride(0)
            plain = plain and logits.is_contiguous() and step >= V and logits.dim() == 2
    except (AttributeError, IndexError):
        plain = False
    if not plain:
        pl, dt, step = _logits(logits, V, "logprobs: logits", stride, dtype)
        pt, pi = _address(tokens, _i32, "logprobs: tokens"), _address(top_ids, _i32, "logprobs: top_ids")
        pp, pe, px = (_address(t, _f32, what) for t, what in (
            (logp, "logprobs: logp"), (entropy, "logprobs: entropy"), (top_logp, "logprobs: top_logp")))
    status = _logprobs(_LOGPROB.pack(pl, pt, pp, pe, pi, px, step, n, V, k, dt, scale), _stream(stream))
    if status:
        _check(status)


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
