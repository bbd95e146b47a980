"""GB300 (sm_103a) windowed prefill attention over a paged int8 KV pool.

A thin ctypes binding over ``libpa.so`` (C ABI in ``include/pa.h``).  The
functions keep the C names; they only marshal arguments (torch tensors for
device memory, the current torch stream) and raise on a non-zero status.
Every step of the computation runs in the library's CUDA kernels; there is no
CPU or PyTorch fallback: if the library is missing this module fails to import.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libpa.so")

if not os.path.exists(_LIB_PATH):
    raise ImportError("libpa.so is not built; run `python -c \"import __graft_entry__ as g; g.build()\"` "
                      "or `python windowed_prefill_attention_gb300/build.py`")

_lib = C.CDLL(_LIB_PATH)

PA_OK, PA_EINVAL, PA_EARCH, PA_ECUDA, PA_ETIMEOUT, PA_EBADPAGE, PA_ENOMEM, PA_ENOSCRATCH = 0, -1, -2, -3, -4, -5, -6, -7
PA_NOALLOC_SCRATCH_BYTES = 32 << 20
# query rows per work unit (PA_UNIT_ROWS in include/pa.h)
UNIT_ROWS = 256
PA_Q_BF16, PA_Q_INT8 = 0, 1
PA_P_F16, PA_P_U8 = 0, 1
PA_ROPE_HALF, PA_ROPE_ADJACENT, PA_ROPE_MAX_AXES = 0, 1, 4

EXPORTED = ("pa_default_options", "pa_create", "pa_device", "pa_destroy", "pa_prefill", "pa_prefill_batch",
            "pa_prefill_batch_gated", "pa_prefill_host", "pa_kv_append", "pa_rope_init", "pa_qk_norm_rope",
            "pa_qkv_append", "pa_decode", "pa_decode_shared", "pa_decode_shared_plan",
            "pa_last_error", "pa_timing", "pa_strerror", "pa_plan", "pa_plan_pairs", "pa_host_chunks", "pa_decode_plan",
            "pa_debug_gather",
            "pa_debug_maskset", "pa_debug_qcodes", "pa_debug_copy_streams_idle", "pa_prefill_noalloc",
            "pa_debug_noalloc_units", "pa_debug_qk_norm_rope_check", "pa_debug_qkv_append_check",
            "pa_debug_qkv_append_pool_check",
            "pa_debug_decode_shared_pass")


class pa_options(C.Structure):
    _fields_ = [("q_mode", C.c_int), ("p_mode", C.c_int), ("wait_timeout_ms", C.c_int), ("record_timing", C.c_int),
                ("debug_stall", C.c_int), ("debug_fail_host", C.c_int)]


class pa_seq(C.Structure):
    _fields_ = [("q_off", C.c_int), ("q_start", C.c_int), ("n_q", C.c_int), ("n_ctx", C.c_int)]


class pa_rope(C.Structure):
    _fields_ = [("rot_dim", C.c_int), ("pairing", C.c_int), ("n_axes", C.c_int), ("reserved", C.c_int),
                ("turn", C.c_uint64 * 128), ("axis", C.c_uint8 * 128)]


class pa_rows(C.Structure):
    _fields_ = [("data", C.c_void_p), ("n_tok", C.c_longlong), ("tok_stride", C.c_longlong),
                ("head_stride", C.c_longlong)]


_vp, _i, _f = C.c_void_p, C.c_int, C.c_float
_lib.pa_default_options.argtypes = [C.POINTER(pa_options)]
_lib.pa_default_options.restype = None
_lib.pa_create.argtypes = [C.POINTER(_vp), _i, _i, _i, _i, _i, _i, C.POINTER(pa_options)]
_lib.pa_destroy.argtypes = [_vp]
_lib.pa_destroy.restype = None
_lib.pa_prefill.argtypes = [_vp] + [_vp] * 6 + [_i] * 5 + [_f, _vp, _vp]
_lib.pa_prefill_batch.argtypes = [_vp, _i, C.POINTER(pa_seq)] + [_vp] * 6 + [_i, _i, _f, _vp, _vp]
_lib.pa_prefill_host.argtypes = _lib.pa_prefill_batch.argtypes
_lib.pa_prefill_batch_gated.argtypes = [_vp, _i, C.POINTER(pa_seq)] + [_vp] * 7 + [_i, _i, _f, _vp, _vp]
_lib.pa_kv_append.argtypes = [_vp, _vp, _vp, _i, _i] + [_vp] * 6
_ll = C.c_longlong
_lib.pa_rope_init.argtypes = [C.POINTER(pa_rope), _i, _i, _i, _vp, _vp]
_lib.pa_qk_norm_rope.argtypes = [_vp, _i, C.POINTER(pa_rows), C.POINTER(pa_rows), _vp, _vp, _f, _f, C.POINTER(pa_rope),
                                 _vp, _ll, _vp, _vp, _vp]
_lib.pa_qkv_append.argtypes = ([_vp, _i, _vp] + [C.POINTER(pa_rows)] * 3
                               + [_vp, _vp, _f, _f, C.POINTER(pa_rope), _vp, _ll] + [_vp] * 7)
_lib.pa_debug_qk_norm_rope_check.argtypes = [_i, _i] + _lib.pa_qk_norm_rope.argtypes[1:-1]
_lib.pa_debug_qkv_append_check.argtypes = [_i, _i, _i] + _lib.pa_qkv_append.argtypes[1:-1]
_lib.pa_debug_qkv_append_pool_check.argtypes = [_i, _i, _i, _i] + _lib.pa_qkv_append.argtypes[1:-1]
_lib.pa_decode.argtypes = _lib.pa_prefill_batch.argtypes
_lib.pa_decode_shared.argtypes = [_vp, _i, _vp, _i, _i] + [_vp] * 6 + [_i, _i, _f, _vp, _vp]
_lib.pa_decode_shared_plan.argtypes = ([_i] * 5 + [C.POINTER(pa_seq)] + [_i] * 4
                                       + [_vp, _i, C.POINTER(_i), _vp, _i, C.POINTER(_i)])
_lib.pa_debug_decode_shared_pass.argtypes = [_vp, _i]
_lib.pa_device.argtypes = [_vp]
_lib.pa_last_error.argtypes = [_vp, _vp]
_lib.pa_timing.argtypes = [_vp, _i, C.POINTER(C.c_double), C.POINTER(C.c_double), C.POINTER(_i)]
_lib.pa_strerror.argtypes = [_i]
_lib.pa_strerror.restype = C.c_char_p
_lib.pa_plan.argtypes = [_i, _i, _i, C.POINTER(pa_seq), _i, _i, _vp, _i, C.POINTER(_i), C.POINTER(C.c_longlong),
                         C.POINTER(_i)]
_lib.pa_plan_pairs.argtypes = [_i, _i, _i, C.POINTER(pa_seq), _i, _i, _i, _vp, _i, _vp, C.POINTER(_i)]
_lib.pa_host_chunks.argtypes = [_i, _i, _i, C.POINTER(pa_seq), _i, _vp, _i, C.POINTER(_i)]
_lib.pa_decode_plan.argtypes = [_i, _i, _i, C.POINTER(pa_seq), _i, _i, _vp, _i, C.POINTER(_i), C.POINTER(_i),
                                C.POINTER(_i), C.POINTER(_i), C.POINTER(C.c_longlong)]
_lib.pa_debug_gather.argtypes = ([_vp, _i, C.POINTER(pa_seq)] + [_vp] * 5 + [_i, _i, _i] + [_vp] * 5
                                 + [_i, C.POINTER(_i), _vp])
_lib.pa_debug_maskset.argtypes = [_vp, _i, C.POINTER(pa_seq), _i, _i, _vp, _vp, _i, _vp, _i, C.POINTER(_i), _vp]
_lib.pa_debug_qcodes.argtypes = [_vp, _i, _vp, _vp, _vp]
_lib.pa_debug_copy_streams_idle.argtypes = [_vp]
_lib.pa_prefill_noalloc.argtypes = [_i] * 4 + [_vp] * 6 + [_i] * 5 + [_f, _vp, _vp]
_lib.pa_debug_noalloc_units.argtypes = [_i, _vp, _vp]


class PAError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__("%s: %s (%d)" % (where, pa_strerror(code), code))
        self.code = code


def pa_strerror(code: int) -> str:
    return _lib.pa_strerror(code).decode()


def _check(code: int, where: str) -> int:
    if code != PA_OK:
        raise PAError(code, where)
    return code


def _seqs(seqs):
    """[(q_off, q_start, n_q, n_ctx), ...] or an int array [n, 4] -> ctypes array."""
    arr = np.asarray(seqs, dtype=np.int64).reshape(-1, 4)
    if arr.size and (int(arr.min()) < -2**31 or int(arr.max()) >= 2**31):
        raise ValueError("sequence fields must fit int32")
    return (pa_seq * arr.shape[0]).from_buffer_copy(np.ascontiguousarray(arr, dtype=np.int32))


def _dev(t, dtype, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return C.c_void_p(t.data_ptr())


def _host(a, name):
    import torch
    if isinstance(a, torch.Tensor):
        if a.is_cuda or not a.is_contiguous():
            raise TypeError("%s must be a contiguous host tensor" % name)
        return C.c_void_p(a.data_ptr())
    a = np.asarray(a)
    if not a.flags["C_CONTIGUOUS"]:
        raise ValueError("%s must be contiguous" % name)
    return a.ctypes.data_as(C.c_void_p)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


_torch_names = None


def _torch():
    """(bfloat16, float32, int8, int32, current raw stream of a device index): looked up once, since the calls of
    a single decode step cost more on the host than on the GPU."""
    global _torch_names
    if _torch_names is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        _torch_names = (torch.bfloat16, torch.float32, torch.int8, torch.int32, raw)
    return _torch_names


def _seq_array(seqs):
    """Sequences as the library reads them, and their number: an int32 array [n, 4] is taken as it is."""
    if not (type(seqs) is np.ndarray and seqs.dtype == np.int32 and seqs.ndim == 2 and seqs.shape[1] == 4
            and seqs.flags.c_contiguous):
        wide = np.asarray(seqs, dtype=np.int64).reshape(-1, 4)
        seqs = np.ascontiguousarray(wide, dtype=np.int32)
        if not np.array_equal(seqs, wide):
            raise ValueError("sequence fields must fit int32")
    return seqs, seqs.shape[0]


def pa_default_options() -> pa_options:
    o = pa_options()
    _lib.pa_default_options(C.byref(o))
    return o


# (q heads, kv heads, pool pages, pages per sequence, device) of the live handles, for the calls that check their tensors
_geometry = {}


def _address(h):
    """Address of a handle: a c_void_p (as pa_create gives it) or a plain integer; None for no handle."""
    return getattr(h, "value", h)


def _geometry_of(h):
    try:
        return _geometry[_address(h)]
    except (KeyError, TypeError):
        raise ValueError("not a live handle") from None


def pa_create(n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq, head_dim=256, page_size=16,
              q_mode=PA_Q_BF16, p_mode=PA_P_F16, wait_timeout_ms=2000, record_timing=False, debug_stall=False,
              debug_fail_host=False):
    o = pa_options(q_mode, p_mode, wait_timeout_ms, 1 if record_timing else 0, 1 if debug_stall else 0,
                   1 if debug_fail_host else 0)
    h = C.c_void_p()
    _check(_lib.pa_create(C.byref(h), n_q_heads, n_kv_heads, head_dim, page_size, n_pool_pages, max_pages_per_seq,
                          C.byref(o)), "pa_create")
    _geometry[h.value] = (n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq, pa_device(h))
    return h


def pa_device(h) -> int:
    """Index of the CUDA device the handle is bound to (-1: no handle)."""
    return _lib.pa_device(h)


def pa_destroy(h) -> None:
    _geometry.pop(_address(h), None)
    _lib.pa_destroy(h)


def _dev_inputs(q, k_pool, v_pool, k_scale, v_scale, block_table):
    import torch
    return [_dev(q, torch.bfloat16, "q"), _dev(k_pool, torch.int8, "k_pool"), _dev(v_pool, torch.int8, "v_pool"),
            _dev(k_scale, torch.float32, "k_scale"), _dev(v_scale, torch.float32, "v_scale"),
            _dev(block_table, torch.int32, "block_table")]


def pa_prefill(h, q, k_pool, v_pool, k_scale, v_scale, block_table, q_start, n_q, n_ctx, n_sink_blk, n_win_blk,
               sm_scale, out, stream=None) -> None:
    import torch
    args = _dev_inputs(q, k_pool, v_pool, k_scale, v_scale, block_table)
    _check(_lib.pa_prefill(h, *args, q_start, n_q, n_ctx, n_sink_blk, n_win_blk, float(sm_scale),
                           _dev(out, torch.bfloat16, "out"), _stream(stream)), "pa_prefill")


def pa_prefill_batch(h, seqs, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, sm_scale,
                     out, stream=None, q_gate=None) -> None:
    """q_gate (bf16, shaped like out) selects pa_prefill_batch_gated."""
    import torch
    s = _seqs(seqs)
    args = _dev_inputs(q, k_pool, v_pool, k_scale, v_scale, block_table)
    if q_gate is None:
        _check(_lib.pa_prefill_batch(h, len(s), s, *args, n_sink_blk, n_win_blk, float(sm_scale),
                                     _dev(out, torch.bfloat16, "out"), _stream(stream)), "pa_prefill_batch")
    else:
        _check(_lib.pa_prefill_batch_gated(h, len(s), s, args[0], _dev(q_gate, torch.bfloat16, "q_gate"), *args[1:],
                                           n_sink_blk, n_win_blk, float(sm_scale), _dev(out, torch.bfloat16, "out"),
                                           _stream(stream)), "pa_prefill_batch_gated")


def pa_decode(h, seqs, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, sm_scale, out,
              stream=None) -> None:
    """One new token per sequence (seqs rows (q_off, n_ctx - 1, 1, n_ctx))."""
    import torch
    s = _seqs(seqs)
    args = _dev_inputs(q, k_pool, v_pool, k_scale, v_scale, block_table)
    _check(_lib.pa_decode(h, len(s), s, *args, n_sink_blk, n_win_blk, float(sm_scale),
                          _dev(out, torch.bfloat16, "out"), _stream(stream)), "pa_decode")


def pa_decode_shared(h, seqs, n_prefix, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk,
                     sm_scale, out, stream=None) -> None:
    """pa_decode for sequences that share their first n_prefix tokens (the pages of block_table row 0).  seqs as
    pa_qkv_append takes them; stream None: the current one of the handle's device."""
    geometry = _geometry_of(h)
    device = geometry[4]
    bf16, _, _, _, raw_stream = _torch()
    s, n_seq = _seq_array(seqs)
    rows = (q.shape[0], geometry[0], 256)
    bt, kp, vp, ks, vs = _pool_args(geometry, n_seq, block_table, k_pool, v_pool, k_scale, v_scale)
    _check(_lib.pa_decode_shared(
        h, n_seq, s.ctypes.data, n_prefix, rows[0], _array(q, bf16, rows, "q", device), kp, vp, ks, vs, bt, n_sink_blk,
        n_win_blk, sm_scale, _array(out, bf16, rows, "out", device),
        raw_stream(device) if stream is None else stream.cuda_stream), "pa_decode_shared")


def pa_kv_append(h, k_new, v_new, tok_start, block_table_row, k_pool, v_pool, k_scale, v_scale,
                 stream=None) -> None:
    """Quantise the new tokens' K/V rows (bf16 [n_new, HKV, 256]) into the pool."""
    import torch
    n_new = int(k_new.shape[0])
    _check(_lib.pa_kv_append(h, _dev(k_new, torch.bfloat16, "k_new"), _dev(v_new, torch.bfloat16, "v_new"), n_new,
                             int(tok_start), _dev(block_table_row, torch.int32, "block_table_row"),
                             _dev(k_pool, torch.int8, "k_pool"), _dev(v_pool, torch.int8, "v_pool"),
                             _dev(k_scale, torch.float32, "k_scale"), _dev(v_scale, torch.float32, "v_scale"),
                             _stream(stream)), "pa_kv_append")


def pa_rope_init(inv_freq, pairing=PA_ROPE_HALF, pair_axis=None) -> pa_rope:
    """A rotation of the first 2 * len(inv_freq) dims of a head: radians per position of each pair, and
    the position axis each pair follows (None: one axis)."""
    freq = np.ascontiguousarray(inv_freq, dtype=np.float64).reshape(-1)
    axis = None if pair_axis is None else np.ascontiguousarray(pair_axis, dtype=np.int32).reshape(-1)
    if axis is not None and axis.size != freq.size:
        raise ValueError("pair_axis and inv_freq must have one entry for each pair")
    n_axes = 1 if axis is None or axis.size == 0 else int(axis.max()) + 1
    r = pa_rope()
    _check(_lib.pa_rope_init(C.byref(r), 2 * freq.size, pairing, n_axes, freq.ctypes.data_as(C.c_void_p),
                             None if axis is None else axis.ctypes.data_as(C.c_void_p)), "pa_rope_init")
    return r


def _wrong(t, dtype, shape, name, device, what="contiguous"):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        return TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != device:
        return ValueError("%s must be on the handle's device %d, got %d" % (name, device, t.get_device()))
    return ValueError("%s must be %s and %s, got %s with strides %s" % (name, what, tuple(shape), tuple(t.shape), t.stride()))


def _array(t, dtype, shape, name, device):
    """Address of a contiguous CUDA tensor of this type and shape on this device."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise _wrong(t, dtype, shape, name, device)


def _rows(t, bf16, shape, name, device):
    """bf16 rows [token, head, 256] at any strides (the 256 values of a row contiguous)."""
    try:
        if t.dtype is bf16 and t.get_device() == device and t.shape == shape:
            ts, hs, one = t.stride()
            if one == 1:
                return pa_rows(t.data_ptr(), shape[0], ts, hs)
    except AttributeError:
        pass
    raise _wrong(t, bf16, shape, name, device, "with contiguous rows")


def _gain(w, bf16, name, device):
    return None if w is None else _array(w, bf16, (256,), name, device)


def _positions(positions, rope, tokens, int32, device):
    """int32 [tokens] or [axes, tokens] -> address and row stride."""
    if positions is None:
        return None, 0
    shape, stride = positions.shape, positions.stride()
    if positions.dtype is not int32 or not positions.is_cuda:
        raise TypeError("positions must be a CUDA int32 tensor")
    if positions.get_device() != device:
        raise ValueError("positions must be on the handle's device %d, got %d" % (device, positions.get_device()))
    n_axes = shape[0] if len(shape) == 2 else 1
    if len(shape) not in (1, 2) or shape[-1] < tokens or (stride[-1] != 1 and shape[-1] > 1):
        raise ValueError("positions must be [tokens] or [axes, tokens], contiguous along the tokens")
    if rope is not None and rope.rot_dim > 0 and n_axes < rope.n_axes:
        raise ValueError("positions must have %d axes, got %d" % (rope.n_axes, n_axes))
    return positions.data_ptr(), stride[0] if n_axes > 1 else shape[-1]


def _pool_args(geometry, n_seq, block_table, k_pool, v_pool, k_scale, v_scale):
    """Addresses of the block table, pools and scales, of the handle's shapes."""
    _, f32, int8, int32, _ = _torch()
    _, hkv, n_pool, max_pages, device = geometry
    if block_table.shape[0] < n_seq:
        raise ValueError("block_table must have a row for each sequence")
    rows, scales = (n_pool, 16, hkv, 256), (n_pool, 16, hkv)
    return (_array(block_table, int32, (block_table.shape[0], max_pages), "block_table", device),
            _array(k_pool, int8, rows, "k_pool", device), _array(v_pool, int8, rows, "v_pool", device),
            _array(k_scale, f32, scales, "k_scale", device), _array(v_scale, f32, scales, "v_scale", device))


def pa_qk_norm_rope(h, q, k, q_weight, k_weight, eps, rope, positions, q_out, k_out, weight_offset=0.0,
                    stream=None) -> None:
    """Norm and rotate query rows q [tokens, HQ, 256] into q_out and key rows k [tokens, HKV, 256] into k_out
    (contiguous; q or k None leaves that kind out).  rope: a pa_rope, or None for the norm alone; positions
    int32 [tokens] or [axes, tokens].  stream None: the current one of the handle's device."""
    some = k if q is None else q
    if some is None:
        raise ValueError("q or k is needed")
    hq, hkv, _, _, device = _geometry_of(h)
    bf16, _, _, int32, raw_stream = _torch()
    n = some.shape[0]
    qs, ks = (n, hq, 256), (n, hkv, 256)
    pos, pos_stride = _positions(positions, rope, n, int32, device)
    _check(_lib.pa_qk_norm_rope(
        h, n, None if q is None else _rows(q, bf16, qs, "q", device),
        None if k is None else _rows(k, bf16, ks, "k", device), _gain(q_weight, bf16, "q_weight", device),
        _gain(k_weight, bf16, "k_weight", device), weight_offset, eps, rope, pos, pos_stride,
        None if q is None else _array(q_out, bf16, qs, "q_out", device),
        None if k is None else _array(k_out, bf16, ks, "k_out", device),
        raw_stream(device) if stream is None else stream.cuda_stream), "pa_qk_norm_rope")


def pa_qkv_append(h, seqs, q, k, v, q_weight, k_weight, eps, rope, positions, block_table, k_pool, v_pool, k_scale,
                  v_scale, q_out, weight_offset=0.0, stream=None) -> None:
    """The new tokens of a batch of sequences (seqs: (q_off, q_start, n_q, n_ctx) each, an int32 array is taken as it
    is; rows q_off .. q_off + n_q of q, k, v): queries normed and rotated into q_out, keys normed, rotated and
    quantised, values quantised into the pool.  positions None: the tokens' own; q None (with q_out None): keys and
    values only.  stream None: the current one of the handle's device."""
    geometry = _geometry_of(h)
    hq, hkv, _, _, device = geometry
    bf16, _, _, int32, raw_stream = _torch()
    s, n_seq = _seq_array(seqs)
    n = k.shape[0]
    pos, pos_stride = _positions(positions, rope, n, int32, device)
    _check(_lib.pa_qkv_append(
        h, n_seq, s.ctypes.data, None if q is None else _rows(q, bf16, (n, hq, 256), "q", device),
        _rows(k, bf16, (n, hkv, 256), "k", device), _rows(v, bf16, (n, hkv, 256), "v", device),
        _gain(q_weight, bf16, "q_weight", device), _gain(k_weight, bf16, "k_weight", device), weight_offset, eps, rope,
        pos, pos_stride, *_pool_args(geometry, n_seq, block_table, k_pool, v_pool, k_scale, v_scale),
        None if q is None else _array(q_out, bf16, (n, hq, 256), "q_out", device),
        raw_stream(device) if stream is None else stream.cuda_stream), "pa_qkv_append")


def pa_prefill_host(h, seqs, q, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, sm_scale,
                    out, stream=None) -> None:
    """Host buffers (numpy arrays or CPU tensors; pinned is fastest); synchronous."""
    s = _seqs(seqs)
    args = [_host(a, n) for a, n in ((q, "q"), (k_pool, "k_pool"), (v_pool, "v_pool"), (k_scale, "k_scale"),
                                     (v_scale, "v_scale"), (block_table, "block_table"))]
    _check(_lib.pa_prefill_host(h, len(s), s, *args, n_sink_blk, n_win_blk, float(sm_scale), _host(out, "out"),
                                _stream(stream)), "pa_prefill_host")


def pa_prefill_noalloc(n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq, q, k_pool, v_pool, k_scale, v_scale,
                       block_table, q_start, n_q, n_ctx, n_sink_blk, n_win_blk, sm_scale, out, stream=None) -> None:
    """Handle-free pa_prefill whose scratch is a static device array (no allocation); synchronous."""
    import torch
    args = _dev_inputs(q, k_pool, v_pool, k_scale, v_scale, block_table)
    _check(_lib.pa_prefill_noalloc(n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq, *args, q_start, n_q, n_ctx,
                                   n_sink_blk, n_win_blk, float(sm_scale), _dev(out, torch.bfloat16, "out"),
                                   _stream(stream)), "pa_prefill_noalloc")


def pa_debug_noalloc_units(n_units, stream=None):
    """The work list (int32 [n_units, 4]) the last pa_prefill_noalloc call on the current device built."""
    units = np.zeros((n_units, 4), dtype=np.int32)
    _check(_lib.pa_debug_noalloc_units(n_units, units.ctypes.data_as(C.c_void_p), _stream(stream)),
           "pa_debug_noalloc_units")
    return units


def pa_debug_copy_streams_idle(h) -> bool:
    """True if the handle's host-path copy streams have no work pending (does not wait)."""
    r = _lib.pa_debug_copy_streams_idle(h)
    if r < 0:
        raise PAError(r, "pa_debug_copy_streams_idle")
    return r == 1


def pa_last_error(h, stream=None) -> int:
    """Synchronise and return the first device-side status since the last call (0 = fine)."""
    return _lib.pa_last_error(h, _stream(stream))


def pa_timing(h, reset=False):
    w, a, n = C.c_double(), C.c_double(), C.c_int()
    _check(_lib.pa_timing(h, 1 if reset else 0, C.byref(w), C.byref(a), C.byref(n)), "pa_timing")
    return w.value, a.value, n.value


def pa_plan(n_q_heads, n_kv_heads, seqs, n_sink_blk, n_win_blk):
    """Host-only work plan: (units int32 [n, 4] = seq, kv head, first token, tiles; total tiles; widened rows)."""
    s = _seqs(seqs)
    n_units, n_tiles, n_rows = C.c_int(), C.c_longlong(), C.c_int()
    _check(_lib.pa_plan(n_q_heads, n_kv_heads, len(s), s, n_sink_blk, n_win_blk, None, 0, C.byref(n_units),
                        C.byref(n_tiles), C.byref(n_rows)), "pa_plan")
    units = np.zeros((n_units.value, 4), dtype=np.int32)
    _check(_lib.pa_plan(n_q_heads, n_kv_heads, len(s), s, n_sink_blk, n_win_blk, units.ctypes.data_as(C.c_void_p),
                        n_units.value, C.byref(n_units), C.byref(n_tiles), C.byref(n_rows)), "pa_plan")
    return units, n_tiles.value, n_rows.value


def pa_plan_pairs(n_q_heads, n_kv_heads, seqs, n_sink_blk, n_win_blk, n_pairs):
    """Host-only: pa_plan's units as a launch hands them to n_pairs SM pairs.  Returns
    (units int32 [n, 4] laid out pair by pair, pair_off int32 [n_pairs + 1])."""
    s = _seqs(seqs)
    n = C.c_int()
    off = np.zeros(n_pairs + 1, dtype=np.int32)
    _check(_lib.pa_plan_pairs(n_q_heads, n_kv_heads, len(s), s, n_sink_blk, n_win_blk, n_pairs, None, 0,
                              off.ctypes.data_as(C.c_void_p), C.byref(n)), "pa_plan_pairs")
    units = np.zeros((n.value, 4), dtype=np.int32)
    _check(_lib.pa_plan_pairs(n_q_heads, n_kv_heads, len(s), s, n_sink_blk, n_win_blk, n_pairs,
                              units.ctypes.data_as(C.c_void_p), n.value, off.ctypes.data_as(C.c_void_p),
                              C.byref(n)), "pa_plan_pairs")
    return units, off


def pa_host_chunks(n_q_heads, n_kv_heads, seqs, n_pairs):
    """Host-only: the chunk ends (rows of the sequences laid end to end) of pa_prefill_host."""
    s = _seqs(seqs)
    n = C.c_int()
    _check(_lib.pa_host_chunks(n_q_heads, n_kv_heads, len(s), s, n_pairs, None, 0, C.byref(n)), "pa_host_chunks")
    ends = np.zeros(n.value, dtype=np.int64)
    _check(_lib.pa_host_chunks(n_q_heads, n_kv_heads, len(s), s, n_pairs, ends.ctypes.data_as(C.c_void_p), n.value,
                               C.byref(n)), "pa_host_chunks")
    return ends


def pa_decode_plan(n_kv_heads, slots, seqs, n_sink_blk, n_win_blk):
    """Host-only: pa_decode's work split of one launch.  Returns (runs int32 [n_cta, 3] =
    first block, sequence, partial slot; per_cta; max_slots; listed; total blocks)."""
    s = _seqs(seqs)
    n_cta, per_cta, max_slots, listed, total = C.c_int(), C.c_int(), C.c_int(), C.c_int(), C.c_longlong()
    args = lambda buf, cap: (n_kv_heads, slots, len(s), s, n_sink_blk, n_win_blk, buf, cap, C.byref(n_cta),  # noqa: E731
                             C.byref(per_cta), C.byref(max_slots), C.byref(listed), C.byref(total))
    _check(_lib.pa_decode_plan(*args(None, 0)), "pa_decode_plan")
    runs = np.zeros((n_cta.value, 3), dtype=np.int32)
    _check(_lib.pa_decode_plan(*args(runs.ctypes.data_as(C.c_void_p), n_cta.value)), "pa_decode_plan")
    return runs, per_cta.value, max_slots.value, bool(listed.value), total.value


def pa_debug_decode_shared_pass(h, prefix_pass) -> None:
    """Test hook: 1 / 0 / -1, whether pa_decode_shared computes the prefix once for all sequences (see include/pa.h)."""
    _check(_lib.pa_debug_decode_shared_pass(h, prefix_pass), "pa_debug_decode_shared_pass")


def pa_decode_shared_plan(n_q_heads, n_kv_heads, max_pages_per_seq, n_sm, seqs, n_prefix, n_sink_blk, n_win_blk,
                          prefix_pass=-1):
    """Host-only: pa_decode_shared's work split of one launch (see include/pa.h): (prefix runs int32 [n, 8],
    own runs int32 [m, 7])."""
    s = _seqs(seqs)
    n, m = C.c_int(), C.c_int()
    args = (n_q_heads, n_kv_heads, max_pages_per_seq, n_sm, len(s), s, n_prefix, n_sink_blk, n_win_blk, prefix_pass)
    _check(_lib.pa_decode_shared_plan(*args, None, 0, C.byref(n), None, 0, C.byref(m)), "pa_decode_shared_plan")
    pre, own = np.zeros((n.value, 8), dtype=np.int32), np.zeros((m.value, 7), dtype=np.int32)
    _check(_lib.pa_decode_shared_plan(*args, pre.ctypes.data_as(C.c_void_p), n.value, C.byref(n),
                                      own.ctypes.data_as(C.c_void_p), m.value, C.byref(m)), "pa_decode_shared_plan")
    return pre, own


def pa_debug_gather(h, seqs, k_pool, v_pool, k_scale, v_scale, block_table, n_sink_blk, n_win_blk, seq, cap,
                    stream=None):
    """Widened rows of sequence `seq` as the kernels see them (int8 codes, scales, logical token of each row)."""
    import torch
    s = _seqs(seqs)
    dev = k_pool.device
    hkv = k_pool.shape[2]
    k_out = torch.empty((hkv, cap, 256), dtype=torch.int8, device=dev)
    v_out = torch.empty_like(k_out)
    ks_out = torch.empty((hkv, cap), dtype=torch.float32, device=dev)
    vs_out = torch.empty_like(ks_out)
    tok = torch.empty((cap,), dtype=torch.int32, device=dev)
    n = C.c_int()
    _check(_lib.pa_debug_gather(h, len(s), s, _dev(k_pool, torch.int8, "k_pool"), _dev(v_pool, torch.int8, "v_pool"),
                                _dev(k_scale, torch.float32, "k_scale"), _dev(v_scale, torch.float32, "v_scale"),
                                _dev(block_table, torch.int32, "block_table"), n_sink_blk, n_win_blk, seq,
                                C.c_void_p(k_out.data_ptr()), C.c_void_p(v_out.data_ptr()),
                                C.c_void_p(ks_out.data_ptr()), C.c_void_p(vs_out.data_ptr()),
                                C.c_void_p(tok.data_ptr()), cap, C.byref(n), _stream(stream)), "pa_debug_gather")
    r = n.value
    # the export packs rows densely as [HKV][n_rows]
    k_flat = k_out.reshape(-1)[: hkv * r * 256].reshape(hkv, r, 256)
    v_flat = v_out.reshape(-1)[: hkv * r * 256].reshape(hkv, r, 256)
    ks = ks_out.reshape(-1)[: hkv * r].reshape(hkv, r)
    vs = vs_out.reshape(-1)[: hkv * r].reshape(hkv, r)
    return k_flat, v_flat, ks, vs, tok[:r]


def pa_debug_maskset(h, seqs, n_sink_blk, n_win_blk, units_cap, cap, stream=None):
    """Per unit: visited key blocks and per-row admitted key counts (see include/pa.h)."""
    import torch
    s = _seqs(seqs)
    counts = torch.empty((units_cap, UNIT_ROWS), dtype=torch.int32, device="cuda")
    blocks = torch.empty((units_cap, cap), dtype=torch.int32, device="cuda")
    units = np.zeros((units_cap, 4), dtype=np.int32)
    n = C.c_int()
    _check(_lib.pa_debug_maskset(h, len(s), s, n_sink_blk, n_win_blk, C.c_void_p(counts.data_ptr()),
                                 C.c_void_p(blocks.data_ptr()), cap, units.ctypes.data_as(C.c_void_p), units_cap,
                                 C.byref(n), _stream(stream)), "pa_debug_maskset")
    k = n.value
    return units[:k], counts[:k], blocks[:k]


def pa_debug_qcodes(q_rows, stream=None):
    """The attention prologue's int8 query grid on bf16 rows [n, 256]: (int8 codes [n, 256], fp32 scales [n])."""
    import torch
    n = int(q_rows.shape[0])
    codes = torch.empty((n, 256), dtype=torch.int8, device=q_rows.device)
    scales = torch.empty((n,), dtype=torch.float32, device=q_rows.device)
    _check(_lib.pa_debug_qcodes(_dev(q_rows, torch.bfloat16, "q_rows"), n, C.c_void_p(codes.data_ptr()),
                                C.c_void_p(scales.data_ptr()), _stream(stream)), "pa_debug_qcodes")
    return codes, scales


class Handle:
    """Owns a pa_handle; ``close()`` (or garbage collection) destroys it."""

    def __init__(self, n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq, **opts):
        self.h = pa_create(n_q_heads, n_kv_heads, n_pool_pages, max_pages_per_seq, **opts)
        self.n_q_heads, self.n_kv_heads = n_q_heads, n_kv_heads

    def close(self):
        if self.h is not None:
            pa_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
