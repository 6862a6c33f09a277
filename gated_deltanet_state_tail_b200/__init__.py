"""Python binding of the Tail-Replay C ABI (``include/gdn_tail_replay.h``).

Argument marshalling only: every step of the replay and the prefill runs in
the CUDA kernels of ``libgdn_tail_replay.so``.  PyTorch provides device
memory and streams.  There is no CPU fallback: if the library is missing the
import fails, and every call checks the status the library returns.

The low-level names mirror the C entry points (``gdn_plan_create_replay``,
``gdn_tail_replay_state``, ``gdn_tail_replay_outputs``, ``gdn_chunk_prefill``,
``gdn_decode_step``, ...).  ``ReplayPlan`` and
``PrefillPlan`` wrap a plan's lifetime; ``tail_replay_state`` and
``chunk_prefill`` are the one-call conveniences on torch tensors.  The
full-attention layers of the hybrid stack have ``qk_norm_rope`` and
``PagedAttention`` (``paged_attention`` in one call).
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
# GDN_DEBUG_BOUNDS=1 in the environment selects the debug build, whose kernels
# check every global index against the plan and report GDN_ERR_BOUNDS.
DEBUG_BOUNDS = os.environ.get("GDN_DEBUG_BOUNDS", "0") not in ("", "0")
LIB_PATH = os.path.join(_PKG, "libgdn_tail_replay_debug.so" if DEBUG_BOUNDS else "libgdn_tail_replay.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT, \
    GDN_ERR_ALLOC, GDN_ERR_MISMATCH, GDN_ERR_BOUNDS = range(8)
GDN_F32, GDN_BF16 = 0, 1
GDN_ROTARY_HALVES, GDN_ROTARY_INTERLEAVED = 0, 1
GDN_KERNEL_AUTO, GDN_KERNEL_RECURRENT, GDN_KERNEL_CHUNKED_TC = 0, 1, 2
# the chunked kernel with the state-only replay pinned to its two-CTA-per-SM kernel (the
# default), its warp-specialised one or its cluster-pair one
GDN_KERNEL_CHUNKED_TC_TWO_CTA, GDN_KERNEL_CHUNKED_TC_WARP_SPEC, GDN_KERNEL_CHUNKED_TC_PAIR = 3, 4, 5

EXPORTED = (
    "gdn_plan_create_replay", "gdn_plan_create_prefill", "gdn_plan_destroy", "gdn_replay_windows",
    "gdn_plan_window",
    "gdn_plan_info", "gdn_plan_launches", "gdn_workspace_bytes", "gdn_tail_replay_state", "gdn_chunk_prefill",
    "gdn_workspace_status", "gdn_status_string", "gdn_version", "gdn_tail_replay_state_noalloc",
    "gdn_tail_replay_outputs", "gdn_decode_step", "gdn_plan_create_fused", "gdn_tail_replay_prefill",
    "gdn_selftest_bounded_wait", "gdn_debug_fail_plan_allocations", "gdn_selftest_index_check",
    "gdn_debug_bounds_enabled", "gdn_qk_norm_rope", "gdn_paged_attention", "gdn_paged_attention_workspace_bytes",
    "gdn_selftest_split_entry",
)


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {gdn_status_string(status)} (status {status})")
        self.status = status


class gdn_varlen_desc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("d_k", ctypes.c_int32),
        ("d_v", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("seq_offsets_host", ctypes.POINTER(ctypes.c_int32)),
        ("row_stride_elems", ctypes.c_int64),
    ]


class gdn_paged_kv(ctypes.Structure):
    _fields_ = [
        ("num_pages", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
        ("page_stride", ctypes.c_int64),
        ("row_stride", ctypes.c_int64),
        ("head_stride", ctypes.c_int64),
    ]


class gdn_qk_desc(ctypes.Structure):
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("num_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("rotary_style", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("q_row_stride", ctypes.c_int64),
        ("k_row_stride", ctypes.c_int64),
        ("v_row_stride", ctypes.c_int64),
    ]


class gdn_attn_desc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_heads", ctypes.c_int32),
        ("rows", ctypes.c_int64),
        ("q_row_stride", ctypes.c_int64),
        ("max_pages", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m gated_deltanet_state_tail_b200.build` "
            "(there is no CPU fallback)")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    pd = ctypes.POINTER(gdn_varlen_desc)
    sig = {
        "gdn_plan_create_replay": (I32, [pd, P, P, ctypes.POINTER(P)]),
        "gdn_plan_create_prefill": (I32, [pd, ctypes.POINTER(P)]),
        "gdn_plan_destroy": (None, [P]),
        "gdn_replay_windows": (I32, [I32, P, P, P, P, P]),
        "gdn_plan_window": (I32, [P, I32, ctypes.POINTER(I64), ctypes.POINTER(I32)]),
        "gdn_plan_info": (I32, [P, ctypes.POINTER(I64), ctypes.POINTER(I64), ctypes.POINTER(I32)]),
        "gdn_plan_launches": (I32, [P, ctypes.POINTER(I32)]),
        "gdn_workspace_bytes": (ctypes.c_size_t, [P]),
        "gdn_tail_replay_state": (I32, [P, P, P, P, P, P, P, P, P, P, P, P]),
        "gdn_chunk_prefill": (I32, [P, P, P, P, P, P, P, P, P, P, P, P]),
        "gdn_workspace_status": (I32, [P, P]),
        "gdn_status_string": (ctypes.c_char_p, [I32]),
        "gdn_version": (I32, []),
        "gdn_tail_replay_state_noalloc": (I32, [pd, P, P, P, P, P, P, P, P, ctypes.POINTER(ctypes.c_uint32)]),
        "gdn_tail_replay_outputs": (I32, [P, P, P, P, P, P, P, P, P, P, P, P, P]),
        "gdn_decode_step": (I32, [I32, I32, I32, I32, I32, P, P, P, P, P, P, P, P, P]),
        "gdn_plan_create_fused": (I32, [pd, P, P, P, ctypes.POINTER(P)]),
        "gdn_tail_replay_prefill": (I32, [P, P, P, P, P, P, P, P, P, P, P, P, P, P, P]),
        "gdn_selftest_bounded_wait": (I32, [ctypes.c_uint64, P, P]),
        "gdn_debug_fail_plan_allocations": (None, [I32]),
        "gdn_selftest_index_check": (I32, [P, P]),
        "gdn_debug_bounds_enabled": (I32, []),
        "gdn_selftest_split_entry": (I32, [ctypes.POINTER(I32), I32, I32, I32, I64, I32]),
        "gdn_qk_norm_rope": (I32, [ctypes.POINTER(gdn_qk_desc), P, P, P, P, P, P, P, ctypes.c_float,
                                   ctypes.POINTER(gdn_paged_kv), P, P, P, P, P, P]),
        "gdn_paged_attention": (I32, [ctypes.POINTER(gdn_attn_desc), ctypes.POINTER(gdn_paged_kv), P, P, P, P, P, P,
                                      P, P, P, P]),
        "gdn_paged_attention_workspace_bytes": (ctypes.c_size_t, [I32, I32, I32]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib_handle = None


def library():
    """The loaded ctypes handle of libgdn_tail_replay.so (loaded on first use;
    raises ImportError if the library has not been built)."""
    global _lib_handle
    if _lib_handle is None:
        _lib_handle = _load()
    return _lib_handle


class _LazyLib:
    def __getattr__(self, name):
        return getattr(library(), name)


_lib = _LazyLib()


def gdn_status_string(status: int) -> str:
    return _lib.gdn_status_string(int(status)).decode()


def gdn_version() -> int:
    return int(_lib.gdn_version())


def _check(status: int, what: str):
    if status != GDN_OK:
        raise GdnError(status, what)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _ptr(t):
    """Device (or host) address of a tensor / numpy array, or None."""
    if t is None:
        return None
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dtype_code(dtype) -> int:
    import torch
    if dtype in (torch.float32, "f32"):
        return GDN_F32
    if dtype in (torch.bfloat16, "bf16"):
        return GDN_BF16
    raise ValueError(f"unsupported dtype {dtype}")


def _make_desc(batch, H, dk, dv, dtype, kernel, offsets: np.ndarray, row_stride=0):
    d = gdn_varlen_desc()
    d.batch, d.num_heads, d.d_k, d.d_v = int(batch), int(H), int(dk), int(dv)
    d.dtype = _dtype_code(dtype)
    d.kernel = int(kernel)
    d.seq_offsets_host = offsets.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
    d.row_stride_elems = int(row_stride)
    return d


def row_stride_of(*tensors) -> int:
    """Row stride (elements) shared by [rows, H, d] views of q, k and v, or 0 when each
    is packed.  Heads must be contiguous inside a row (strides (., d, 1))."""
    ts = [t for t in tensors if t is not None]
    for t in ts:
        if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError("q/k/v must be [rows, H, d] views with contiguous heads inside a row")
        if t.shape[0] > 1 and t.stride(0) == 0:   # 0 would read as packed
            raise ValueError("q, k and v must not be one row expanded to many")
    if all(t.stride(0) == t.shape[1] * t.shape[2] for t in ts):
        return 0
    rs = {t.stride(0) for t in ts}
    if len(rs) != 1:
        raise ValueError("q, k and v must share one row stride (or all be packed)")
    return rs.pop()


def gdn_plan_create_replay(H, dk, dv, dtype, seq_offsets, match_len, R, kernel=GDN_KERNEL_AUTO, row_stride=0):
    """Create a replay plan; returns the raw handle (int).  Host int arrays."""
    off, ml, rr = _i32(seq_offsets), _i32(match_len), _i32(R)
    if len(off) != len(ml) + 1 or len(rr) != len(ml):
        raise ValueError("seq_offsets must have batch + 1 entries, match_len and R batch entries")
    d = _make_desc(len(ml), H, dk, dv, dtype, kernel, off, row_stride)
    h = ctypes.c_void_p()
    _check(_lib.gdn_plan_create_replay(ctypes.byref(d), ml.ctypes.data, rr.ctypes.data,
                                       ctypes.byref(h)), "gdn_plan_create_replay")
    return h.value


def gdn_plan_create_prefill(H, dk, dv, dtype, cu_seqlens, kernel=GDN_KERNEL_AUTO, row_stride=0):
    off = _i32(cu_seqlens)
    d = _make_desc(len(off) - 1, H, dk, dv, dtype, kernel, off, row_stride)
    h = ctypes.c_void_p()
    _check(_lib.gdn_plan_create_prefill(ctypes.byref(d), ctypes.byref(h)), "gdn_plan_create_prefill")
    return h.value


def gdn_plan_create_fused(H, dk, dv, dtype, seq_offsets, match_len, R, suffix_offsets,
                          kernel=GDN_KERNEL_AUTO, row_stride=0):
    """Create a fused replay + suffix plan; returns the raw handle (int).  Host int arrays."""
    off, ml, rr, so = _i32(seq_offsets), _i32(match_len), _i32(R), _i32(suffix_offsets)
    if len(off) != len(ml) + 1 or len(rr) != len(ml) or len(so) != len(ml) + 1:
        raise ValueError("seq_offsets and suffix_offsets need batch + 1 entries, match_len and R batch")
    d = _make_desc(len(ml), H, dk, dv, dtype, kernel, off, row_stride)
    h = ctypes.c_void_p()
    _check(_lib.gdn_plan_create_fused(ctypes.byref(d), ml.ctypes.data, rr.ctypes.data, so.ctypes.data,
                                      ctypes.byref(h)), "gdn_plan_create_fused")
    return h.value


def gdn_replay_windows(seq_offsets, match_len, R):
    """Host-side replay windows: (row0 int64 [B], len int32 [B])."""
    off, ml, rr = _i32(seq_offsets), _i32(match_len), _i32(R)
    if len(off) != len(ml) + 1 or len(rr) != len(ml):
        raise ValueError("seq_offsets must have batch + 1 entries, match_len and R batch entries")
    row0 = np.zeros(len(ml), np.int64)
    ln = np.zeros(len(ml), np.int32)
    _check(_lib.gdn_replay_windows(len(ml), off.ctypes.data, ml.ctypes.data, rr.ctypes.data,
                                   row0.ctypes.data, ln.ctypes.data), "gdn_replay_windows")
    return row0, ln


def gdn_plan_destroy(handle):
    _lib.gdn_plan_destroy(handle)


def gdn_plan_window(handle, b):
    r0, ln = ctypes.c_int64(), ctypes.c_int32()
    _check(_lib.gdn_plan_window(handle, int(b), ctypes.byref(r0), ctypes.byref(ln)), "gdn_plan_window")
    return r0.value, ln.value


def gdn_plan_info(handle):
    u, t, k = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int32()
    _check(_lib.gdn_plan_info(handle, ctypes.byref(u), ctypes.byref(t), ctypes.byref(k)), "gdn_plan_info")
    return {"units": u.value, "total_tokens": t.value, "kernel": k.value}


def gdn_plan_launches(handle) -> int:
    n = ctypes.c_int32()
    _check(_lib.gdn_plan_launches(handle, ctypes.byref(n)), "gdn_plan_launches")
    return n.value


def gdn_workspace_bytes(handle) -> int:
    return int(_lib.gdn_workspace_bytes(handle))


def gdn_tail_replay_state(handle, q, k, v, alpha, beta, seq_offsets, match_len, R, state_out,
                          workspace, stream=None):
    """Launch the tail replay (tensors on the plan's device; any may be a raw int address)."""
    _check(_lib.gdn_tail_replay_state(handle, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                      _ptr(seq_offsets), _ptr(match_len), _ptr(R), _ptr(state_out),
                                      _ptr(workspace), _stream_handle(stream)),
           "gdn_tail_replay_state")


def gdn_tail_replay_outputs(handle, q, k, v, alpha, beta, seq_offsets, match_len, R, o_out, state_out,
                            workspace, stream=None):
    """Tail replay that also writes o_t = S_t^T q_t for every window row (rows of o_out
    outside the windows are left untouched)."""
    _check(_lib.gdn_tail_replay_outputs(handle, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                        _ptr(seq_offsets), _ptr(match_len), _ptr(R), _ptr(o_out),
                                        _ptr(state_out), _ptr(workspace), _stream_handle(stream)),
           "gdn_tail_replay_outputs")


def gdn_tail_replay_prefill(handle, k, v, alpha, beta, sq, sk, sv, salpha, sbeta, o_out, state_mid,
                            state_out, workspace, stream=None):
    """Fused rebuild of the states and prefill of the suffixes (one launch on the
    tensor-core kernel)."""
    _check(_lib.gdn_tail_replay_prefill(handle, _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(sq), _ptr(sk),
                                        _ptr(sv), _ptr(salpha), _ptr(sbeta), _ptr(o_out), _ptr(state_mid),
                                        _ptr(state_out), _ptr(workspace), _stream_handle(stream)),
           "gdn_tail_replay_prefill")


def gdn_decode_step(q, k, v, alpha, beta, state_in, state_out, o_out, stream=None):
    """One decode step on dense [B, H, d] tensors (state [B, H, dk, dv] fp32; state_out may be
    state_in for an in-place update)."""
    B, H, dk = k.shape
    dv = v.shape[2]
    _check(_lib.gdn_decode_step(int(B), int(H), int(dk), int(dv), _dtype_code(k.dtype), _ptr(q), _ptr(k),
                                _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state_in), _ptr(state_out),
                                _ptr(o_out), _stream_handle(stream)),
           "gdn_decode_step")


def gdn_chunk_prefill(handle, q, k, v, alpha, beta, cu_seqlens, state_in, o_out, state_out,
                      workspace, stream=None):
    _check(_lib.gdn_chunk_prefill(handle, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                  _ptr(cu_seqlens), _ptr(state_in), _ptr(o_out), _ptr(state_out),
                                  _ptr(workspace), _stream_handle(stream)),
           "gdn_chunk_prefill")


def gdn_tail_replay_state_noalloc(H, dk, dv, dtype, seq_offsets, match_len, R, k, v, alpha, beta,
                                  state_out, kernel=GDN_KERNEL_AUTO, stream=None, wait_status=True,
                                  row_stride=0):
    """Replay without any device allocation (schedule in the library's fixed
    device array).  Returns the device status word when wait_status is set."""
    off, ml, rr = _i32(seq_offsets), _i32(match_len), _i32(R)
    if len(off) != len(ml) + 1 or len(rr) != len(ml):
        raise ValueError("seq_offsets must have batch + 1 entries, match_len and R batch entries")
    d = _make_desc(len(ml), H, dk, dv, dtype, kernel, off, row_stride)
    st = ctypes.c_uint32(0xFFFFFFFF)
    _check(_lib.gdn_tail_replay_state_noalloc(ctypes.byref(d), ml.ctypes.data, rr.ctypes.data,
                                              _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                              _ptr(state_out), _stream_handle(stream),
                                              ctypes.byref(st) if wait_status else None),
           "gdn_tail_replay_state_noalloc")
    return st.value if wait_status else None


def gdn_selftest_bounded_wait(limit_ns, workspace, stream=None):
    """Launch the failure-path self-test: a device wait bounded by limit_ns that runs out."""
    _check(_lib.gdn_selftest_bounded_wait(int(limit_ns), _ptr(workspace), _stream_handle(stream)),
           "gdn_selftest_bounded_wait")


def gdn_selftest_index_check(workspace, stream=None):
    """Debug build only: run one failing index check (access skipped); the workspace
    status then reads GDN_ERR_BOUNDS."""
    _check(_lib.gdn_selftest_index_check(_ptr(workspace), _stream_handle(stream)), "gdn_selftest_index_check")


def gdn_selftest_split_entry(entry, index, parts, most_tokens, rows, num_kv_heads) -> bool:
    """Whether the paged attention's merging kernel would merge a table entry (5 host ints) at `index`."""
    return bool(_lib.gdn_selftest_split_entry((ctypes.c_int32 * 5)(*entry), index, parts, most_tokens, rows, num_kv_heads))


def gdn_debug_bounds_enabled() -> bool:
    return bool(_lib.gdn_debug_bounds_enabled())


def gdn_debug_fail_plan_allocations(count):
    """Make the next `count` plan creations fail with GDN_ERR_ALLOC (0 clears it)."""
    _lib.gdn_debug_fail_plan_allocations(int(count))


def gdn_workspace_status(workspace, stream=None) -> int:
    """Synchronise the stream and return the device-side status of the last call."""
    return int(_lib.gdn_workspace_status(_ptr(workspace), _stream_handle(stream)))


# The operators below are called once per layer and token, so their argument checks are
# written to cost little: no torch import, stream object or library lookup per call.

_torch_module = None
_codes = {}


def _torch():
    """torch, imported at the first call that needs it."""
    global _torch_module
    if _torch_module is None:
        import torch
        _codes.update({torch.float32: GDN_F32, torch.bfloat16: GDN_BF16})
        _torch_module = torch
    return _torch_module


def _code(dtype):
    code = _codes.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def _row_stride(shape, stride, name):
    """Row stride (elements; 0 = packed) of a [rows, heads, dim] view with contiguous heads inside a row."""
    rows, heads, dim = shape
    if rows and (stride[2] != 1 or (heads > 1 and stride[1] != dim)):
        raise ValueError(f"{name} must have contiguous heads inside a row")
    if rows > 1 and stride[0] == 0:   # the descriptors' 0 means packed rows
        raise ValueError(f"{name} must not be one row expanded to many")
    return stride[0] if rows > 1 else 0


def _dense(t, shape, dtype, name):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")


def _launch_device(*tensors):
    """The current CUDA device, where the call launches and every tensor must be."""
    here = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            here = -1
    if here < 0 or here != _torch().cuda.current_device():
        raise ValueError("every tensor must be on the current CUDA device")
    return here


def _launch_stream(stream, device):
    if stream is not None:
        if stream.device_index != device:
            raise ValueError("the stream belongs to another device")
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # the current stream without an object around it
    return raw(device) if raw is not None else torch.cuda.current_stream().cuda_stream


def _refused(status, what, **tensors):
    """Raises for a call's status, naming the tensors that start off a 16-byte boundary: a slice of an index array
    (``positions[1:]``) is the likeliest refusal that a program meets."""
    off = [name for name, t in tensors.items() if t is not None and t.data_ptr() % 16]
    if status == GDN_ERR_INVALID_ARG and off:
        what = f"{what}: {', '.join(off)} must start on a 16-byte boundary"
    raise GdnError(status, what)


_entry = {}


def _fn(name):
    """The library's entry point, looked up once."""
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(library(), name)
    return f


# Descriptors by their fields: a program's calls repeat a few shapes.  The structures are never changed.
@functools.lru_cache(maxsize=256)
def _kv_desc(shape, stride, packed, code):
    if len(shape) != 4 or stride[3] != 1:
        raise ValueError("k_cache and v_cache must be [num_pages, page_size, num_kv_heads, head_dim] with contiguous "
                         "elements inside a head")
    if any(n > 1 and s == 0 for n, s in zip(shape, stride)):   # the descriptor's three zeros mean packed
        raise ValueError("k_cache and v_cache must not be expanded")
    return gdn_paged_kv(*shape, code, 0, *((0, 0, 0) if packed else stride[:3]))


@functools.lru_cache(maxsize=256)
def _qk_desc(*fields):
    return gdn_qk_desc(*fields)


@functools.lru_cache(maxsize=256)
def _attn_desc(batch, num_heads, rows, q_row_stride, max_pages, window, scale):
    if not 0 <= window < 2 ** 31:   # ctypes would take its low 32 bits
        raise ValueError("window must be 0 (all keys) to 2^31 - 1")
    return gdn_attn_desc(batch, num_heads, rows, q_row_stride, max_pages, window, scale, 0)


def _paged_kv(k_cache, v_cache):
    """Descriptor of [num_pages, page_size, num_kv_heads, head_dim] key and value pools (any strides with
    contiguous elements inside a head, the same for both)."""
    shape, stride, dtype = k_cache.shape, k_cache.stride(), k_cache.dtype
    if shape != v_cache.shape or dtype is not v_cache.dtype:
        raise ValueError("k_cache and v_cache must be alike")
    if stride != v_cache.stride():
        raise ValueError("k_cache and v_cache must share their strides")
    _torch()
    return _kv_desc(shape, stride, k_cache.is_contiguous(), _code(dtype))


def gdn_qk_norm_rope(q, k, v, positions, inv_freq, q_weight, k_weight, eps, k_cache, v_cache, slots, q_out, k_out,
                     interleaved=False, stream=None):
    """Norm, rotation and cache append (see ``qk_norm_rope``); every output is given."""
    torch = _torch()
    device = _launch_device(q, k, v, positions, inv_freq, q_weight, k_weight, k_cache, v_cache, slots, q_out, k_out)
    q_shape, k_shape, dtype = q.shape, k.shape, q.dtype
    if len(q_shape) != 3 or len(k_shape) != 3 or q_shape[0] != k_shape[0] or q_shape[2] != k_shape[2]:
        raise ValueError("q must be [rows, num_heads, head_dim] and k [rows, num_kv_heads, head_dim]")
    rows, heads, dim = q_shape
    if k.dtype is not dtype or (v is not None and v.dtype is not dtype):
        raise ValueError("q, k and v must have one dtype")
    half, pos_ptr, freq_ptr, qw_ptr, kw_ptr, ko_ptr = 0, None, None, None, None, None
    if inv_freq is not None:
        half = inv_freq.numel()
        _dense(inv_freq, (half,), torch.float64, "inv_freq")
        _dense(positions, (rows,), torch.int64, "positions")
        pos_ptr, freq_ptr = positions.data_ptr(), inv_freq.data_ptr()
    if q_weight is not None:
        _dense(q_weight, (dim,), torch.float32, "q_weight")
        qw_ptr = q_weight.data_ptr()
    if k_weight is not None:
        _dense(k_weight, (dim,), torch.float32, "k_weight")
        kw_ptr = k_weight.data_ptr()
    _dense(q_out, q_shape, dtype, "q_out")
    if k_out is not None:
        _dense(k_out, k_shape, dtype, "k_out")
        ko_ptr = k_out.data_ptr()
    cache, v_stride, v_ptr, k_pages, v_pages, slot_ptr = None, 0, None, None, None, None
    if k_cache is not None:
        if v is None or v_cache is None or slots is None or v.shape != k_shape:
            raise ValueError("a cache needs v (shaped like k), v_cache and slots")
        v_stride = _row_stride(k_shape, v.stride(), "v")
        _dense(slots, (rows,), torch.int64, "slots")
        if k_cache.dtype is not dtype:
            raise ValueError("the cache must have the dtype of q, k and v")
        cache = ctypes.byref(_paged_kv(k_cache, v_cache))
        v_ptr, k_pages, v_pages, slot_ptr = v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), slots.data_ptr()
    elif slots is not None or v_cache is not None:
        raise ValueError("slots and v_cache need k_cache")
    d = _qk_desc(rows, heads, k_shape[1], dim, 2 * half, GDN_ROTARY_INTERLEAVED if interleaved else GDN_ROTARY_HALVES,
                 _code(dtype), _row_stride(q_shape, q.stride(), "q"), _row_stride(k_shape, k.stride(), "k"), v_stride)
    status = _fn("gdn_qk_norm_rope")(
        ctypes.byref(d), q.data_ptr(), k.data_ptr(), v_ptr, pos_ptr, freq_ptr, qw_ptr, kw_ptr, eps, cache, slot_ptr,
        k_pages, v_pages, q_out.data_ptr(), ko_ptr, _launch_stream(stream, device))
    if status:
        _refused(status, "gdn_qk_norm_rope", q=q, k=k, v=v, positions=positions, inv_freq=inv_freq, q_weight=q_weight,
                 k_weight=k_weight, k_cache=k_cache, v_cache=v_cache, slots=slots, q_out=q_out, k_out=k_out)


def gdn_paged_attention_workspace_bytes(dtype, head_dim, max_batch) -> int:
    return int(_fn("gdn_paged_attention_workspace_bytes")(_dtype_code(dtype), int(head_dim), int(max_batch)))


@functools.lru_cache(maxsize=256)
def _attention_bytes(code, dim, batch):
    return int(_fn("gdn_paged_attention_workspace_bytes")(code, dim, batch))


def gdn_paged_attention(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out, workspace, scale=None,
                        window=0, stream=None):
    """Causal attention of new tokens over a paged cache (see ``PagedAttention.run``)."""
    device = _launch_device(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out, workspace)
    _attend(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out, workspace, scale, window,
            _launch_stream(stream, device))


def _attend(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out, workspace, scale, window, stream):
    """gdn_paged_attention on tensors of the current device and a raw stream."""
    torch = _torch()
    c = _paged_kv(k_cache, v_cache)
    q_shape, t_shape = q.shape, page_table.shape
    if len(q_shape) != 3 or q.dtype is not k_cache.dtype:
        raise ValueError("q must be [rows, num_heads, head_dim] of the cache's dtype")
    rows, heads, dim = q_shape
    if dim != c.head_dim:
        raise ValueError("q and the cache must have one head_dim")
    if len(t_shape) != 2:
        raise ValueError("page_table must be [batch, max_pages]")
    batch, width = t_shape
    _dense(page_table, t_shape, torch.int32, "page_table")
    _dense(cu_seqlens, (batch + 1,), torch.int32, "cu_seqlens")
    _dense(context_len, (batch,), torch.int32, "context_len")
    _dense(o_out, q_shape, q.dtype, "o_out")
    lse_ptr = None
    if lse_out is not None:
        _dense(lse_out, (rows, heads), torch.float32, "lse_out")
        lse_ptr = lse_out.data_ptr()
    need = _attention_bytes(c.dtype, dim, batch)
    if not workspace.is_contiguous() or workspace.numel() * workspace.element_size() < need:
        raise ValueError(f"the workspace must be contiguous and have at least {need} bytes")
    d = _attn_desc(batch, heads, rows, _row_stride(q_shape, q.stride(), "q"), width, int(window),
                   dim ** -0.5 if scale is None else scale)
    status = _fn("gdn_paged_attention")(
        ctypes.byref(d), ctypes.byref(c), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(),
        cu_seqlens.data_ptr(), context_len.data_ptr(), o_out.data_ptr(), lse_ptr, workspace.data_ptr(), stream)
    if status:
        _refused(status, "gdn_paged_attention", q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table,
                 cu_seqlens=cu_seqlens, context_len=context_len, o_out=o_out, lse_out=lse_out, workspace=workspace)


class _Plan:
    def __init__(self, handle, H, dk, dv, dtype, batch):
        import torch
        self.handle, self.H, self.dk, self.dv, self.dtype, self.batch = handle, H, dk, dv, dtype, batch
        self.info = gdn_plan_info(handle)
        self.launches = gdn_plan_launches(handle)   # kernel launches per call
        self.workspace = torch.zeros(gdn_workspace_bytes(handle), dtype=torch.uint8, device="cuda")

    def window(self, b):
        return gdn_plan_window(self.handle, b)

    def status(self, stream=None) -> int:
        return gdn_workspace_status(self.workspace, stream)

    def check(self, stream=None):
        _check(self.status(stream), "device status")

    def close(self):
        if self.handle:
            gdn_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class ReplayPlan(_Plan):
    """Plan of a tail replay over a packed varlen cache (host int arrays)."""

    def __init__(self, H, dk, dv, dtype, seq_offsets, match_len, R, kernel=GDN_KERNEL_AUTO, row_stride=0):
        h = gdn_plan_create_replay(H, dk, dv, dtype, seq_offsets, match_len, R, kernel, row_stride)
        super().__init__(h, H, dk, dv, dtype, len(match_len))

    def run(self, k, v, alpha, beta, state_out, q=None, seq_offsets=None, match_len=None, R=None,
            stream=None, workspace=None):
        gdn_tail_replay_state(self.handle, q, k, v, alpha, beta, seq_offsets, match_len, R,
                              state_out, self.workspace if workspace is None else workspace, stream)

    def run_outputs(self, q, k, v, alpha, beta, o_out, state_out=None, seq_offsets=None, match_len=None,
                    R=None, stream=None, workspace=None):
        """Replay that also writes the window rows of o_out (see gdn_tail_replay_outputs)."""
        gdn_tail_replay_outputs(self.handle, q, k, v, alpha, beta, seq_offsets, match_len, R, o_out,
                                state_out, self.workspace if workspace is None else workspace, stream)


class PrefillPlan(_Plan):
    """Plan of a chunked prefill over whole packed sequences (host cu_seqlens)."""

    def __init__(self, H, dk, dv, dtype, cu_seqlens, kernel=GDN_KERNEL_AUTO, row_stride=0):
        h = gdn_plan_create_prefill(H, dk, dv, dtype, cu_seqlens, kernel, row_stride)
        super().__init__(h, H, dk, dv, dtype, len(cu_seqlens) - 1)

    def run(self, q, k, v, alpha, beta, o_out, state_in=None, state_out=None, cu_seqlens=None,
            stream=None, workspace=None):
        gdn_chunk_prefill(self.handle, q, k, v, alpha, beta, cu_seqlens, state_in, o_out, state_out,
                          self.workspace if workspace is None else workspace, stream)


class FusedPlan(_Plan):
    """Plan of a fused replay + suffix prefill (host int arrays)."""

    def __init__(self, H, dk, dv, dtype, seq_offsets, match_len, R, suffix_offsets, kernel=GDN_KERNEL_AUTO,
                 row_stride=0):
        h = gdn_plan_create_fused(H, dk, dv, dtype, seq_offsets, match_len, R, suffix_offsets, kernel,
                                  row_stride)
        super().__init__(h, H, dk, dv, dtype, len(match_len))

    def run(self, k, v, alpha, beta, sq, sk, sv, salpha, sbeta, o_out, state_out, state_mid=None, stream=None,
            workspace=None):
        gdn_tail_replay_prefill(self.handle, k, v, alpha, beta, sq, sk, sv, salpha, sbeta, o_out, state_mid,
                                state_out, self.workspace if workspace is None else workspace, stream)


def tail_replay_state(k, v, alpha, beta, seq_offsets, match_len, R, kernel=GDN_KERNEL_AUTO):
    """One-shot replay on torch CUDA tensors; returns state [B, H, dk, dv] fp32.  k and v
    may be row-strided views (e.g. slices of one fused projection buffer)."""
    import torch
    rows, H, dk = k.shape
    dv = v.shape[2]
    plan = ReplayPlan(H, dk, dv, k.dtype, seq_offsets, match_len, R, kernel, row_stride_of(k, v))
    out = torch.empty((plan.batch, H, dk, dv), dtype=torch.float32, device=k.device)
    plan.run(k, v, alpha, beta, out)
    plan.check()
    plan.close()
    return out


def chunk_prefill(q, k, v, alpha, beta, cu_seqlens, state_in=None, kernel=GDN_KERNEL_AUTO):
    """One-shot prefill on torch CUDA tensors; returns (o, state_out).  q, k and v may be
    row-strided views sharing one row stride; o is packed."""
    import torch
    rows, H, dk = k.shape
    dv = v.shape[2]
    plan = PrefillPlan(H, dk, dv, k.dtype, cu_seqlens, kernel, row_stride_of(q, k, v))
    o = torch.empty((rows, H, dv), dtype=k.dtype, device=k.device)
    st = torch.empty((plan.batch, H, dk, dv), dtype=torch.float32, device=k.device)
    plan.run(q, k, v, alpha, beta, o, state_in=state_in, state_out=st)
    plan.check()
    plan.close()
    return o, st


def decode_step(q, k, v, alpha, beta, state, o=None, in_place=True):
    """One decode step on torch CUDA tensors ([B, H, d], state [B, H, dk, dv] fp32).
    Updates `state` in place (or returns a new one) and returns (o, state)."""
    import torch
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    out = state if in_place else torch.empty_like(state)
    gdn_decode_step(q, k, v, alpha, beta, state, out, o)
    return o, out


class PagedAttention:
    """Causal attention of new tokens over a paged key/value cache, with the workspace that its calls share
    (calls that may run at the same time, or captured ones that may, need one each; it lives as long as graphs that
    captured its calls).

    Lengths and pages are device tensors read when the call runs, so a captured ``run`` may be replayed with new
    ones.  The cache already holds the new tokens (``qk_norm_rope`` appends them).
    """

    def __init__(self, num_heads, num_kv_heads, head_dim, dtype, max_batch, max_rows=None):
        import torch
        self.num_heads, self.num_kv_heads, self.head_dim = int(num_heads), int(num_kv_heads), int(head_dim)
        self.dtype, self.max_batch = _dtype_code(dtype), int(max_batch)
        self.max_rows = None if max_rows is None else int(max_rows)
        n = gdn_paged_attention_workspace_bytes(dtype, head_dim, max_batch)
        if n == 0 or num_kv_heads < 1 or num_heads < 1 or num_heads % num_kv_heads:
            raise GdnError(GDN_ERR_UNSUPPORTED, "PagedAttention")
        self.workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.workspace[:256].zero_()   # the status, for status() before the first run
        made_on = torch.cuda.current_stream()
        self._made = None if torch.cuda.is_current_stream_capturing() else made_on.record_event()
        self._ordered = {made_on.cuda_stream}   # streams that are behind the workspace's making

    def run(self, q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out=None, scale=None, window=0,
            stream=None, workspace=None):
        """q [rows, H, d] (row-strided views too); k_cache, v_cache [num_pages, page_size, Hkv, d]; page_table
        [B, max_pages], cu_seqlens [B + 1], context_len [B] int32; o_out [rows, H, d] and lse_out [rows, H] fp32
        are written at the rows that sequences own.  Row i of a sequence with n new tokens and context L is
        position L - n + i and sees the keys up to it, with a window only the last `window` of them.  Every tensor
        starts on a 16-byte boundary (copy an odd slice of an index array)."""
        rows, heads, dim = q.shape
        if heads != self.num_heads or dim != self.head_dim or k_cache.shape[2] != self.num_kv_heads:
            raise ValueError("q or the cache has other heads than this PagedAttention")
        if page_table.shape[0] > self.max_batch or (self.max_rows is not None and rows > self.max_rows):
            raise ValueError("more sequences or rows than this PagedAttention was made for")
        if workspace is None:
            workspace = self.workspace
        device = _launch_device(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out, workspace)
        handle = _launch_stream(stream, device)
        if handle not in self._ordered and workspace is self.workspace:
            self._order(stream, handle)
        _attend(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o_out, lse_out, workspace, scale, window, handle)

    def _order(self, stream, handle):
        """The first run on a stream other than the one that the workspace was made on: behind what that one had
        queued then (the memory's earlier owner, the zeroed status), and with the memory kept until this stream is done
        with it.  torch.cuda.graph waits for the device before it captures, and the caller keeps what it captured."""
        torch = _torch()
        if self._made is None or torch.cuda.is_current_stream_capturing():
            return
        stream = torch.cuda.current_stream() if stream is None else stream
        stream.wait_event(self._made)
        self.workspace.record_stream(stream)
        self._ordered.add(handle)

    def status(self, stream=None) -> int:
        return gdn_workspace_status(self.workspace, stream)

    def check(self, stream=None):
        _check(self.status(stream), "device status")


def paged_attention(q, k_cache, v_cache, page_table, cu_seqlens, context_len, scale=None, window=0, with_lse=False):
    """One-shot paged attention; returns o [rows, H, d], or (o, lse) with `with_lse`.  Rows that no sequence owns
    are zero (lse -inf)."""
    import torch
    attn = PagedAttention(q.shape[1], k_cache.shape[2], q.shape[2], q.dtype, page_table.shape[0])
    o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
    lse = torch.full(q.shape[:2], float("-inf"), dtype=torch.float32, device=q.device) if with_lse else None
    attn.run(q, k_cache, v_cache, page_table, cu_seqlens, context_len, o, lse, scale, window)
    attn.check()
    return (o, lse) if with_lse else o


def qk_norm_rope(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps=1e-6, interleaved=False, v=None,
                 k_cache=None, v_cache=None, slots=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every query and key head (where its weight is given), rotation of the first
    2 * inv_freq.numel() elements by position * inv_freq (fp64, radians), and, with a paged cache, the append of
    keys and values at `slots` (int64 page * page_size + row; a negative one writes nothing).

    q, k and v are [rows, heads, d] (row-strided views too).  Every tensor starts on a 16-byte boundary (copy an odd
    slice of an index array).  Returns (q_out, k_out); k_out is made only where there is no cache and none was given."""
    if q_out is None or (k_out is None and k_cache is None):
        torch = _torch()
        with torch.cuda.stream(stream):   # what is made here is made on the stream that fills it
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if k_out is None and k_cache is None:
                k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    gdn_qk_norm_rope(q, k, v, positions, inv_freq, q_weight, k_weight, eps, k_cache, v_cache, slots, q_out, k_out,
                     interleaved, stream)
    return q_out, k_out
