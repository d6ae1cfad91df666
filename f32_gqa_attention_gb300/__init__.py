"""Python binding of the GB300 f32 attention library (``libvtmu.so``).

Argument marshalling only: every step of the ops runs in the library's CUDA
kernels.  The binding exposes the C ABI of ``include/vtmu_attention.h`` under
the same names (``vtmu_attention``, ``vtmu_cache_write``, ...) plus two
conveniences for PyTorch CUDA tensors, ``attention`` and ``cache_write``,
whose keyword names follow the op catalog (vtmu.mpakt.dev/api/ops, ops
"attention" and "cache_write").  PyTorch only provides device memory and
streams.

There is no fallback: if ``libvtmu.so`` is not built, loading raises.
Build it with ``python -m f32_gqa_attention_gb300._build``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libvtmu.so")

VTMU_OK = 0
VTMU_ERR_INVALID = 1
VTMU_ERR_UNSUPPORTED = 2
VTMU_ERR_RANGE = 3
VTMU_ERR_WORKSPACE = 4
VTMU_ERR_CUDA = 5

VTMU_ALIBI_NONE, VTMU_ALIBI_BLOOM, VTMU_ALIBI_MPT, VTMU_ALIBI_SLOPES = 0, 1, 2, 3
VTMU_BIAS_NONE, VTMU_BIAS_TS, VTMU_BIAS_HTS = 0, 1, 2
VTMU_KERNEL_AUTO, VTMU_KERNEL_DECODE, VTMU_KERNEL_PREFILL_FFMA, VTMU_KERNEL_PREFILL_TF32X3 = 0, 1, 2, 3
VTMU_KERNEL_DECODE_TF32X3 = 4

EXPORTED = ("vtmu_attention_params_init", "vtmu_attention_workspace_size", "vtmu_attention",
            "vtmu_cache_write", "vtmu_features", "vtmu_last_error", "vtmu_attention_decode_noalloc",
            "vtmu_device_error", "vtmu_decode_step", "vtmu_decode_step_host_workspace_size",
            "vtmu_decode_step_host", "vtmu_rope_params_init", "vtmu_rope", "vtmu_decode_step_rope",
            "vtmu_mla_params_init", "vtmu_mla_workspace_size", "vtmu_mla_attention", "vtmu_mla_decode_step",
            "vtmu_mla_decode_step_host_workspace_size", "vtmu_mla_decode_step_host",
            "vtmu_page_map", "vtmu_tree_plan", "vtmu_rope_at", "vtmu_paged_write", "vtmu_paged_params_init",
            "vtmu_paged_workspace_size", "vtmu_paged_attention")
NOALLOC_SCRATCH_BYTES = 8 << 20  # VTMU_NOALLOC_SCRATCH_BYTES


class VtmuError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"vtmu status {status}: {message}")
        self.status = status


class vtmu_attention_params(ctypes.Structure):
    """Mirror of ``vtmu_attention_params`` (include/vtmu_attention.h)."""
    _fields_ = [
        ("T", ctypes.c_int64),
        ("S", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("v_head_dim", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("has_scale", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("pos_offset", ctypes.c_int64),
        ("window", ctypes.c_int64),
        ("alibi", ctypes.c_int32),
        ("alibi_max", ctypes.c_float),
        ("alibi_slopes", ctypes.POINTER(ctypes.c_float)),
        ("bias_kind", ctypes.c_int32),
        ("kernel", ctypes.c_int32),
        ("decode_splits", ctypes.c_int32),
        ("sinks", ctypes.c_int64),
    ]


VTMU_ROPE_SCALING_NONE, VTMU_ROPE_SCALING_LINEAR = 0, 1


class vtmu_rope_params(ctypes.Structure):
    """Mirror of ``vtmu_rope_params`` (include/vtmu_attention.h)."""
    _fields_ = [
        ("head_dim", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("scaling", ctypes.c_int32),
        ("base", ctypes.c_float),
        ("scaling_factor", ctypes.c_float),
        ("attention_factor", ctypes.c_float),
        ("inv_freq", ctypes.POINTER(ctypes.c_float)),
    ]


class vtmu_mla_params(ctypes.Structure):
    """Mirror of ``vtmu_mla_params`` (include/vtmu_attention.h)."""
    _fields_ = [
        ("T", ctypes.c_int64),
        ("S", ctypes.c_int64),
        ("heads", ctypes.c_int32),
        ("kv_rank", ctypes.c_int32),
        ("qk_nope", ctypes.c_int32),
        ("qk_rope", ctypes.c_int32),
        ("v_head_dim", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("has_scale", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("pos_offset", ctypes.c_int64),
        ("window", ctypes.c_int64),
        ("sinks", ctypes.c_int64),
        ("kernel", ctypes.c_int32),
    ]


class vtmu_paged_params(ctypes.Structure):
    """Mirror of ``vtmu_paged_params`` (include/vtmu_attention.h)."""
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("pages", ctypes.c_int64),
        ("requests", ctypes.c_int32),
        ("max_rows", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("heads", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("tree", ctypes.c_int32),
        ("has_scale", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("kernel", ctypes.c_int32),
        ("window", ctypes.c_int64),
        ("sinks", ctypes.c_int64),
    ]


VTMU_PAGED_AUTO, VTMU_PAGED_CUDA_CORES, VTMU_PAGED_TENSOR_CORES = 0, 1, 2
TREE_MAX_ROWS = 64  # VTMU_TREE_MAX_ROWS

MLA_KERNEL_AUTO, MLA_KERNEL_CUDA_CORES, MLA_KERNEL_TENSOR_CORES = 0, 1, 2

_lib = None
_lib_lock = threading.Lock()


def load_library():
    """Load libvtmu.so (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run `python -m f32_gqa_attention_gb300._build`")
        lib = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(vtmu_attention_params)
        vp = ctypes.c_void_p
        lib.vtmu_attention_params_init.argtypes = [P]
        lib.vtmu_attention_params_init.restype = None
        lib.vtmu_attention_workspace_size.argtypes = [P, ctypes.POINTER(ctypes.c_size_t)]
        lib.vtmu_attention_workspace_size.restype = ctypes.c_int
        lib.vtmu_attention.argtypes = [vp, vp, vp, vp, vp, P, vp, ctypes.c_size_t, vp]
        lib.vtmu_attention.restype = ctypes.c_int
        lib.vtmu_cache_write.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, vp, ctypes.c_int64,
                                         ctypes.c_int64, vp]
        lib.vtmu_cache_write.restype = ctypes.c_int
        lib.vtmu_features.argtypes = []
        lib.vtmu_features.restype = ctypes.c_char_p
        lib.vtmu_last_error.argtypes = []
        lib.vtmu_last_error.restype = ctypes.c_char_p
        lib.vtmu_decode_step.argtypes = [vp, vp, ctypes.c_int64, vp, vp, ctypes.c_int64, ctypes.c_int64,
                                         vp, vp, vp, P, vp, ctypes.c_size_t, vp]
        lib.vtmu_decode_step.restype = ctypes.c_int
        lib.vtmu_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        lib.vtmu_device_error.restype = ctypes.c_int
        lib.vtmu_attention_decode_noalloc.argtypes = [vp, vp, vp, vp, vp, P, vp]
        lib.vtmu_attention_decode_noalloc.restype = ctypes.c_int
        R = ctypes.POINTER(vtmu_rope_params)
        lib.vtmu_rope_params_init.argtypes = [R]
        lib.vtmu_rope_params_init.restype = None
        lib.vtmu_rope.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int64, R, vp]
        lib.vtmu_rope.restype = ctypes.c_int
        lib.vtmu_decode_step_rope.argtypes = [vp, vp, ctypes.c_int64, vp, vp, ctypes.c_int64, ctypes.c_int64,
                                              vp, vp, vp, P, R, vp, ctypes.c_size_t, vp]
        lib.vtmu_decode_step_rope.restype = ctypes.c_int
        lib.vtmu_decode_step_host_workspace_size.argtypes = [P, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]
        lib.vtmu_decode_step_host_workspace_size.restype = ctypes.c_int
        lib.vtmu_decode_step_host.argtypes = [vp, vp, ctypes.c_int64, vp, vp, ctypes.c_int64, ctypes.c_int64,
                                              vp, vp, vp, P, vp, ctypes.c_size_t, vp]
        lib.vtmu_decode_step_host.restype = ctypes.c_int
        M = ctypes.POINTER(vtmu_mla_params)
        lib.vtmu_mla_params_init.argtypes = [M]
        lib.vtmu_mla_params_init.restype = None
        lib.vtmu_mla_workspace_size.argtypes = [M, ctypes.POINTER(ctypes.c_size_t)]
        lib.vtmu_mla_workspace_size.restype = ctypes.c_int
        lib.vtmu_mla_attention.argtypes = [vp, vp, vp, vp, vp, M, vp, ctypes.c_size_t, vp]
        lib.vtmu_mla_attention.restype = ctypes.c_int
        lib.vtmu_mla_decode_step.argtypes = [vp, ctypes.c_int64, vp, ctypes.c_int64, ctypes.c_int64, vp, vp, vp, vp,
                                             M, vp, ctypes.c_size_t, vp]
        lib.vtmu_mla_decode_step.restype = ctypes.c_int
        lib.vtmu_mla_decode_step_host_workspace_size.argtypes = [M, ctypes.c_int64, ctypes.POINTER(ctypes.c_size_t)]
        lib.vtmu_mla_decode_step_host_workspace_size.restype = ctypes.c_int
        lib.vtmu_mla_decode_step_host.argtypes = [vp, ctypes.c_int64, vp, ctypes.c_int64, ctypes.c_int64, vp, vp,
                                                  vp, vp, M, vp, ctypes.c_size_t, vp]
        lib.vtmu_mla_decode_step_host.restype = ctypes.c_int
        i32, i64 = ctypes.c_int32, ctypes.c_int64
        lib.vtmu_page_map.argtypes = [vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, i64, i32, i32, vp]
        lib.vtmu_page_map.restype = ctypes.c_int
        lib.vtmu_tree_plan.argtypes = [vp, vp, vp, vp, vp, i32, i64, vp]
        lib.vtmu_tree_plan.restype = ctypes.c_int
        lib.vtmu_rope_at.argtypes = [vp, vp, i64, i32, vp, R, vp]
        lib.vtmu_rope_at.restype = ctypes.c_int
        lib.vtmu_paged_write.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp, i64, vp]
        lib.vtmu_paged_write.restype = ctypes.c_int
        G = ctypes.POINTER(vtmu_paged_params)
        lib.vtmu_paged_params_init.argtypes = [G]
        lib.vtmu_paged_params_init.restype = None
        lib.vtmu_paged_workspace_size.argtypes = [G, ctypes.POINTER(ctypes.c_size_t)]
        lib.vtmu_paged_workspace_size.restype = ctypes.c_int
        lib.vtmu_paged_attention.argtypes = [vp] * 11 + [G, vp, ctypes.c_size_t, vp]
        lib.vtmu_paged_attention.restype = ctypes.c_int
        _lib = lib
        return lib


def _check(status: int):
    if status != VTMU_OK:
        raise VtmuError(status, load_library().vtmu_last_error().decode())


def _addr(x):
    """Device address of a torch tensor, or an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _haddr(x):
    """Host address of a contiguous f32 numpy array or CPU tensor, an int, or None."""
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if x.device.type != "cpu" or not x.is_contiguous() or x.element_size() != 4:
            raise ValueError("host buffer: expected a contiguous f32 CPU tensor")
        return x.data_ptr()
    if x.dtype.itemsize != 4 or x.dtype.kind != "f" or not x.flags["C_CONTIGUOUS"]:
        raise ValueError("host buffer: expected a C-contiguous float32 array")
    return x.ctypes.data


# ---------------------------------------------------------------- C ABI names
def vtmu_attention_params_init() -> vtmu_attention_params:
    p = vtmu_attention_params()
    load_library().vtmu_attention_params_init(ctypes.byref(p))
    return p


def vtmu_attention_workspace_size(p: vtmu_attention_params) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().vtmu_attention_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def vtmu_attention(q, k, v, bias, out, p: vtmu_attention_params, workspace, workspace_bytes: int,
                   stream: int = 0) -> None:
    _check(load_library().vtmu_attention(_addr(q), _addr(k), _addr(v), _addr(bias), _addr(out),
                                         ctypes.byref(p), _addr(workspace), int(workspace_bytes),
                                         stream or None))


def vtmu_decode_step(k_cache, v_cache, max_rows: int, k_new, v_new, new_rows: int, offset: int, q, bias, out,
                     p: vtmu_attention_params, workspace, workspace_bytes: int, stream: int = 0) -> None:
    _check(load_library().vtmu_decode_step(_addr(k_cache), _addr(v_cache), int(max_rows), _addr(k_new),
                                           _addr(v_new), int(new_rows), int(offset), _addr(q), _addr(bias),
                                           _addr(out), ctypes.byref(p), _addr(workspace), int(workspace_bytes),
                                           stream or None))


def vtmu_decode_step_host_workspace_size(p: vtmu_attention_params, new_rows: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().vtmu_decode_step_host_workspace_size(ctypes.byref(p), int(new_rows), ctypes.byref(n)))
    return int(n.value)


def vtmu_decode_step_host(k_cache, v_cache, max_rows: int, k_new_host, v_new_host, new_rows: int, offset: int,
                          q_host, bias_host, out_host, p: vtmu_attention_params, workspace, workspace_bytes: int,
                          stream: int = 0) -> None:
    """vtmu_decode_step with q / new rows / bias / out in host memory (numpy
    arrays or CPU tensors, f32, contiguous; pinned memory copies
    asynchronously).  Returns once out_host holds the result."""
    _check(load_library().vtmu_decode_step_host(_addr(k_cache), _addr(v_cache), int(max_rows), _haddr(k_new_host),
                                                _haddr(v_new_host), int(new_rows), int(offset), _haddr(q_host),
                                                _haddr(bias_host), _haddr(out_host), ctypes.byref(p),
                                                _addr(workspace), int(workspace_bytes), stream or None))


def vtmu_rope_params_init() -> vtmu_rope_params:
    r = vtmu_rope_params()
    load_library().vtmu_rope_params_init(ctypes.byref(r))
    return r


def vtmu_rope(x, out, T: int, heads: int, offset: int, r: vtmu_rope_params, stream: int = 0) -> None:
    _check(load_library().vtmu_rope(_addr(x), _addr(out), int(T), int(heads), int(offset), ctypes.byref(r),
                                    stream or None))


def vtmu_decode_step_rope(k_cache, v_cache, max_rows: int, k_new, v_new, new_rows: int, offset: int, q, bias, out,
                          p: vtmu_attention_params, r: vtmu_rope_params, workspace, workspace_bytes: int,
                          stream: int = 0) -> None:
    _check(load_library().vtmu_decode_step_rope(_addr(k_cache), _addr(v_cache), int(max_rows), _addr(k_new),
                                                _addr(v_new), int(new_rows), int(offset), _addr(q), _addr(bias),
                                                _addr(out), ctypes.byref(p), ctypes.byref(r), _addr(workspace),
                                                int(workspace_bytes), stream or None))


def vtmu_cache_write(cache, max_rows: int, width: int, values, rows: int, offset: int, stream: int = 0) -> None:
    _check(load_library().vtmu_cache_write(_addr(cache), int(max_rows), int(width), _addr(values),
                                           int(rows), int(offset), stream or None))


def vtmu_attention_decode_noalloc(q, k, v, bias, out, p: vtmu_attention_params, stream: int = 0) -> None:
    """Decode (T == 1) with the library's static scratch: no workspace, no
    allocation, for callers that cannot allocate device memory.  The first
    call on a device looks up the scratch address (do it before any stream
    capture); calls that overlap on the GPU race on the shared scratch."""
    _check(load_library().vtmu_attention_decode_noalloc(_addr(q), _addr(k), _addr(v), _addr(bias), _addr(out),
                                                        ctypes.byref(p), stream or None))


def vtmu_mla_params_init() -> vtmu_mla_params:
    p = vtmu_mla_params()
    load_library().vtmu_mla_params_init(ctypes.byref(p))
    return p


def vtmu_mla_workspace_size(p: vtmu_mla_params) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().vtmu_mla_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def vtmu_mla_attention(q, state, k_b, v_b, out, p: vtmu_mla_params, workspace, workspace_bytes: int,
                       stream: int = 0) -> None:
    _check(load_library().vtmu_mla_attention(_addr(q), _addr(state), _addr(k_b), _addr(v_b), _addr(out),
                                             ctypes.byref(p), _addr(workspace), int(workspace_bytes),
                                             stream or None))


def vtmu_mla_decode_step(state, max_rows: int, state_new, new_rows: int, offset: int, q, k_b, v_b, out,
                         p: vtmu_mla_params, workspace, workspace_bytes: int, stream: int = 0) -> None:
    _check(load_library().vtmu_mla_decode_step(_addr(state), int(max_rows), _addr(state_new), int(new_rows),
                                               int(offset), _addr(q), _addr(k_b), _addr(v_b), _addr(out),
                                               ctypes.byref(p), _addr(workspace), int(workspace_bytes),
                                               stream or None))


def vtmu_mla_decode_step_host_workspace_size(p: vtmu_mla_params, new_rows: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().vtmu_mla_decode_step_host_workspace_size(ctypes.byref(p), int(new_rows), ctypes.byref(n)))
    return int(n.value)


def vtmu_mla_decode_step_host(state, max_rows: int, state_new_host, new_rows: int, offset: int, q_host, k_b, v_b,
                              out_host, p: vtmu_mla_params, workspace, workspace_bytes: int, stream: int = 0) -> None:
    """vtmu_mla_decode_step with q / new latent rows / out in host memory
    (numpy arrays or CPU tensors, f32, contiguous; pinned buffers are used in
    place).  Returns once out_host holds the result."""
    _check(load_library().vtmu_mla_decode_step_host(_addr(state), int(max_rows), _haddr(state_new_host),
                                                    int(new_rows), int(offset), _haddr(q_host), _addr(k_b),
                                                    _addr(v_b), _haddr(out_host), ctypes.byref(p), _addr(workspace),
                                                    int(workspace_bytes), stream or None))


def vtmu_page_map(lens, cu_rows, accept, block_table, free_pages, free_capacity: int, n_free, slots, positions,
                  new_lens, n_free_out, requests: int, rows: int, page_size: int, max_pages: int,
                  stream: int = 0) -> None:
    _check(load_library().vtmu_page_map(_addr(lens), _addr(cu_rows), _addr(accept), _addr(block_table),
                                        _addr(free_pages), int(free_capacity), _addr(n_free), _addr(slots),
                                        _addr(positions), _addr(new_lens), _addr(n_free_out), int(requests),
                                        int(rows), int(page_size), int(max_pages), stream or None))


def vtmu_tree_plan(parents, cu_rows, lens, masks, positions, requests: int, rows: int, stream: int = 0) -> None:
    _check(load_library().vtmu_tree_plan(_addr(parents), _addr(cu_rows), _addr(lens), _addr(masks),
                                         _addr(positions), int(requests), int(rows), stream or None))


def vtmu_rope_at(x, out, T: int, heads: int, positions, r: vtmu_rope_params, stream: int = 0) -> None:
    _check(load_library().vtmu_rope_at(_addr(x), _addr(out), int(T), int(heads), _addr(positions), ctypes.byref(r),
                                       stream or None))


def vtmu_paged_write(k_pool, v_pool, pool_rows: int, k_width: int, v_width: int, k_new, v_new, slots, rows: int,
                     stream: int = 0) -> None:
    _check(load_library().vtmu_paged_write(_addr(k_pool), _addr(v_pool), int(pool_rows), int(k_width),
                                           int(v_width), _addr(k_new), _addr(v_new), _addr(slots), int(rows),
                                           stream or None))


def vtmu_paged_params_init() -> vtmu_paged_params:
    p = vtmu_paged_params()
    load_library().vtmu_paged_params_init(ctypes.byref(p))
    return p


def vtmu_paged_workspace_size(p: vtmu_paged_params) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().vtmu_paged_workspace_size(ctypes.byref(p), ctypes.byref(n)))
    return int(n.value)


def vtmu_paged_attention(q, k_pool, v_pool, block_table, lens, cu_rows, k_new, v_new, masks, positions, out,
                         p: vtmu_paged_params, workspace, workspace_bytes: int, stream: int = 0) -> None:
    _check(load_library().vtmu_paged_attention(_addr(q), _addr(k_pool), _addr(v_pool), _addr(block_table),
                                               _addr(lens), _addr(cu_rows), _addr(k_new), _addr(v_new),
                                               _addr(masks), _addr(positions), _addr(out), ctypes.byref(p),
                                               _addr(workspace), int(workspace_bytes), stream or None))


def vtmu_device_error() -> int:
    """Synchronises the device; returns and clears the kernels' wait-timeout
    flags (0 when no bounded wait gave up)."""
    v = ctypes.c_uint(0)
    _check(load_library().vtmu_device_error(ctypes.byref(v)))
    return int(v.value)


def vtmu_features() -> str:
    return load_library().vtmu_features().decode()


def vtmu_last_error() -> str:
    return load_library().vtmu_last_error().decode()


# ------------------------------------------------------------ torch helpers
def make_params(T, S, *, heads, headDim, kvHeads=None, vHeadDim=None, causal=True, posOffset=0,
                scale=None, softcap=None, window=None, alibi=False, alibiMax=None, alibiSlopes=None,
                bias_kind=VTMU_BIAS_NONE, kernel=VTMU_KERNEL_AUTO, decode_splits=0, sinks=None):
    """A params struct from the op catalog's parameter names.  ALiBi
    precedence: alibiSlopes, then alibiMax, then alibi.  The returned struct
    keeps any slope array alive as ``_slopes``."""
    p = vtmu_attention_params_init()
    p.T, p.S = int(T), int(S)
    p.heads = int(heads)
    p.kv_heads = 0 if kvHeads is None else int(kvHeads)
    p.head_dim = int(headDim)
    p.v_head_dim = 0 if vHeadDim is None else int(vHeadDim)
    p.causal = 1 if causal else 0
    p.pos_offset = int(posOffset)
    if scale is not None:
        p.has_scale, p.scale = 1, float(scale)
    p.softcap = 0.0 if softcap is None else float(softcap)
    p.window = 0 if window is None else int(window)
    if alibiSlopes is not None:
        arr = (ctypes.c_float * len(alibiSlopes))(*[float(s) for s in alibiSlopes])
        p.alibi, p.alibi_slopes = VTMU_ALIBI_SLOPES, ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
        p._slopes = arr
    elif alibiMax is not None:
        p.alibi, p.alibi_max = VTMU_ALIBI_MPT, float(alibiMax)
    elif alibi:
        p.alibi = VTMU_ALIBI_BLOOM
    p.bias_kind = int(bias_kind)
    p.kernel = int(kernel)
    p.decode_splits = int(decode_splits)
    p.sinks = 0 if sinks is None else int(sinks)
    return p


def make_rope_params(*, headDim, base=None, rotaryDim=None, interleaved=False, scaling=None, invFreq=None,
                     attentionFactor=None):
    """A rope params struct from op "rope"'s parameter names.  ``scaling`` is
    config.json's rope_scaling object; "linear" maps to the library's linear
    scaling and any other kind is passed on so that the library refuses it
    with "rope.scaling" named.  Keeps an invFreq array alive as ``_inv``."""
    r = vtmu_rope_params_init()
    r.head_dim = int(headDim)
    r.rotary_dim = 0 if rotaryDim is None else int(rotaryDim)
    r.interleaved = 1 if interleaved else 0
    r.base = 0.0 if base is None else float(base)
    if scaling is not None:
        kind = scaling.get("rope_type", scaling.get("type"))
        r.scaling = VTMU_ROPE_SCALING_LINEAR if kind == "linear" else 100
        r.scaling_factor = float(scaling.get("factor", 0.0))
    r.attention_factor = 0.0 if attentionFactor is None else float(attentionFactor)
    if invFreq is not None:
        arr = (ctypes.c_float * len(invFreq))(*[float(f) for f in invFreq])
        r.inv_freq = ctypes.cast(arr, ctypes.POINTER(ctypes.c_float))
        r._inv = arr
    return r


_HERE = contextlib.nullcontext()
WORKSPACE_HEADER_BYTES = 64 << 10  # the decode kernels' arrival counters, zero between calls


def _on(device):
    """The device as the current one; nothing to do where it is (the usual case)."""
    import torch
    return _HERE if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw_stream(device) -> int:
    """The device's current stream as the library takes it."""
    import torch
    return torch._C._cuda_getCurrentRawStream(device.index)


def _at(device, stream: int):
    """The stream as torch's current one."""
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if stream
                             else torch.cuda.default_stream(device))


class Workspace:
    """A zero-initialised device scratch buffer (torch-allocated) that grows
    on demand.  One per concurrent stream, and one for each captured graph
    whose replays may overlap other calls.  Inside a capture it does not grow:
    a call that needs more gets a buffer of the graph's own.  A buffer that a
    graph was captured with stays allocated as long as the Workspace."""

    def __init__(self, device=None):
        import torch
        self.device = torch.device("cuda") if device is None else torch.device(device)
        self.buf = None
        self._captured = False  # a graph holds buf's address
        self._kept = []

    def get(self, nbytes: int):
        import torch
        if nbytes == 0:
            return None, 0
        capturing = torch.cuda.is_current_stream_capturing()
        if self.buf is None or self.buf.numel() < nbytes:
            if capturing:
                return _graph_scratch(self.device, nbytes)
            if self._captured:
                self._kept.append(self.buf)
            self.buf, self._captured = torch.zeros(nbytes, dtype=torch.uint8, device=self.device), False
        self._captured = self._captured or capturing
        return self.buf, self.buf.numel()


def _graph_scratch(device, nbytes: int, counters: bool = True):
    """A buffer out of the memory of the graph that is being captured, its counters cleared
    by the graph.  Given back at the end of the call, it serves later calls on the stream."""
    import torch
    buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if counters:
        buf[:WORKSPACE_HEADER_BYTES].zero_()
    return buf, nbytes


_ws = threading.local()  # per host thread: two threads' launches on one stream may alternate


def _default_scratch(device, stream: int, nbytes: int, counters: bool):
    """The scratch of a call without a workspace: the buffer that this thread has for the
    stream; in a capture one of the graph's, so that no graph shares it with other calls."""
    import torch
    if nbytes == 0:
        return None, 0
    if torch.cuda.current_device() != device.index or stream != _raw_stream(device):
        with _on(device), _at(device, stream):
            return _default_scratch(device, stream, nbytes, counters)
    if torch.cuda.is_current_stream_capturing():
        return _graph_scratch(device, nbytes, counters)
    spaces = _ws.__dict__
    key = (device.index, stream)
    if key not in spaces:
        spaces[key] = Workspace(device)
    return spaces[key].get(nbytes)


def _scratch(workspace, device, stream: int, nbytes: int, counters: bool = True):
    """(buffer, its bytes) of a call: the caller's workspace, or the default one
    (`counters`: with the decode kernels' arrival counters, cleared)."""
    return workspace.get(nbytes) if workspace is not None else _default_scratch(device, stream, nbytes, counters)


def attention(q, k, v, bias=None, *, heads, headDim, out=None, workspace=None, stream=None, **params):
    """op "attention" on CUDA tensors: q [T, heads*headDim], k [S, kvHeads*headDim],
    v [S, kvHeads*vHeadDim], optional bias [T, S] or [heads, T, S]; returns
    out [T, heads*vHeadDim] (float32).  Keyword names as in the op catalog."""
    import torch
    T, S = q.shape[0], k.shape[0]
    vhd = params.get("vHeadDim") or headDim
    bias_kind = VTMU_BIAS_NONE
    if bias is not None:
        bias_kind = VTMU_BIAS_TS if bias.dim() == 2 else VTMU_BIAS_HTS
    p = make_params(T, S, heads=heads, headDim=headDim, bias_kind=bias_kind, **params)
    for name, t in (("q", q), ("k", k), ("v", v), ("bias", bias)):
        if t is not None and (not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    if out is None:
        out = torch.empty((T, heads * vhd), dtype=torch.float32, device=q.device)
    nbytes = vtmu_attention_workspace_size(p)
    st = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    buf, cap = _scratch(workspace, q.device, st, nbytes)
    vtmu_attention(q, k, v, bias, out, p, buf, cap, st)
    return out


def decode_step(k_cache, v_cache, k_new, v_new, offset: int, q, bias=None, *, heads, headDim, out=None,
                workspace=None, stream=None, **params):
    """A decode step on CUDA tensors: cache_write of k_new / v_new into the
    caches at row ``offset``, then attention of q over the updated caches
    (all of their rows, posOffset defaulting to the last new row).  One launch
    when the decode kernel covers the shape.  Returns out."""
    import torch
    T, S = q.shape[0], k_cache.shape[0]
    vhd = params.get("vHeadDim") or headDim
    params.setdefault("posOffset", offset + k_new.shape[0] - T)
    bias_kind = VTMU_BIAS_NONE
    if bias is not None:
        bias_kind = VTMU_BIAS_TS if bias.dim() == 2 else VTMU_BIAS_HTS
    p = make_params(T, S, heads=heads, headDim=headDim, bias_kind=bias_kind, **params)
    if out is None:
        out = torch.empty((T, heads * vhd), dtype=torch.float32, device=q.device)
    nbytes = vtmu_attention_workspace_size(p)
    st = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    buf, cap = _scratch(workspace, q.device, st, nbytes)
    vtmu_decode_step(k_cache, v_cache, S, k_new, v_new, k_new.shape[0], offset, q, bias, out, p, buf, cap, st)
    return out


def rope(x, *, headDim, offset=0, out=None, stream=None, **params):
    """op "rope" on a CUDA tensor x [T, heads*headDim]; ``out=x`` turns it in
    place.  Params as make_rope_params.  Returns out."""
    import torch
    T, width = x.shape
    if out is None:
        out = torch.empty_like(x)
    r = make_rope_params(headDim=headDim, **params)
    st = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
    vtmu_rope(x, out, T, width // headDim, offset, r, st)
    return out


def decode_step_rope(k_cache, v_cache, k_new, v_new, offset: int, q, bias=None, *, heads, headDim, rope: dict,
                     out=None, workspace=None, stream=None, **params):
    """decode_step with the rotary embedding ``rope`` (make_rope_params
    names, headDim taken from the call) fused in: q and the new keys are
    turned inside the one decode launch, the caches receive turned keys."""
    import torch
    T, S = q.shape[0], k_cache.shape[0]
    vhd = params.get("vHeadDim") or headDim
    params.setdefault("posOffset", offset + k_new.shape[0] - T)
    bias_kind = VTMU_BIAS_NONE
    if bias is not None:
        bias_kind = VTMU_BIAS_TS if bias.dim() == 2 else VTMU_BIAS_HTS
    p = make_params(T, S, heads=heads, headDim=headDim, bias_kind=bias_kind, **params)
    r = make_rope_params(headDim=headDim, **rope)
    if out is None:
        out = torch.empty((T, heads * vhd), dtype=torch.float32, device=q.device)
    nbytes = vtmu_attention_workspace_size(p)
    st = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    buf, cap = _scratch(workspace, q.device, st, nbytes)
    vtmu_decode_step_rope(k_cache, v_cache, S, k_new, v_new, k_new.shape[0], offset, q, bias, out, p, r, buf, cap,
                          st)
    return out


def cache_write(cache, values, offset: int, stream=None):
    """op "cache_write" on CUDA tensors: cache [maxRows, width] is updated in
    place with values [rows, width] at row ``offset``; returns cache."""
    import torch
    for name, t in (("cache", cache), ("values", values)):
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 2:
            raise ValueError(f"{name} must be a contiguous 2-D float32 CUDA tensor")
    if values.shape[1] != cache.shape[1]:
        raise ValueError("values must be as wide as the cache")
    st = stream if stream is not None else torch.cuda.current_stream(cache.device).cuda_stream
    vtmu_cache_write(cache, cache.shape[0], cache.shape[1], values, values.shape[0], offset, st)
    return cache


def make_mla_params(T, S, *, heads, kv_rank=512, qk_nope, qk_rope=64, v_head_dim, scale=None, causal=True,
                    posOffset=0, window=None, sinks=None, kernel=0):
    """An mla params struct from the IR page's parameter names (mla_attention)."""
    p = vtmu_mla_params_init()
    p.T, p.S = int(T), int(S)
    p.heads, p.kv_rank, p.qk_nope, p.qk_rope, p.v_head_dim = (int(heads), int(kv_rank), int(qk_nope), int(qk_rope),
                                                              int(v_head_dim))
    p.causal = 1 if causal else 0
    if scale is not None:
        p.has_scale, p.scale = 1, float(scale)
    p.pos_offset = int(posOffset)
    p.window = 0 if window is None else int(window)
    p.sinks = 0 if sinks is None else int(sinks)
    p.kernel = int(kernel)
    return p


def mla_attention(q, state, k_b, v_b, *, heads, qk_nope, v_head_dim, out=None, workspace=None, stream=None,
                  S=None, **params):
    """mla_attention on CUDA tensors: q [T, heads*(qk_nope+qk_rope)], state
    [rows, kv_rank+qk_rope] (its first S rows are read; all by default),
    k_b [heads*qk_nope, kv_rank], v_b [heads*v_head_dim, kv_rank]; returns
    out [T, heads*v_head_dim] (float32)."""
    import torch
    T = q.shape[0]
    p = make_mla_params(T, state.shape[0] if S is None else S, heads=heads, qk_nope=qk_nope,
                        v_head_dim=v_head_dim, **params)
    for name, t in (("q", q), ("state", state), ("k_b", k_b), ("v_b", v_b)):
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor")
    if out is None:
        out = torch.empty((T, heads * v_head_dim), dtype=torch.float32, device=q.device)
    nbytes = vtmu_mla_workspace_size(p)
    st = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    buf, cap = _scratch(workspace, q.device, st, nbytes, counters=False)
    vtmu_mla_attention(q, state, k_b, v_b, out, p, buf, cap, st)
    return out


def mla_decode_step(state, state_new, offset: int, q, k_b, v_b, *, heads, qk_nope, v_head_dim, out=None,
                    workspace=None, stream=None, **params):
    """A latent-attention decode step on CUDA tensors: cache_write of
    state_new into state at row ``offset``, then mla_attention over the
    first offset + new rows of the cache (posOffset defaulting to the last
    new row).  Returns out."""
    import torch
    T, R = q.shape[0], state_new.shape[0]
    params.setdefault("posOffset", offset + R - T)
    p = make_mla_params(T, offset + R, heads=heads, qk_nope=qk_nope, v_head_dim=v_head_dim, **params)
    if out is None:
        out = torch.empty((T, heads * v_head_dim), dtype=torch.float32, device=q.device)
    nbytes = vtmu_mla_workspace_size(p)
    st = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    buf, cap = _scratch(workspace, q.device, st, nbytes, counters=False)
    vtmu_mla_decode_step(state, state.shape[0], state_new, R, offset, q, k_b, v_b, out, p, buf, cap, st)
    return out


# ------------------------------------------------------------- paged caches
def _need(name, t, dtype, device=None):
    """A contiguous CUDA tensor of the type, on the call's device."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or (device is not None and t.device != device):
        where = "" if device is None else f" on {device}"
        raise ValueError(f"{name} must be a contiguous {str(dtype).removeprefix('torch.')} CUDA tensor{where}")


def page_map(lens, cu_rows, block_table, free_pages, n_free, *, rows: int, pageSize: int, accept=None, stream=None):
    """Block tables, slot maps and positions of a step's new rows on CUDA
    tensors (vtmu_page_map): lens [requests] and cu_rows [requests + 1] int32,
    block_table [requests, maxPages] int32 (completed in place), the stack
    free_pages [n] with n_free [1] pages on it, accept [requests] int64 bit
    masks of the rows to add (None: all).  Returns (slots [rows],
    positions [rows], new_lens [requests], n_free [1]), all int32.  A negative
    n_free says that as many pages were missing: call again with the same
    lens and n_free once pages are back on the stack."""
    import torch
    dev, n = lens.device, lens.shape[0]
    i32 = torch.int32
    for name, t in (("lens", lens), ("cu_rows", cu_rows), ("block_table", block_table), ("free_pages", free_pages),
                    ("n_free", n_free)):
        _need(name, t, i32, dev)
    if accept is not None:
        _need("accept", accept, torch.int64, dev)
    if (cu_rows.shape != (n + 1,) or block_table.dim() != 2 or block_table.shape[0] != n or n_free.numel() != 1 or
            (accept is not None and accept.shape != (n,)) or pageSize >= 1 << 31):
        raise ValueError("page_map: pageSize below 2^31, cu_rows [requests + 1], block_table [requests, maxPages], "
                         "n_free [1], accept [requests]")
    slots, positions, new_lens, left = torch.empty(2 * rows + n + 1, dtype=i32, device=dev).split([rows, rows, n, 1])
    with _on(dev):
        st = _raw_stream(dev) if stream is None else stream
        vtmu_page_map(lens, cu_rows, accept, block_table, free_pages, free_pages.numel(), n_free, slots, positions,
                      new_lens, left, n, rows, pageSize, block_table.shape[1], st)
    return slots, positions, new_lens, left


def tree_plan(parents, cu_rows, lens, *, stream=None):
    """Ancestor masks and positions of drafted trees on CUDA tensors
    (vtmu_tree_plan): parents [rows], cu_rows [requests + 1] and lens
    [requests] int32.  Returns (masks [rows] int64, positions [rows] int32)."""
    import torch
    dev = parents.device
    for name, t in (("parents", parents), ("cu_rows", cu_rows), ("lens", lens)):
        _need(name, t, torch.int32, dev)
    if cu_rows.shape != (lens.shape[0] + 1,):
        raise ValueError("tree_plan: cu_rows [requests + 1], lens [requests]")
    masks = torch.empty(parents.shape[0], dtype=torch.int64, device=dev)
    positions = torch.empty(parents.shape[0], dtype=torch.int32, device=dev)
    with _on(dev):
        st = _raw_stream(dev) if stream is None else stream
        vtmu_tree_plan(parents, cu_rows, lens, masks, positions, lens.shape[0], parents.shape[0], st)
    return masks, positions


def rope_at(x, positions, *, headDim, out=None, stream=None, **params):
    """op "rope" on a CUDA tensor x [T, heads*headDim] whose row t sits at
    positions[t] (int32; a row at a negative position is left as it was in
    out, so without ``out`` it is unset); ``out=x`` turns it in place.  Params as make_rope_params."""
    import torch
    dev = x.device
    _need("x", x, torch.float32)
    _need("positions", positions, torch.int32, dev)
    if out is None:
        out = torch.empty_like(x)
    _need("out", out, torch.float32, dev)
    if headDim < 1 or x.dim() != 2 or x.shape[1] % headDim or positions.shape != (x.shape[0],) or out.shape != x.shape:
        raise ValueError("rope_at: x and out [T, heads*headDim], positions [T]")
    r = make_rope_params(headDim=headDim, **params)
    with _on(dev):
        st = _raw_stream(dev) if stream is None else stream
        vtmu_rope_at(x, out, x.shape[0], x.shape[1] // headDim, positions, r, st)
    return out


def paged_write(k_pool, v_pool, k_new, v_new, slots, *, stream=None):
    """op "cache_write" through a slot map on CUDA tensors: rows of k_new and
    v_new into the pools at the rows that slots (int32) names; rows whose slot
    is outside the pool are skipped.  Returns (k_pool, v_pool)."""
    import torch
    dev = k_pool.device
    for name, t in (("k_pool", k_pool), ("v_pool", v_pool), ("k_new", k_new), ("v_new", v_new)):
        _need(name, t, torch.float32, dev)
    _need("slots", slots, torch.int32, dev)
    n = slots.shape[0]
    if (k_pool.dim() != 2 or v_pool.dim() != 2 or k_pool.shape[0] != v_pool.shape[0] or
            k_new.shape != (n, k_pool.shape[1]) or v_new.shape != (n, v_pool.shape[1])):
        raise ValueError("paged_write: pools [poolRows, width], k_new and v_new [rows, width], slots [rows]")
    with _on(dev):
        st = _raw_stream(dev) if stream is None else stream
        vtmu_paged_write(k_pool, v_pool, k_pool.shape[0], k_pool.shape[1], v_pool.shape[1], k_new, v_new, slots, n, st)
    return k_pool, v_pool


def paged_attention(q, k_pool, v_pool, block_table, lens, cu_rows, *, heads, headDim, pageSize, maxRows, kvHeads=None,
                    tree=None, scale=None, softcap=None, window=None, sinks=None, kernel=VTMU_PAGED_AUTO, out=None,
                    workspace=None, stream=None):
    """op "attention" of a ragged batch over a paged cache on CUDA tensors
    (vtmu_paged_attention): q [rows, heads*headDim], pools [pages*pageSize,
    kvHeads*headDim], block_table [requests, maxPages], lens [requests] and
    cu_rows [requests + 1] int32; maxRows bounds the rows of one request.
    ``tree=(k_new, v_new, masks, positions)`` attends to drafted rows beside
    the cache (positions may be None without a window); with a window the
    cache's first ``sinks`` rows stay visible, drafted ones do not.  Returns
    out [rows, heads*headDim]; rows of no request are not written."""
    import torch
    dev = q.device
    f32, i32 = torch.float32, torch.int32
    for name, t in (("q", q), ("k_pool", k_pool), ("v_pool", v_pool)):
        _need(name, t, f32, dev)
    for name, t in (("block_table", block_table), ("lens", lens), ("cu_rows", cu_rows)):
        _need(name, t, i32, dev)
    hk = heads if kvHeads is None else kvHeads
    rows, n = q.shape[0], lens.shape[0]
    if (not 0 < pageSize < 1 << 31 or q.shape != (rows, heads * headDim) or k_pool.dim() != 2 or
            k_pool.shape[1] != hk * headDim or k_pool.shape != v_pool.shape or k_pool.shape[0] % pageSize or
            block_table.dim() != 2 or block_table.shape[0] != n or cu_rows.shape != (n + 1,)):
        raise ValueError("paged_attention: pageSize in 1 .. 2^31 - 1, q [rows, heads*headDim], pools [pages*pageSize, "
                         "kvHeads*headDim], block_table [requests, maxPages], lens [requests], cu_rows [requests + 1]")
    k_new = v_new = masks = positions = None
    if tree is not None:
        k_new, v_new, masks, positions = tree
        for name, t in (("k_new", k_new), ("v_new", v_new)):
            _need(name, t, f32, dev)
        _need("masks", masks, torch.int64, dev)
        if positions is not None:
            _need("positions", positions, i32, dev)
        if (k_new.shape != (rows, hk * headDim) or v_new.shape != k_new.shape or masks.shape != (rows,) or
                (positions is not None and positions.shape != (rows,))):
            raise ValueError("paged_attention: k_new and v_new [rows, kvHeads*headDim], masks and positions [rows]")
    if out is None:
        out = torch.empty_like(q)
    _need("out", out, f32, dev)
    if out.shape != q.shape:
        raise ValueError("paged_attention: out [rows, heads*headDim]")
    p = vtmu_paged_params(rows=rows, pages=k_pool.shape[0] // pageSize, requests=n,
                          max_rows=max(min(maxRows, rows), -1), page_size=pageSize,
                          max_pages=block_table.shape[1], heads=heads, kv_heads=hk, head_dim=headDim,
                          tree=0 if tree is None else 1, has_scale=0 if scale is None else 1,
                          scale=0.0 if scale is None else scale, softcap=softcap or 0.0, kernel=kernel,
                          window=window or 0, sinks=sinks or 0)
    with _on(dev):
        nbytes = vtmu_paged_workspace_size(p)
        st = _raw_stream(dev) if stream is None else stream
        buf, cap = _scratch(workspace, dev, st, nbytes, counters=False)
        vtmu_paged_attention(q, k_pool, v_pool, block_table, lens, cu_rows, k_new, v_new, masks, positions, out, p,
                             buf, cap, st)
    return out
