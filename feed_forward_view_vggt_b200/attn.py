"""ctypes binding of ``libvggt_attn.so`` -- argument marshalling only.

Every function named ``vggt_*`` mirrors the C entry point of the same name in
``include/vggt_attn.h`` and returns its status code (an int; 0 = VGGT_OK).
Tensor arguments may be CUDA ``torch`` tensors (their ``data_ptr()`` is
passed) or raw integer device addresses; ``stream`` may be a
``torch.cuda.Stream``, a raw ``cudaStream_t`` integer, or None for torch's
current stream.  The library is loaded on first use; if it has not been
built this raises -- there is no CPU fallback.

Tensors given to a call on another stream than torch's current one must live
until that stream is past the call (or be recorded on it).

The helpers at the bottom (``frame``, ``global_``, ``sga``, ``cached``, ...) allocate the
outputs with torch, call the entry points and raise ``VggtError`` on a
non-zero status.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libvggt_attn.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "libvggt_attn_debug.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "vggt_attn.h")

# The ABI this binding marshals for (VGGT_ABI_VERSION of include/vggt_attn.h);
# a library reporting another version is refused at load.
ABI_VERSION = 3

VGGT_OK = 0
VGGT_ERR_INVALID_ARG = 1
VGGT_ERR_UNSUPPORTED = 2
VGGT_ERR_WORKSPACE = 3
VGGT_ERR_CUDA = 4
VGGT_ERR_TIMEOUT = 5
VGGT_ERR_BOUNDS = 6


class VggtError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = int(status)
        super().__init__(f"{what}: {vggt_status_string(status)} ({status})" if what else
                         f"{vggt_status_string(status)} ({status})")


class vggt_shape(ctypes.Structure):
    _fields_ = [("n_frames", ctypes.c_int32), ("n_special", ctypes.c_int32),
                ("patch_h", ctypes.c_int32), ("patch_w", ctypes.c_int32),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class vggt_layer(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("s_h", ctypes.c_int32), ("s_w", ctypes.c_int32)]


class vggt_cache(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class vggt_norm(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_cols", ctypes.c_int32), ("kind", ctypes.c_int32),
                ("x_fp32", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("rows_per_gate", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("h_stride", ctypes.c_int64)]


VGGT_NORM_LAYER, VGGT_NORM_RMS = 0, 1
_NORM_KINDS = {"layer": VGGT_NORM_LAYER, "rms": VGGT_NORM_RMS}

VGGT_LAYER_FRAME, VGGT_LAYER_GLOBAL, VGGT_LAYER_SGA, VGGT_LAYER_REGISTER = 0, 1, 2, 3
_LAYER_KINDS = {"frame": VGGT_LAYER_FRAME, "global": VGGT_LAYER_GLOBAL, "sga": VGGT_LAYER_SGA,
                "register": VGGT_LAYER_REGISTER}

_lib = None


def load():
    """Loads the in-tree library (raises if it is missing).  With the
    environment variable VGGT_DEBUG=1 the library with device index checks
    (libvggt_attn_debug.so) is loaded instead."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = load_library(DEBUG_LIB_PATH if os.environ.get("VGGT_DEBUG") == "1" else LIB_PATH)
    return _lib


def load_library(path: str):
    """A separate ctypes handle on one build of the library, with every
    entry point's signature set (raises if it is missing)."""
    if not os.path.exists(path):
        flag = " --debug" if path == DEBUG_LIB_PATH else ""
        raise RuntimeError(f"{path} is not built; run `python -m feed_forward_view_vggt_b200.build{flag}`")
    lib = ctypes.CDLL(path)
    i32, i64, sz, vp, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_float
    S, CA = vggt_shape, vggt_cache
    sigs = {
        "vggt_status_string": ([i32], ctypes.c_char_p),
        "vggt_abi_version": ([], i32),
        "vggt_num_tokens": ([S], i64),
        "vggt_sga_num_kept": ([S, i32, i32], i64),
        "vggt_sga_num_dropped": ([S, i32, i32], i64),
        "vggt_sga_workspace_bytes": ([S, i32, i32], sz),
        "vggt_sga_build_index": ([S, i32, i32, vp, vp, vp], i32),
        "vggt_attn_frame": ([vp, vp, vp, vp, vp, S, f32, vp], i32),
        "vggt_attn_global": ([vp, vp, vp, vp, vp, S, f32, vp], i32),
        "vggt_attn_sga": ([vp, vp, vp, vp, vp, S, i32, i32, vp, vp, vp, sz, f32, vp], i32),
        "vggt_attn_sga_noalloc": ([vp, vp, vp, vp, vp, S, i32, i32, vp, vp, f32, vp], i32),
        "vggt_attn_global_rows": ([vp, i32, vp, vp, vp, vp, S, f32, vp], i32),
        "vggt_attn_sga_rows": ([vp, i32, i32, vp, vp, vp, vp, S, i32, i32, vp, vp, vp, sz, f32, vp], i32),
        "vggt_attn_register": ([vp, vp, vp, vp, vp, S, f32, vp], i32),
        "vggt_sga_partial_workspace_bytes": ([S], sz),
        "vggt_sga_gather_partial": ([vp, vp, S, i32, i32, vp, vp, vp, vp, sz, vp], i32),
        "vggt_attn_sga_gathered": ([vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, S, i32, i32, f32, vp], i32),
        "vggt_test_attn_global_stall": ([vp, vp, vp, vp, S, f32, ctypes.c_uint64, vp], i32),
        "vggt_check": ([vp, vp], i32),
        "vggt_schedule_workspace_bytes": ([S, vp, i32], i64),
        "vggt_qkv_rope": ([vp, vp, vp, vp, vp, vp, S, f32, vp], i32),
        "vggt_out_proj": ([vp, vp, vp, vp, S, vp], i32),
        "vggt_attn_schedule": ([vp, vp, vp, vp, S, vp, i32, f32, vp, sz, vp], i32),
        "vggt_debug_checks": ([], i32),
        "vggt_cache_plan": ([CA, vp, vp, vp, i32, vp, vp, i32, vp, vp, vp, vp, vp], i32),
        "vggt_cache_append": ([CA, vp, vp, i64, i64, vp, i32, vp, vp, vp], i32),
        "vggt_attn_cached_workspace_bytes": ([CA, i32], sz),
        "vggt_attn_cached": ([CA, vp, i64, i64, vp, vp, vp, vp, vp, i32, i32, vp, vp, vp, sz, f32, vp], i32),
        "vggt_norm_residual": ([vggt_norm, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
    }
    for name, (args, res) in sigs.items():
        # entry points were added without a new version: an older library may report the same one
        fn = getattr(lib, name, None)
        if fn is None:
            raise RuntimeError(f"{path} has no {name}; rebuild it")
        fn.argtypes = args
        fn.restype = res
    if lib.vggt_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{path} has ABI version {lib.vggt_abi_version()}, the binding expects {ABI_VERSION}; "
                           "rebuild it")
    return lib


def declared_symbols(header: str = HEADER_PATH):
    """Names of the functions declared in the public header."""
    text = open(header).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(vggt_[a-z0-9_]+)\s*\(", text)))


# ------------------------------------------------------------- marshalling

def _shape(shape) -> vggt_shape:
    if isinstance(shape, vggt_shape):
        return shape
    if isinstance(shape, (tuple, list)):
        return vggt_shape(*[int(x) for x in shape])
    # objects with N, n_special, h, w, H, d (synth.Workload, oracle.Shape)
    return vggt_shape(int(shape.N), int(shape.n_special), int(shape.h), int(shape.w), int(shape.H),
                      int(shape.d))


def _ptr(x, dtype=None, name="argument"):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    import torch

    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name}: expected a CUDA tensor or an integer device address")
    if not x.is_cuda:
        raise ValueError(f"{name}: tensor must live on a CUDA device")
    if not x.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    if dtype is not None and x.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {x.dtype}")
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _bf16():
    import torch

    return torch.bfloat16


def _i32():
    import torch

    return torch.int32


def _f32():
    import torch

    return torch.float32


def _layers(layers):
    """ctypes array of vggt_layer from descriptors: a vggt_layer, a kind name
    ("frame", "global", "register"), or a tuple (kind[, s_h, s_w])."""
    out = (vggt_layer * max(len(layers), 1))()
    for i, ly in enumerate(layers):
        if isinstance(ly, vggt_layer):
            out[i] = ly
            continue
        if isinstance(ly, str):
            ly = (ly,)
        kind = _LAYER_KINDS[ly[0]] if isinstance(ly[0], str) else int(ly[0])
        s_h, s_w = (int(ly[1]), int(ly[2])) if len(ly) >= 3 else (0, 0)
        out[i] = vggt_layer(kind, s_h, s_w)
    return out


def _ptr_array(xs, dtype, name):
    return (ctypes.c_void_p * max(len(xs), 1))(*[_ptr(x, dtype, name) for x in xs])


# ------------------------------------------------- entry points, same names

def vggt_status_string(status: int) -> str:
    return load().vggt_status_string(int(status)).decode()


def vggt_abi_version() -> int:
    return int(load().vggt_abi_version())


def vggt_num_tokens(shape) -> int:
    return int(load().vggt_num_tokens(_shape(shape)))


def vggt_sga_num_kept(shape, s_h: int, s_w: int) -> int:
    return int(load().vggt_sga_num_kept(_shape(shape), s_h, s_w))


def vggt_sga_num_dropped(shape, s_h: int, s_w: int) -> int:
    return int(load().vggt_sga_num_dropped(_shape(shape), s_h, s_w))


def vggt_sga_workspace_bytes(shape, s_h: int, s_w: int) -> int:
    return int(load().vggt_sga_workspace_bytes(_shape(shape), s_h, s_w))


def vggt_sga_build_index(shape, s_h, s_w, kept_idx, mult, stream=None) -> int:
    return int(load().vggt_sga_build_index(_shape(shape), s_h, s_w, _ptr(kept_idx, _i32(), "kept_idx"),
                                           _ptr(mult, _i32(), "mult"), _stream(stream)))


def vggt_attn_frame(q, k, v, o, lse, shape, scale, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_frame(_ptr(q, b, "q"), _ptr(k, b, "k"), _ptr(v, b, "v"), _ptr(o, b, "o"),
                                      _ptr(lse, _f32(), "lse"), _shape(shape), float(scale), _stream(stream)))


def vggt_attn_global(q, k, v, o, lse, shape, scale, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_global(_ptr(q, b, "q"), _ptr(k, b, "k"), _ptr(v, b, "v"), _ptr(o, b, "o"),
                                       _ptr(lse, _f32(), "lse"), _shape(shape), float(scale), _stream(stream)))


def vggt_attn_sga(q, k, v, o, lse, shape, s_h, s_w, kept_idx, mult, workspace, workspace_bytes, scale,
                  stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_sga(_ptr(q, b, "q"), _ptr(k, b, "k"), _ptr(v, b, "v"), _ptr(o, b, "o"),
                                    _ptr(lse, _f32(), "lse"), _shape(shape), int(s_h), int(s_w),
                                    _ptr(kept_idx, _i32(), "kept_idx"), _ptr(mult, _i32(), "mult"),
                                    _ptr(workspace, None, "workspace"), int(workspace_bytes), float(scale),
                                    _stream(stream)))


def vggt_attn_sga_noalloc(q, k, v, o, lse, shape, s_h, s_w, kept_idx, mult, scale, stream=None) -> int:
    """SGA for callers that cannot allocate: the library's built-in 16 MiB
    device scratch array stands in for the workspace (see the header)."""
    b = _bf16()
    return int(load().vggt_attn_sga_noalloc(_ptr(q, b, "q"), _ptr(k, b, "k"), _ptr(v, b, "v"),
                                            _ptr(o, b, "o"), _ptr(lse, _f32(), "lse"), _shape(shape),
                                            int(s_h), int(s_w), _ptr(kept_idx, _i32(), "kept_idx"),
                                            _ptr(mult, _i32(), "mult"), float(scale), _stream(stream)))


def vggt_attn_global_rows(q_rows, n_rows, k, v, o_rows, lse_rows, shape, scale, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_global_rows(_ptr(q_rows, b, "q_rows"), int(n_rows), _ptr(k, b, "k"), _ptr(v, b, "v"),
                                            _ptr(o_rows, b, "o_rows"), _ptr(lse_rows, _f32(), "lse_rows"),
                                            _shape(shape), float(scale), _stream(stream)))


def vggt_attn_sga_rows(q_rows, row0, n_rows, k, v, o_rows, lse_rows, shape, s_h, s_w, kept_idx, mult, workspace,
                       workspace_bytes, scale, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_sga_rows(_ptr(q_rows, b, "q_rows"), int(row0), int(n_rows), _ptr(k, b, "k"),
                                         _ptr(v, b, "v"), _ptr(o_rows, b, "o_rows"), _ptr(lse_rows, _f32(), "lse_rows"),
                                         _shape(shape), int(s_h), int(s_w), _ptr(kept_idx, _i32(), "kept_idx"),
                                         _ptr(mult, _i32(), "mult"), _ptr(workspace, None, "workspace"),
                                         int(workspace_bytes), float(scale), _stream(stream)))


def vggt_sga_partial_workspace_bytes(local_shape) -> int:
    return int(load().vggt_sga_partial_workspace_bytes(_shape(local_shape)))


def vggt_sga_gather_partial(k, v, local_shape, s_h, s_w, kept_k, kept_v, dropped_sums, workspace, workspace_bytes,
                            stream=None) -> int:
    b = _bf16()
    return int(load().vggt_sga_gather_partial(_ptr(k, b, "k"), _ptr(v, b, "v"), _shape(local_shape), int(s_h),
                                              int(s_w), _ptr(kept_k, b, "kept_k"), _ptr(kept_v, b, "kept_v"),
                                              _ptr(dropped_sums, _f32(), "dropped_sums"),
                                              _ptr(workspace, None, "workspace"), int(workspace_bytes),
                                              _stream(stream)))


def vggt_attn_sga_gathered(q_rows, row0, n_rows, k_rows, v_rows, kept_k, kept_v, dropped_sums, mult, means, o_rows,
                           lse_rows, shape, s_h, s_w, scale, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_sga_gathered(_ptr(q_rows, b, "q_rows"), int(row0), int(n_rows),
                                             _ptr(k_rows, b, "k_rows"), _ptr(v_rows, b, "v_rows"),
                                             _ptr(kept_k, b, "kept_k"), _ptr(kept_v, b, "kept_v"),
                                             _ptr(dropped_sums, _f32(), "dropped_sums"), _ptr(mult, _i32(), "mult"),
                                             _ptr(means, _f32(), "means"), _ptr(o_rows, b, "o_rows"),
                                             _ptr(lse_rows, _f32(), "lse_rows"), _shape(shape), int(s_h), int(s_w),
                                             float(scale), _stream(stream)))


def vggt_test_attn_global_stall(q, k, v, o, shape, scale, wait_limit_ns, stream=None) -> int:
    """Failure-path test hook: global attention whose first scores are never
    signalled, with in-kernel waits bounded by wait_limit_ns (see header)."""
    b = _bf16()
    return int(load().vggt_test_attn_global_stall(_ptr(q, b, "q"), _ptr(k, b, "k"), _ptr(v, b, "v"),
                                                  _ptr(o, b, "o"), _shape(shape), float(scale),
                                                  int(wait_limit_ns), _stream(stream)))


def vggt_attn_register(q, k, v, o, lse, shape, scale, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_attn_register(_ptr(q, b, "q"), _ptr(k, b, "k"), _ptr(v, b, "v"), _ptr(o, b, "o"),
                                         _ptr(lse, _f32(), "lse"), _shape(shape), float(scale), _stream(stream)))


def vggt_schedule_workspace_bytes(shape, layers) -> int:
    return int(load().vggt_schedule_workspace_bytes(_shape(shape), _layers(layers), len(layers)))


def vggt_attn_schedule(qs, ks, vs, os_, shape, layers, scale, workspace, workspace_bytes, stream=None) -> int:
    b = _bf16()
    n = len(layers)
    return int(load().vggt_attn_schedule(_ptr_array(qs, b, "q"), _ptr_array(ks, b, "k"), _ptr_array(vs, b, "v"),
                                         _ptr_array(os_, b, "o"), _shape(shape), _layers(layers), n, scale,
                                         _ptr(workspace, None, "workspace"), workspace_bytes, _stream(stream)))


def vggt_qkv_rope(x, w, bias, q, k, v, shape, rope_base, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_qkv_rope(_ptr(x, b, "x"), _ptr(w, b, "w"), _ptr(bias, _f32(), "bias"), _ptr(q, b, "q"),
                                    _ptr(k, b, "k"), _ptr(v, b, "v"), _shape(shape), rope_base, _stream(stream)))


def vggt_out_proj(o, w, bias, y, shape, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_out_proj(_ptr(o, b, "o"), _ptr(w, b, "w"), _ptr(bias, _f32(), "bias"), _ptr(y, b, "y"),
                                    _shape(shape), _stream(stream)))


def _rows_ptr(x, dtype, name):
    """As _ptr for a tensor whose rows may be strided (the last dimension is contiguous)."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError(f"{name}: tensor must live on a CUDA device")
    if x.stride(-1) != 1 and x.shape[-1] != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if x.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {x.dtype}")
    return x.data_ptr()


def vggt_cache_plan(cache, cached_lens, new_lens, free_pages, free_capacity, n_free, block_table, n_rows, cu_rows,
                    kv_lens, slots, counts, stream=None) -> int:
    i = _i32()
    return int(load().vggt_cache_plan(cache, _ptr(cached_lens, i, "cached_lens"), _ptr(new_lens, i, "new_lens"),
                                      _ptr(free_pages, i, "free_pages"), int(free_capacity),
                                      _ptr(n_free, i, "n_free"), _ptr(block_table, i, "block_table"), int(n_rows),
                                      _ptr(cu_rows, i, "cu_rows"), _ptr(kv_lens, i, "kv_lens"),
                                      _ptr(slots, i, "slots"), _ptr(counts, i, "counts"), _stream(stream)))


def vggt_cache_append(cache, k, v, row_stride, in_head_stride, slots, n_rows, k_pages, v_pages, stream=None) -> int:
    b = _bf16()
    return int(load().vggt_cache_append(cache, _rows_ptr(k, b, "k"), _rows_ptr(v, b, "v"), int(row_stride),
                                        int(in_head_stride), _ptr(slots, _i32(), "slots"), int(n_rows),
                                        _rows_ptr(k_pages, b, "k_pages"), _rows_ptr(v_pages, b, "v_pages"),
                                        _stream(stream)))


def vggt_attn_cached_workspace_bytes(cache, n_rows) -> int:
    return int(load().vggt_attn_cached_workspace_bytes(cache, int(n_rows)))


def vggt_attn_cached(cache, q, q_row_stride, q_head_stride, k_pages, v_pages, block_table, cu_rows, kv_lens, n_rows,
                     causal_unit, o, lse, workspace, workspace_bytes, scale, stream=None) -> int:
    b, i = _bf16(), _i32()
    return int(load().vggt_attn_cached(cache, _rows_ptr(q, b, "q"), int(q_row_stride), int(q_head_stride),
                                       _rows_ptr(k_pages, b, "k_pages"), _rows_ptr(v_pages, b, "v_pages"),
                                       _ptr(block_table, i, "block_table"), _ptr(cu_rows, i, "cu_rows"),
                                       _ptr(kv_lens, i, "kv_lens"), int(n_rows), int(causal_unit), _ptr(o, b, "o"),
                                       _ptr(lse, _f32(), "lse"), _ptr(workspace, None, "workspace"),
                                       int(workspace_bytes), float(scale), _stream(stream)))


def vggt_norm_residual(norm, x, y, post_w, post_b, scale, gate, w, b, x_out, h, stream=None) -> int:
    f, t = _f32(), _f32() if norm.x_fp32 else _bf16()
    return int(load().vggt_norm_residual(norm, _rows_ptr(x, t, "x"), _rows_ptr(y, _bf16(), "y"),
                                         _ptr(post_w, f, "post_w"), _ptr(post_b, f, "post_b"),
                                         _ptr(scale, f, "scale"), _ptr(gate, _bf16(), "gate"), _ptr(w, f, "w"),
                                         _ptr(b, f, "b"), _rows_ptr(x_out, t, "x_out"),
                                         _rows_ptr(h, _bf16(), "h"), _stream(stream)))


def vggt_check(stream=None):
    """(status, detail word); synchronises the stream."""
    detail = ctypes.c_uint32(0)
    st = int(load().vggt_check(_stream(stream), ctypes.byref(detail)))
    return st, int(detail.value)


# ----------------------------------------------------------- conveniences

def _raise(status: int, what: str):
    if status != VGGT_OK:
        raise VggtError(status, what)


def default_scale(head_dim: int = 64) -> float:
    return 1.0 / math.sqrt(head_dim)


def frame(q, k, v, shape, scale=None, want_lse=False, stream=None):
    import torch

    o = torch.empty_like(q)
    sh = _shape(shape)
    lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device) if want_lse else None
    _raise(vggt_attn_frame(q, k, v, o, lse, sh, default_scale(sh.head_dim) if scale is None else scale, stream), "vggt_attn_frame")
    return (o, lse) if want_lse else o


def global_(q, k, v, shape, scale=None, want_lse=False, stream=None):
    import torch

    o = torch.empty_like(q)
    sh = _shape(shape)
    lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device) if want_lse else None
    _raise(vggt_attn_global(q, k, v, o, lse, sh, default_scale(sh.head_dim) if scale is None else scale, stream),
           "vggt_attn_global")
    return (o, lse) if want_lse else o


class SgaIndex:
    """Device-side SGA index (kept list + multiplicities) for one shape and
    stride, built once by vggt_sga_build_index and reusable across heads and
    layers; also owns a workspace of vggt_sga_workspace_bytes."""

    def __init__(self, shape, s_h: int, s_w: int, device=None, stream=None):
        import torch

        self.shape = _shape(shape)
        self.s_h, self.s_w = int(s_h), int(s_w)
        self.n_kept = vggt_sga_num_kept(self.shape, s_h, s_w)
        self.n_dropped = vggt_sga_num_dropped(self.shape, s_h, s_w)
        if self.n_kept < 0:
            raise VggtError(VGGT_ERR_INVALID_ARG, "SgaIndex")
        S = vggt_num_tokens(self.shape)
        device = device or torch.device("cuda")
        self.kept_idx = torch.empty(max(self.n_kept, 1), dtype=torch.int32, device=device)
        self.mult = torch.empty(S, dtype=torch.int32, device=device)
        self.workspace_bytes = vggt_sga_workspace_bytes(self.shape, s_h, s_w)
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
        _raise(vggt_sga_build_index(self.shape, s_h, s_w, self.kept_idx, self.mult, stream),
               "vggt_sga_build_index")

    def means(self):
        """(kbar, vbar) fp32 [H, 64] as left in the workspace by the last call."""
        hd = self.shape.n_heads * 64
        f = self.workspace[: 8 * hd].view(_f32())
        return f[:hd].view(self.shape.n_heads, 64), f[hd:2 * hd].view(self.shape.n_heads, 64)


def sga(q, k, v, index: SgaIndex, scale=None, want_lse=False, stream=None):
    import torch

    o = torch.empty_like(q)
    lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device) if want_lse else None
    _raise(vggt_attn_sga(q, k, v, o, lse, index.shape, index.s_h, index.s_w, index.kept_idx, index.mult,
                         index.workspace, index.workspace_bytes,
                         default_scale(index.shape.head_dim) if scale is None else scale, stream), "vggt_attn_sga")
    return (o, lse) if want_lse else o


def register(q, k, v, shape, scale=None, want_lse=False, o=None, stream=None):
    """Register attention; returns O (patch-token rows are those of ``o`` if
    given, else uninitialised)."""
    import torch

    sh = _shape(shape)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device) if want_lse else None
    _raise(vggt_attn_register(q, k, v, o, lse, sh, default_scale(sh.head_dim) if scale is None else scale, stream),
           "vggt_attn_register")
    return (o, lse) if want_lse else o


def schedule(qs, ks, vs, shape, layers, os_=None, scale=None, stream=None):
    """Runs a layer schedule: layer i reads qs[i], ks[i], vs[i] and writes
    os_[i] (allocated if not given; register layers write only the
    special-token rows).  Returns the list of outputs."""
    import torch

    sh = _shape(shape)
    n = len(layers)
    if not (len(qs) == len(ks) == len(vs) == n):
        raise ValueError("one q, k and v per layer")
    os_ = [torch.empty_like(q) for q in qs] if os_ is None else os_
    nbytes = vggt_schedule_workspace_bytes(sh, layers)
    if nbytes < 0:
        raise VggtError(VGGT_ERR_INVALID_ARG, "vggt_schedule_workspace_bytes")
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=qs[0].device) if n else None
    _raise(vggt_attn_schedule(qs, ks, vs, os_, sh, layers, default_scale(sh.head_dim) if scale is None else scale,
                              ws, nbytes, stream), "vggt_attn_schedule")
    return os_


def qkv_rope(x, w, shape, bias=None, rope_base=100.0, stream=None):
    """Fused QKV projection + 2D RoPE; returns (q, k, v), each [S, H, 64]."""
    import torch

    sh = _shape(shape)
    S = x.shape[0]
    q, k, v = (torch.empty(S, sh.n_heads, sh.head_dim, dtype=x.dtype, device=x.device) for _ in range(3))
    _raise(vggt_qkv_rope(x, w, bias, q, k, v, sh, rope_base, stream), "vggt_qkv_rope")
    return q, k, v


def out_proj(o, w, shape, bias=None, stream=None):
    """Output projection y = o W^T + b; returns y, [S, C]."""
    import torch

    sh = _shape(shape)
    y = torch.empty(o.shape[0], sh.n_heads * sh.head_dim, dtype=o.dtype, device=o.device)
    _raise(vggt_out_proj(o, w, bias, y, sh, stream), "vggt_out_proj")
    return y


# ------------------------------------------------------- streaming (paged cache)
#
# A streaming step makes many small calls, so their cost on the host counts: the
# tensors are looked at, and what a call returns is allocated, in a compiled
# module (csrc/streaming_binding.cpp); `stream` is that of the other calls.

_host = None
_entries = {}


def _call(what, function, *args):
    """`function` of the compiled module on the entry point `what` of the loaded library."""
    global _host
    if _host is None:
        _torch()  # the module needs torch's libraries
        try:
            from . import _streaming
        except ImportError as e:
            raise RuntimeError(f"_streaming.so is not built, or not for this torch ({e}); run "
                               "`python -m feed_forward_view_vggt_b200.build`") from e
        _host = _streaming
    result = getattr(_host, function)(_entry(what), *args)
    status = result if isinstance(result, int) else result[0]
    if status != VGGT_OK:
        raise VggtError(status, what)
    return result


def _entry(name):
    """The address of an entry point of the loaded library."""
    lib = load()
    known = _entries.get(name)
    if known is None or known[0] is not lib:
        known = _entries[name] = (lib, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
    return known[1]


def _torch():
    import torch

    return torch


def _torch_stream(stream, device):
    """``stream``, as the calls take it, as one of torch's."""
    cuda = _torch().cuda
    return stream if isinstance(stream, cuda.Stream) else cuda.ExternalStream(_stream(stream), device=device)


def _expect(ok, what):
    if not ok:
        raise ValueError(what)


def cache_plan(cached_lens, new_lens, free_pages, n_free, block_table, page_size, n_rows, n_pages=None, stream=None):
    """Plans a step: writes the pages it takes into block_table and returns
    (cu_rows, kv_lens, slots, counts), all int32 on the device; counts is
    [free pages left, sequences refused] and counts[:1] the next step's n_free.
    n_rows: rows of the step's packed buffers (>= the new rows).  n_pages: pages
    of the cache (default: as many as 32-bit slots allow)."""
    if n_pages is None:
        n_pages = (2 ** 31 - 1) // page_size if page_size > 0 else 1
    return _call("vggt_cache_plan", "plan", cached_lens, new_lens, free_pages, n_free, block_table, page_size, n_rows,
                 n_pages, stream, None, None)[1:]


def cache_append(k, v, slots, k_pages, v_pages, stream=None):
    """Writes the rows of k and v ([n_rows, n_kv_heads, 64], rows and heads may
    be strided, alike in both) into their slots of k_pages and v_pages."""
    _call("vggt_cache_append", "append", k, v, slots, k_pages, v_pages, stream)


def cached(q, k_pages, v_pages, block_table, cu_rows, kv_lens, causal_unit=0, scale=None, want_lse=False,
           workspace=None, o=None, stream=None):
    """Attention of the new rows q ([n_rows, H, 64], rows and heads may be
    strided) over a paged cache; see vggt_attn_cached for the mask.  Rows
    behind cu_rows[-1] keep what ``o`` holds (uninitialised if not given)."""
    _, o, lse = _call("vggt_attn_cached", "attend", _entry("vggt_attn_cached_workspace_bytes"), q, k_pages, v_pages,
                      block_table, cu_rows, kv_lens, causal_unit,
                      default_scale(q.shape[-1]) if scale is None else scale, want_lse, workspace, o, stream)
    return (o, lse) if want_lse else o


def norm_residual(x, y=None, kind="layer", eps=1e-6, scale=None, gate=None, rows_per_gate=0, post_norm=False,
                  post_weight=None, post_bias=None, weight=None, bias=None, want_h=True, inplace=False, stream=None):
    """x' = x + scale * gate * N_post(y) and h = N_pre(x') in one pass over the
    rows of x and y ([n_rows, n_cols]); returns (x', h).  Without y x' is x;
    with want_h false h is None; with inplace x' overwrites x."""
    _expect(kind in _NORM_KINDS, "kind: 'layer' or 'rms'")
    return _call("vggt_norm_residual", "norm", x, y, _NORM_KINDS[kind], eps, scale, gate, rows_per_gate, post_norm,
                 post_weight, post_bias, weight, bias, want_h, inplace, stream)[1:]


class PagedCache:
    """The paged K/V cache of a streaming trunk: pages for ``n_layers`` layers
    that share one block table, the sequences' lengths and the free list, all
    on the device.  A step is ``plan(new_lens, n_rows)``, then per layer
    ``append(layer, k, v)`` and ``attend(layer, q)``, with the rows of the
    sequences packed one after another.

    Everything stays where it is: ``plan`` updates the lengths in place, and
    two plans with the same n_rows write the same ``cu_rows`` and ``slots``.  A
    step may therefore be captured into a graph, with its plan or only its
    layers; every replay goes on from the cache's present state."""

    def __init__(self, n_pages, page_size, n_kv_heads, n_seqs, max_pages, n_layers=1, head_dim=64, device=None):
        import torch

        _expect(min(n_pages, page_size, n_kv_heads, n_seqs, max_pages, n_layers) >= 1, "sizes must be >= 1")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = int(page_size)
        self.pages = [tuple(torch.zeros(n_pages, n_kv_heads, page_size, head_dim, dtype=torch.bfloat16, device=device)
                            for _ in range(2)) for _ in range(n_layers)]
        self.block_table = torch.full((n_seqs, max_pages), -1, **i32)
        # of the last step: free pages, sequences refused, and the sequences' lengths
        self._state = torch.zeros(2 + n_seqs, **i32)
        self._state[0] = n_pages
        self.n_free, self.kv_lens = self._state[:1], self._state[2:]
        # one entry more than the pages: where release() drops what it must not write
        self.free_pages = torch.arange(n_pages + 1, **i32)
        self._free = self.free_pages[:n_pages]
        self.cu_rows = self.slots = None
        self._steps = {}  # by rows, rounded up to a power of two: a step's row offsets and slots

    def plan(self, new_lens, n_rows, stream=None):
        """Plans a step of new_lens rows (int32 [n_seqs], on the device) in buffers of n_rows rows; returns the
        number of refused sequences (int32 [1], on the device).  A refused sequence keeps its length, its rows are
        not appended, and what attend() returns for them is to be discarded."""
        size = 1 << max(int(n_rows) - 1, 0).bit_length()
        step, device = self._steps.get(size), self._state.device
        if step is None:
            # on the call's stream: memory that the current one has freed may still be in use on it
            with _torch().cuda.stream(None if stream is None else _torch_stream(stream, device)):
                step = self._steps[size] = self._state.new_empty(self.kv_lens.numel() + 1 + size)
        _, self.cu_rows, _, self.slots, counts = _call(
            "vggt_cache_plan", "plan", self.kv_lens, new_lens, self._free, self.n_free, self.block_table,
            self.page_size, n_rows, self.pages[0][0].shape[0], stream, step, self._state)
        if stream is not None:
            self._used_on(stream, self._state, self.free_pages, self.block_table)
            step.record_stream(_torch().cuda.current_stream(device))
        return counts[1:]

    def _used_on(self, stream, *tensors):
        """When the cache goes, these and its step buffers are given to nobody before ``stream`` is past its work."""
        if stream is not None:
            stream = _torch_stream(stream, self.kv_lens.device)
            for t in (*tensors, *self._steps.values()):
                t.record_stream(stream)

    def append(self, layer, k, v, stream=None):
        """Writes the step's rows of a layer."""
        cache_append(k, v, self.slots, *self.pages[layer], stream=stream)
        self._used_on(stream, *self.pages[layer])

    def attend(self, layer, q, causal_unit=0, stream=None, **more):
        """Attention of the step's rows over a layer's cache (see ``cached``)."""
        result = cached(q, *self.pages[layer], self.block_table, self.cu_rows, self.kv_lens, causal_unit,
                        stream=stream, **more)
        self._used_on(stream, *self.pages[layer], self.block_table, self.kv_lens)
        return result

    def release(self, seq):
        """Gives the pages of sequence ``seq`` back and empties it (on torch's current stream)."""
        import torch

        row, held = self.block_table[seq], (self.kv_lens[seq] + self.page_size - 1) // self.page_size
        col = torch.arange(row.numel(), device=row.device)
        at = torch.where(col < held, self.n_free + col, self.free_pages.numel() - 1)
        self.free_pages.index_put_((at,), row)
        self.n_free += held
        self.kv_lens[seq] = 0
