"""ctypes binding of ``libvggt_attn.so`` -- argument marshalling only.

Every function named ``vggt_*`` mirrors the C entry point of the same name in
``include/vggt_attn.h`` and returns its status code (an int; 0 = VGGT_OK).
Tensor arguments may be CUDA ``torch`` tensors (their ``data_ptr()`` is
passed) or raw integer device addresses; ``stream`` may be a
``torch.cuda.Stream``, a raw ``cudaStream_t`` integer, or None for torch's
current stream.  The library is loaded on first use; if it has not been
built this raises -- there is no CPU fallback.

The helpers at the bottom (``frame``, ``global_``, ``sga``, ``cached``, ...) allocate the
outputs with torch, call the entry points and raise ``VggtError`` on a
non-zero status.
"""
from __future__ import annotations

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
        fn = getattr(lib, name)
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
# A streaming step makes many small calls, so their cost on the host counts:
# each tensor is looked at once (_use), the arguments go to the C entry point as
# integers, and nothing is imported or looked up twice.

_T = None  # torch, once a call has needed it


def _torch():
    global _T
    if _T is None:
        import torch

        _T = torch
    return _T


def _use(x, dtype, device, name, contiguous=True):
    """The address of a tensor of a call on CUDA device ``device`` (an index); None stays None."""
    if x is None:
        return None
    if x.get_device() != device:
        if not x.is_cuda:
            raise ValueError(f"{name}: tensor must live on a CUDA device")
        raise ValueError(f"{name}: tensor on cuda:{x.get_device()}, the call runs on cuda:{device}")
    if x.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {x.dtype}")
    if contiguous and not x.is_contiguous():
        raise ValueError(f"{name}: tensor must be contiguous")
    return x.data_ptr()


def _device(x, name):
    """The index of the CUDA device of a call: that of its first tensor."""
    device = x.get_device()
    if device < 0:
        raise ValueError(f"{name}: tensor must live on a CUDA device")
    return device


def _launch(status_of, device, args, stream, what):
    """Calls an entry point on its device and on `stream` (None: torch's current stream of that device)."""
    torch = _torch()
    raw = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    if torch.cuda.current_device() == device:
        status = status_of(*args, raw)
    else:
        with torch.cuda.device(device):
            status = status_of(*args, raw)
    if status != VGGT_OK:
        raise VggtError(status, what)


def _new(shape, dtype, device, stream, returned=True):
    """A buffer of a call on `stream`: allocated there, since memory that was freed on torch's current stream may still
    be in use on it, and (if it is returned) freed only after the work of the current stream that reads it."""
    torch = _torch()
    device = torch.device("cuda", device)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        x = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        x.record_stream(torch.cuda.current_stream(device))
    return x


def _expect(ok, what):
    if not ok:
        raise ValueError(what)


def _page_layout(k_pages, v_pages, n_heads, n_seqs, max_pages):
    shape, stride = k_pages.shape, k_pages.stride()
    _expect(len(shape) == 4 and shape == v_pages.shape and stride == v_pages.stride() and
            (stride[3] == 1 or shape[3] == 1),
            "k_pages, v_pages: [n_pages, n_kv_heads, page_size, head_dim] of the same strides, the last one 1")
    n_pages, n_kv_heads, page_size, head_dim = shape
    sp, sh, st, _ = stride
    if n_pages == 1:  # a single page or head has no stride
        sp = 64
    if n_kv_heads == 1:
        sh = 64
    return vggt_cache(n_seqs, n_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages, sp, sh, st)


def cache_plan(cached_lens, new_lens, free_pages, n_free, block_table, page_size, n_rows, n_pages=None, stream=None):
    """Plans a step: writes the pages it takes into block_table and returns
    (cu_rows, kv_lens, slots, counts), all int32 on the device; counts is
    [free pages left, sequences refused] and counts[:1] the next step's n_free.
    n_rows: rows of the step's packed buffers (>= the new rows).  n_pages: pages
    of the cache (default: as many as 32-bit slots allow)."""
    torch = _torch()
    _expect(block_table.dim() == 2 and cached_lens.numel() == new_lens.numel() == block_table.shape[0]
            and n_free.numel() == 1, "one cached length, new length and row of block_table per sequence, one n_free")
    seqs, max_pages = block_table.shape
    if n_pages is None:
        n_pages = (2 ** 31 - 1) // page_size if page_size > 0 else 1
    d, i32 = _device(block_table, "block_table"), torch.int32
    inputs = (_use(cached_lens, i32, d, "cached_lens"), _use(new_lens, i32, d, "new_lens"),
              _use(free_pages, i32, d, "free_pages"), free_pages.numel(), _use(n_free, i32, d, "n_free"),
              _use(block_table, i32, d, "block_table"), n_rows)
    # one buffer: every part starts on 4 bytes, which is all that is asked
    out = _new(2 * seqs + 3 + max(n_rows, 0), i32, d, stream)
    at = out.data_ptr()
    cu, kv = at + 8, at + 12 + 4 * seqs
    slots = kv + 4 * seqs
    _launch(load().vggt_cache_plan, d, (vggt_cache(seqs, 1, 1, 64, page_size, n_pages, max_pages, 64, 64, 64), *inputs,
                                        cu, kv, slots, at), stream, "vggt_cache_plan")
    counts, cu_rows, kv_lens, slots = torch.split_with_sizes(out, (2, seqs + 1, seqs, n_rows))
    return cu_rows, kv_lens, slots, counts


def cache_append(k, v, slots, k_pages, v_pages, stream=None):
    """Writes the rows of k and v ([n_rows, n_kv_heads, 64], rows and heads may
    be strided) into their slots of k_pages and v_pages."""
    shape = k.shape
    _expect(len(shape) == 3 and shape == v.shape and k.stride() == v.stride() and slots.shape == shape[:1],
            "k, v: [n_rows, n_kv_heads, head_dim] of the same strides, one slot per row")
    cache = _page_layout(k_pages, v_pages, shape[1], 1, 1)
    _expect(shape[1] == cache.n_kv_heads and shape[2] == cache.head_dim, "k, v: the heads and head_dim of the pages")
    d, bf16 = _device(k_pages, "k_pages"), _torch().bfloat16
    row, head = _row_strides(k)
    _launch(load().vggt_cache_append, d,
            (cache, _use(k, bf16, d, "k", False), _use(v, bf16, d, "v", False), row, head,
             _use(slots, _T.int32, d, "slots"), shape[0], _use(k_pages, bf16, d, "k_pages", False),
             _use(v_pages, bf16, d, "v_pages", False)), stream, "vggt_cache_append")


def _row_strides(x):
    row, head, last = x.stride()
    rows, heads, dim = x.shape
    _expect(last == 1 or dim == 1, "the last dimension must be contiguous")
    # a dimension of one element has no stride of its own: any valid one does
    if heads <= 1:
        head = 64
    if rows <= 1:
        row = max(64, head * heads)
    return row, head


def cached(q, k_pages, v_pages, block_table, cu_rows, kv_lens, causal_unit=0, scale=None, want_lse=False,
           workspace=None, o=None, stream=None):
    """Attention of the new rows q ([n_rows, H, 64], rows and heads may be
    strided) over a paged cache; see vggt_attn_cached for the mask.  Rows
    behind cu_rows[-1] keep what ``o`` holds (uninitialised if not given)."""
    torch = _torch()
    shape, tables = q.shape, block_table.shape
    _expect(len(shape) == 3 and shape[2] == k_pages.shape[-1], "q: [n_rows, n_heads, head_dim]")
    _expect(len(tables) == 2 and kv_lens.numel() == tables[0] == cu_rows.numel() - 1,
            "one row of block_table and one length per sequence, one row offset more")
    _expect(o is None or o.shape == shape, "o: the shape of q")
    rows, heads, _ = shape
    cache = _page_layout(k_pages, v_pages, heads, *tables)
    d, bf16, i32 = _device(q, "q"), torch.bfloat16, torch.int32
    row, head = _row_strides(q)
    inputs = (cache, _use(q, bf16, d, "q", False), row, head, _use(k_pages, bf16, d, "k_pages", False),
              _use(v_pages, bf16, d, "v_pages", False), _use(block_table, i32, d, "block_table"),
              _use(cu_rows, i32, d, "cu_rows"), _use(kv_lens, i32, d, "kv_lens"), rows, causal_unit)
    lib, lse = load(), None
    if o is None:
        o = _new(shape, bf16, d, stream)
    if want_lse:
        lse = _new((rows, heads), torch.float32, d, stream)
    if workspace is None:
        nbytes = lib.vggt_attn_cached_workspace_bytes(cache, rows)
        if nbytes:
            workspace = _new(nbytes, torch.uint8, d, stream, returned=False)
    else:
        nbytes = workspace.numel() * workspace.element_size()
    _launch(lib.vggt_attn_cached, d,
            (*inputs, _use(o, bf16, d, "o"), None if lse is None else lse.data_ptr(),
             None if workspace is None else _use(workspace, workspace.dtype, d, "workspace"), nbytes,
             default_scale(shape[2]) if scale is None else scale), stream, "vggt_attn_cached")
    return (o, lse) if want_lse else o


def norm_residual(x, y=None, kind="layer", eps=1e-6, scale=None, gate=None, rows_per_gate=0, post_norm=False,
                  post_weight=None, post_bias=None, weight=None, bias=None, want_h=True, inplace=False, stream=None):
    """x' = x + scale * gate * N_post(y) and h = N_pre(x') in one pass over the
    rows of x and y ([n_rows, n_cols]); returns (x', h).  Without y x' is x;
    with want_h false h is None; with inplace x' overwrites x."""
    torch = _torch()
    shape = x.shape
    _expect(len(shape) == 2 and (y is None or y.shape == shape), "x, y: [n_rows, n_cols]")
    _expect(kind in _NORM_KINDS, "kind: 'layer' or 'rms'")
    rows, cols = shape
    if gate is None:
        rows_per_gate = 0
    else:
        _expect(rows_per_gate >= 1 and gate.shape == (-(-rows // rows_per_gate), cols),
                "gate: [ceil(n_rows / rows_per_gate), n_cols]")
    xt, f32, bf16 = x.dtype, torch.float32, torch.bfloat16
    _expect(xt == f32 or xt == bf16, "x: float32 or bfloat16")
    d = _device(x, "x")

    def factors(t, name):
        _expect(t is None or t.shape == (cols,), f"{name}: [n_cols]")
        return _use(t, f32, d, name)

    def stride(t, name):
        if t is None:
            return cols
        row, col = t.stride()
        _expect(col == 1 or cols == 1, f"{name}: the last dimension must be contiguous")
        return row if rows > 1 else cols

    inputs = (_use(x, xt, d, "x", False), _use(y, bf16, d, "y", False), factors(post_weight, "post_weight"),
              factors(post_bias, "post_bias"), factors(scale, "scale"), _use(gate, bf16, d, "gate"),
              factors(weight, "weight"), factors(bias, "bias"))
    xs, ys = stride(x, "x"), stride(y, "y")
    out = None
    if y is not None:
        out = x if inplace else _new(shape, xt, d, stream)
    h = _new(shape, bf16, d, stream) if want_h else None
    norm = vggt_norm(rows, cols, _NORM_KINDS[kind], xt == f32, bool(post_norm), rows_per_gate, eps, xs, ys,
                     xs if inplace else cols, cols)
    _launch(load().vggt_norm_residual, d, (norm, *inputs, None if out is None else out.data_ptr(),
                                           None if h is None else h.data_ptr()), stream, "vggt_norm_residual")
    return (x if out is None else out), h


class PagedCache:
    """The paged K/V cache of a streaming trunk: pages for ``n_layers`` layers
    that share one block table, the sequences' lengths and the free list, all
    on the device.  A step is ``plan(new_lens, n_rows)``, then per layer
    ``append(layer, k, v)`` and ``attend(layer, q)``, with the rows of the
    sequences packed one after another."""

    def __init__(self, n_pages, page_size, n_kv_heads, n_seqs, max_pages, n_layers=1, head_dim=64, device=None):
        import torch

        _expect(min(n_pages, page_size, n_kv_heads, n_seqs, max_pages, n_layers) >= 1, "sizes must be >= 1")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        i32 = dict(dtype=torch.int32, device=device)
        self.page_size = int(page_size)
        self.pages = [tuple(torch.zeros(n_pages, n_kv_heads, page_size, head_dim, dtype=torch.bfloat16, device=device)
                            for _ in range(2)) for _ in range(n_layers)]
        self.block_table = torch.full((n_seqs, max_pages), -1, **i32)
        self.kv_lens = torch.zeros(n_seqs, **i32)
        # one entry more than the pages: where release() drops what it must not write
        self.free_pages = torch.arange(n_pages + 1, **i32)
        self.n_free = torch.full((1,), n_pages, **i32)
        self.cu_rows = self.slots = None

    def plan(self, new_lens, n_rows, stream=None):
        """Plans a step of new_lens rows (int32 [n_seqs], on the device) in buffers of n_rows rows; returns the
        number of refused sequences (int32 [1], on the device)."""
        n_pages = self.pages[0][0].shape[0]
        self.cu_rows, self.kv_lens, self.slots, counts = cache_plan(
            self.kv_lens, new_lens, self.free_pages[:n_pages], self.n_free, self.block_table, self.page_size, n_rows,
            n_pages=n_pages, stream=stream)
        self.n_free = counts[:1]
        return counts[1:]

    def append(self, layer, k, v, stream=None):
        """Writes the step's rows of a layer."""
        cache_append(k, v, self.slots, *self.pages[layer], stream=stream)

    def attend(self, layer, q, causal_unit=0, **more):
        """Attention of the step's rows over a layer's cache (see ``cached``)."""
        return cached(q, *self.pages[layer], self.block_table, self.cu_rows, self.kv_lens, causal_unit, **more)

    def release(self, seq):
        """Gives the pages of sequence ``seq`` back and empties it (on torch's current stream)."""
        import torch

        row, held = self.block_table[seq], (self.kv_lens[seq] + self.page_size - 1) // self.page_size
        col = torch.arange(row.numel(), device=row.device)
        at = torch.where(col < held, self.n_free + col, self.free_pages.numel() - 1)
        self.free_pages = self.free_pages.index_put((at,), row)
        self.n_free = (self.n_free + held).to(torch.int32)
        self.kv_lens = self.kv_lens.clone()
        self.kv_lens[seq] = 0
