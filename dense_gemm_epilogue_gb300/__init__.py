"""Python binding of the tg_gemm C ABI (``include/tg_gemm.h``).

Argument marshalling only: every step of the GEMM runs in the CUDA library
``_lib/libtg_gemm.so`` built from ``csrc/`` by ``build.py``.  There is no
fallback: if the library is missing, ``load()`` raises.

Pointers may be given as integers, as objects with ``data_ptr()`` (torch
tensors) or as None (NULL).  Streams may be integers (a ``cudaStream_t``),
objects with a ``cuda_stream`` attribute (``torch.cuda.Stream``) or None (the
legacy default stream).
"""

from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading
import warnings

from .build import LIB as LIBRARY_PATH
from .build import PYCALL as _PYCALL_PATH
from .build import build, gemm_source_hash, source_hash  # noqa: F401

TG_OK = 0
TG_ERR_INVALID_VALUE = 1
TG_ERR_UNSUPPORTED = 2
TG_ERR_CUDA = 3
TG_ERR_DEVICE_TIMEOUT = 4

TG_BF16 = 0
TG_FP16 = 1
TG_TF32 = 2
TG_E4M3 = 3
TG_E5M2 = 4
TG_E2M1 = 5
TG_NVF4 = 6
DTYPE_CODES = {"bf16": TG_BF16, "fp16": TG_FP16, "tf32": TG_TF32, "e4m3": TG_E4M3,
               "e5m2": TG_E5M2, "e2m1": TG_E2M1, "nvf4": TG_NVF4}

TG_EPILOGUE_NONE = 0
TG_EPILOGUE_RELU = 1

TG_OUT_F32 = 0
TG_OUT_BF16 = 1
TG_OUT_F16 = 2
TG_ACT_NONE = 0
TG_ACT_RELU = 1
TG_ACT_SILU = 2
TG_ACT_GELU_TANH = 3
ACT_CODES = {"none": TG_ACT_NONE, "relu": TG_ACT_RELU, "silu": TG_ACT_SILU,
             "gelu_tanh": TG_ACT_GELU_TANH}

TG_PRODUCT_LINEAR = 0
TG_PRODUCT_GATED = 1
TG_PRODUCT_LINEAR_DX = 2
TG_PRODUCT_GATED_DX = 3
TG_PRODUCT_LINEAR_DW = 4
TG_PRODUCT_GATED_DW = 5
PRODUCT_CODES = {"linear": TG_PRODUCT_LINEAR, "gated": TG_PRODUCT_GATED,
                 "linear_dx": TG_PRODUCT_LINEAR_DX, "gated_dx": TG_PRODUCT_GATED_DX,
                 "linear_dw": TG_PRODUCT_LINEAR_DW, "gated_dw": TG_PRODUCT_GATED_DW}

TG_ROTARY_HALVES = 0
TG_ROTARY_PAIRS = 1
ROTARY_LAYOUTS = {"halves": TG_ROTARY_HALVES, "pairs": TG_ROTARY_PAIRS}
TG_ROTARY_NONE = 0
TG_ROTARY_LINEAR = 1
TG_ROTARY_BASE = 2
TG_ROTARY_BANDS = 3
ROTARY_SCALINGS = {"none": TG_ROTARY_NONE, "linear": TG_ROTARY_LINEAR, "base": TG_ROTARY_BASE,
                   "bands": TG_ROTARY_BANDS}

OUT_CODES = {"f32": TG_OUT_F32, "bf16": TG_OUT_BF16, "fp16": TG_OUT_F16}

# Every symbol include/tg_gemm.h declares.
EXPORTED = (
    "tg_gemm",
    "tg_gemm_ex",
    "tg_plan",
    "tg_plan_describe",
    "tg_status_string",
    "tg_check_device_status",
    "tg_set_wait_limit_ns",
    "tg_selftest_wait_timeout",
    "tg_version",
    "tg_gemm_noalloc",
    "tg_gemm_batched",
    "tg_gemm_epilogue",
    "tg_gemm_mx",
    "tg_gemm_mx_batched",
    "tg_plan_mx",
    "tg_mx_scale_bytes",
    "tg_mx_pack_scales",
    "tg_bs_scale_bytes",
    "tg_bs_pack_scales",
    "tg_linear_workspace_bytes",
    "tg_linear",
    "tg_linear_backward_workspace_bytes",
    "tg_linear_backward",
    "tg_gated_workspace_bytes",
    "tg_gated",
    "tg_gated_backward_workspace_bytes",
    "tg_gated_backward",
    "tg_layer_norm",
    "tg_layer_norm_backward_workspace_bytes",
    "tg_layer_norm_backward",
    "tg_product_plan_describe",
    "tg_rotary_steps",
    "tg_rotary",
    "tg_rotary_backward",
    "tg_attention_workspace_bytes",
    "tg_attention",
    "tg_attention_plan_describe",
    "tg_attention_backward_workspace_bytes",
    "tg_attention_backward",
)


class TgError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {tg_status_string(status)} ({status})" if what else
                         f"{tg_status_string(status)} ({status})")


class tg_options(ctypes.Structure):
    _fields_ = [
        ("block_n", ctypes.c_int32),
        ("producer", ctypes.c_int32),
        ("swap_ab", ctypes.c_int32),
        ("raster_group", ctypes.c_int32),
        ("max_ctas", ctypes.c_int32),
        ("cta_pair", ctypes.c_int32),
        ("split_k", ctypes.c_int32),
        ("l2_hint", ctypes.c_int32),
        ("prefetch_k", ctypes.c_int32),
        ("multicast", ctypes.c_int32),
        ("schedule", ctypes.c_int32),
        ("reserved", ctypes.c_int32 * 1),
    ]


EPI_KINDS = {"scale": 0, "add": 1, "relu": 2, "leaky_relu": 3, "clamp": 4, "sigmoid": 5,
             "silu": 6, "gelu_tanh": 7, "bias_row": 8, "bias_col": 9}


class tg_epi_op(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("a", ctypes.c_float),
        ("b", ctypes.c_float),
        ("bias", ctypes.c_void_p),
    ]


class tg_plan_info(ctypes.Structure):
    _fields_ = [
        ("block_m", ctypes.c_int32),
        ("block_n", ctypes.c_int32),
        ("block_k", ctypes.c_int32),
        ("stages", ctypes.c_int32),
        ("producer", ctypes.c_int32),
        ("swap_ab", ctypes.c_int32),
        ("raster_group", ctypes.c_int32),
        ("grid", ctypes.c_int32),
        ("tiles", ctypes.c_int64),
        ("threads", ctypes.c_int32),
        ("smem_bytes", ctypes.c_int32),
        ("tmem_cols", ctypes.c_int32),
        ("vector_store", ctypes.c_int32),
        ("cta_pair", ctypes.c_int32),
        ("split_tiles", ctypes.c_int32),
        ("split_segs", ctypes.c_int32),
        ("multicast", ctypes.c_int32),
        ("stream_k", ctypes.c_int32),
        ("schedule", ctypes.c_int32),
        ("k_rotate", ctypes.c_int32),
        ("k_snake", ctypes.c_int32),
    ]


_lock = threading.Lock()
_lib = None
_call = None  # the hot calls without ctypes (csrc/tg_pycall.c), when built
_CALLS = ("tg_linear_workspace_bytes", "tg_linear", "tg_gated_workspace_bytes", "tg_gated",
          "tg_layer_norm", "tg_layer_norm_backward_workspace_bytes", "tg_layer_norm_backward",
          "tg_rotary", "tg_rotary_backward", "tg_attention_workspace_bytes", "tg_attention",
          "tg_attention_backward_workspace_bytes", "tg_attention_backward")


def _load_calls(lib):
    """The marshalling module bound to this library's entry points, or None.
    It only saves time: one that does not load, or does not take these entry
    points, is named in a warning and the ctypes wrappers serve."""
    if not os.path.exists(_PYCALL_PATH):
        return None
    try:
        loader = importlib.machinery.ExtensionFileLoader("_tgcall", _PYCALL_PATH)
        spec = importlib.util.spec_from_loader("_tgcall", loader)
        mod = importlib.util.module_from_spec(spec)
        loader.exec_module(mod)
        mod.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _CALLS},
                 DTYPE_CODES, ACT_CODES, OUT_CODES)
    except (ImportError, SystemError, AttributeError, KeyError, TypeError, ValueError) as e:
        warnings.warn(f"{_PYCALL_PATH} is left out, calls go through ctypes: {e}", RuntimeWarning,
                      stacklevel=3)
        return None
    return mod


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib, _call
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIBRARY_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"tg_gemm library not built ({p} missing); run "
                               "dense_gemm_epilogue_gb300.build.build() first")
        lib = ctypes.CDLL(p)
        i64, i32, f32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p
        lib.tg_gemm.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, ctypes.c_int,
                                ctypes.c_int, vp]
        lib.tg_gemm.restype = ctypes.c_int
        lib.tg_gemm_ex.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, ctypes.c_int,
                                   ctypes.c_int, ctypes.POINTER(tg_options), vp]
        lib.tg_gemm_ex.restype = ctypes.c_int
        lib.tg_plan.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, ctypes.c_int,
                                ctypes.POINTER(tg_options), i32, ctypes.POINTER(tg_plan_info)]
        lib.tg_plan.restype = ctypes.c_int
        lib.tg_plan_describe.argtypes = [i64, i64, i64, ctypes.c_int, i64, i64, i64, i32,
                                         ctypes.c_char_p, ctypes.c_size_t]
        lib.tg_plan_describe.restype = ctypes.c_int
        lib.tg_status_string.argtypes = [ctypes.c_int]
        lib.tg_status_string.restype = ctypes.c_char_p
        lib.tg_check_device_status.argtypes = [vp, ctypes.POINTER(i32)]
        lib.tg_check_device_status.restype = ctypes.c_int
        lib.tg_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
        lib.tg_set_wait_limit_ns.restype = ctypes.c_int
        lib.tg_selftest_wait_timeout.argtypes = [ctypes.c_uint64, vp]
        lib.tg_selftest_wait_timeout.restype = ctypes.c_int
        lib.tg_gemm_noalloc.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64,
                                        ctypes.c_int, ctypes.c_int, vp]
        lib.tg_gemm_noalloc.restype = ctypes.c_int
        lib.tg_gemm_batched.argtypes = [i64, i64, i64, f32, vp, i64, i64, vp, i64, i64, vp, i64,
                                        i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.POINTER(tg_options), vp]
        lib.tg_gemm_batched.restype = ctypes.c_int
        lib.tg_gemm_epilogue.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64,
                                         ctypes.c_int, ctypes.c_int, ctypes.POINTER(tg_epi_op),
                                         i32, ctypes.POINTER(tg_options), vp]
        lib.tg_gemm_epilogue.restype = ctypes.c_int
        lib.tg_gemm_mx.argtypes = [i64, i64, i64, f32, vp, i64, vp, vp, i64, vp, vp, i64,
                                   ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                   ctypes.POINTER(tg_options), vp]
        lib.tg_gemm_mx.restype = ctypes.c_int
        lib.tg_gemm_mx_batched.argtypes = [i64, i64, i64, f32, vp, i64, i64, vp, i64, vp, i64,
                                           i64, vp, i64, vp, i64, i64, i64, ctypes.c_int,
                                           ctypes.c_int, ctypes.POINTER(tg_epi_op), i32,
                                           ctypes.POINTER(tg_options), vp]
        lib.tg_gemm_mx_batched.restype = ctypes.c_int
        lib.tg_plan_mx.argtypes = [i64, i64, i64, i64, i64, i64, ctypes.c_int,
                                   ctypes.POINTER(tg_options), i32, ctypes.POINTER(tg_plan_info)]
        lib.tg_plan_mx.restype = ctypes.c_int
        lib.tg_mx_scale_bytes.argtypes = [i64, i64]
        lib.tg_mx_scale_bytes.restype = i64
        lib.tg_mx_pack_scales.argtypes = [i64, i64, vp, i64, vp, vp]
        lib.tg_mx_pack_scales.restype = ctypes.c_int
        lib.tg_bs_scale_bytes.argtypes = [i64, i64, ctypes.c_int]
        lib.tg_bs_scale_bytes.restype = i64
        lib.tg_bs_pack_scales.argtypes = [i64, i64, ctypes.c_int, vp, i64, vp, vp]
        lib.tg_bs_pack_scales.restype = ctypes.c_int
        c = ctypes.c_int
        lib.tg_linear_workspace_bytes.argtypes = [i64, i64, i64, vp, i64, vp, i64, c]
        lib.tg_linear_workspace_bytes.restype = i64
        lib.tg_linear.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, c, vp, i64, vp, i64, vp,
                                  i64, c, vp, i64, vp]
        lib.tg_linear.restype = c
        lib.tg_linear_backward_workspace_bytes.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp,
                                                           i64, c, c]
        lib.tg_linear_backward_workspace_bytes.restype = i64
        lib.tg_linear_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, c,
                                           vp, i64, vp, i64, c, vp, c, vp, i64, vp]
        lib.tg_linear_backward.restype = c
        lib.tg_gated_workspace_bytes.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, c]
        lib.tg_gated_workspace_bytes.restype = i64
        lib.tg_gated.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, c, vp, i64, vp, i64,
                                 vp, i64, c, vp, i64, vp]
        lib.tg_gated.restype = c
        lib.tg_gated_backward_workspace_bytes.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp,
                                                          i64, c]
        lib.tg_gated_backward_workspace_bytes.restype = i64
        lib.tg_gated_backward.argtypes = [i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, vp,
                                          i64, vp, i64, c, vp, i64, vp, i64, vp, i64, c, c, vp,
                                          i64, vp]
        lib.tg_gated_backward.restype = c
        lib.tg_layer_norm.argtypes = [i64, i64, vp, i64, vp, vp, f32, vp, i64, vp, vp, c, vp]
        lib.tg_layer_norm.restype = c
        lib.tg_layer_norm_backward_workspace_bytes.argtypes = [i64, i64]
        lib.tg_layer_norm_backward_workspace_bytes.restype = i64
        lib.tg_layer_norm_backward.argtypes = [i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, i64,
                                               vp, vp, c, vp, i64, vp]
        lib.tg_layer_norm_backward.restype = c
        lib.tg_product_plan_describe.argtypes = [c, i64, i64, i64, i32, ctypes.c_char_p,
                                                 ctypes.c_size_t]
        lib.tg_product_plan_describe.restype = c
        f64 = ctypes.c_double
        lib.tg_rotary_steps.argtypes = [i64, f64, c, f64, f64, f64, f64,
                                        ctypes.POINTER(ctypes.c_uint64)]
        lib.tg_rotary_steps.restype = c
        lib.tg_rotary.argtypes = [i64, i64, i64, i64, vp, i64, i64, vp, i64, i64, i64, vp, vp, vp, c,
                                  f32, c, vp]
        lib.tg_rotary.restype = c
        lib.tg_rotary_backward.argtypes = [i64, i64, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, c,
                                           f32, c, vp]
        lib.tg_rotary_backward.restype = c
        lib.tg_attention_workspace_bytes.argtypes = [i64] * 8 + [c]
        lib.tg_attention_workspace_bytes.restype = i64
        lib.tg_attention.argtypes = ([i64] * 6 + [vp, i64, i64] * 3 + [vp] * 4 + [i64, i64, i32, f32]
                                     + [vp, i64, i64, vp, c, vp, i64, vp])
        lib.tg_attention.restype = c
        lib.tg_attention_backward_workspace_bytes.argtypes = [i64] * 8 + [c]
        lib.tg_attention_backward_workspace_bytes.restype = i64
        lib.tg_attention_backward.argtypes = ([i64] * 6 + [vp, i64, i64] * 5 + [vp] * 5
                                              + [i64, i64, i32, f32] + [vp, i64, i64] * 3
                                              + [c, vp, i64, vp])
        lib.tg_attention_backward.restype = c
        lib.tg_attention_plan_describe.argtypes = [i64] * 8 + [c, i32, ctypes.c_char_p, ctypes.c_size_t]
        lib.tg_attention_plan_describe.restype = c
        lib.tg_version.argtypes = []
        lib.tg_version.restype = i32
        if path is None:
            _call = _load_calls(lib)
            _lib = lib
        return lib


def _ptr(x):
    if x is None:
        return None
    try:
        return x.data_ptr()
    except AttributeError:
        pass
    if isinstance(x, int):
        return x
    raise TypeError(f"cannot pass {type(x).__name__} as a pointer")


def _stream(s):
    if s is None:
        return None
    try:
        return s.cuda_stream
    except AttributeError:
        pass
    if isinstance(s, int):
        return s
    raise TypeError(f"cannot pass {type(s).__name__} as a stream")


def _dtype(d):
    return DTYPE_CODES[d] if isinstance(d, str) else int(d)


def _epi(e):
    if isinstance(e, str):
        return {"none": TG_EPILOGUE_NONE, "relu": TG_EPILOGUE_RELU}[e]
    if isinstance(e, bool):
        return TG_EPILOGUE_RELU if e else TG_EPILOGUE_NONE
    return int(e)


def _options(opts):
    if opts is None:
        return None
    if isinstance(opts, tg_options):
        return ctypes.byref(opts)
    o = tg_options()
    for k, v in dict(opts).items():
        if k == "reserved":
            for i, r in enumerate(v):
                o.reserved[i] = int(r)
        else:
            setattr(o, k, int(v))
    return ctypes.byref(o)


def tg_gemm(M, N, K, alpha, A, lda, B, ldb, D, ldc, in_dtype, epilogue, stream=None) -> int:
    """D = epi(alpha * A * B); returns the tg_status code (enqueue only)."""
    return load().tg_gemm(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldc,
                          _dtype(in_dtype), _epi(epilogue), _stream(stream))


def tg_gemm_ex(M, N, K, alpha, A, lda, B, ldb, D, ldc, in_dtype, epilogue, opts=None,
               stream=None) -> int:
    """tg_gemm with planner overrides (dict of tg_options fields)."""
    return load().tg_gemm_ex(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldc,
                             _dtype(in_dtype), _epi(epilogue), _options(opts), _stream(stream))


def tg_gemm_noalloc(M, N, K, alpha, A, lda, B, ldb, D, ldc, in_dtype, epilogue,
                    stream=None) -> int:
    """tg_gemm for callers that cannot allocate device memory (the library
    allocates nothing in this call; see include/tg_gemm.h)."""
    return load().tg_gemm_noalloc(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldc,
                                  _dtype(in_dtype), _epi(epilogue), _stream(stream))


def tg_gemm_batched(M, N, K, alpha, A, lda, stride_a, B, ldb, stride_b, D, ldc, stride_d, batch,
                    in_dtype, out_dtype, epilogue, opts=None, stream=None) -> int:
    """Strided batch of GEMMs with an output type (f32, bf16 or fp16)."""
    out = OUT_CODES[out_dtype] if isinstance(out_dtype, str) else int(out_dtype)
    return load().tg_gemm_batched(M, N, K, alpha, _ptr(A), lda, stride_a, _ptr(B), ldb, stride_b,
                                  _ptr(D), ldc, stride_d, batch, _dtype(in_dtype), out,
                                  _epi(epilogue), _options(opts), _stream(stream))


def tg_plan(M, N, K, A, lda, B, ldb, D, ldc, in_dtype, opts=None, num_sms=0):
    """The planner's choice as a dict; raises TgError on invalid arguments."""
    info = tg_plan_info()
    st = load().tg_plan(M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldc, _dtype(in_dtype),
                        _options(opts), num_sms, ctypes.byref(info))
    if st != TG_OK:
        raise TgError(st, "tg_plan")
    return {name: getattr(info, name) for name, _ in tg_plan_info._fields_}


def tg_plan_describe(M, N, K, in_dtype, lda, ldb, ldc, num_sms=0, size=256):
    """The planner's choice as one line of text; raises TgError on invalid
    arguments or when the text does not fit in `size` bytes."""
    buf = ctypes.create_string_buffer(size)
    st = load().tg_plan_describe(M, N, K, _dtype(in_dtype), lda, ldb, ldc, num_sms, buf, size)
    if st != TG_OK:
        raise TgError(st, "tg_plan_describe")
    return buf.value.decode()


def _epi_ops(ops):
    arr = (tg_epi_op * max(len(ops), 1))()
    for q, (kind, a, b, bias) in enumerate(ops):
        arr[q].kind = EPI_KINDS[kind] if isinstance(kind, str) else int(kind)
        arr[q].a = float(a)
        arr[q].b = float(b)
        arr[q].bias = _ptr(bias)
    return arr


def tg_gemm_epilogue(M, N, K, alpha, A, lda, B, ldb, D, ldc, in_dtype, out_dtype, ops,
                     opts=None, stream=None) -> int:
    """D = out(op_n(... op_1(alpha * A B))); ops: sequence of (kind, a, b, bias)
    with kind a name of EPI_KINDS (or its code) and bias a device tensor or None."""
    out = OUT_CODES[out_dtype] if isinstance(out_dtype, str) else int(out_dtype)
    arr = _epi_ops(ops)
    return load().tg_gemm_epilogue(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, _ptr(D), ldc,
                                   _dtype(in_dtype), out, arr, len(ops), _options(opts),
                                   _stream(stream))


def tg_gemm_mx(M, N, K, alpha, A, lda, SFA, B, ldb, SFB, D, ldc, in_dtype, out_dtype, epilogue,
               opts=None, stream=None) -> int:
    """Block-scaled FP8 GEMM; SFA / SFB are scale-atom buffers (see
    include/tg_gemm.h, tg_gemm_mx)."""
    out = OUT_CODES[out_dtype] if isinstance(out_dtype, str) else int(out_dtype)
    return load().tg_gemm_mx(M, N, K, alpha, _ptr(A), lda, _ptr(SFA), _ptr(B), ldb, _ptr(SFB),
                             _ptr(D), ldc, _dtype(in_dtype), out, _epi(epilogue), _options(opts),
                             _stream(stream))


def tg_gemm_mx_batched(M, N, K, alpha, A, lda, stride_a, SFA, stride_sfa, B, ldb, stride_b, SFB,
                       stride_sfb, D, ldc, stride_d, batch, in_dtype, out_dtype, ops=(),
                       opts=None, stream=None) -> int:
    """Strided batch of block-scaled GEMMs with a composed epilogue (see
    include/tg_gemm.h, tg_gemm_mx_batched); scale strides in bytes."""
    out = OUT_CODES[out_dtype] if isinstance(out_dtype, str) else int(out_dtype)
    arr = _epi_ops(ops)
    return load().tg_gemm_mx_batched(M, N, K, alpha, _ptr(A), lda, stride_a, _ptr(SFA),
                                     stride_sfa, _ptr(B), ldb, stride_b, _ptr(SFB), stride_sfb,
                                     _ptr(D), ldc, stride_d, batch, _dtype(in_dtype), out, arr,
                                     len(ops), _options(opts), _stream(stream))


def tg_plan_mx(M, N, K, lda, ldb, ldc, in_dtype, opts=None, num_sms=0):
    """The block-scaled planner's choice as a dict; raises TgError on invalid arguments."""
    info = tg_plan_info()
    st = load().tg_plan_mx(M, N, K, lda, ldb, ldc, _dtype(in_dtype), _options(opts), num_sms,
                           ctypes.byref(info))
    if st != TG_OK:
        raise TgError(st, "tg_plan_mx")
    return {name: getattr(info, name) for name, _ in tg_plan_info._fields_}


def tg_mx_scale_bytes(rows, K) -> int:
    return int(load().tg_mx_scale_bytes(rows, K))


def tg_mx_pack_scales(rows, K, src, ld_src, dst, stream=None) -> int:
    """Row-major scale codes (device) -> scale atoms (device)."""
    return load().tg_mx_pack_scales(rows, K, _ptr(src), ld_src, _ptr(dst), _stream(stream))


def tg_bs_scale_bytes(rows, K, in_dtype) -> int:
    return int(load().tg_bs_scale_bytes(rows, K, _dtype(in_dtype)))


def tg_bs_pack_scales(rows, K, in_dtype, src, ld_src, dst, stream=None) -> int:
    """Row-major scale codes (device) -> scale atoms (device), for in_dtype's
    block size (32 K per scale; nvf4: 16)."""
    return load().tg_bs_pack_scales(rows, K, _dtype(in_dtype), _ptr(src), ld_src, _ptr(dst),
                                    _stream(stream))


def _act(a):
    return ACT_CODES[a] if isinstance(a, str) else int(a)


def _out(d):
    return OUT_CODES[d] if isinstance(d, str) else int(d)


def _space(w):
    """(pointer, bytes) of a workspace: None, a tensor, or such a pair."""
    if w is None:
        return None, 0
    if isinstance(w, tuple):
        return _ptr(w[0]), int(w[1])
    return w.data_ptr(), w.numel() * w.element_size()


def tg_linear_workspace_bytes(M, N, K, X, ldx, W, ldw, dtype) -> int:
    if _call is not None:
        return _call.tg_linear_workspace_bytes(M, N, K, X, ldx, W, ldw, dtype)
    return load().tg_linear_workspace_bytes(M, N, K, _ptr(X), ldx, _ptr(W), ldw, _dtype(dtype))


def tg_linear(M, N, K, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, Z, ldz, dtype, workspace=None,
              stream=None) -> int:
    """Y = act(X W^T + bias) + R and, when Z is given, Z = X W^T + bias (row-major; bias, R and Z
    may be None; act a name of ACT_CODES).  workspace: None, a tensor or (pointer, bytes)."""
    if _call is not None:
        return _call.tg_linear(M, N, K, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, Z, ldz, dtype,
                               workspace, stream)
    ws, n = _space(workspace)
    return load().tg_linear(M, N, K, _ptr(X), ldx, _ptr(W), ldw, _ptr(bias), _act(act), _ptr(R),
                            ldr, _ptr(Y), ldy, _ptr(Z), ldz, _dtype(dtype), ws, n, _stream(stream))


def tg_linear_backward_workspace_bytes(M, N, K, dY, lddy, X, ldx, W, ldw, act, dtype) -> int:
    return load().tg_linear_backward_workspace_bytes(M, N, K, _ptr(dY), lddy, _ptr(X), ldx,
                                                     _ptr(W), ldw, _act(act), _dtype(dtype))


def tg_linear_backward(M, N, K, dY, lddy, X, ldx, W, ldw, Z, ldz, act, dX, lddx, dW, lddw,
                       dw_dtype, db, dtype, workspace=None, stream=None) -> int:
    """dZ = dY act'(Z); dX = dZ W, dW = dZ^T X (of type dw_dtype), db = sum over rows of dZ;
    each of the three may be None."""
    ws, n = _space(workspace)
    return load().tg_linear_backward(M, N, K, _ptr(dY), lddy, _ptr(X), ldx, _ptr(W), ldw, _ptr(Z),
                                     ldz, _act(act), _ptr(dX), lddx, _ptr(dW), lddw,
                                     _out(dw_dtype), _ptr(db), _dtype(dtype), ws, n,
                                     _stream(stream))


def tg_gated_workspace_bytes(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, dtype) -> int:
    if _call is not None:
        return _call.tg_gated_workspace_bytes(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, dtype)
    return load().tg_gated_workspace_bytes(M, N, K, _ptr(X), ldx, _ptr(Wg), ldwg, _ptr(Wu), ldwu,
                                           _dtype(dtype))


def tg_gated(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, act, H, ldh, G, ldg, U, ldu, dtype,
             workspace=None, stream=None) -> int:
    """H = act(X Wg^T) * (X Wu^T) in one kernel; G and U (the two products) are stored when
    given."""
    if _call is not None:
        return _call.tg_gated(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, act, H, ldh, G, ldg, U, ldu, dtype,
                              workspace, stream)
    ws, n = _space(workspace)
    return load().tg_gated(M, N, K, _ptr(X), ldx, _ptr(Wg), ldwg, _ptr(Wu), ldwu, _act(act),
                           _ptr(H), ldh, _ptr(G), ldg, _ptr(U), ldu, _dtype(dtype), ws, n,
                           _stream(stream))


def tg_gated_backward_workspace_bytes(M, N, K, X, ldx, Wg, ldwg, Wu, ldwu, dtype) -> int:
    return load().tg_gated_backward_workspace_bytes(M, N, K, _ptr(X), ldx, _ptr(Wg), ldwg,
                                                    _ptr(Wu), ldwu, _dtype(dtype))


def tg_gated_backward(M, N, K, dH, lddh, X, ldx, Wg, ldwg, Wu, ldwu, G, ldg, U, ldu, act, dX, lddx,
                      dWg, lddwg, dWu, lddwu, dw_dtype, dtype, workspace=None, stream=None) -> int:
    """dX = dG Wg + dU Wu, dWg = dG^T X, dWu = dU^T X with dG = dH U act'(G), dU = dH act(G);
    each of the three may be None."""
    ws, n = _space(workspace)
    return load().tg_gated_backward(M, N, K, _ptr(dH), lddh, _ptr(X), ldx, _ptr(Wg), ldwg,
                                    _ptr(Wu), ldwu, _ptr(G), ldg, _ptr(U), ldu, _act(act),
                                    _ptr(dX), lddx, _ptr(dWg), lddwg, _ptr(dWu), lddwu,
                                    _out(dw_dtype), _dtype(dtype), ws, n, _stream(stream))


def tg_layer_norm(M, N, X, ldx, gamma, beta, eps, Y, ldy, mean, rstd, dtype, stream=None) -> int:
    """Y = (X - mean) rstd gamma + beta per row; gamma, beta, mean and rstd may be None; dtype a
    name of OUT_CODES."""
    if _call is not None:
        return _call.tg_layer_norm(M, N, X, ldx, gamma, beta, eps, Y, ldy, mean, rstd, dtype, stream)
    return load().tg_layer_norm(M, N, _ptr(X), ldx, _ptr(gamma), _ptr(beta), eps, _ptr(Y), ldy,
                                _ptr(mean), _ptr(rstd), _out(dtype), _stream(stream))


def tg_layer_norm_backward_workspace_bytes(M, N) -> int:
    if _call is not None:
        return _call.tg_layer_norm_backward_workspace_bytes(M, N)
    return load().tg_layer_norm_backward_workspace_bytes(M, N)


def tg_layer_norm_backward(M, N, dY, lddy, X, ldx, gamma, mean, rstd, dX, lddx, dgamma, dbeta,
                           dtype, workspace=None, stream=None) -> int:
    """dX, dgamma and dbeta (each may be None) of tg_layer_norm."""
    if _call is not None:
        return _call.tg_layer_norm_backward(M, N, dY, lddy, X, ldx, gamma, mean, rstd, dX, lddx, dgamma,
                                            dbeta, dtype, workspace, stream)
    ws, n = _space(workspace)
    return load().tg_layer_norm_backward(M, N, _ptr(dY), lddy, _ptr(X), ldx, _ptr(gamma),
                                         _ptr(mean), _ptr(rstd), _ptr(dX), lddx, _ptr(dgamma),
                                         _ptr(dbeta), _out(dtype), ws, n, _stream(stream))


def tg_rotary_steps(rot, base, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192.0):
    """Frequencies as 64-bit fractions of a turn a position, in a list of rot/2 integers as int64
    holds them (a tensor of them on the device is what tg_rotary reads); raises TgError on invalid
    arguments.  scaling is a name of ROTARY_SCALINGS."""
    # (room for every rot that the library takes: 4096 at most)
    out = (ctypes.c_uint64 * min(max(int(rot) // 2, 1), 2048))()
    code = ROTARY_SCALINGS[scaling] if isinstance(scaling, str) else int(scaling)
    check(load().tg_rotary_steps(rot, base, code, factor, low, high, original, out), "tg_rotary_steps")
    return [v - (1 << 64) if v >> 63 else v for v in out]


def _rotary_layout(n):
    return ROTARY_LAYOUTS[n] if isinstance(n, str) else int(n)


def tg_rotary(tokens, heads, dim, rot, X, ldx, hx, Y, ldy, hy, y_rows, positions, rows, steps, layout,
              amplitude, dtype, stream=None) -> int:
    """Rotary positions on the first rot values of each head (rows of Y by `rows` when given);
    positions and rows may be None; layout a name of ROTARY_LAYOUTS, dtype of OUT_CODES."""
    if _call is not None:
        return _call.tg_rotary(tokens, heads, dim, rot, X, ldx, hx, Y, ldy, hy, y_rows, positions, rows,
                               steps, _rotary_layout(layout), amplitude, dtype, stream)
    return load().tg_rotary(tokens, heads, dim, rot, _ptr(X), ldx, hx, _ptr(Y), ldy, hy, y_rows,
                            _ptr(positions), _ptr(rows), _ptr(steps), _rotary_layout(layout),
                            amplitude, _out(dtype), _stream(stream))


def tg_rotary_backward(tokens, heads, dim, rot, dY, lddy, hdy, dX, lddx, hdx, positions, steps, layout,
                       amplitude, dtype, stream=None) -> int:
    """The transposed map, from dY to dX (which may be dY)."""
    if _call is not None:
        return _call.tg_rotary_backward(tokens, heads, dim, rot, dY, lddy, hdy, dX, lddx, hdx, positions,
                                        steps, _rotary_layout(layout), amplitude, dtype, stream)
    return load().tg_rotary_backward(tokens, heads, dim, rot, _ptr(dY), lddy, hdy, _ptr(dX), lddx, hdx,
                                     _ptr(positions), _ptr(steps), _rotary_layout(layout), amplitude,
                                     _out(dtype), _stream(stream))


def tg_attention_workspace_bytes(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype) -> int:
    if _call is not None:
        return _call.tg_attention_workspace_bytes(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k,
                                                  dtype)
    return load().tg_attention_workspace_bytes(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k,
                                               _dtype(dtype))


def tg_attention(seqs, q_rows, k_rows, heads, kv_heads, dim, Q, ldq, hq, K, ldk, hk, V, ldv, hv,
                 q_starts, q_lengths, k_starts, k_lengths, max_q, max_k, causal, scale, O, ldo, ho, LSE,
                 dtype, workspace=None, stream=None) -> int:
    """O = softmax(scale Q K^T) V over packed sequences, and the rows' LSE; the lengths and LSE may be
    None."""
    if _call is not None:
        return _call.tg_attention(seqs, q_rows, k_rows, heads, kv_heads, dim, Q, ldq, hq, K, ldk, hk, V, ldv,
                                  hv, q_starts, q_lengths, k_starts, k_lengths, max_q, max_k, causal, scale,
                                  O, ldo, ho, LSE, dtype, workspace, stream)
    ws, n = _space(workspace)
    return load().tg_attention(seqs, q_rows, k_rows, heads, kv_heads, dim, _ptr(Q), ldq, hq, _ptr(K),
                               ldk, hk, _ptr(V), ldv, hv, _ptr(q_starts), _ptr(q_lengths),
                               _ptr(k_starts), _ptr(k_lengths), max_q, max_k, int(causal), scale,
                               _ptr(O), ldo, ho, _ptr(LSE), _dtype(dtype), ws, n, _stream(stream))


def tg_attention_plan_describe(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k, dtype, num_sms=0,
                               size=256) -> str:
    """The plan of a tg_attention call as text; raises TgError on invalid arguments."""
    buf = ctypes.create_string_buffer(size)
    check(load().tg_attention_plan_describe(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k,
                                            _dtype(dtype), num_sms, buf, size),
          "tg_attention_plan_describe")
    return buf.value.decode()


def tg_attention_backward_workspace_bytes(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q, max_k,
                                          dtype) -> int:
    if _call is not None:
        return _call.tg_attention_backward_workspace_bytes(seqs, q_rows, k_rows, heads, kv_heads, dim,
                                                           max_q, max_k, dtype)
    return load().tg_attention_backward_workspace_bytes(seqs, q_rows, k_rows, heads, kv_heads, dim, max_q,
                                                        max_k, _dtype(dtype))


def tg_attention_backward(seqs, q_rows, k_rows, heads, kv_heads, dim, Q, ldq, hq, K, ldk, hk, V, ldv, hv,
                          O, ldo, ho, dO, lddo, hdo, LSE, q_starts, q_lengths, k_starts, k_lengths,
                          max_q, max_k, causal, scale, dQ, lddq, hdq, dK, lddk, hdk, dV, lddv, hdv, dtype,
                          workspace=None, stream=None) -> int:
    """dQ, dK and dV (each may be None) of tg_attention, from dO, O and LSE."""
    if _call is not None:
        return _call.tg_attention_backward(
            seqs, q_rows, k_rows, heads, kv_heads, dim, Q, ldq, hq, K, ldk, hk, V, ldv, hv, O, ldo, ho, dO,
            lddo, hdo, LSE, q_starts, q_lengths, k_starts, k_lengths, max_q, max_k, causal, scale, dQ, lddq,
            hdq, dK, lddk, hdk, dV, lddv, hdv, dtype, workspace, stream)
    ws, n = _space(workspace)
    return load().tg_attention_backward(
        seqs, q_rows, k_rows, heads, kv_heads, dim, _ptr(Q), ldq, hq, _ptr(K), ldk, hk, _ptr(V), ldv, hv,
        _ptr(O), ldo, ho, _ptr(dO), lddo, hdo, _ptr(LSE), _ptr(q_starts), _ptr(q_lengths), _ptr(k_starts),
        _ptr(k_lengths), max_q, max_k, int(causal), scale, _ptr(dQ), lddq, hdq, _ptr(dK), lddk, hdk,
        _ptr(dV), lddv, hdv, _dtype(dtype), ws, n, _stream(stream))


def tg_product_plan_describe(product, M, N, K, num_sms=0, size=256) -> str:
    """The planner's choice for a feed-forward product (a name of PRODUCT_CODES) as text."""
    buf = ctypes.create_string_buffer(size)
    code = PRODUCT_CODES[product] if isinstance(product, str) else int(product)
    check(load().tg_product_plan_describe(code, M, N, K, num_sms, buf, size),
          "tg_product_plan_describe")
    return buf.value.decode()


def tg_status_string(status: int) -> str:
    return load().tg_status_string(int(status)).decode()


def tg_check_device_status(stream=None):
    """(status, where): synchronises the stream and reads/clears the status word."""
    where = ctypes.c_int32(0)
    st = load().tg_check_device_status(_stream(stream), ctypes.byref(where))
    return st, where.value


def tg_set_wait_limit_ns(ns: int) -> int:
    return load().tg_set_wait_limit_ns(int(ns))


def tg_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return load().tg_selftest_wait_timeout(int(limit_ns), _stream(stream))


def tg_version() -> int:
    return load().tg_version()


def check(status: int, what: str = "tg_gemm") -> None:
    if status != TG_OK:
        raise TgError(status, what)
