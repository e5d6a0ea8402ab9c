"""ctypes binding of libtpmlp, with the C ABI's names (argument marshalling
only: every step of the block runs in the library's CUDA kernels).

Tensor arguments may be torch tensors (their ``data_ptr()`` is passed), raw
integer device addresses, or None for the C ABI's nullable pointers.  Status
codes other than TPMLP_OK raise :class:`TPMLPError`, except from
``tp_mlp_check`` and the plain queries, which return the code.  There is no
fallback: if the shared library is missing, loading it raises.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

# TPMLP_LIB selects another build of the library (e.g. the debug variant
# libtpmlp_checks.so); by default the in-tree libtpmlp.so.
LIB_PATH = os.environ.get("TPMLP_LIB") or _build.LIB_PATH

TPMLP_OK = 0
TPMLP_ERR_ARG = -1
TPMLP_ERR_SHAPE = -2
TPMLP_ERR_ALIGN = -3
TPMLP_ERR_ARCH = -4
TPMLP_ERR_CUDA = -5
TPMLP_ERR_TIMEOUT = -6
TPMLP_ERR_WORKSPACE = -7
TPMLP_ERR_CHECK = -8

TPMLP_BF16 = 0
TPMLP_FP32 = 1
TPMLP_GELU_ERF = 0
TPMLP_GELU_TANH = 1

# Every function the header declares, for the export check.
EXPORTED = (
    "tp_mlp_create", "tp_mlp_destroy", "tp_mlp_workspace_bytes",
    "tp_mlp_forward", "tp_mlp_backward", "tp_mlp_check",
    "tp_mlp_status_string", "tp_mlp_last_detail", "tp_mlp_launch_count",
    "tp_mlp_set_timing", "tp_mlp_timing_get", "tp_mlp_timing_reset",
    "tp_mlp_set_wait_budget", "tp_mlp_set_nvtx", "tp_mlp_set_ln_prologue",
    "tp_mlp_bias_grad_noalloc",
    "tp_mlp_set_dropout_seed",
    "tp_mlp_fp8_weights_bytes", "tp_mlp_fp8_pack_weights",
    "tp_mlp_fp8_workspace_bytes", "tp_mlp_forward_fp8", "tp_mlp_fp8_offset",
    "tp_mlp_fp8_train_workspace_bytes", "tp_mlp_forward_fp8_train",
    "tp_mlp_backward_fp8",
    "tp_mlp_probe_mma_cycles",
    "tp_mlp_probe_gelu",
    "tp_attn_create", "tp_attn_destroy", "tp_attn_workspace_bytes",
    "tp_attn_forward", "tp_attn_backward", "tp_attn_check",
    "tp_attn_launch_count", "tp_attn_set_timing", "tp_attn_timing_get",
    "tp_attn_timing_reset", "tp_attn_set_wait_budget", "tp_attn_set_nvtx",
    "tp_attn_set_ln_prologue",
    "tp_attn_workspace_offset", "tp_attn_set_rope", "tp_attn_set_qk_norm",
    "tp_attn_forward_qk", "tp_attn_backward_qk",
)

# The same for tp_rope.h, tp_grad.h and tp_fp4.h.
EXPORTED_ROPE = (
    "tp_rope_create", "tp_rope_destroy", "tp_rope_frequencies",
    "tp_rope_apply", "tp_qk_norm_forward", "tp_qk_norm_workspace_bytes",
    "tp_qk_norm_backward",
)
EXPORTED_GRAD = ("tp_grad_workspace_bytes", "tp_grad_norm", "tp_grad_clip")
EXPORTED_FP4 = (
    "tp_fp4_bytes", "tp_fp4_offset", "tp_fp4_quantize",
    "tp_fp4_colsum_workspace_bytes", "tp_fp4_quantize_both", "tp_fp4_dequantize",
    "tp_fp4_matmul", "tp_fp4_linear", "tp_fp4_check", "tp_fp4_mlp_weights_bytes",
    "tp_fp4_mlp_pack_weights", "tp_fp4_mlp_workspace_bytes",
    "tp_fp4_mlp_set_status", "tp_fp4_mlp_forward",
)

TPROPE_MAX_HEAD_DIM = 256
TPROPE_SCALE_NONE = 0
TPROPE_SCALE_LINEAR = 1
TPROPE_SCALE_NTK = 2
TPROPE_SCALE_YARN = 3
TPROPE_SCALE_CUSTOM = 4
TPQK_RMSNORM = 1
TPQK_LAYERNORM = 2

TPFP4_NV = 0
TPFP4_MX = 1
TPFP4_CODES = 0
TPFP4_SCALES = 1

TPMLP_FP8_PACK_SCALES = 0
TPMLP_FP8_PACK_AQT = 1
TPMLP_FP8_PACK_BQT = 2
TPMLP_FP8_WS_SCALES = 3
TPMLP_FP8_WS_XQ = 4
TPMLP_FP8_WS_Y = 5
TPMLP_FP8_WS_YQ = 6
TPMLP_FP8_PACK_AQ = 7
TPMLP_FP8_PACK_BQ = 8
TPMLP_FP8_WS_H = 9
TPMLP_FP8_WS_XQT = 10
TPMLP_FP8_WS_YQT = 11
TPMLP_FP8_WS_BSCALES = 12
TPMLP_FP8_WS_DZQ = 13
TPMLP_FP8_WS_DZQT = 14
TPMLP_FP8_WS_DH = 15
TPMLP_FP8_WS_DHQ = 16
TPMLP_FP8_WS_DHQT = 17

TPATTN_WS_QKV = 0
TPATTN_WS_CTX = 1
TPATTN_WS_LSE = 2
TPATTN_WS_DQKV = 3
TPATTN_WS_QKR = 4

TPMLP_NOALLOC_SCRATCH_FLOATS = 1 << 20


class tp_mlp_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("ffn", ctypes.c_int),
                ("shards", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("dtype", ctypes.c_int), ("use_layernorm", ctypes.c_int),
                ("ln_eps", ctypes.c_float), ("gelu_mode", ctypes.c_int),
                ("use_residual", ctypes.c_int), ("dropout_p", ctypes.c_float)]


class tp_attn_config(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int), ("heads", ctypes.c_int),
                ("shards", ctypes.c_int), ("max_tokens", ctypes.c_int),
                ("seq_len", ctypes.c_int), ("causal", ctypes.c_int),
                ("use_layernorm", ctypes.c_int), ("ln_eps", ctypes.c_float),
                ("use_residual", ctypes.c_int)]


class tp_rope_config(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int), ("scaling", ctypes.c_int),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_double),
                ("slow_turns", ctypes.c_double),
                ("fast_turns", ctypes.c_double),
                ("amplitude", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class tp_heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_longlong),
                ("group_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("heads", ctypes.c_int),
                ("group", ctypes.c_int)]


class tp_positions(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("is_int64", ctypes.c_int),
                ("offset", ctypes.c_longlong), ("seq_len", ctypes.c_longlong)]


class tp_qk_norm(ctypes.Structure):
    _fields_ = [("norm", ctypes.c_int), ("eps", ctypes.c_float),
                ("q_gamma", ctypes.c_void_p), ("q_beta", ctypes.c_void_p),
                ("k_gamma", ctypes.c_void_p), ("k_beta", ctypes.c_void_p)]


class tp_qk_norm_grads(ctypes.Structure):
    _fields_ = [("q_gamma", ctypes.c_void_p), ("q_beta", ctypes.c_void_p),
                ("k_gamma", ctypes.c_void_p), ("k_beta", ctypes.c_void_p)]


class tp_attn_qk(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p),
                ("positions_int64", ctypes.c_int),
                ("q_gamma", ctypes.c_void_p), ("q_beta", ctypes.c_void_p),
                ("k_gamma", ctypes.c_void_p), ("k_beta", ctypes.c_void_p)]


class tp_grad_tensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("numel", ctypes.c_longlong), ("dtype", ctypes.c_int)]


class TPMLPError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(message)
        self.code = code


_lib = None
_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load libtpmlp.so (once) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with "
            "tensor_transformer_mlp_tcgen05_gb300.build.build() (nvcc, sm_103a)")
    L = ctypes.CDLL(p)
    L.tp_mlp_create.argtypes = [ctypes.POINTER(tp_mlp_config),
                                ctypes.POINTER(_vp)]
    L.tp_mlp_create.restype = _i
    L.tp_mlp_destroy.argtypes = [_vp]
    L.tp_mlp_destroy.restype = _i
    L.tp_mlp_workspace_bytes.argtypes = [_vp, _i, _i]
    L.tp_mlp_workspace_bytes.restype = _sz
    L.tp_mlp_forward.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                 _vp, _vp, _sz, _i, _vp]
    L.tp_mlp_forward.restype = _i
    L.tp_mlp_backward.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                  _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    L.tp_mlp_backward.restype = _i
    L.tp_mlp_check.argtypes = [_vp, _vp, _vp]
    L.tp_mlp_check.restype = _i
    L.tp_mlp_status_string.argtypes = [_i]
    L.tp_mlp_status_string.restype = ctypes.c_char_p
    L.tp_mlp_last_detail.argtypes = []
    L.tp_mlp_last_detail.restype = ctypes.c_char_p
    L.tp_mlp_launch_count.argtypes = [_vp]
    L.tp_mlp_launch_count.restype = ctypes.c_longlong
    L.tp_mlp_set_timing.argtypes = [_vp, _i]
    L.tp_mlp_set_timing.restype = _i
    L.tp_mlp_timing_get.argtypes = [_vp, _i, ctypes.POINTER(ctypes.c_char_p),
                                    ctypes.POINTER(ctypes.c_longlong),
                                    ctypes.POINTER(ctypes.c_double)]
    L.tp_mlp_timing_get.restype = _i
    L.tp_mlp_timing_reset.argtypes = [_vp]
    L.tp_mlp_timing_reset.restype = _i
    L.tp_mlp_set_wait_budget.argtypes = [_vp, ctypes.c_ulonglong]
    L.tp_mlp_set_wait_budget.restype = _i
    L.tp_mlp_set_nvtx.argtypes = [_vp, _i]
    L.tp_mlp_set_nvtx.restype = _i
    L.tp_mlp_set_ln_prologue.argtypes = [_vp, _i]
    L.tp_mlp_set_ln_prologue.restype = _i
    L.tp_mlp_set_dropout_seed.argtypes = [_vp, ctypes.c_ulonglong,
                                          ctypes.c_ulonglong]
    L.tp_mlp_set_dropout_seed.restype = _i
    L.tp_mlp_bias_grad_noalloc.argtypes = [_i, _i, _i, _vp, _vp, _vp]
    L.tp_mlp_bias_grad_noalloc.restype = _i
    L.tp_mlp_fp8_weights_bytes.argtypes = [_vp]
    L.tp_mlp_fp8_weights_bytes.restype = _sz
    L.tp_mlp_fp8_pack_weights.argtypes = [_vp, _vp, _vp, _vp, _sz, _vp]
    L.tp_mlp_fp8_pack_weights.restype = _i
    L.tp_mlp_fp8_workspace_bytes.argtypes = [_vp, _i]
    L.tp_mlp_fp8_workspace_bytes.restype = _sz
    L.tp_mlp_forward_fp8.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp, _vp, _sz, _vp]
    L.tp_mlp_forward_fp8.restype = _i
    L.tp_mlp_fp8_train_workspace_bytes.argtypes = [_vp, _i]
    L.tp_mlp_fp8_train_workspace_bytes.restype = _sz
    L.tp_mlp_forward_fp8_train.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _sz, _vp]
    L.tp_mlp_forward_fp8_train.restype = _i
    L.tp_mlp_backward_fp8.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _sz,
                                      _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    L.tp_mlp_backward_fp8.restype = _i
    L.tp_mlp_fp8_offset.argtypes = [_vp, _i, _i]
    L.tp_mlp_fp8_offset.restype = ctypes.c_longlong
    L.tp_mlp_probe_mma_cycles.argtypes = [_i, _i, _i, _vp, _vp, _vp]
    L.tp_mlp_probe_mma_cycles.restype = _i
    L.tp_mlp_probe_gelu.argtypes = [_vp, _vp, _vp, _i, _i, _vp]
    L.tp_mlp_probe_gelu.restype = _i
    L.tp_attn_create.argtypes = [ctypes.POINTER(tp_attn_config),
                                 ctypes.POINTER(_vp)]
    L.tp_attn_create.restype = _i
    L.tp_attn_destroy.argtypes = [_vp]
    L.tp_attn_destroy.restype = _i
    L.tp_attn_workspace_bytes.argtypes = [_vp, _i, _i]
    L.tp_attn_workspace_bytes.restype = _sz
    L.tp_attn_workspace_offset.argtypes = [_vp, _i, _i, _i]
    L.tp_attn_workspace_offset.restype = ctypes.c_longlong
    L.tp_attn_forward.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                  _vp, _vp, _sz, _i, _vp]
    L.tp_attn_forward.restype = _i
    L.tp_attn_backward.argtypes = [_vp, _i, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                   _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
    L.tp_attn_backward.restype = _i
    L.tp_attn_check.argtypes = [_vp, _vp, _vp]
    L.tp_attn_check.restype = _i
    L.tp_attn_launch_count.argtypes = [_vp]
    L.tp_attn_launch_count.restype = ctypes.c_longlong
    L.tp_attn_set_timing.argtypes = [_vp, _i]
    L.tp_attn_set_timing.restype = _i
    L.tp_attn_timing_get.argtypes = [_vp, _i, ctypes.POINTER(ctypes.c_char_p),
                                     ctypes.POINTER(ctypes.c_longlong),
                                     ctypes.POINTER(ctypes.c_double)]
    L.tp_attn_timing_get.restype = _i
    L.tp_attn_timing_reset.argtypes = [_vp]
    L.tp_attn_timing_reset.restype = _i
    L.tp_attn_set_nvtx.argtypes = [_vp, _i]
    L.tp_attn_set_nvtx.restype = _i
    L.tp_attn_set_ln_prologue.argtypes = [_vp, _i]
    L.tp_attn_set_ln_prologue.restype = _i
    L.tp_attn_set_wait_budget.argtypes = [_vp, ctypes.c_ulonglong]
    L.tp_attn_set_wait_budget.restype = _i
    L.tp_attn_set_rope.argtypes = [_vp, ctypes.POINTER(tp_rope_config)]
    L.tp_attn_set_rope.restype = _i
    L.tp_attn_set_qk_norm.argtypes = [_vp, _i, ctypes.c_float]
    L.tp_attn_set_qk_norm.restype = _i
    L.tp_attn_forward_qk.argtypes = (L.tp_attn_forward.argtypes[:-1] +
                                     [_vp, _vp])
    L.tp_attn_forward_qk.restype = _i
    L.tp_attn_backward_qk.argtypes = (L.tp_attn_backward.argtypes[:-1] +
                                      [_vp, _vp, _vp])
    L.tp_attn_backward_qk.restype = _i
    # Structures travel as addresses: ctypes.byref of the classes above.
    L.tp_rope_create.argtypes = [ctypes.POINTER(tp_rope_config),
                                 ctypes.POINTER(_vp)]
    L.tp_rope_create.restype = _i
    L.tp_rope_destroy.argtypes = [_vp]
    L.tp_rope_destroy.restype = _i
    L.tp_rope_frequencies.argtypes = [_vp, ctypes.POINTER(ctypes.c_double),
                                      ctypes.POINTER(ctypes.c_double)]
    L.tp_rope_frequencies.restype = _i
    L.tp_rope_apply.argtypes = [_vp, _i, _i, _i] + [_vp] * 6
    L.tp_rope_apply.restype = _i
    L.tp_qk_norm_forward.argtypes = [_vp, _i, _i] + [_vp] * 7
    L.tp_qk_norm_forward.restype = _i
    L.tp_qk_norm_workspace_bytes.argtypes = [_vp]
    L.tp_qk_norm_workspace_bytes.restype = _sz
    L.tp_qk_norm_backward.argtypes = ([_vp, _i, _i] + [_vp] * 10 + [_sz, _vp])
    L.tp_qk_norm_backward.restype = _i
    L.tp_grad_workspace_bytes.argtypes = [_i]
    L.tp_grad_workspace_bytes.restype = _sz
    L.tp_grad_norm.argtypes = [_i, _vp, _vp, _vp, _sz, _vp]
    L.tp_grad_norm.restype = _i
    L.tp_grad_clip.argtypes = [_i, _vp, ctypes.c_double, ctypes.c_double, _vp,
                               _vp, _sz, _vp]
    L.tp_grad_clip.restype = _i
    ll, dbl = ctypes.c_longlong, ctypes.c_double
    L.tp_fp4_bytes.argtypes = [ll, ll, _i]
    L.tp_fp4_bytes.restype = _sz
    L.tp_fp4_offset.argtypes = [ll, ll, _i, _i]
    L.tp_fp4_offset.restype = ll
    L.tp_fp4_colsum_workspace_bytes.argtypes = [ll, ll]
    L.tp_fp4_colsum_workspace_bytes.restype = _sz
    L.tp_fp4_quantize.argtypes = [ll, ll, _i, _vp, ll, _i, _i, dbl, _vp, _vp,
                                  _sz, _vp, _vp, _sz, _vp]
    L.tp_fp4_quantize.restype = _i
    L.tp_fp4_quantize_both.argtypes = [ll, ll, _i, _vp, ll, _i, dbl, _vp, _sz, _vp,
                                       _sz, _vp, _vp, _sz, _vp]
    L.tp_fp4_quantize_both.restype = _i
    L.tp_fp4_dequantize.argtypes = [ll, ll, _i, _vp, _sz, _i, _vp, ll, _vp]
    L.tp_fp4_dequantize.restype = _i
    L.tp_fp4_matmul.argtypes = [ll, ll, ll, _i, _vp, _sz, _vp, _sz, _vp, _i,
                                _vp, ll, _vp, _vp]
    L.tp_fp4_matmul.restype = _i
    L.tp_fp4_linear.argtypes = [ll, ll, ll, _i, _vp, ll, _i, dbl, _vp, _sz,
                                _vp, _sz, _vp, _i, _vp, ll, _vp, _vp]
    L.tp_fp4_linear.restype = _i
    L.tp_fp4_check.argtypes = [_vp, _vp]
    L.tp_fp4_check.restype = _i
    L.tp_fp4_mlp_weights_bytes.argtypes = [_vp, _i]
    L.tp_fp4_mlp_weights_bytes.restype = _sz
    L.tp_fp4_mlp_pack_weights.argtypes = [_vp, _i, _vp, _vp, _vp, _sz, _vp]
    L.tp_fp4_mlp_pack_weights.restype = _i
    L.tp_fp4_mlp_workspace_bytes.argtypes = [_vp, _i, _i]
    L.tp_fp4_mlp_workspace_bytes.restype = _sz
    L.tp_fp4_mlp_set_status.argtypes = [_vp, _vp]
    L.tp_fp4_mlp_set_status.restype = _i
    L.tp_fp4_mlp_forward.argtypes = [_vp, _i, _i, _vp, _vp, _vp, _vp, _vp, _vp,
                                     dbl, dbl, _vp, _vp, _sz, _vp]
    L.tp_fp4_mlp_forward.restype = _i
    if path is None:
        _lib = L
    return L


_calls = None


def tensor_calls():
    """The module _pycall (csrc/pycall.cpp) that was built for this Python and
    torch, bound to the loaded library."""
    global _calls
    if _calls is None:
        from importlib import machinery, util
        path = _build.pycall_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with "
                "tensor_transformer_mlp_tcgen05_gb300.build.build()")
        loader = machinery.ExtensionFileLoader(f"{__package__}._pycall", path)
        m = util.module_from_spec(
            util.spec_from_file_location(loader.name, path, loader=loader))
        loader.exec_module(m)
        L = lib()
        m.bind(_check, *[
            ctypes.cast(getattr(L, n), ctypes.c_void_p).value
            for n in ("tp_rope_apply", "tp_qk_norm_forward",
                      "tp_qk_norm_workspace_bytes", "tp_qk_norm_backward",
                      "tp_grad_workspace_bytes", "tp_grad_norm",
                      "tp_grad_clip", "tp_fp4_bytes", "tp_fp4_quantize",
                      "tp_fp4_colsum_workspace_bytes", "tp_fp4_quantize_both",
                      "tp_fp4_dequantize", "tp_fp4_matmul", "tp_fp4_linear",
                      "tp_fp4_mlp_workspace_bytes", "tp_fp4_mlp_forward",
                      "tp_fp4_mlp_weights_bytes", "tp_fp4_mlp_pack_weights")])
        _calls = m
    return _calls


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s):
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def tp_mlp_status_string(code: int) -> str:
    return lib().tp_mlp_status_string(code).decode()


def tp_mlp_last_detail() -> str:
    return lib().tp_mlp_last_detail().decode()


def _check(code: int, what: str):
    if code != TPMLP_OK:
        raise TPMLPError(code, f"{what}: {tp_mlp_status_string(code)} "
                               f"[{tp_mlp_last_detail()}]")


def tp_mlp_create(config: tp_mlp_config) -> int:
    h = _vp()
    _check(lib().tp_mlp_create(ctypes.byref(config), ctypes.byref(h)),
           "tp_mlp_create")
    return h.value


def tp_mlp_destroy(handle: int) -> None:
    _check(lib().tp_mlp_destroy(handle), "tp_mlp_destroy")


def tp_mlp_workspace_bytes(handle: int, tokens: int, training: int) -> int:
    return int(lib().tp_mlp_workspace_bytes(handle, tokens, training))


def tp_mlp_forward(handle, tokens, X, A, B, bias1, bias2, ln_gamma, ln_beta,
                   Z, workspace, workspace_bytes, training, stream=None):
    _check(lib().tp_mlp_forward(
        handle, tokens, _ptr(X), _ptr(A), _ptr(B), _ptr(bias1), _ptr(bias2),
        _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(workspace),
        workspace_bytes, training, _stream(stream)), "tp_mlp_forward")


def tp_mlp_backward(handle, tokens, dZ, X, A, B, ln_gamma, workspace,
                    workspace_bytes, dX, dA, dB, dbias1, dbias2, dgamma, dbeta,
                    stream=None):
    _check(lib().tp_mlp_backward(
        handle, tokens, _ptr(dZ), _ptr(X), _ptr(A), _ptr(B), _ptr(ln_gamma),
        _ptr(workspace), workspace_bytes, _ptr(dX), _ptr(dA), _ptr(dB),
        _ptr(dbias1), _ptr(dbias2), _ptr(dgamma), _ptr(dbeta),
        _stream(stream)), "tp_mlp_backward")


def tp_mlp_check(handle, workspace, stream=None) -> int:
    return int(lib().tp_mlp_check(handle, _ptr(workspace), _stream(stream)))


def tp_mlp_launch_count(handle) -> int:
    return int(lib().tp_mlp_launch_count(handle))


def tp_mlp_set_timing(handle, enable: bool) -> None:
    _check(lib().tp_mlp_set_timing(handle, 1 if enable else 0),
           "tp_mlp_set_timing")


def tp_mlp_timing_get(handle):
    """All per-kernel totals: list of (name, launches, total_ms)."""
    out = []
    i = 0
    while True:
        name = ctypes.c_char_p()
        n = ctypes.c_longlong()
        ms = ctypes.c_double()
        rc = lib().tp_mlp_timing_get(handle, i, ctypes.byref(name),
                                     ctypes.byref(n), ctypes.byref(ms))
        if rc == TPMLP_ERR_ARG:
            break
        _check(rc, "tp_mlp_timing_get")
        out.append((name.value.decode(), n.value, ms.value))
        i += 1
    return out


def tp_mlp_timing_reset(handle) -> None:
    _check(lib().tp_mlp_timing_reset(handle), "tp_mlp_timing_reset")


def tp_mlp_set_dropout_seed(handle, seed: int, offset: int = 0) -> None:
    _check(lib().tp_mlp_set_dropout_seed(handle, seed, offset),
           "tp_mlp_set_dropout_seed")


def tp_mlp_set_wait_budget(handle, ns: int) -> None:
    _check(lib().tp_mlp_set_wait_budget(handle, ns), "tp_mlp_set_wait_budget")


def tp_mlp_set_nvtx(handle, enable: bool) -> None:
    _check(lib().tp_mlp_set_nvtx(handle, 1 if enable else 0), "tp_mlp_set_nvtx")


def tp_mlp_set_ln_prologue(handle, enable: bool) -> None:
    _check(lib().tp_mlp_set_ln_prologue(handle, 1 if enable else 0),
           "tp_mlp_set_ln_prologue")


def tp_mlp_bias_grad_noalloc(tokens, cols, dtype, grad, dbias, stream=None):
    """Column sums of a [tokens, cols] gradient into dbias, with the partial
    sums in the library's static device scratch instead of a workspace (for
    callers that cannot allocate device memory)."""
    _check(lib().tp_mlp_bias_grad_noalloc(tokens, cols, dtype, _ptr(grad),
                                          _ptr(dbias), _stream(stream)),
           "tp_mlp_bias_grad_noalloc")


# ------------------------------------------------------------------ fp8 --

def tp_mlp_fp8_weights_bytes(handle) -> int:
    return int(lib().tp_mlp_fp8_weights_bytes(handle))


def tp_mlp_fp8_pack_weights(handle, A, B, packed, packed_bytes, stream=None):
    _check(lib().tp_mlp_fp8_pack_weights(handle, _ptr(A), _ptr(B),
                                         _ptr(packed), packed_bytes,
                                         _stream(stream)),
           "tp_mlp_fp8_pack_weights")


def tp_mlp_fp8_workspace_bytes(handle, tokens: int) -> int:
    return int(lib().tp_mlp_fp8_workspace_bytes(handle, tokens))


def tp_mlp_forward_fp8(handle, tokens, X, packed, bias1, bias2, ln_gamma,
                       ln_beta, Z, workspace, workspace_bytes, stream=None):
    _check(lib().tp_mlp_forward_fp8(
        handle, tokens, _ptr(X), _ptr(packed), _ptr(bias1), _ptr(bias2),
        _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(workspace),
        workspace_bytes, _stream(stream)), "tp_mlp_forward_fp8")


def tp_mlp_fp8_train_workspace_bytes(handle, tokens: int) -> int:
    return int(lib().tp_mlp_fp8_train_workspace_bytes(handle, tokens))


def tp_mlp_forward_fp8_train(handle, tokens, X, packed, bias1, bias2,
                             ln_gamma, ln_beta, Z, workspace, workspace_bytes,
                             stream=None):
    _check(lib().tp_mlp_forward_fp8_train(
        handle, tokens, _ptr(X), _ptr(packed), _ptr(bias1), _ptr(bias2),
        _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(workspace),
        workspace_bytes, _stream(stream)), "tp_mlp_forward_fp8_train")


def tp_mlp_backward_fp8(handle, tokens, dZ, X, packed, ln_gamma, workspace,
                        workspace_bytes, dX, dA, dB, dbias1, dbias2, dgamma,
                        dbeta, stream=None):
    _check(lib().tp_mlp_backward_fp8(
        handle, tokens, _ptr(dZ), _ptr(X), _ptr(packed), _ptr(ln_gamma),
        _ptr(workspace), workspace_bytes, _ptr(dX), _ptr(dA), _ptr(dB),
        _ptr(dbias1), _ptr(dbias2), _ptr(dgamma), _ptr(dbeta),
        _stream(stream)), "tp_mlp_backward_fp8")


def tp_mlp_fp8_offset(handle, tokens: int, which: int) -> int:
    return int(lib().tp_mlp_fp8_offset(handle, tokens, which))


def tp_mlp_probe_mma_cycles(n, ctas, n_mma, cycles, status, stream=None):
    _check(lib().tp_mlp_probe_mma_cycles(n, ctas, n_mma, _ptr(cycles),
                                         _ptr(status), _stream(stream)),
           "tp_mlp_probe_mma_cycles")


def tp_mlp_probe_gelu(x, y, dy, n, mode, stream=None):
    _check(lib().tp_mlp_probe_gelu(_ptr(x), _ptr(y), _ptr(dy), int(n),
                                   int(mode), _stream(stream)),
           "tp_mlp_probe_gelu")


def device_gelu(x, mode=None):
    """(GeLU(x), GeLU'(x)) as the library's GEMM epilogues compute them, for
    a contiguous fp32 CUDA tensor x."""
    import torch
    mode = TPMLP_GELU_ERF if mode is None else mode
    x = x.contiguous()
    y = torch.empty_like(x)
    dy = torch.empty_like(x)
    tp_mlp_probe_gelu(x, y, dy, x.numel(), mode)
    return y, dy


def mma_flops_per_cycle(n=256, n_mma=4096, device=None):
    """Measured per-SM dense bf16 tensor rate (flops per SM cycle), one CTA
    per SM, averaged over the SMs."""
    import torch
    dev = torch.device(device or "cuda")
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    cycles = torch.zeros(sms, dtype=torch.int64, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    tp_mlp_probe_mma_cycles(n, sms, n_mma, cycles, status)
    torch.cuda.synchronize(dev)
    if int(status.item()) != 0:
        raise TPMLPError(int(status.item()), "mma probe: completion wait gave up")
    mean = float(cycles.double().mean().item())
    return 2.0 * 128 * n * 16 * n_mma / mean, sms


# ------------------------------------------------------------- attention --

def tp_attn_create(config: tp_attn_config) -> int:
    h = _vp()
    _check(lib().tp_attn_create(ctypes.byref(config), ctypes.byref(h)),
           "tp_attn_create")
    return h.value


def tp_attn_destroy(handle: int) -> None:
    _check(lib().tp_attn_destroy(handle), "tp_attn_destroy")


def tp_attn_workspace_bytes(handle: int, tokens: int, training: int) -> int:
    return int(lib().tp_attn_workspace_bytes(handle, tokens, training))


def tp_attn_workspace_offset(handle: int, tokens: int, training: int,
                             which: int) -> int:
    return int(lib().tp_attn_workspace_offset(handle, tokens, training, which))


def tp_attn_forward(handle, tokens, X, Wqkv, Wo, bqkv, bo, ln_gamma, ln_beta,
                    Z, workspace, workspace_bytes, training, stream=None):
    _check(lib().tp_attn_forward(
        handle, tokens, _ptr(X), _ptr(Wqkv), _ptr(Wo), _ptr(bqkv), _ptr(bo),
        _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(workspace),
        workspace_bytes, training, _stream(stream)), "tp_attn_forward")


def tp_attn_backward(handle, tokens, dZ, X, Wqkv, Wo, ln_gamma, workspace,
                     workspace_bytes, dX, dWqkv, dWo, dbqkv, dbo, dgamma,
                     dbeta, stream=None):
    _check(lib().tp_attn_backward(
        handle, tokens, _ptr(dZ), _ptr(X), _ptr(Wqkv), _ptr(Wo),
        _ptr(ln_gamma), _ptr(workspace), workspace_bytes, _ptr(dX),
        _ptr(dWqkv), _ptr(dWo), _ptr(dbqkv), _ptr(dbo), _ptr(dgamma),
        _ptr(dbeta), _stream(stream)), "tp_attn_backward")


def tp_attn_set_rope(handle, config) -> None:
    """config: a tp_rope_config, or None."""
    _check(lib().tp_attn_set_rope(
        handle, None if config is None else ctypes.byref(config)),
        "tp_attn_set_rope")


def tp_attn_set_qk_norm(handle, norm: int, eps: float) -> None:
    _check(lib().tp_attn_set_qk_norm(handle, norm, eps), "tp_attn_set_qk_norm")


def tp_attn_forward_qk(handle, tokens, X, Wqkv, Wo, bqkv, bo, ln_gamma,
                       ln_beta, Z, workspace, workspace_bytes, training, qk,
                       stream=None):
    """qk: a tp_attn_qk, or None."""
    _check(lib().tp_attn_forward_qk(
        handle, tokens, _ptr(X), _ptr(Wqkv), _ptr(Wo), _ptr(bqkv), _ptr(bo),
        _ptr(ln_gamma), _ptr(ln_beta), _ptr(Z), _ptr(workspace),
        workspace_bytes, training, _ref(qk), _stream(stream)),
        "tp_attn_forward_qk")


def tp_attn_backward_qk(handle, tokens, dZ, X, Wqkv, Wo, ln_gamma, workspace,
                        workspace_bytes, dX, dWqkv, dWo, dbqkv, dbo, dgamma,
                        dbeta, qk, qk_grads, stream=None):
    """qk: a tp_attn_qk, qk_grads: a tp_qk_norm_grads, or None."""
    _check(lib().tp_attn_backward_qk(
        handle, tokens, _ptr(dZ), _ptr(X), _ptr(Wqkv), _ptr(Wo),
        _ptr(ln_gamma), _ptr(workspace), workspace_bytes, _ptr(dX),
        _ptr(dWqkv), _ptr(dWo), _ptr(dbqkv), _ptr(dbo), _ptr(dgamma),
        _ptr(dbeta), _ref(qk), _ref(qk_grads), _stream(stream)),
        "tp_attn_backward_qk")


def tp_attn_check(handle, workspace, stream=None) -> int:
    return int(lib().tp_attn_check(handle, _ptr(workspace), _stream(stream)))


def tp_attn_launch_count(handle) -> int:
    return int(lib().tp_attn_launch_count(handle))


def tp_attn_set_timing(handle, enable: bool) -> None:
    _check(lib().tp_attn_set_timing(handle, 1 if enable else 0),
           "tp_attn_set_timing")


def tp_attn_timing_get(handle):
    """All per-kernel totals: list of (name, launches, total_ms)."""
    out = []
    i = 0
    while True:
        name = ctypes.c_char_p()
        n = ctypes.c_longlong()
        ms = ctypes.c_double()
        rc = lib().tp_attn_timing_get(handle, i, ctypes.byref(name),
                                      ctypes.byref(n), ctypes.byref(ms))
        if rc == TPMLP_ERR_ARG:
            break
        _check(rc, "tp_attn_timing_get")
        out.append((name.value.decode(), n.value, ms.value))
        i += 1
    return out


def tp_attn_timing_reset(handle) -> None:
    _check(lib().tp_attn_timing_reset(handle), "tp_attn_timing_reset")


def tp_attn_set_nvtx(handle, enable: bool) -> None:
    _check(lib().tp_attn_set_nvtx(handle, 1 if enable else 0), "tp_attn_set_nvtx")


def tp_attn_set_ln_prologue(handle, enable: bool) -> None:
    _check(lib().tp_attn_set_ln_prologue(handle, 1 if enable else 0),
           "tp_attn_set_ln_prologue")


def tp_attn_set_wait_budget(handle, ns: int) -> None:
    _check(lib().tp_attn_set_wait_budget(handle, ns), "tp_attn_set_wait_budget")


# ---------------------------------------------------------- queries, keys --

def tp_rope_create(config: tp_rope_config) -> int:
    h = _vp()
    _check(lib().tp_rope_create(ctypes.byref(config), ctypes.byref(h)),
           "tp_rope_create")
    return h.value


def tp_rope_destroy(handle: int) -> None:
    _check(lib().tp_rope_destroy(handle), "tp_rope_destroy")


def tp_rope_frequencies(handle, rot_dim: int):
    """(list of the rot_dim / 2 frequencies, amplitude)."""
    f = (ctypes.c_double * max(1, rot_dim // 2))()
    amp = ctypes.c_double()
    _check(lib().tp_rope_frequencies(handle, f, ctypes.byref(amp)),
           "tp_rope_frequencies")
    return list(f)[:rot_dim // 2], amp.value


def _ref(s):
    """The address of a structure, or None."""
    return None if s is None else ctypes.byref(s)


def tp_rope_apply(handle, tokens, dtype, inverse, q_in, q_out, k_in, k_out,
                  positions, stream=None):
    _check(lib().tp_rope_apply(
        handle, tokens, dtype, inverse, _ref(q_in), _ref(q_out), _ref(k_in),
        _ref(k_out), _ref(positions), _stream(stream)), "tp_rope_apply")


def tp_qk_norm_forward(handle, tokens, dtype, norm, q_in, q_out, k_in, k_out,
                       positions, stream=None):
    _check(lib().tp_qk_norm_forward(
        handle, tokens, dtype, _ref(norm), _ref(q_in), _ref(q_out), _ref(k_in),
        _ref(k_out), _ref(positions), _stream(stream)), "tp_qk_norm_forward")


def tp_qk_norm_workspace_bytes(handle) -> int:
    return int(lib().tp_qk_norm_workspace_bytes(handle))


def tp_qk_norm_backward(handle, tokens, dtype, norm, dq, q_in, dq_out, dk,
                        k_in, dk_out, positions, grads, workspace,
                        workspace_bytes, stream=None):
    _check(lib().tp_qk_norm_backward(
        handle, tokens, dtype, _ref(norm), _ref(dq), _ref(q_in), _ref(dq_out),
        _ref(dk), _ref(k_in), _ref(dk_out), _ref(positions), _ref(grads),
        _ptr(workspace), workspace_bytes, _stream(stream)),
        "tp_qk_norm_backward")


# ------------------------------------------------------------- gradients --

def tp_grad_workspace_bytes(count: int) -> int:
    return int(lib().tp_grad_workspace_bytes(count))


def tp_grad_norm(count, tensors, norm, workspace, workspace_bytes,
                 stream=None):
    """tensors: a ctypes array of tp_grad_tensor."""
    _check(lib().tp_grad_norm(count, tensors, _ptr(norm), _ptr(workspace),
                              workspace_bytes, _stream(stream)),
           "tp_grad_norm")


def tp_grad_clip(count, tensors, max_norm, eps, norm, workspace,
                 workspace_bytes, stream=None):
    """tensors: a ctypes array of tp_grad_tensor."""
    _check(lib().tp_grad_clip(count, tensors, max_norm, eps, _ptr(norm),
                              _ptr(workspace), workspace_bytes,
                              _stream(stream)), "tp_grad_clip")


# ------------------------------------------------------------- four bits --

def tp_fp4_bytes(rows: int, cols: int, format: int) -> int:
    return int(lib().tp_fp4_bytes(rows, cols, format))


def tp_fp4_offset(rows: int, cols: int, format: int, which: int) -> int:
    return int(lib().tp_fp4_offset(rows, cols, format, which))


def tp_fp4_colsum_workspace_bytes(rows: int, cols: int) -> int:
    return int(lib().tp_fp4_colsum_workspace_bytes(rows, cols))


def tp_fp4_quantize(rows, cols, dtype, x, row_stride, transpose, format, scale,
                    like, packed, packed_bytes, colsum=None, workspace=None,
                    workspace_bytes=0, stream=None):
    _check(lib().tp_fp4_quantize(
        rows, cols, dtype, _ptr(x), row_stride, transpose, format, scale,
        _ptr(like), _ptr(packed), packed_bytes, _ptr(colsum), _ptr(workspace),
        workspace_bytes, _stream(stream)), "tp_fp4_quantize")


def tp_fp4_quantize_both(rows, cols, dtype, x, row_stride, format, scale, packed,
                         packed_bytes, packed_t, packed_t_bytes, colsum=None,
                         workspace=None, workspace_bytes=0, stream=None):
    _check(lib().tp_fp4_quantize_both(
        rows, cols, dtype, _ptr(x), row_stride, format, scale, _ptr(packed),
        packed_bytes, _ptr(packed_t), packed_t_bytes, _ptr(colsum), _ptr(workspace),
        workspace_bytes, _stream(stream)), "tp_fp4_quantize_both")


def tp_fp4_dequantize(rows, cols, format, packed, packed_bytes, dtype, out,
                      row_stride, stream=None):
    _check(lib().tp_fp4_dequantize(
        rows, cols, format, _ptr(packed), packed_bytes, dtype, _ptr(out),
        row_stride, _stream(stream)), "tp_fp4_dequantize")


def tp_fp4_matmul(T, N, K, format, A, a_bytes, B, b_bytes, bias, dtype, C, ldc,
                  status=None, stream=None):
    _check(lib().tp_fp4_matmul(
        T, N, K, format, _ptr(A), a_bytes, _ptr(B), b_bytes, _ptr(bias), dtype,
        _ptr(C), ldc, _ptr(status), _stream(stream)), "tp_fp4_matmul")


def tp_fp4_linear(T, N, K, x_dtype, x, x_stride, format, x_scale, xq, xq_bytes,
                  W, w_bytes, bias, dtype, C, ldc, status=None, stream=None):
    _check(lib().tp_fp4_linear(
        T, N, K, x_dtype, _ptr(x), x_stride, format, x_scale, _ptr(xq), xq_bytes,
        _ptr(W), w_bytes, _ptr(bias), dtype, _ptr(C), ldc, _ptr(status),
        _stream(stream)), "tp_fp4_linear")


def tp_fp4_check(status, stream=None) -> int:
    return int(lib().tp_fp4_check(_ptr(status), _stream(stream)))


def tp_fp4_mlp_weights_bytes(handle, format: int) -> int:
    return int(lib().tp_fp4_mlp_weights_bytes(handle, format))


def tp_fp4_mlp_pack_weights(handle, format, A, B, packed, packed_bytes,
                            stream=None):
    _check(lib().tp_fp4_mlp_pack_weights(
        handle, format, _ptr(A), _ptr(B), _ptr(packed), packed_bytes,
        _stream(stream)), "tp_fp4_mlp_pack_weights")


def tp_fp4_mlp_workspace_bytes(handle, tokens: int, format: int) -> int:
    return int(lib().tp_fp4_mlp_workspace_bytes(handle, tokens, format))


def tp_fp4_mlp_set_status(handle, status):
    _check(lib().tp_fp4_mlp_set_status(handle, _ptr(status)),
           "tp_fp4_mlp_set_status")


def tp_fp4_mlp_forward(handle, tokens, format, X, packed, bias1, bias2,
                       ln_gamma, ln_beta, x_scale, y_scale, Z, workspace,
                       workspace_bytes, stream=None):
    _check(lib().tp_fp4_mlp_forward(
        handle, tokens, format, _ptr(X), _ptr(packed), _ptr(bias1),
        _ptr(bias2), _ptr(ln_gamma), _ptr(ln_beta), x_scale, y_scale, _ptr(Z),
        _ptr(workspace), workspace_bytes, _stream(stream)),
        "tp_fp4_mlp_forward")
