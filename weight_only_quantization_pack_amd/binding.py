"""ctypes binding of libawq.so (C ABI in include/awq.h).

Argument marshalling only: every step of the computation runs in the HIP
library.  Tensors are torch tensors on the GPU; the binding checks dtype,
device, shape and contiguity, allocates outputs with torch and passes raw
device pointers and the current HIP stream.  A missing library raises
``AwqError`` on first use; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "libawq.so"

_c_void_p = ctypes.c_void_p
_c_int = ctypes.c_int
_c_size_t = ctypes.c_size_t
_c_float = ctypes.c_float
_c_double = ctypes.c_double
_c_int64 = ctypes.c_int64

# (name, restype, argtypes) for every exported symbol of include/awq.h
SIGNATURES = [
    ("awq_status_str", ctypes.c_char_p, [_c_int]),
    ("awq_pack_format_version", _c_int, []),
    ("awq_packed_words_per_row", _c_size_t, [_c_int, _c_int]),
    ("awq_packed_words", _c_size_t, [_c_int, _c_int, _c_int]),
    ("awq_quantize_pack", _c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                   _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    ("awq_scale_activations", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_void_p]),
    ("awq_search_workspace_bytes", _c_size_t, [_c_int, _c_int, _c_int, _c_int]),
    ("awq_search_workspace_bytes_fused", _c_size_t, [_c_int, _c_int, _c_int, _c_int]),
    ("awq_search_scale", _c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_void_p, _c_int,
                                  _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                  _c_void_p, _c_size_t, _c_void_p]),
    ("awq_search_scale_shared", _c_int, [_c_void_p, _c_void_p, _c_int, _c_void_p, _c_int, _c_int,
                                         _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p,
                                         _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    ("awq_search_mlp_workspace_bytes", _c_size_t, [_c_int, _c_int, _c_int, _c_int, _c_int]),
    ("awq_search_scale_mlp", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int,
                                      _c_int, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p,
                                      _c_void_p, _c_void_p, _c_void_p, _c_size_t, _c_void_p]),
    ("awq_gemv", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int,
                          _c_int, _c_int, _c_int, _c_void_p]),
    ("awq_gemm", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int,
                          _c_int, _c_int, _c_int, _c_void_p]),
    ("awq_dequantize", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int,
                                _c_int, _c_void_p]),
    ("awq_gemv_scaled", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                 _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    ("awq_gemv_gate_up", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                  _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                  _c_int, _c_void_p]),
    ("awq_gemm_splitk_workspace_bytes", _c_size_t, [_c_int, _c_int, _c_int]),
    ("awq_gemm_splitk", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                                 _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    ("awq_gemm_scaled", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                 _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_size_t,
                                 _c_void_p]),
    ("awq_gemm_splitk_noalloc_max_bytes", _c_size_t, []),
    ("awq_gemm_splitk_noalloc", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                         _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    ("awq_norm_gate_residual", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                                        _c_float, _c_void_p, _c_void_p, _c_int, _c_float, _c_int, _c_int,
                                        _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    ("awq_quantize_rows", _c_int, [_c_void_p, _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p]),
    ("awq_gemm_w8a8_workspace_bytes", _c_size_t, [_c_int, _c_int, _c_int]),
    ("awq_gemm_w8a8", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                               _c_int, _c_int, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    ("awq_linear_w8a8_workspace_bytes", _c_size_t, [_c_int, _c_int, _c_int]),
    ("awq_linear_w8a8", _c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int,
                                 _c_int, _c_int, _c_void_p, _c_size_t, _c_void_p]),
    ("awq_moe_workspace_bytes", _c_size_t, [_c_int] * 5),
    ("awq_moe", _c_int, [_c_void_p] * 13 + [_c_int] * 8 + [_c_void_p, _c_size_t, _c_void_p]),
    ("awq_rope_frequencies", _c_int, [_c_int, _c_double, _c_int, _c_double, _c_double, _c_double, _c_double,
                                      _c_void_p, _c_void_p]),
    ("awq_rope", _c_int, [_c_void_p, _c_int64, _c_void_p, _c_void_p, _c_float, _c_void_p, _c_int64] + [_c_int] * 7
     + [_c_void_p]),
    ("awq_cache_append", _c_int, [_c_void_p, _c_int64] * 3 + [_c_void_p, _c_void_p, _c_float, _c_int, _c_int]
     + [_c_void_p] * 7 + [_c_int] * 9 + [_c_void_p]),
    ("awq_cache_read", _c_int, [_c_void_p] * 7 + [_c_int] * 8 + [_c_void_p] * 3),
    ("awq_cache_attention_workspace_bytes", _c_size_t, [_c_int] * 7),
    ("awq_cache_attention", _c_int, [_c_void_p, _c_int64] + [_c_void_p] * 9 + [_c_float, _c_int, _c_float]
     + [_c_int] * 11 + [_c_void_p, _c_size_t, _c_void_p]),
    ("awq_cache_fork", _c_int, [_c_void_p] * 6 + [_c_int] * 5 + [_c_void_p]),
    ("awq_cache_reserve", _c_int, [_c_void_p] * 6 + [_c_int] * 4 + [_c_void_p]),
    ("awq_cache_compact", _c_int, [_c_void_p] * 5 + [_c_int] * 4 + [_c_void_p]),
    ("awq_cache_copy_pages", _c_int, [_c_void_p, _c_void_p, _c_int, _c_int, _c_void_p, _c_void_p, _c_int, _c_int,
                                      _c_void_p]),
]

STATUS = {0: "AWQ_OK", 1: "AWQ_ERR_NULL", 2: "AWQ_ERR_SHAPE", 3: "AWQ_ERR_UNSUPPORTED",
          4: "AWQ_ERR_ALIGN", 5: "AWQ_ERR_WORKSPACE", 6: "AWQ_ERR_HIP"}

GROUP_SIZE = 128


class AwqError(RuntimeError):
    """A non-zero status from the library, or the library is missing."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


_lib = None


def library_path() -> str:
    return os.environ.get("AWQ_MI355X_LIB", os.path.join(_HERE, "lib", LIB_NAME))


def load_library():
    """Load libawq.so once; raise AwqError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise AwqError(f"HIP library not built: {path} is missing "
                       "(run __graft_entry__.build() or python -m "
                       "weight_only_quantization_pack_amd.build)")
    lib = ctypes.CDLL(path)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        name = STATUS.get(status, str(status))
        raise AwqError(f"{what} failed: {name}", status)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_ptr(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need(t, dtype, shape, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def pack_format_version() -> int:
    return int(load_library().awq_pack_format_version())


def packed_words_per_row(K: int, bits: int) -> int:
    return int(load_library().awq_packed_words_per_row(K, bits))


def packed_words(N: int, K: int, bits: int) -> int:
    """uint32 words of a packed N x K matrix (format 3: rows padded to 16)."""
    return int(load_library().awq_packed_words(N, K, bits))


def quantize_pack(W, s=None, bits: int = 4, group_size: int = GROUP_SIZE,
                  zero_point: bool = True, out=None):
    """Quantize fp16 W [N][K] (times s [K] if given) and pack.

    Returns (qweight int32 [packed_words(N, K, bits)], scales fp16
    [ceil(N/16)][G][16], zeros fp16 [ceil(N/16)][G][16]) in packed format 3.
    """
    torch = _torch()
    lib = load_library()
    N, K = W.shape
    _need(W, torch.float16, (N, K), "W")
    if s is not None:
        _need(s, torch.float32, (K,), "s")
    G = K // group_size if group_size > 0 else 0
    if out is None:
        words = int(lib.awq_packed_words(N, K, bits))
        qweight = torch.empty((words,), dtype=torch.int32, device=W.device)
        NB = (N + 15) // 16
        scales = torch.empty((NB, G, 16), dtype=torch.float16, device=W.device)
        zeros = torch.empty((NB, G, 16), dtype=torch.float16, device=W.device)
    else:
        qweight, scales, zeros = out
    st = lib.awq_quantize_pack(_ptr(W), _ptr(s), N, K, bits, group_size, int(zero_point),
                               _ptr(qweight), _ptr(scales), _ptr(zeros), _stream_ptr(W))
    _check(st, "awq_quantize_pack")
    return qweight, scales, zeros


def fake_quantize(qweight, scales, zeros, N: int, K: int, bits: int = 4, group_size: int = GROUP_SIZE,
                  out=None):
    """w_hat fp16 [N][K] = fp16((q - z) * D) from the packed layer (awq_dequantize)."""
    torch = _torch()
    lib = load_library()
    _need_layer(qweight, scales, zeros, N, K, bits, group_size)
    if out is None:
        out = torch.empty((N, K), dtype=torch.float16, device=qweight.device)
    else:
        _need(out, torch.float16, (N, K), "out")
    st = lib.awq_dequantize(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out), N, K, bits,
                            group_size, _stream_ptr(qweight))
    _check(st, "awq_dequantize")
    return out


def scale_activations(x, s, out=None):
    """x' = fp16(x / s) per input channel."""
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    _need(x, torch.float16, (M, K), "x")
    _need(s, torch.float32, (K,), "s")
    if out is None:
        out = torch.empty_like(x)
    st = lib.awq_scale_activations(_ptr(x), _ptr(s), _ptr(out), M, K, _stream_ptr(x))
    _check(st, "awq_scale_activations")
    return out


def search_workspace_bytes(T: int, N: int, K: int, n_alpha: int, fused: bool = True) -> int:
    """Workspace of the search's fused path (the default: the loss kernel forms
    W - w_hat / s in registers), or (fused=False) the larger one with which the
    search writes those differences out per chunk of alphas and runs a loss GEMM."""
    lib = load_library()
    f = lib.awq_search_workspace_bytes_fused if fused else lib.awq_search_workspace_bytes
    return int(f(T, N, K, n_alpha))


def search_scale(W, X_cal, alphas, bits: int = 4, group_size: int = GROUP_SIZE,
                 zero_point: bool = True, workspace=None, fused: bool = True):
    """AWQ alpha-grid search.  Returns (s fp32 [K], loss fp32 [n_alpha], best int32 [1]).
    The path follows the workspace size (awq_search_workspace_bytes[_fused]);
    without a workspace, the one of the path `fused` names is allocated."""
    torch = _torch()
    lib = load_library()
    N, K = W.shape
    T = X_cal.shape[0]
    _need(W, torch.float16, (N, K), "W")
    _need(X_cal, torch.float16, (T, K), "X_cal")
    a = (ctypes.c_float * len(alphas))(*[float(v) for v in alphas])
    n_alpha = len(alphas)
    need = search_workspace_bytes(T, N, K, n_alpha, fused)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=W.device)
    s_out = torch.empty(K, dtype=torch.float32, device=W.device)
    loss = torch.empty(max(n_alpha, 1), dtype=torch.float32, device=W.device)
    best = torch.empty(1, dtype=torch.int32, device=W.device)
    st = lib.awq_search_scale(_ptr(W), _ptr(X_cal), T, N, K, ctypes.cast(a, _c_void_p), n_alpha,
                              bits, group_size, int(zero_point), _ptr(s_out), _ptr(loss),
                              _ptr(best), _ptr(workspace), workspace.numel(), _stream_ptr(W))
    _check(st, "awq_search_scale")
    return s_out, loss[:n_alpha], best


def search_mlp_workspace_bytes(T: int, K: int, I: int, K_out: int, n_alpha: int) -> int:
    return int(load_library().awq_search_mlp_workspace_bytes(T, K, I, K_out, n_alpha))


def search_scale_mlp(W_gate, W_up, W_down, X_cal, alphas, bits: int = 4, group_size: int = GROUP_SIZE,
                     zero_point: bool = True, workspace=None):
    """The gate/up pair's shared scale searched on the MLP block's output
    (awq_search_scale_mlp).  W_gate, W_up fp16 [I][K], W_down fp16 [K_out][I],
    X_cal fp16 [T][K].  Returns (s fp32 [K], loss fp32 [n_alpha], best int32 [1])."""
    torch = _torch()
    lib = load_library()
    I, K = W_gate.shape
    K_out = W_down.shape[0]
    T = X_cal.shape[0]
    _need(W_gate, torch.float16, (I, K), "W_gate")
    _need(W_up, torch.float16, (I, K), "W_up")
    _need(W_down, torch.float16, (K_out, I), "W_down")
    _need(X_cal, torch.float16, (T, K), "X_cal")
    n_alpha = len(alphas)
    a = (ctypes.c_float * n_alpha)(*[float(v) for v in alphas])
    need = search_mlp_workspace_bytes(T, K, I, K_out, n_alpha)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=W_gate.device)
    s_out = torch.empty(K, dtype=torch.float32, device=W_gate.device)
    loss = torch.empty(max(n_alpha, 1), dtype=torch.float32, device=W_gate.device)
    best = torch.empty(1, dtype=torch.int32, device=W_gate.device)
    st = lib.awq_search_scale_mlp(_ptr(W_gate), _ptr(W_up), _ptr(W_down), _ptr(X_cal), T, K, I, K_out,
                                  ctypes.cast(a, _c_void_p), n_alpha, bits, group_size, int(zero_point),
                                  _ptr(s_out), _ptr(loss), _ptr(best), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(), _stream_ptr(W_gate))
    _check(st, "awq_search_scale_mlp")
    return s_out, loss[:n_alpha], best


def _need_layer(qweight, scales, zeros, N, K, bits, group_size, what=""):
    torch = _torch()
    words = int(load_library().awq_packed_words(N, K, bits))
    _need(qweight, torch.int32, (words,), what + "qweight")
    G = K // group_size if group_size > 0 else 0
    NB = (N + 15) // 16
    _need(scales, torch.float16, (NB, G, 16), what + "scales")
    _need(zeros, torch.float16, (NB, G, 16), what + "zeros")


def search_scale_shared(Ws, X_cal, alphas, bits: int = 4, group_size: int = GROUP_SIZE,
                        zero_point: bool = True, workspace=None, fused: bool = True):
    """One s for several layers reading X_cal (awq_search_scale_shared): the
    layers' rows together form the searched layer.  Returns (s fp32 [K],
    losses fp32 [n_alpha], best int32 [1]) as search_scale (workspace and
    fused as there)."""
    torch = _torch()
    lib = load_library()
    Ws = list(Ws)
    if not Ws:
        raise ValueError("Ws must hold at least one layer")
    T, K = X_cal.shape
    _need(X_cal, torch.float16, (T, K), "X_cal")
    for i, W in enumerate(Ws):
        _need(W, torch.float16, (W.shape[0], K), f"Ws[{i}]")
    n = len(Ws)
    ptrs = (_c_void_p * n)(*[W.data_ptr() for W in Ws])
    Ns = (ctypes.c_int * n)(*[int(W.shape[0]) for W in Ws])
    a = (ctypes.c_float * len(alphas))(*[float(v) for v in alphas])
    n_alpha = len(alphas)
    need = search_workspace_bytes(T, sum(Ns), K, n_alpha, fused)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=X_cal.device)
    s_out = torch.empty(K, dtype=torch.float32, device=X_cal.device)
    loss = torch.empty(max(n_alpha, 1), dtype=torch.float32, device=X_cal.device)
    best = torch.empty(1, dtype=torch.int32, device=X_cal.device)
    st = lib.awq_search_scale_shared(ctypes.cast(ptrs, _c_void_p), ctypes.cast(Ns, _c_void_p), n,
                                     _ptr(X_cal), T, K, ctypes.cast(a, _c_void_p), n_alpha, bits,
                                     group_size, int(zero_point), _ptr(s_out), _ptr(loss), _ptr(best),
                                     _ptr(workspace), workspace.numel(), _stream_ptr(X_cal))
    _check(st, "awq_search_scale_shared")
    return s_out, loss[:n_alpha], best


def _matmul(fn_name, x, qweight, scales, zeros, N, bits, group_size, out, workspace=None):
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    _need(x, torch.float16, (M, K), "x")
    _need_layer(qweight, scales, zeros, N, K, bits, group_size)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=x.device)
    else:
        _need(out, torch.float16, (M, N), "out")
    if fn_name == "awq_gemm_splitk":
        st = lib.awq_gemm_splitk(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out),
                                 M, N, K, bits, group_size, _ptr(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                 _stream_ptr(x))
    else:
        st = getattr(lib, fn_name)(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out),
                                   M, N, K, bits, group_size, _stream_ptr(x))
    _check(st, fn_name)
    return out


def _gemm_scaled(x, inv_s, qweight, scales, zeros, N, bits, group_size, out, split_k, workspace):
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    _need(x, torch.float16, (M, K), "x")
    _need(inv_s, torch.float32, (K,), "inv_s")
    _need_layer(qweight, scales, zeros, N, K, bits, group_size)
    out = _out(out, M, N, x.device)
    need = gemm_splitk_workspace_bytes(M, N, K) if split_k else 0
    if need == 0:
        workspace = None
    elif workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    st = lib.awq_gemm_scaled(_ptr(x), _ptr(inv_s), _ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out),
                             M, N, K, bits, group_size, _ptr(workspace),
                             0 if workspace is None else workspace.numel() * workspace.element_size(),
                             _stream_ptr(x))
    _check(st, "awq_gemm_scaled")
    return out


def gemm_splitk_noalloc(x, qweight, scales, zeros, N: int, bits: int = 4,
                        group_size: int = GROUP_SIZE, out=None):
    """awq_gemm_splitk_noalloc: the split-K prefill product with its fp32
    partials in the library's fixed per-GPU array (the call allocates no device
    memory; `out` is allocated here only when not given).  Calls overlapping on
    one GPU race on that array."""
    return _matmul("awq_gemm_splitk_noalloc", x, qweight, scales, zeros, N, bits, group_size, out)


def gemm_splitk_noalloc_max_bytes() -> int:
    """Size of the fixed partial-sum array of awq_gemm_splitk_noalloc."""
    return int(load_library().awq_gemm_splitk_noalloc_max_bytes())


def gemv(x, qweight, scales, zeros, N: int, bits: int = 4, group_size: int = GROUP_SIZE, out=None,
         inv_s=None):
    """Decode product y = x . w_hat^T for 1 <= M <= 16 rows of x; N output columns.

    inv_s (fp32 [K] device tensor, the reciprocal of the AWQ scale) folds the
    activation scale into the load: y = fp16(x * inv_s) . w_hat^T through
    awq_gemv_scaled."""
    if inv_s is None:
        return _matmul("awq_gemv", x, qweight, scales, zeros, N, bits, group_size, out)
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    _need(x, torch.float16, (M, K), "x")
    _need(inv_s, torch.float32, (K,), "inv_s")
    _need_layer(qweight, scales, zeros, N, K, bits, group_size)
    out = _out(out, M, N, x.device)
    st = lib.awq_gemv_scaled(_ptr(x), _ptr(inv_s), _ptr(qweight), _ptr(scales), _ptr(zeros),
                             _ptr(out), M, N, K, bits, group_size, _stream_ptr(x))
    _check(st, "awq_gemv_scaled")
    return out


def gemv_gate_up(x, gate, up, N: int, bits: int = 4, group_size: int = GROUP_SIZE, inv_s=None,
                 out=None):
    """Gate/up half of a fused MLP in one launch: h = SiLU(x' . w_gate^T) * (x' . w_up^T).

    gate, up: (qweight, scales, zeros) of two N x K layers; x' = fp16(x * inv_s)
    when inv_s (fp32 [K]) is given, else x.  h fp16 [M][N] (awq_gemv_gate_up)."""
    torch = _torch()
    lib = load_library()
    M, K = x.shape
    _need(x, torch.float16, (M, K), "x")
    if inv_s is not None:
        _need(inv_s, torch.float32, (K,), "inv_s")
    _need_layer(*gate, N, K, bits, group_size, "gate ")
    _need_layer(*up, N, K, bits, group_size, "up ")
    out = _out(out, M, N, x.device)
    st = lib.awq_gemv_gate_up(_ptr(x), _ptr(inv_s), _ptr(gate[0]), _ptr(gate[1]), _ptr(gate[2]),
                              _ptr(up[0]), _ptr(up[1]), _ptr(up[2]), _ptr(out), M, N, K, bits,
                              group_size, _stream_ptr(x))
    _check(st, "awq_gemv_gate_up")
    return out


def _out(out, M, N, device):
    torch = _torch()
    if out is None:
        return torch.empty((M, N), dtype=torch.float16, device=device)
    _need(out, torch.float16, (M, N), "out")
    return out


def gemm_splitk_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes awq_gemm_splitk needs for this shape (0: no split)."""
    return int(load_library().awq_gemm_splitk_workspace_bytes(M, N, K))


def gemm(x, qweight, scales, zeros, N: int, bits: int = 4, group_size: int = GROUP_SIZE, out=None,
         split_k: bool = True, workspace=None, inv_s=None):
    """Prefill product y = x . w_hat^T for any M >= 1 rows of x (bits 4 or 3); N output columns.

    With split_k (default) shapes with few output tiles run through
    awq_gemm_splitk; its fp32 workspace is `workspace` (a device tensor of at
    least gemm_splitk_workspace_bytes bytes) or allocated here.  split_k=False
    always calls awq_gemm.  inv_s (fp32 [K] device tensor, the reciprocal of
    the AWQ scale) folds the activation scale into the product through
    awq_gemm_scaled: y = fp16(x * inv_s) . w_hat^T.
    """
    if inv_s is not None:
        return _gemm_scaled(x, inv_s, qweight, scales, zeros, N, bits, group_size, out, split_k,
                            workspace)
    if split_k and x.dim() == 2:
        need = gemm_splitk_workspace_bytes(x.shape[0], N, x.shape[1])
        if need > 0:
            if workspace is None:
                workspace = _torch().empty(need, dtype=_torch().uint8, device=x.device)
            return _matmul("awq_gemm_splitk", x, qweight, scales, zeros, N, bits, group_size, out,
                           workspace)
    return _matmul("awq_gemm", x, qweight, scales, zeros, N, bits, group_size, out)


# ---------------------------------------------------------------------------
# operators beside the packed products in a decoder block
#
# A decode step calls these per token, so their checks are kept short: _arg
# accepts a right argument with one chain of comparisons and gives its address;
# only a wrong one goes on to the checks that name what is wrong with it.
# ---------------------------------------------------------------------------
NORM_KINDS = {"rms": 0, "layer": 1}


def _arg(t, dtype, shape, device, name):
    """The address of t, a contiguous tensor of this type and shape on GPU
    `device` (its index)."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _need(t, dtype, shape, name)
    raise ValueError(f"{name} must be on GPU {device}, got {t.device}")


def _optional(t, dtype, shape, device, name):
    """_arg, or NULL for None."""
    return None if t is None else _arg(t, dtype, shape, device, name)


def _dtype_code(dtype, name):
    """awq_dtype of a 16-bit torch dtype."""
    torch = _torch()
    if dtype is torch.float16:
        return 0
    if dtype is torch.bfloat16:
        return 1
    raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {dtype}")


def _rows2d(t, name):
    """(shape, GPU index) of a 2-dimensional GPU tensor."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{name} must have 2 dimensions, got shape {tuple(t.shape)}")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on the GPU")
    return t.shape, device


def _raw_stream(device):
    """The current stream of GPU `device` as an integer handle."""
    return _torch()._C._cuda_getCurrentRawStream(device)


def _workspace(workspace, need, like):
    """(tensor kept alive, address, bytes) of a call's scratch memory."""
    if need == 0:
        return None, None, 0
    if workspace is None:
        workspace = like.new_empty(need, dtype=_torch().uint8)
    elif workspace.get_device() != like.get_device() or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {like.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def norm_gate_residual(block, residual, pre_weight, post_weight=None, gate=None, residual_scale: float = 1.0,
                       kind: str = "rms", pre_bias=None, post_bias=None, eps: float = 1e-6,
                       quantize: bool = False, out=None):
    """Norms before and after a block with its gate and the scaled residual
    (awq_norm_gate_residual), one launch:

        t  = post(block)                            (block itself without post_weight)
        r' = residual_scale * residual + gate * t
        h  = pre(r')

    block, residual: fp16 or bf16 [T][H], contiguous, H a multiple of 8, at
    most 32768; weights and biases [H] and gate [H] or [B][H] (B divides T: one
    gate row for each T / B rows) of the same type.  kind "rms" or "layer" for
    both norms.  Returns (r', h), or with quantize=True (r', codes int8 [T][H],
    scales fp32 [T]) for gemm_w8a8.  out: the tensors to write, in that order;
    the first may be `residual`.
    """
    torch = _torch()
    lib = load_library()
    shape, dev = _rows2d(block, "block")
    T, H = shape
    dtype = block.dtype
    code = _dtype_code(dtype, "block")
    row = shape[1:]
    residual_at = _arg(residual, dtype, shape, dev, "residual")
    if post_bias is not None and post_weight is None:
        raise ValueError("post_bias needs post_weight")
    if kind not in NORM_KINDS:
        raise ValueError(f"kind must be one of {sorted(NORM_KINDS)}, got {kind!r}")
    gate_rows, gate_shape = 0, row
    if gate is not None:
        gate_rows = 1
        if gate.dim() != 1:
            gate_rows = gate.shape[0]
            gate_shape = (gate_rows, H)
            if gate_rows == 0 or T % gate_rows:
                raise ValueError(f"gate rows ({gate_rows}) must divide the rows of block ({T})")
    scales = scales_at = None
    if out is None:
        r = torch.empty_like(residual)
        if quantize:
            h = block.new_empty(shape, dtype=torch.int8)
            scales = block.new_empty(T, dtype=torch.float32)
            scales_at = scales.data_ptr()
        else:
            h = torch.empty_like(residual)
        r_at, h_at = r.data_ptr(), h.data_ptr()
    else:
        if quantize:
            r, h, scales = out
            scales_at = _arg(scales, torch.float32, shape[:1], dev, "out[2]")
        else:
            r, h = out
        r_at = _arg(r, dtype, shape, dev, "out[0]")
        h_at = _arg(h, torch.int8 if quantize else dtype, shape, dev, "out[1]")
    st = lib.awq_norm_gate_residual(
        _arg(block, dtype, shape, dev, "block"), residual_at,
        _optional(post_weight, dtype, row, dev, "post_weight"), _optional(post_bias, dtype, row, dev, "post_bias"),
        _optional(gate, dtype, gate_shape, dev, "gate"), gate_rows, residual_scale,
        _arg(pre_weight, dtype, row, dev, "pre_weight"), _optional(pre_bias, dtype, row, dev, "pre_bias"),
        NORM_KINDS[kind], eps, T, H, code, r_at, h_at, scales_at, _raw_stream(dev))
    _check(st, "awq_norm_gate_residual")
    return (r, h, scales) if quantize else (r, h)


def quantize_rows(x, out=None):
    """8-bit codes with one scale per row (awq_quantize_rows): (int8 [M][K],
    fp32 [M]) with scale = max|row| / 127 and q = rint(127 x / max|row|).  Rows
    are tokens of activations or output channels of weights; x fp16 or bf16, K
    a multiple of 16."""
    torch = _torch()
    lib = load_library()
    shape, dev = _rows2d(x, "x")
    code = _dtype_code(x.dtype, "x")
    if out is None:
        q = x.new_empty(shape, dtype=torch.int8)
        scales = x.new_empty(shape[0], dtype=torch.float32)
    else:
        q, scales = out
    st = lib.awq_quantize_rows(_arg(x, x.dtype, shape, dev, "x"), shape[0], shape[1], code,
                               _arg(q, torch.int8, shape, dev, "out[0]"),
                               _arg(scales, torch.float32, shape[:1], dev, "out[1]"), _raw_stream(dev))
    _check(st, "awq_quantize_rows")
    return q, scales


def gemm_w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes of gemm_w8a8 (0: none) on the current device."""
    return int(load_library().awq_gemm_w8a8_workspace_bytes(M, N, K))


def linear_w8a8_workspace_bytes(M: int, N: int, K: int) -> int:
    """Workspace bytes of linear_w8a8 (0: none) on the current device."""
    return int(load_library().awq_linear_w8a8_workspace_bytes(M, N, K))


def gemm_w8a8(q, q_scales, weight, weight_scales, bias=None, dtype=None, out=None, workspace=None):
    """y = q_scales[m] * weight_scales[n] * (q . weight^T) + bias in 8-bit
    integers (awq_gemm_w8a8): q int8 [M][K] and weight int8 [N][K] with their
    fp32 scales, as quantize_rows gives them; bias fp32 [N].  y is fp16 or bf16
    [M][N]: dtype (default torch.float16), or out's."""
    torch = _torch()
    lib = load_library()
    (M, K), dev = _rows2d(q, "q")
    N = _rows2d(weight, "weight")[0][0]
    if dtype is None:
        dtype = torch.float16 if out is None else out.dtype
    code = _dtype_code(dtype, "dtype")
    if out is None:
        out = q.new_empty((M, N), dtype=dtype)
        out_at = out.data_ptr()
    else:
        out_at = _arg(out, dtype, (M, N), dev, "out")
    keep, ws, ws_bytes = _workspace(workspace, lib.awq_gemm_w8a8_workspace_bytes(M, N, K), q)
    st = lib.awq_gemm_w8a8(_arg(q, torch.int8, (M, K), dev, "q"), _arg(q_scales, torch.float32, (M,), dev, "q_scales"),
                           _arg(weight, torch.int8, (N, K), dev, "weight"),
                           _arg(weight_scales, torch.float32, (N,), dev, "weight_scales"),
                           _optional(bias, torch.float32, (N,), dev, "bias"), out_at,
                           M, N, K, code, ws, ws_bytes, _raw_stream(dev))
    _check(st, "awq_gemm_w8a8")
    return out


def linear_w8a8(x, weight, weight_scales, bias=None, out=None, workspace=None):
    """gemm_w8a8 of the quantized rows of x (awq_linear_w8a8): x fp16 or bf16
    [M][K], y of the same type.  One call: short decode rows are quantized
    inside the product's launch."""
    torch = _torch()
    lib = load_library()
    (M, K), dev = _rows2d(x, "x")
    dtype = x.dtype
    code = _dtype_code(dtype, "x")
    N = _rows2d(weight, "weight")[0][0]
    if out is None:
        out = x.new_empty((M, N))
        out_at = out.data_ptr()
    else:
        out_at = _arg(out, dtype, (M, N), dev, "out")
    keep, ws, ws_bytes = _workspace(workspace, lib.awq_linear_w8a8_workspace_bytes(M, N, K), x)
    st = lib.awq_linear_w8a8(_arg(x, dtype, (M, K), dev, "x"), _arg(weight, torch.int8, (N, K), dev, "weight"),
                             _arg(weight_scales, torch.float32, (N,), dev, "weight_scales"),
                             _optional(bias, torch.float32, (N,), dev, "bias"), out_at,
                             M, N, K, code, ws, ws_bytes, _raw_stream(dev))
    _check(st, "awq_linear_w8a8")
    return out


def moe_workspace_bytes(M: int, K: int, I: int, E: int, top_k: int) -> int:
    """Workspace bytes of moe for M tokens of K channels, E experts of I channels."""
    return int(load_library().awq_moe_workspace_bytes(M, K, I, E, top_k))


def moe(x, router, gate, up, down, inter: int, top_k: int, bits: int = 4, group_size: int = GROUP_SIZE,
        renormalize: bool = True, inv_s=None, out=None, workspace=None):
    """A whole mixture-of-experts layer for a few tokens over packed experts
    (awq_moe): y[m] = sum_j p_j down_j(SiLU(gate_j x') * up_j x') over the top_k
    experts of x . router^T.

    x fp16 [M][K], M <= 64; router fp16 [E][K]; gate, up: (qweight int32
    [E][packed_words(inter, K, bits)], scales, zeros fp16
    [E][ceil(inter / 16)][K / group_size][16]) -- the E layers of quantize_pack,
    stacked; down the same of K x inter layers.  p = softmax over the chosen
    experts (renormalize) or over all.  inv_s (fp32 [K], the reciprocal of the
    AWQ scale of gate and up): x' = x * inv_s; the router reads x.  A token whose
    x' or SiLU(gate) * up passes the fp16 maximum (65504) has a row of NaN.
    """
    torch = _torch()
    lib = load_library()
    shape, dev = _rows2d(x, "x")
    M, K = shape
    E = _rows2d(router, "router")[0][0]
    half, I = torch.float16, inter
    if bits not in (3, 4) or group_size not in (64, 128):
        _check(3, "awq_moe")                                 # AWQ_ERR_UNSUPPORTED
    x_at = _arg(x, half, shape, dev, "x")
    if out is None:
        out = torch.empty_like(x)
        out_at = out.data_ptr()
    else:
        out_at = _arg(out, half, shape, dev, "out")
    keep, ws, ws_bytes = _workspace(workspace, lib.awq_moe_workspace_bytes(M, K, I, E, top_k), x)
    args = [x_at, _optional(inv_s, torch.float32, shape[1:], dev, "inv_s"),
            _arg(router, half, (E, K), dev, "router")]
    for layer, n, k, name in ((gate, I, K, "gate"), (up, I, K, "up"), (down, K, I, "down")):
        qweight, scales, zeros = layer
        blocks = (n + 15) // 16
        params = (E, blocks, k // group_size, 16)
        args += [_arg(qweight, torch.int32, (E, blocks * 16 * (k // 32 * bits)), dev, name + " qweight"),
                 _arg(scales, half, params, dev, name + " scales"), _arg(zeros, half, params, dev, name + " zeros")]
    st = lib.awq_moe(*args, out_at, M, K, I, E, top_k, bits, group_size,
                     int(renormalize), ws, ws_bytes, _raw_stream(dev))
    _check(st, "awq_moe")
    return out


# ---------------------------------------------------------------------------
# rotary positions and the paged 8-bit cache
#
# A layer's cache is (k_codes int8 [pages][kv][page][dim], k_scales fp32
# [pages][kv], v_codes, v_scales); a call's sequences are tables int32 [B][W],
# lens int32 [B] and starts int32 [B + 1] (or None: one row each), as in awq.h.
# ---------------------------------------------------------------------------
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
ROPE_SCALINGS = {None: 0, "linear": 1, "base": 2, "yarn": 3, "bands": 4, "yarn_rounded": 3 | 16}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling=None, factor: float = 1.0,
                     original_length: float = 0.0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """(inv_freq fp32 [rotary_dim / 2] on `device`, magnitude) of a rotary
    embedding (awq_rope_frequencies): scaling None, "linear", "base" (a larger
    base), "yarn_rounded", "yarn" or "bands" (frequencies that turn `high` times or more in
    original_length are kept, those that turn `low` times or fewer are divided by
    factor; a ramp over the channels, or over the number of turns).  The channels'
    ramp begins and ends at whole channels in "yarn_rounded", as in YaRN's released
    code: it is the one for a checkpoint that does not say otherwise; "yarn" does
    not round its ends."""
    torch = _torch()
    if scaling not in ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALINGS)}, got {scaling!r}")
    inv_freq, magnitude = (_c_float * max(rotary_dim // 2, 1))(), _c_float()
    st = load_library().awq_rope_frequencies(rotary_dim, base, ROPE_SCALINGS[scaling], factor, original_length, low,
                                             high, inv_freq, ctypes.byref(magnitude))
    _check(st, "awq_rope_frequencies")
    return torch.tensor(list(inv_freq), dtype=torch.float32).to(device), float(magnitude.value)


def _heads3d(t, dtype, device, name):
    """(address, row stride) of a GPU tensor [T][heads][dim] of dense rows."""
    try:
        if t.dtype is dtype and t.dim() == 3 and t.get_device() == device >= 0:
            T, h, d = t.shape
            row, head, channel = t.stride()
            if (channel == 1 or d == 1) and (head == d or h == 1):
                return t.data_ptr(), row if T > 1 else -(-h * d // 8) * 8
    except AttributeError:
        pass
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3:
        raise ValueError(f"{name} must have 3 dimensions [rows][heads][channels], got shape {tuple(t.shape)}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name} must be on the GPU" + (f" {device}, got {t.device}" if device >= 0 else ""))
    raise ValueError(f"{name}'s rows must be dense (heads x channels), got strides {t.stride()}")


def _gpu_of(t, name):
    """The index of the GPU that t is on."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    device = t.get_device()
    if device < 0:
        raise ValueError(f"{name} must be on the GPU")
    return device


def _layout(layout):
    if layout not in ROPE_LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(ROPE_LAYOUTS)}, got {layout!r}")
    return ROPE_LAYOUTS[layout]


def rope(x, positions, inv_freq, layout: str = "half", magnitude: float = 1.0, inverse: bool = False, out=None):
    """Rows turned by their positions (awq_rope): x fp16 or bf16 [T][heads][dim]
    (dense rows, which may be apart: a part of a fused projection), positions
    int32 [T], inv_freq fp32 [rotary / 2] as rope_frequencies gives it; the first
    rotary channels of each head are turned.  inverse turns back, which is also
    the gradient.  out may be x."""
    torch = _torch()
    dev = _gpu_of(x, "x")
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return rope(x, positions, inv_freq, layout, magnitude, inverse, out)
    lib = load_library()
    dtype = x.dtype
    code = _dtype_code(dtype, "x")
    x_at, x_stride = _heads3d(x, dtype, dev, "x")
    T, heads, dim = x.shape
    if out is None:
        out = x.new_empty((T, heads, dim))
        out_at, out_stride = out.data_ptr(), heads * dim
    else:
        if out.shape != x.shape:
            raise ValueError(f"out must have shape {tuple(x.shape)}, got {tuple(out.shape)}")
        out_at, out_stride = _heads3d(out, dtype, dev, "out")
    n = inv_freq.numel()
    st = lib.awq_rope(x_at, x_stride, _arg(positions, torch.int32, (T,), dev, "positions"),
                      _arg(inv_freq, torch.float32, (n,), dev, "inv_freq"), magnitude, out_at, out_stride, T, heads,
                      dim, 2 * n, _layout(layout), int(inverse), code, _raw_stream(dev))
    if st:
        _check(st, "awq_rope")
    return out


def empty_cache(pages: int, kv_heads: int, page_size: int, head_dim: int, layers=None, device="cuda"):
    """(k_codes, k_scales, v_codes, v_scales) of zeros, with a leading dimension of
    `layers` if given (a layer's cache is then each tensor's slice of it)."""
    torch = _torch()
    lead = (pages,) if layers is None else (layers, pages)
    return tuple(t for _ in range(2) for t in (
        torch.zeros((*lead, kv_heads, page_size, head_dim), dtype=torch.int8, device=device),
        torch.zeros((*lead, kv_heads), dtype=torch.float32, device=device)))


def _cache_args(cache, device):
    """(addresses, (pages, kv heads, page size, head dim)) of a layer's cache on GPU `device`."""
    torch = _torch()
    i8, f32 = torch.int8, torch.float32
    k, ks, v, vs = cache
    try:
        shape, few = k.shape, ks.shape
        pages, kv, page, dim = shape
        if (few == (pages, kv) and v.shape == shape and vs.shape == few and k.dtype is i8 and v.dtype is i8
                and ks.dtype is f32 and vs.dtype is f32 and k.get_device() == device and ks.get_device() == device
                and v.get_device() == device and vs.get_device() == device and k.is_contiguous()
                and ks.is_contiguous() and v.is_contiguous() and vs.is_contiguous()):
            return (k.data_ptr(), ks.data_ptr(), v.data_ptr(), vs.data_ptr()), shape
    except (AttributeError, ValueError):
        pass
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("cache must be (k_codes [pages][kv][page][dim], k_scales [pages][kv], v_codes, v_scales)")
    shape = k.shape
    few = shape[:2]
    return (_arg(k, i8, shape, device, "k_codes"), _arg(ks, f32, few, device, "k_scales"),
            _arg(v, i8, shape, device, "v_codes"), _arg(vs, f32, few, device, "v_scales")), shape


def _sequence_args(tables, lens, starts, device):
    """(addresses, B, W) of a call's sequences."""
    torch = _torch()
    i32 = torch.int32
    try:
        B, W = tables.shape
        if (tables.dtype is i32 and lens.dtype is i32 and lens.shape == (B,) and tables.get_device() == device
                and lens.get_device() == device and tables.is_contiguous() and lens.is_contiguous()):
            return (tables.data_ptr(), lens.data_ptr(), None if starts is None else
                    _arg(starts, i32, (B + 1,), device, "starts")), B, W
    except (AttributeError, ValueError):
        pass                                     # said below, argument by argument
    if not isinstance(tables, torch.Tensor) or tables.dim() != 2:
        raise ValueError("tables must be an int32 tensor [sequences][pages]")
    B, W = tables.shape
    return (_arg(tables, i32, (B, W), device, "tables"), _arg(lens, i32, (B,), device, "lens"),
            _optional(starts, i32, (B + 1,), device, "starts")), B, W


def cache_append(q, k, v, cache, tables, lens, starts=None, inv_freq=None, layout: str = "half",
                 magnitude: float = 1.0, out=None):
    """New tokens into the cache (awq_cache_append): k, v fp16 or bf16
    [T][kv][dim] become codes with one scale for each page and head, k turned by
    its place in the sequence if inv_freq is given, as is q [T][heads][dim] (or
    None).  lens counts the new tokens.  Returns the turned q (`out` if given)."""
    torch = _torch()
    dev = _gpu_of(k, "k")
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_append(q, k, v, cache, tables, lens, starts, inv_freq, layout, magnitude, out)
    lib = load_library()
    dtype = k.dtype
    code = _dtype_code(dtype, "k")
    k_at, k_stride = _heads3d(k, dtype, dev, "k")
    T, kv, dim = k.shape
    v_at, v_stride = _heads3d(v, dtype, dev, "v")
    if v.shape != k.shape:
        raise ValueError(f"v must have shape {tuple(k.shape)}, got {tuple(v.shape)}")
    codes, (pages, c_kv, page, c_dim) = _cache_args(cache, dev)
    if (c_kv, c_dim) != (kv, dim):
        raise ValueError(f"k has {kv} heads of {dim}, the cache {c_kv} of {c_dim}")
    seqs, B, W = _sequence_args(tables, lens, starts, dev)
    q_at = out_at = None
    q_stride = heads = 0
    if q is not None:
        q_at, q_stride = _heads3d(q, dtype, dev, "q")
        heads = q.shape[1]
        if q.shape[0] != T or q.shape[2] != dim:
            raise ValueError(f"q must have shape ({T}, heads, {dim}), got {tuple(q.shape)}")
        if out is None:
            out = q.new_empty((T, heads, dim))
            out_at = out.data_ptr()
        else:
            out_at = _arg(out, dtype, (T, heads, dim), dev, "out")
    freq_at, rotary = None, 0
    if inv_freq is not None:
        rotary = 2 * inv_freq.numel()
        freq_at = _arg(inv_freq, torch.float32, (rotary // 2,), dev, "inv_freq")
    st = lib.awq_cache_append(q_at, q_stride, k_at, k_stride, v_at, v_stride, out_at, freq_at, magnitude, rotary,
                              _layout(layout), *codes, *seqs, T, B, W, heads, kv, dim, pages, page, code,
                              _raw_stream(dev))
    if st:
        _check(st, "awq_cache_append")
    return out if q is not None else None


def cache_read(cache, tables, lens, starts=None, tokens=None, dtype=None, out=None):
    """The last starts[b + 1] - starts[b] tokens of each sequence as the values the
    cache holds (awq_cache_read): (k, v) of `dtype` (default torch.float16)
    [tokens][kv][dim].  tokens: the rows of the call (default: one a sequence)."""
    torch = _torch()
    dev = _gpu_of(tables, "tables")
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_read(cache, tables, lens, starts, tokens, dtype, out)
    lib = load_library()
    codes, (pages, kv, page, dim) = _cache_args(cache, dev)
    seqs, B, W = _sequence_args(tables, lens, starts, dev)
    if tokens is None:
        if starts is not None:
            raise ValueError("starts needs tokens, the number of rows")
        tokens = B
    if out is None:
        dtype = dtype or torch.float16
        code = _dtype_code(dtype, "dtype")
        shape = (tokens, kv, dim)
        k, v = cache[0].new_empty(shape, dtype=dtype), cache[0].new_empty(shape, dtype=dtype)
        k_at, v_at = k.data_ptr(), v.data_ptr()
    else:
        k, v = out
        dtype = k.dtype
        code = _dtype_code(dtype, "out[0]")
        k_at = _arg(k, dtype, (tokens, kv, dim), dev, "out[0]")
        v_at = _arg(v, dtype, (tokens, kv, dim), dev, "out[1]")
    st = lib.awq_cache_read(*codes, *seqs, tokens, B, W, kv, dim, pages, page, code, k_at, v_at, _raw_stream(dev))
    if st:
        _check(st, "awq_cache_read")
    return k, v


def cache_attention_workspace_bytes(tokens: int, sequences: int, heads: int, kv_heads: int, head_dim: int,
                                    max_new: int, max_len: int) -> int:
    """Workspace bytes of cache_attention (0: none) on the current device."""
    return int(load_library().awq_cache_attention_workspace_bytes(tokens, sequences, heads, kv_heads, head_dim,
                                                                  max_new, max_len))


def cache_attention(q, cache, tables, lens, starts=None, scale=None, window: int = 0, softcap: float = 0.0,
                    max_new=None, max_len=None, lse=None, out=None, workspace=None):
    """Attention of each sequence's last tokens over its cached keys and values
    (awq_cache_attention): q fp16 or bf16 [T][heads][dim], causal, within `window`
    keys (0: all), scores scale * q.k (default dim^-1/2) capped by softcap (0:
    not).  max_new, max_len: the most rows and tokens of a sequence, if known (they
    choose the kernel; default T, or 1 without starts, and the table's).  Give max_new
    with starts: 63 single rows over up to 8000 tokens take 107 us with max_new=1 and 432
    as what could be one prompt of 63.  lse: fp32 [T][heads] to write, or None.  Returns out, [T][heads][dim] like q."""
    torch = _torch()
    dev = _gpu_of(q, "q")
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_attention(q, cache, tables, lens, starts, scale, window, softcap, max_new, max_len, lse, out,
                                   workspace)
    lib = load_library()
    dtype = q.dtype
    code = _dtype_code(dtype, "q")
    q_at, q_stride = _heads3d(q, dtype, dev, "q")
    T, heads, dim = q.shape
    codes, (pages, kv, page, c_dim) = _cache_args(cache, dev)
    if c_dim != dim:
        raise ValueError(f"q has heads of {dim} channels, the cache of {c_dim}")
    seqs, B, W = _sequence_args(tables, lens, starts, dev)
    if max_new is None:
        max_new = max(T, 1) if starts is not None else 1
    if max_len is None:
        max_len = min(W * page, 0x7FFFFFFF)
    if out is None:
        out = q.new_empty((T, heads, dim))
        out_at = out.data_ptr()
    else:
        out_at = _arg(out, dtype, (T, heads, dim), dev, "out")
    lse_at = _optional(lse, torch.float32, (T, heads), dev, "lse")
    need = lib.awq_cache_attention_workspace_bytes(T, B, heads, kv, dim, max_new, max_len)
    keep, ws, ws_bytes = _workspace(workspace, need, q)
    st = lib.awq_cache_attention(q_at, q_stride, *codes, *seqs, out_at, lse_at,
                                 dim ** -0.5 if scale is None else scale, max(min(window, 1 << 30), -1), softcap, T, B, W,
                                 heads, kv, dim, pages, page, max_new, max_len, code, ws, ws_bytes, _raw_stream(dev))
    if st:
        _check(st, "awq_cache_attention")
    return out


def _book_args(tables, lens, refs):
    """(addresses, device, B, W, pages) of a cache's book."""
    torch = _torch()
    dev = _gpu_of(tables, "tables")
    (t_at, l_at, _), B, W = _sequence_args(tables, lens, None, dev)
    return (t_at, l_at, _arg(refs, torch.int32, (refs.numel(),), dev, "refs")), dev, B, W, refs.numel()


def cache_fork(tables, lens, refs, parents, page_size: int, out=None):
    """Table rows from their parents, all at once (awq_cache_fork): row b of the
    result is row parents[b] (-1: an empty row).  refs, int32 [pages], follows in
    place.  Returns (tables, lens) of parents' length (`out` if given)."""
    torch = _torch()
    book, dev, B, W, pages = _book_args(tables, lens, refs)
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_fork(tables, lens, refs, parents, page_size, out)
    lib = load_library()
    n = parents.numel()
    if out is None:
        new_tables, new_lens = tables.new_empty((n, W)), lens.new_empty(n)
        out_at = new_tables.data_ptr(), new_lens.data_ptr()
    else:
        new_tables, new_lens = out
        out_at = (_arg(new_tables, torch.int32, (n, W), dev, "out[0]"), _arg(new_lens, torch.int32, (n,), dev, "out[1]"))
    st = lib.awq_cache_fork(*book, _arg(parents, torch.int32, (n,), dev, "parents"), *out_at, B, n, W, pages, page_size,
                            _raw_stream(dev))
    if st:
        _check(st, "awq_cache_fork")
    return new_tables, new_lens


def cache_reserve(tables, lens, refs, counts, page_size: int, out=None):
    """Room for counts[b] more tokens in every row, in place (awq_cache_reserve).
    Returns (pairs int32 [B][2]: the pages to copy before they are written, for
    cache_copy_pages; status int32 [2]: pages missing, rows past the table -- if
    either is not 0 nothing has changed)."""
    torch = _torch()
    book, dev, B, W, pages = _book_args(tables, lens, refs)
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_reserve(tables, lens, refs, counts, page_size, out)
    lib = load_library()
    if out is None:
        pairs, status = tables.new_empty((B, 2)), lens.new_empty(2)
        out_at = pairs.data_ptr(), status.data_ptr()
    else:
        pairs, status = out
        out_at = _arg(pairs, torch.int32, (B, 2), dev, "out[0]"), _arg(status, torch.int32, (2,), dev, "out[1]")
    st = lib.awq_cache_reserve(*book, _arg(counts, torch.int32, (B,), dev, "counts"), *out_at, B, W, pages, page_size,
                               _raw_stream(dev))
    if st:
        _check(st, "awq_cache_reserve")
    return pairs, status


def cache_compact(tables, lens, refs, page_size: int, out=None):
    """Used pages moved to the front of the cache (awq_cache_compact); tables and
    refs follow in place.  Returns (moves int32 [pages][2], count int32 [1]) for
    cache_copy_pages."""
    torch = _torch()
    book, dev, B, W, pages = _book_args(tables, lens, refs)
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_compact(tables, lens, refs, page_size, out)
    lib = load_library()
    moves, count = (refs.new_empty((pages, 2)), refs.new_empty(1)) if out is None else out
    st = lib.awq_cache_compact(*book, _arg(moves, torch.int32, (pages, 2), dev, "out[0]"),
                               _arg(count, torch.int32, (1,), dev, "out[1]"), B, W, pages, page_size, _raw_stream(dev))
    if st:
        _check(st, "awq_cache_compact")
    return moves, count


def cache_copy_pages(tensors, pairs, count=None, layers=None):
    """Page pairs[i][0] to page pairs[i][1] in every tensor, in place
    (awq_cache_copy_pages).  tensors: up to 8, each [pages][...], or
    [layers][pages][...] with layers given; pairs int32 [n][2], entries outside
    the cache are passed over; count int32 [1] on the GPU: how many pairs there
    are (None: all)."""
    torch = _torch()
    tensors = list(tensors)
    shape, dev = _rows2d(pairs, "pairs")
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return cache_copy_pages(tensors, pairs, count, layers)
    lib = load_library()
    lead = 0 if layers is None else 1
    if not tensors or tensors[0].dim() <= lead or 0 in tensors[0].shape:
        raise ValueError("tensors must hold at least one tensor of at least one page")
    n = len(tensors)
    at, size = (_c_void_p * n)(), (_c_size_t * n)()
    pages = tensors[0].shape[lead]
    for i, t in enumerate(tensors):
        if t.dim() <= lead or t.shape[lead] != pages or (lead and t.shape[0] != layers):
            raise ValueError(f"tensors[{i}] must be [{'layers][' if lead else ''}pages][...], got {tuple(t.shape)}")
        at[i] = _arg(t, t.dtype, t.shape, dev, f"tensors[{i}]")
        size[i] = t.numel() // (pages * (layers if lead else 1)) * t.element_size()
    st = lib.awq_cache_copy_pages(at, size, n, layers if lead else 1,
                                  _arg(pairs, torch.int32, (shape[0], 2), dev, "pairs"),
                                  _optional(count, torch.int32, (1,), dev, "count"), shape[0], pages, _raw_stream(dev))
    if st:
        _check(st, "awq_cache_copy_pages")
