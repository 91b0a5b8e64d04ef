"""Python binding of libtttmlp.so (the C ABI in include/tttmlp.h).

Argument marshalling only: every function forwards to the C entry point of
the same name; all arithmetic runs in the library's CUDA kernels.  PyTorch
is used for device memory and streams.  There is no fallback: if the
library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from operator import index

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtttmlp.so")
_lib = None

TTT_OK, TTT_ERR_INVALID_ARG, TTT_ERR_UNSUPPORTED, TTT_ERR_CUDA, TTT_ERR_NONFINITE, TTT_ERR_TIMEOUT = range(6)
STATUS_NAMES = {0: "TTT_OK", 1: "TTT_ERR_INVALID_ARG", 2: "TTT_ERR_UNSUPPORTED", 3: "TTT_ERR_CUDA",
                4: "TTT_ERR_NONFINITE", 5: "TTT_ERR_TIMEOUT"}
TTT_FWD, TTT_REV, TTT_BIDIR = 0, 1, 2
TTT_F32, TTT_BF16 = 0, 1
TTT_PHASE_FWD, TTT_PHASE_REV = 0, 1
DIRS = {"fwd": TTT_FWD, "rev": TTT_REV, "bidir": TTT_BIDIR}

EXPORTED = ["ttt_mlp_workspace_size", "ttt_mlp_forward", "ttt_mlp_status", "ttt_mlp_host_io_workspace_size",
            "ttt_mlp_forward_host", "ttt_mlp_select_kernels", "ttt_last_error", "ttt_launch_count",
            "ttt_kernel_timing", "ttt_kernel_times", "ttt_mlp_forward_noalloc", "ttt_mlp_noalloc_status", "ttt_debug_inject_wait_timeout",
            "ttt_linear_workspace_size", "ttt_linear_forward", "ttt_debug_pipe_segments",
            "ttt_mlp_backward_workspace_size", "ttt_mlp_backward", "ttt_mlp_heads_workspace_size",
            "ttt_mlp_forward_heads", "ttt_seg_attention_workspace_size", "ttt_seg_attention",
            "ttt_block_workspace_size", "ttt_block_forward", "ttt_debug_set_block_front",
            "ttt_linear_host_io_workspace_size", "ttt_linear_forward_host", "ttt_debug_set_backward_ctas",
            "ttt_rope", "ttt_window_attention_workspace_size", "ttt_window_attention",
            "ttt_window_attention_backward_workspace_size", "ttt_window_attention_backward",
            "ttt_window_attention_decode_workspace_size", "ttt_window_attention_decode",
            "ttt_gated_scan_workspace_size", "ttt_gated_scan_chunk_states_size", "ttt_gated_scan",
            "ttt_gated_scan_backward", "ttt_gated_scan_step"]


class TTTError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {ttt_last_error()}")


TTT_ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
TTT_ROPE_SCALINGS = {"none": 0, "linear": 1, "base": 2, "ramp": 3}
TTT_GATE_FORMS = {"sum": 0, "convex": 1, "unit": 2}


class ttt_rope_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int), ("rot", ctypes.c_int),
                ("layout", ctypes.c_int), ("x_dtype", ctypes.c_int), ("scaling", ctypes.c_int),
                ("base", ctypes.c_double), ("factor", ctypes.c_double), ("length", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double), ("amplitude", ctypes.c_double)]


class ttt_window_desc(ctypes.Structure):
    _fields_ = [("Tq", ctypes.c_int), ("Tk", ctypes.c_int), ("n_seq", ctypes.c_int), ("Hq", ctypes.c_int),
                ("Hk", ctypes.c_int), ("d", ctypes.c_int), ("left", ctypes.c_int), ("right", ctypes.c_int),
                ("sinks", ctypes.c_int), ("scale", ctypes.c_float)]


class ttt_window_decode_desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("Hq", ctypes.c_int), ("Hk", ctypes.c_int), ("d", ctypes.c_int),
                ("slots", ctypes.c_int), ("left", ctypes.c_int), ("sinks", ctypes.c_int), ("scale", ctypes.c_float),
                ("ld_request", ctypes.c_longlong), ("ld_slot", ctypes.c_longlong), ("ld_head", ctypes.c_longlong)]


class ttt_gated_scan_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("D", ctypes.c_int), ("n_seq", ctypes.c_int), ("form", ctypes.c_int),
                ("dir", ctypes.c_int), ("x_dtype", ctypes.c_int)]


class ttt_mlp_desc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int), ("H", ctypes.c_int), ("d", ctypes.c_int), ("m", ctypes.c_int),
                ("D", ctypes.c_int), ("per_head_input", ctypes.c_int), ("x_dtype", ctypes.c_int)]


def make_desc(T: int, H: int, d: int, per_head: bool, bf16: bool) -> ttt_mlp_desc:
    return ttt_mlp_desc(T, H, d, 4 * d, H * d, 1 if per_head else 0, TTT_BF16 if bf16 else TTT_F32)


def library_path() -> str:
    return _LIB_PATH


def lib():
    """Load libtttmlp.so (raises if it is missing: there is no fallback path)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with python -m test_rnn_layer_b200.build")
        L = ctypes.CDLL(_LIB_PATH)
        vp, sz, i, f = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
        dp = ctypes.POINTER(ttt_mlp_desc)
        L.ttt_mlp_workspace_size.restype = sz
        L.ttt_mlp_workspace_size.argtypes = [dp, i, i]
        L.ttt_mlp_host_io_workspace_size.restype = sz
        L.ttt_mlp_host_io_workspace_size.argtypes = [dp, i, i]
        L.ttt_mlp_forward.restype = i
        L.ttt_mlp_forward.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, i, i, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.ttt_mlp_forward_host.restype = i
        L.ttt_mlp_forward_host.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, i, i, vp, vp, vp, vp, sz, vp]
        L.ttt_mlp_forward_noalloc.restype = i
        L.ttt_mlp_forward_noalloc.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, i, i, vp, vp, vp, vp, vp, vp, vp]
        L.ttt_mlp_backward_workspace_size.restype = sz
        L.ttt_mlp_backward_workspace_size.argtypes = [dp, i, i]
        L.ttt_mlp_backward.restype = i
        L.ttt_mlp_backward.argtypes = [dp, vp, vp, vp, vp, vp, vp, f, i, i, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                       vp, sz, vp]
        L.ttt_mlp_heads_workspace_size.restype = sz
        L.ttt_mlp_heads_workspace_size.argtypes = [dp, i, i]
        L.ttt_mlp_forward_heads.restype = i
        L.ttt_mlp_forward_heads.argtypes = [dp, i, i, i, vp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, vp, sz, vp]
        L.ttt_seg_attention_workspace_size.restype = sz
        L.ttt_seg_attention_workspace_size.argtypes = []
        L.ttt_seg_attention.restype = i
        L.ttt_seg_attention.argtypes = [i, i, i, i, vp, vp, vp, i, vp, vp, i, i, i, vp, sz, vp]
        L.ttt_block_workspace_size.restype = sz
        L.ttt_block_workspace_size.argtypes = [dp, i]
        L.ttt_block_forward.restype = i
        L.ttt_block_forward.argtypes = [dp, i, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, f, i, vp, vp, vp, vp, sz, vp]
        L.ttt_debug_set_block_front.restype = i
        L.ttt_debug_set_block_front.argtypes = [i]
        L.ttt_debug_set_backward_ctas.restype = i
        L.ttt_debug_set_backward_ctas.argtypes = [i]
        L.ttt_mlp_noalloc_status.restype = i
        L.ttt_mlp_noalloc_status.argtypes = [vp]
        L.ttt_linear_workspace_size.restype = sz
        L.ttt_linear_workspace_size.argtypes = [dp, i, i]
        L.ttt_linear_host_io_workspace_size.restype = sz
        L.ttt_linear_host_io_workspace_size.argtypes = [dp, i, i]
        L.ttt_linear_forward_host.restype = i
        L.ttt_linear_forward_host.argtypes = [dp, vp, vp, vp, vp, vp, f, i, i, vp, vp, vp, vp, sz, vp]
        L.ttt_linear_forward.restype = i
        L.ttt_linear_forward.argtypes = [dp, vp, vp, vp, vp, vp, f, i, i, vp, vp, vp, vp, vp, vp, sz, vp]
        rp, wp, ep, gp = (ctypes.POINTER(c) for c in (ttt_rope_desc, ttt_window_desc, ttt_window_decode_desc,
                                                      ttt_gated_scan_desc))
        for name, res, args in (
                ("ttt_rope", i, [rp, vp, i, vp, i, vp, i, i, vp]),
                ("ttt_window_attention_workspace_size", sz, [wp]),
                ("ttt_window_attention", i, [wp, vp, vp, vp, i, vp, i, vp, i, vp, vp, i, vp, vp, sz, vp]),
                ("ttt_window_attention_backward_workspace_size", sz, [wp]),
                ("ttt_window_attention_backward", i, [wp, vp, vp, vp, i, vp, i, vp, i, vp, i, vp, vp, i, vp, i, vp, i,
                                                      vp, i, vp, sz, vp]),
                ("ttt_window_attention_decode_workspace_size", sz, [ep]),
                ("ttt_window_attention_decode", i, [ep, vp, i, vp, vp, i, vp, vp, vp, vp, i, vp, sz, vp]),
                ("ttt_gated_scan_workspace_size", sz, [gp]),
                ("ttt_gated_scan_chunk_states_size", sz, [gp]),
                ("ttt_gated_scan", i, [gp, vp, vp, i, vp, i, vp, vp, i, vp, vp, vp, sz, vp]),
                ("ttt_gated_scan_backward", i, [gp, vp, vp, i, vp, i, vp, vp, vp, i, vp, vp, i, vp, i, vp, vp, sz, vp]),
                ("ttt_gated_scan_step", i, [i, i, i, i, vp, i, vp, i, vp, vp, vp, i, vp])):
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        L.ttt_mlp_status.restype = i
        L.ttt_mlp_status.argtypes = [vp, vp]
        L.ttt_mlp_select_kernels.restype = i
        L.ttt_mlp_select_kernels.argtypes = [i, i]
        L.ttt_last_error.restype = ctypes.c_char_p
        L.ttt_last_error.argtypes = []
        L.ttt_launch_count.restype = ctypes.c_uint64
        L.ttt_launch_count.argtypes = []
        L.ttt_debug_pipe_segments.restype = i
        L.ttt_debug_pipe_segments.argtypes = [i, ctypes.POINTER(ctypes.c_int), i]
        L.ttt_debug_inject_wait_timeout.restype = i
        L.ttt_debug_inject_wait_timeout.argtypes = [i]
        L.ttt_kernel_timing.restype = i
        L.ttt_kernel_timing.argtypes = [i]
        L.ttt_kernel_times.restype = i
        L.ttt_kernel_times.argtypes = [i, ctypes.c_char_p, sz, ctypes.POINTER(ctypes.c_double),
                                       ctypes.POINTER(ctypes.c_uint64)]
        _lib = L
    return _lib


def _p(x):
    if x is None:
        return None
    return x.data_ptr() if isinstance(x, torch.Tensor) else int(x)


def _stream(stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())   # current_stream() builds an object
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


# ------------------------------------------------------------------ the C entry points
def ttt_last_error() -> str:
    return lib().ttt_last_error().decode()


def ttt_launch_count() -> int:
    return int(lib().ttt_launch_count())


def ttt_debug_inject_wait_timeout(enable: bool) -> int:
    return int(lib().ttt_debug_inject_wait_timeout(1 if enable else 0))


def ttt_debug_pipe_segments(nchunks: int, max_segments: int = 256) -> list:
    """Chunk segments [(begin, end), ...] of the pipelined full-width layer (tests)."""
    buf = (ctypes.c_int * (2 * max_segments))()
    n = int(lib().ttt_debug_pipe_segments(int(nchunks), buf, max_segments))
    if n < 0:
        raise TTTError(TTT_ERR_INVALID_ARG, "ttt_debug_pipe_segments")
    return [(buf[2 * k], buf[2 * k + 1]) for k in range(min(n, max_segments))]


def ttt_kernel_timing(enable: bool) -> int:
    return int(lib().ttt_kernel_timing(1 if enable else 0))


def ttt_kernel_times(max_kernels: int = 32) -> dict:
    """{kernel name: (total ms, launches)} recorded since ttt_kernel_timing(True)."""
    names = ctypes.create_string_buffer(4096)
    ms = (ctypes.c_double * max_kernels)()
    cnt = (ctypes.c_uint64 * max_kernels)()
    n = lib().ttt_kernel_times(max_kernels, names, 4096, ms, cnt)
    if n < 0:
        raise TTTError(TTT_ERR_CUDA, "ttt_kernel_times")
    keys = names.value.decode().split("\n")[:min(n, max_kernels)]
    return {k: (ms[i], int(cnt[i])) for i, k in enumerate(keys)}


def ttt_mlp_workspace_size(desc: ttt_mlp_desc, b: int, direction: int) -> int:
    return int(lib().ttt_mlp_workspace_size(ctypes.byref(desc), b, direction))


def ttt_mlp_host_io_workspace_size(desc: ttt_mlp_desc, b: int, direction: int) -> int:
    return int(lib().ttt_mlp_host_io_workspace_size(ctypes.byref(desc), b, direction))


def ttt_mlp_select_kernels(scan_impl: int, proj_impl: int) -> int:
    return int(lib().ttt_mlp_select_kernels(scan_impl, proj_impl))


def ttt_mlp_forward(desc, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, direction, alpha_f, alpha_r, Y,
                    Z_out, W1_T, W2_T, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_mlp_forward(ctypes.byref(desc), _p(X), _p(theta_q), _p(theta_k), _p(theta_v), _p(W1_0),
                                     _p(W2_0), float(eta), int(b), int(direction), _p(alpha_f), _p(alpha_r), _p(Y),
                                     _p(Z_out), _p(W1_T), _p(W2_T), _p(workspace), int(workspace_bytes),
                                     _stream(stream)))


def ttt_mlp_forward_host(desc, X_host, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, direction, alpha_f, alpha_r,
                         Y_host, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_mlp_forward_host(ctypes.byref(desc), _p(X_host), _p(theta_q), _p(theta_k), _p(theta_v),
                                          _p(W1_0), _p(W2_0), float(eta), int(b), int(direction), _p(alpha_f),
                                          _p(alpha_r), _p(Y_host), _p(workspace), int(workspace_bytes),
                                          _stream(stream)))


def ttt_mlp_forward_noalloc(desc, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, direction, alpha_f, alpha_r,
                            Y, Z_out, W1_T, W2_T, stream=None) -> int:
    """ttt_mlp_forward without a workspace argument: for callers that cannot
    allocate device memory (the library uses its own fixed 32 MiB scratch)."""
    return int(lib().ttt_mlp_forward_noalloc(ctypes.byref(desc), _p(X), _p(theta_q), _p(theta_k), _p(theta_v),
                                             _p(W1_0), _p(W2_0), float(eta), int(b), int(direction), _p(alpha_f),
                                             _p(alpha_r), _p(Y), _p(Z_out), _p(W1_T), _p(W2_T), _stream(stream)))


def ttt_mlp_backward_workspace_size(desc: ttt_mlp_desc, b: int, direction: int) -> int:
    return int(lib().ttt_mlp_backward_workspace_size(ctypes.byref(desc), b, direction))


def ttt_mlp_backward(desc, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, direction, alpha_f, alpha_r, dY, dX,
                     dtheta_q, dtheta_k, dtheta_v, dW1_0, dW2_0, dalpha_f, dalpha_r, workspace, workspace_bytes,
                     stream=None) -> int:
    return int(lib().ttt_mlp_backward(ctypes.byref(desc), _p(X), _p(theta_q), _p(theta_k), _p(theta_v), _p(W1_0),
                                      _p(W2_0), float(eta), int(b), int(direction), _p(alpha_f), _p(alpha_r), _p(dY),
                                      _p(dX), _p(dtheta_q), _p(dtheta_k), _p(dtheta_v), _p(dW1_0), _p(dW2_0),
                                      _p(dalpha_f), _p(dalpha_r), _p(workspace), int(workspace_bytes),
                                      _stream(stream)))


def layer_backward(X, theta_q, theta_k, theta_v, W1_0, W2_0, eta: float, b: int, dirs: str, alpha_f, alpha_r, dY,
                   per_head: bool = True, workspace: torch.Tensor | None = None, check_status: bool = True,
                   stream=None) -> dict:
    """Allocate gradient outputs (fp32, on X's device) and call ttt_mlp_backward once."""
    dev = X.device
    if per_head:
        H, T, d = X.shape
    else:
        T, _ = X.shape
        H, d = W1_0.shape[0], W1_0.shape[2]
    desc = make_desc(T, H, d, per_head, X.dtype == torch.bfloat16)
    direction = DIRS[dirs]
    if workspace is None:
        n = ttt_mlp_backward_workspace_size(desc, b, direction)
        if n == 0:
            raise TTTError(TTT_ERR_INVALID_ARG, "backward workspace size")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    out = {"dX": torch.empty(X.shape, **f32), "dtheta_q": torch.empty(theta_q.shape, **f32),
           "dtheta_k": torch.empty(theta_k.shape, **f32), "dtheta_v": torch.empty(theta_v.shape, **f32),
           "dW1_0": torch.empty(W1_0.shape, **f32), "dW2_0": torch.empty(W2_0.shape, **f32),
           "dalpha_f": torch.zeros(alpha_f.shape, **f32), "dalpha_r": torch.zeros(alpha_r.shape, **f32)}
    st = ttt_mlp_backward(desc, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, direction, alpha_f, alpha_r,
                          dY.float().contiguous(), out["dX"], out["dtheta_q"], out["dtheta_k"], out["dtheta_v"],
                          out["dW1_0"], out["dW2_0"], out["dalpha_f"], out["dalpha_r"], workspace, workspace.numel(),
                          stream)
    check(st, "ttt_mlp_backward")
    if check_status:
        check(ttt_mlp_status(workspace, stream), "ttt_mlp_status")
    out["workspace"] = workspace
    return out


def ttt_mlp_heads_workspace_size(desc: ttt_mlp_desc, hn: int, b: int) -> int:
    return int(lib().ttt_mlp_heads_workspace_size(ctypes.byref(desc), hn, b))


def ttt_mlp_forward_heads(desc, h0, hn, phase, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, alpha, delta_all,
                          Xp, delta_or_y, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_mlp_forward_heads(ctypes.byref(desc), h0, hn, phase, _p(X), _p(theta_q), _p(theta_k),
                                           _p(theta_v), _p(W1_0), _p(W2_0), float(eta), b, _p(alpha),
                                           _p(delta_all), _p(Xp), _p(delta_or_y), _p(workspace), workspace_bytes,
                                           _stream(stream)))


def ttt_seg_attention_workspace_size() -> int:
    return int(lib().ttt_seg_attention_workspace_size())


def ttt_seg_attention(T, H, d, L, Q, K, V, ld_qkv, Xres, Out, ld_out, row0, row1, workspace, workspace_bytes,
                      stream=None) -> int:
    return int(lib().ttt_seg_attention(T, H, d, L, _p(Q), _p(K), _p(V), ld_qkv, _p(Xres), _p(Out), ld_out, row0,
                                       row1, _p(workspace), workspace_bytes, _stream(stream)))


def ttt_block_workspace_size(desc: ttt_mlp_desc, b: int) -> int:
    return int(lib().ttt_block_workspace_size(ctypes.byref(desc), b))


def ttt_block_forward(desc, seg_len, Qa, Ka, Va, ld_qkv, Xres, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b,
                      alpha_f, alpha_r, Y, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_block_forward(ctypes.byref(desc), seg_len, _p(Qa), _p(Ka), _p(Va), ld_qkv, _p(Xres), _p(X),
                                       _p(theta_q), _p(theta_k), _p(theta_v), _p(W1_0), _p(W2_0), float(eta), b,
                                       _p(alpha_f), _p(alpha_r), _p(Y), _p(workspace), workspace_bytes,
                                       _stream(stream)))


def ttt_debug_set_block_front(percent: int) -> int:
    return int(lib().ttt_debug_set_block_front(percent))


def ttt_debug_set_backward_ctas(ctas: int) -> int:
    return int(lib().ttt_debug_set_backward_ctas(ctas))


def ttt_mlp_noalloc_status(stream=None) -> int:
    """ttt_mlp_status for the no-alloc entry point (its status word lives in
    the library's fixed scratch array on the current device)."""
    return int(lib().ttt_mlp_noalloc_status(_stream(stream)))


def ttt_linear_workspace_size(desc: ttt_mlp_desc, b: int, direction: int) -> int:
    return int(lib().ttt_linear_workspace_size(ctypes.byref(desc), b, direction))


def ttt_linear_host_io_workspace_size(desc: ttt_mlp_desc, b: int, direction: int) -> int:
    return int(lib().ttt_linear_host_io_workspace_size(ctypes.byref(desc), b, direction))


def ttt_linear_forward_host(desc, X_host, theta_q, theta_k, theta_v, W_0, eta, b, direction, alpha_f, alpha_r,
                            Y_host, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_linear_forward_host(ctypes.byref(desc), _p(X_host), _p(theta_q), _p(theta_k), _p(theta_v),
                                             _p(W_0), float(eta), b, direction, _p(alpha_f), _p(alpha_r),
                                             _p(Y_host), _p(workspace), workspace_bytes, _stream(stream)))


def ttt_linear_forward(desc, X, theta_q, theta_k, theta_v, W_0, eta, b, direction, alpha_f, alpha_r, Y, Z_out,
                       W_T, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_linear_forward(ctypes.byref(desc), _p(X), _p(theta_q), _p(theta_k), _p(theta_v), _p(W_0),
                                        float(eta), int(b), int(direction), _p(alpha_f), _p(alpha_r), _p(Y),
                                        _p(Z_out), _p(W_T), _p(workspace), int(workspace_bytes), _stream(stream)))


def ttt_mlp_status(workspace, stream=None) -> int:
    return int(lib().ttt_mlp_status(_p(workspace), _stream(stream)))


# ------------------------------------------------------------------ tensor-level convenience
def check(status: int, where: str) -> None:
    if status != TTT_OK:
        raise TTTError(status, where)


def alloc_workspace(desc: ttt_mlp_desc, b: int, direction: int, device, host_io: bool = False) -> torch.Tensor:
    n = (ttt_mlp_host_io_workspace_size if host_io else ttt_mlp_workspace_size)(desc, b, direction)
    if n == 0:
        raise TTTError(TTT_ERR_INVALID_ARG, "workspace size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def layer_forward(X, theta_q, theta_k, theta_v, W1_0, W2_0, eta: float, b: int, dirs: str, alpha_f=None,
                  alpha_r=None, per_head: bool = True, want_z: bool = False, want_state: bool = False,
                  workspace: torch.Tensor | None = None, check_status: bool = True, stream=None) -> dict:
    """Allocate outputs (torch, on X's device) and call ttt_mlp_forward once."""
    dev = X.device
    if per_head:
        H, T, d = X.shape
    else:
        T, D = X.shape
        d = W1_0.shape[2]
        H = W1_0.shape[0]
    desc = make_desc(T, H, d, per_head, X.dtype == torch.bfloat16)
    direction = DIRS[dirs]
    nd = 2 if dirs == "bidir" else 1
    ws = workspace if workspace is not None else alloc_workspace(desc, b, direction, dev)
    Y = torch.empty_like(X)
    Z = torch.empty((nd,) + tuple(X.shape), dtype=torch.float32, device=dev) if want_z else None
    W1T = torch.empty((nd,) + tuple(W1_0.shape), dtype=torch.float32, device=dev) if want_state else None
    W2T = torch.empty((nd,) + tuple(W2_0.shape), dtype=torch.float32, device=dev) if want_state else None
    st = ttt_mlp_forward(desc, X, theta_q, theta_k, theta_v, W1_0, W2_0, eta, b, direction, alpha_f, alpha_r, Y, Z,
                         W1T, W2T, ws, ws.numel(), stream)
    check(st, "ttt_mlp_forward")
    out = {"Y": Y, "Z": Z, "W1_T": W1T, "W2_T": W2T, "workspace": ws}
    if check_status:
        st = ttt_mlp_status(ws, stream)
        out["status"] = st
        check(st, "ttt_mlp_status")
    return out


def linear_layer_forward(X, theta_q, theta_k, theta_v, W_0, eta: float, b: int, dirs: str, alpha_f=None,
                         alpha_r=None, per_head: bool = True, want_z: bool = False, want_state: bool = False,
                         workspace: torch.Tensor | None = None, check_status: bool = True, stream=None) -> dict:
    """Allocate outputs (torch, on X's device) and call ttt_linear_forward once."""
    dev = X.device
    if per_head:
        H, T, d = X.shape
    else:
        T, _ = X.shape
        H, d = W_0.shape[0], W_0.shape[2]
    desc = make_desc(T, H, d, per_head, X.dtype == torch.bfloat16)
    direction = DIRS[dirs]
    nd = 2 if dirs == "bidir" else 1
    if workspace is None:
        n = ttt_linear_workspace_size(desc, b, direction)
        if n == 0:
            raise TTTError(TTT_ERR_INVALID_ARG, "workspace size")
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    Y = torch.empty_like(X)
    Z = torch.empty((nd,) + tuple(X.shape), dtype=torch.float32, device=dev) if want_z else None
    WT = torch.empty((nd,) + tuple(W_0.shape), dtype=torch.float32, device=dev) if want_state else None
    st = ttt_linear_forward(desc, X, theta_q, theta_k, theta_v, W_0, eta, b, direction, alpha_f, alpha_r, Y, Z, WT,
                            workspace, workspace.numel(), stream)
    check(st, "ttt_linear_forward")
    out = {"Y": Y, "Z": Z, "W_T": WT, "workspace": workspace}
    if check_status:
        st = ttt_mlp_status(workspace, stream)
        out["status"] = st
        check(st, "ttt_mlp_status")
    return out


# ------------------------------------------------------------------ sequence operators
# The C entry points of the same names (pointers as tensors or integers), then
# tensor-level functions that take row strides from the tensors' own, allocate
# what is not given and run on the tensors' device.
def ttt_rope(desc, X, ld_x, Y, ld_y, positions, pos0, inverse, stream=None) -> int:
    return int(lib().ttt_rope(ctypes.byref(desc), _p(X), ld_x, _p(Y), ld_y, _p(positions), pos0, int(inverse),
                              _stream(stream)))


def ttt_window_attention_workspace_size(desc) -> int:
    return int(lib().ttt_window_attention_workspace_size(ctypes.byref(desc)))


def ttt_window_attention(desc, cu_q, cu_k, Q, ld_q, K, ld_k, V, ld_v, Xres, Out, ld_out, Lse, workspace,
                         workspace_bytes, stream=None) -> int:
    return int(lib().ttt_window_attention(ctypes.byref(desc), _p(cu_q), _p(cu_k), _p(Q), ld_q, _p(K), ld_k, _p(V),
                                          ld_v, _p(Xres), _p(Out), ld_out, _p(Lse), _p(workspace), workspace_bytes,
                                          _stream(stream)))


def ttt_window_attention_backward_workspace_size(desc) -> int:
    return int(lib().ttt_window_attention_backward_workspace_size(ctypes.byref(desc)))


def ttt_window_attention_backward(desc, cu_q, cu_k, Q, ld_q, K, ld_k, V, ld_v, Out, ld_out, Lse, dOut, ld_do, dQ,
                                  ld_dq, dK, ld_dk, dV, ld_dv, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_window_attention_backward(ctypes.byref(desc), _p(cu_q), _p(cu_k), _p(Q), ld_q, _p(K), ld_k,
                                                   _p(V), ld_v, _p(Out), ld_out, _p(Lse), _p(dOut), ld_do, _p(dQ),
                                                   ld_dq, _p(dK), ld_dk, _p(dV), ld_dv, _p(workspace),
                                                   workspace_bytes, _stream(stream)))


def ttt_window_attention_decode_workspace_size(desc) -> int:
    return int(lib().ttt_window_attention_decode_workspace_size(ctypes.byref(desc)))


def ttt_window_attention_decode(desc, Q, ld_q, K_new, V_new, ld_new, K_cache, V_cache, lens, Out, ld_out, workspace,
                                workspace_bytes, stream=None) -> int:
    return int(lib().ttt_window_attention_decode(ctypes.byref(desc), _p(Q), ld_q, _p(K_new), _p(V_new), ld_new,
                                                 _p(K_cache), _p(V_cache), _p(lens), _p(Out), ld_out, _p(workspace),
                                                 workspace_bytes, _stream(stream)))


def ttt_gated_scan_workspace_size(desc) -> int:
    return int(lib().ttt_gated_scan_workspace_size(ctypes.byref(desc)))


def ttt_gated_scan_chunk_states_size(desc) -> int:
    return int(lib().ttt_gated_scan_chunk_states_size(ctypes.byref(desc)))


def ttt_gated_scan(desc, cu, F, ld_f, X, ld_x, H_0, Y, ld_y, H_T, chunk_states, workspace, workspace_bytes,
                   stream=None) -> int:
    return int(lib().ttt_gated_scan(ctypes.byref(desc), _p(cu), _p(F), ld_f, _p(X), ld_x, _p(H_0), _p(Y), ld_y,
                                    _p(H_T), _p(chunk_states), _p(workspace), workspace_bytes, _stream(stream)))


def ttt_gated_scan_backward(desc, cu, F, ld_f, X, ld_x, H_0, chunk_states, dY, ld_dy, dH_T, dF, ld_df, dX, ld_dx,
                            dH_0, workspace, workspace_bytes, stream=None) -> int:
    return int(lib().ttt_gated_scan_backward(ctypes.byref(desc), _p(cu), _p(F), ld_f, _p(X), ld_x, _p(H_0),
                                             _p(chunk_states), _p(dY), ld_dy, _p(dH_T), _p(dF), ld_df, _p(dX), ld_dx,
                                             _p(dH_0), _p(workspace), workspace_bytes, _stream(stream)))


def ttt_gated_scan_step(B, D, form, x_dtype, F, ld_f, X, ld_x, H, H_out, Y, ld_y, stream=None) -> int:
    return int(lib().ttt_gated_scan_step(B, D, form, x_dtype, _p(F), ld_f, _p(X), ld_x, _p(H), _p(H_out), _p(Y), ld_y,
                                         _stream(stream)))


class _Elsewhere:
    """The tensors' device current and, if one is given, `stream` (new tensors then belong to it and are filled on it)."""

    __slots__ = ("stack",)

    def __init__(self, device, stream):
        self.stack = [torch.cuda.device(device)]
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):   # a handle; 0 and 1 name the default stream
                handle = int(stream)
                stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
            self.stack.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.stack:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.stack):
            c.__exit__(*exc)
        return False


_HERE = contextlib.nullcontext()


def _place(device, stream):
    """What a call on tensors of `device` runs within."""
    return _HERE if stream is None and device == torch.cuda.current_device() else _Elsewhere(device, stream)


# The checks run on every call of a few microseconds: messages are put together only for a refusal.
def _ask(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows(x, shape, dtype, device, name) -> int:
    """Row stride of a tensor of `shape` whose rows are dense (checked with its type and device)."""
    if x.dtype is not dtype or x.get_device() != device:
        raise ValueError(f"{name}: {x.dtype} on {x.device}, wanted {dtype} on GPU {device}")
    if x.shape != shape:
        raise ValueError(f"{name}: shape {tuple(x.shape)}, wanted {tuple(shape)}")
    strides = x.stride()
    ld = strides[0]
    if len(strides) == 3:
        dense = strides[2] == 1 and strides[1] == shape[2]
    else:
        dense = len(strides) == 2 and strides[1] == 1
    if not dense or shape[0] < 2 or ld >= 2 ** 31:     # an axis of one element may have any stride
        width = 1
        for k in range(len(shape) - 1, 0, -1):
            if strides[k] != width and shape[k] > 1:
                raise ValueError(f"{name}: the columns of a row must be dense, strides {strides}")
            width *= shape[k]
        if shape[0] < 2:
            ld = -(-width // 8) * 8
        if ld >= 2 ** 31:
            raise ValueError(f"{name}: row stride {ld}")
    return ld


def _offsets(cu, device, name):
    if cu is None:
        return 1
    if not (cu.dtype is torch.int32 and cu.get_device() == device and cu.dim() == 1 and cu.numel() >= 2 and cu.is_contiguous()):
        raise ValueError(f"{name}: a dense int32 vector of n_seq + 1 offsets on GPU {device} is wanted")
    return cu.numel() - 1


def _dense(x, shape, dtype, device, name):
    if not (x.dtype is dtype and x.get_device() == device and x.shape == shape and x.is_contiguous()):
        raise ValueError(f"{name}: a dense {dtype} tensor of shape {tuple(shape)} on GPU {device} is wanted")
    return x


def _space(workspace, size, device):
    """The given workspace (the call checks its size), or a new one of size() bytes."""
    if workspace is None:
        n = size()
        if n == 0:
            raise TTTError(TTT_ERR_INVALID_ARG, "workspace size")
        return torch.empty(n, dtype=torch.uint8, device=device)
    if workspace.get_device() != device:
        raise ValueError(f"workspace on {workspace.device}, wanted GPU {device}")
    return workspace


def _dtype_code(x, name) -> int:
    if not (x.is_cuda and (x.dtype is torch.bfloat16 or x.dtype is torch.float32)):
        raise ValueError(f"{name}: float32 or bfloat16 on a GPU is wanted")
    return TTT_BF16 if x.dtype == torch.bfloat16 else TTT_F32


_ROPE_KEYS = {"kind", "factor", "length", "low", "high", "amplitude"}
# Descriptors by their sizes, with a reference for the call: building one costs as much as a launch.  They are looked up
# by Python's own numbers, which do not change: a tensor of one element would be found again whatever it holds by then.
def _descriptor(_type, *args):
    for (name, kind), n in zip(_type._fields_, args):
        _ask(kind is not ctypes.c_int or -2 ** 31 <= n < 2 ** 31, f"{name}={n} does not fit 32 bits")   # ctypes cuts it
    desc = _type(*args)
    desc.ref = ctypes.byref(desc)
    return desc


_rope_desc, _window_sizes, _decode_sizes, _gated_sizes = (
    functools.lru_cache(maxsize=256)(functools.partial(_descriptor, c))
    for c in (ttt_rope_desc, ttt_window_desc, ttt_window_decode_desc, ttt_gated_scan_desc))


def _at(x):
    return None if x is None else x.data_ptr()


def rope(x, positions=None, *, pos0: int = 0, rot: int | None = None, layout: str = "half", base: float = 10000.0,
         scaling: dict | None = None, inverse: bool = False, out=None, stream=None):
    """Rotary positions of x [T, H, d] (ttt_rope).  `scaling`: {"kind": "linear" | "base", "factor": f} or
    {"kind": "ramp", "factor": f, "length": n, "low": l, "high": h}, with "amplitude" optional.  `out` may be x."""
    code, shape, dev = _dtype_code(x, "x"), x.shape, x.get_device()
    T, H, d = shape
    sc = scaling or {}
    if not (_ROPE_KEYS >= sc.keys() and sc.get("kind", "none") in TTT_ROPE_SCALINGS):
        raise ValueError(f"scaling {scaling}")
    desc = _rope_desc(T, H, d, d if rot is None else index(rot), TTT_ROPE_LAYOUTS[layout], code,
                      TTT_ROPE_SCALINGS[sc.get("kind", "none")], float(base), float(sc.get("factor", 1.0)),
                      float(sc.get("length", 0.0)), float(sc.get("low", 0.0)), float(sc.get("high", 0.0)),
                      float(sc.get("amplitude", 1.0)))
    _ask(-2 ** 31 <= pos0 < 2 ** 31, "pos0 does not fit 32 bits")
    if positions is not None:
        _dense(positions, (T,), torch.int32, dev, "positions")
    with _place(dev, stream):
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=dev)
        check(lib().ttt_rope(desc.ref, x.data_ptr(), _rows(x, shape, x.dtype, dev, "x"), out.data_ptr(),
                             _rows(out, shape, x.dtype, dev, "out"), _at(positions), pos0, int(inverse), _stream(stream)),
              "ttt_rope")
    return out


def _window_desc(q, k, n_seq, left, right, sinks, scale):
    _ask(q.is_cuda and q.dim() == 3 and k.dim() == 3 and q.shape[2] == k.shape[2], "q and k: [T, H, 64] on a GPU")
    (Tq, Hq, d), (Tk, Hk, _) = q.shape, k.shape
    return _window_sizes(Tq, Tk, index(n_seq), Hq, Hk, d, index(left), index(right), index(sinks),
                         d ** -0.5 if scale is None else float(scale))


def window_attention_workspace(q, k, n_seq: int = 1, backward: bool = False) -> torch.Tensor:
    """A workspace that window_attention (and, with backward, window_attention_backward) can use."""
    desc = _window_desc(q, k, n_seq, 0, 0, 0, None)
    size = ttt_window_attention_backward_workspace_size if backward else ttt_window_attention_workspace_size
    return _space(None, lambda: size(desc), q.get_device())


def window_attention(q, k, v, *, left: int, right: int = 0, sinks: int = 0, cu_q=None, cu_k=None, scale=None,
                     residual=None, out=None, lse=None, want_lse: bool = False, workspace=None,
                     check_status: bool = True, stream=None) -> dict:
    """Window attention of q [Tq, Hq, 64] on k, v [Tk, Hk, 64] (ttt_window_attention)."""
    dev, bf = q.get_device(), torch.bfloat16
    n_seq = _offsets(cu_q, dev, "cu_q")
    _ask((cu_q is None) == (cu_k is None) and _offsets(cu_k, dev, "cu_k") == n_seq,
         "cu_q and cu_k: both or neither, of the same length")
    desc = _window_desc(q, k, n_seq, left, right, sinks, scale)
    lds = [_rows(q, q.shape, bf, dev, "q"), _rows(k, k.shape, bf, dev, "k"), _rows(v, k.shape, bf, dev, "v")]
    with _place(dev, stream):
        ws = _space(workspace, lambda: ttt_window_attention_workspace_size(desc), dev)
        if out is None:   # rows outside the sequences are not written: they start as zeros
            out = (torch.empty if cu_q is None else torch.zeros)(q.shape, dtype=bf, device=dev)
        if lse is None and want_lse:
            lse = (torch.empty if cu_q is None else torch.zeros)((q.shape[1], q.shape[0]), dtype=torch.float32, device=dev)
        if lse is not None:
            _dense(lse, (q.shape[1], q.shape[0]), torch.float32, dev, "lse")
        ld_out = _rows(out, q.shape, bf, dev, "out")
        if residual is not None:
            _ask(_rows(residual, q.shape, bf, dev, "residual") == ld_out, "residual and out need the same row stride")
        check(lib().ttt_window_attention(desc.ref, _at(cu_q), _at(cu_k), q.data_ptr(), lds[0], k.data_ptr(), lds[1],
                                         v.data_ptr(), lds[2], _at(residual), out.data_ptr(), ld_out, _at(lse),
                                         ws.data_ptr(), ws.numel(), _stream(stream)), "ttt_window_attention")
        if check_status:
            check(ttt_mlp_status(ws, stream), "ttt_mlp_status")
    return {"out": out, "lse": lse, "workspace": ws}


def window_attention_backward(q, k, v, out, lse, dout, *, left: int, right: int = 0, sinks: int = 0, cu_q=None,
                              cu_k=None, scale=None, dq=None, dk=None, dv=None, workspace=None,
                              check_status: bool = True, stream=None) -> dict:
    """Gradients of window_attention (without a residual) from its out and lse (ttt_window_attention_backward)."""
    dev, bf = q.get_device(), torch.bfloat16
    n_seq = _offsets(cu_q, dev, "cu_q")
    _ask((cu_q is None) == (cu_k is None) and _offsets(cu_k, dev, "cu_k") == n_seq,
         "cu_q and cu_k: both or neither, of the same length")
    desc = _window_desc(q, k, n_seq, left, right, sinks, scale)
    _dense(lse, (q.shape[1], q.shape[0]), torch.float32, dev, "lse")
    with _place(dev, stream):
        ws = _space(workspace, lambda: ttt_window_attention_backward_workspace_size(desc), dev)
        new = torch.empty if cu_q is None else torch.zeros
        dq = new(q.shape, dtype=bf, device=dev) if dq is None else dq
        dk = new(k.shape, dtype=bf, device=dev) if dk is None else dk
        dv = new(k.shape, dtype=bf, device=dev) if dv is None else dv
        sq, sk = q.shape, k.shape
        check(lib().ttt_window_attention_backward(
            desc.ref, _at(cu_q), _at(cu_k), q.data_ptr(), _rows(q, sq, bf, dev, "q"), k.data_ptr(),
            _rows(k, sk, bf, dev, "k"), v.data_ptr(), _rows(v, sk, bf, dev, "v"), out.data_ptr(),
            _rows(out, sq, bf, dev, "out"), lse.data_ptr(), dout.data_ptr(), _rows(dout, sq, bf, dev, "dout"),
            dq.data_ptr(), _rows(dq, sq, bf, dev, "dq"), dk.data_ptr(), _rows(dk, sk, bf, dev, "dk"), dv.data_ptr(),
            _rows(dv, sk, bf, dev, "dv"), ws.data_ptr(), ws.numel(), _stream(stream)), "ttt_window_attention_backward")
        if check_status:
            check(ttt_mlp_status(ws, stream), "ttt_mlp_status")
    return {"dq": dq, "dk": dk, "dv": dv, "workspace": ws}


def _decode_desc(q, cache, left, sinks, scale):
    _ask(q.is_cuda and q.dim() == 3 and cache.dim() == 4 and cache.shape[0] == q.shape[0] and
         cache.shape[3] == q.shape[2], "q [B, Hq, 64] and a cache [B, slots, Hk, 64] on a GPU")
    _ask(cache.stride(3) == 1, "the cache's last axis must be dense")
    B, slots, Hk, d = cache.shape
    s0, s1, s2, _ = cache.stride()
    return _decode_sizes(B, q.shape[1], Hk, d, slots, index(left), index(sinks), d ** -0.5 if scale is None else float(scale),
                         s0 if B > 1 else 0, s1 if slots > 1 else d, s2 if Hk > 1 else 0)   # (axes of one: any stride)


def window_attention_decode_workspace(q, cache) -> torch.Tensor:
    """A zeroed workspace for window_attention_decode."""
    desc = _decode_desc(q, cache, 0, 0, None)
    return _space(None, lambda: ttt_window_attention_decode_workspace_size(desc), q.get_device()).zero_()


def window_attention_decode(q, cache_k, cache_v, lens, *, left: int, sinks: int = 0, scale=None, k_new=None,
                            v_new=None, out=None, workspace=None, check_status: bool = True, stream=None) -> dict:
    """One token of each request on its cache (ttt_window_attention_decode): q [B, Hq, 64], caches
    [B, slots, Hk, 64] with any strides, lens int32 [B]; k_new, v_new [B, Hk, 64] are stored first.
    A given workspace must have been zeroed once (window_attention_decode_workspace)."""
    dev, bf = q.get_device(), torch.bfloat16
    desc = _decode_desc(q, cache_k, left, sinks, scale)
    if not (cache_k.dtype is bf and cache_v.dtype is bf and cache_k.get_device() == dev and cache_v.get_device() == dev and
            cache_k.shape == cache_v.shape and cache_k.stride() == cache_v.stride()):
        raise ValueError(f"the caches: bfloat16 on GPU {dev}, of the same shape and strides")
    _dense(lens, (q.shape[0],), torch.int32, dev, "lens")
    ld_q = _rows(q, q.shape, bf, dev, "q")
    ld_new = 0
    if k_new is not None or v_new is not None:
        _ask(k_new is not None and v_new is not None, "k_new and v_new: both or neither")
        shape = (q.shape[0], cache_k.shape[2], q.shape[2])
        ld_new = _rows(k_new, shape, bf, dev, "k_new")
        _ask(_rows(v_new, shape, bf, dev, "v_new") == ld_new, "k_new and v_new need the same row stride")
    with _place(dev, stream):
        if workspace is None:
            workspace = _space(None, lambda: ttt_window_attention_decode_workspace_size(desc), dev).zero_()
        if out is None:
            out = torch.empty(q.shape, dtype=bf, device=dev)
        check(lib().ttt_window_attention_decode(
            desc.ref, q.data_ptr(), ld_q, _at(k_new), _at(v_new), ld_new, cache_k.data_ptr(), cache_v.data_ptr(),
            lens.data_ptr(), out.data_ptr(), _rows(out, q.shape, bf, dev, "out"), workspace.data_ptr(),
            workspace.numel(), _stream(stream)), "ttt_window_attention_decode")
        if check_status:
            check(ttt_mlp_status(workspace, stream), "ttt_mlp_status")
    return {"out": out, "workspace": workspace}


def _gated_desc(x, n_seq, form, dirs):
    _ask(x.dim() == 2, "x: [T, D]")
    T, D = x.shape
    return _gated_sizes(T, D, index(n_seq), TTT_GATE_FORMS[form], DIRS[dirs], _dtype_code(x, "x"))


def gated_scan_workspace(x, n_seq: int = 1) -> torch.Tensor:
    """A workspace for gated_scan and gated_scan_backward on tensors of x's shape and type."""
    desc = _gated_desc(x, n_seq, "sum", "fwd")
    return _space(None, lambda: ttt_gated_scan_workspace_size(desc), x.get_device())


def gated_scan(f, x, *, form: str = "convex", dirs: str = "fwd", cu=None, h0=None, y=None, h_T=None,
               want_state: bool = False, want_chunk_states: bool = False, chunk_states=None, workspace=None,
               check_status: bool = True, stream=None) -> dict:
    """Gated linear recurrence of the gate logits f and inputs x [T, D] (ttt_gated_scan)."""
    dev = x.get_device()
    n_seq = _offsets(cu, dev, "cu")
    desc = _gated_desc(x, n_seq, form, dirs)
    ld_f, ld_x = _rows(f, x.shape, x.dtype, dev, "f"), _rows(x, x.shape, x.dtype, dev, "x")
    state = (n_seq, x.shape[1])
    if h0 is not None:
        _dense(h0, state, torch.float32, dev, "h0")
    with _place(dev, stream):
        ws = _space(workspace, lambda: ttt_gated_scan_workspace_size(desc), dev)
        if y is None:
            y = (torch.empty if cu is None else torch.zeros)(x.shape, dtype=x.dtype, device=dev)
        if h_T is None and want_state:
            h_T = torch.empty(state, dtype=torch.float32, device=dev)
        if h_T is not None:
            _dense(h_T, state, torch.float32, dev, "h_T")
        if chunk_states is not None:
            _dense(chunk_states, (ttt_gated_scan_chunk_states_size(desc) // 4,), torch.float32, dev, "chunk_states")
        elif want_chunk_states:
            chunk_states = torch.empty(ttt_gated_scan_chunk_states_size(desc) // 4, dtype=torch.float32, device=dev)
        check(lib().ttt_gated_scan(desc.ref, _at(cu), f.data_ptr(), ld_f, x.data_ptr(), ld_x, _at(h0), y.data_ptr(),
                                   _rows(y, x.shape, x.dtype, dev, "y"), _at(h_T), _at(chunk_states), ws.data_ptr(),
                                   ws.numel(), _stream(stream)), "ttt_gated_scan")
        if check_status:
            check(ttt_mlp_status(ws, stream), "ttt_mlp_status")
    return {"y": y, "h_T": h_T, "chunk_states": chunk_states, "workspace": ws}


def gated_scan_backward(f, x, dy, chunk_states, *, form: str = "convex", dirs: str = "fwd", cu=None, h0=None,
                        dh_T=None, df=None, dx=None, dh0=None, want_dh0: bool = False, workspace=None,
                        check_status: bool = True, stream=None) -> dict:
    """Gradients of gated_scan from its inputs and chunk states (ttt_gated_scan_backward)."""
    dev = x.get_device()
    n_seq = _offsets(cu, dev, "cu")
    desc = _gated_desc(x, n_seq, form, dirs)
    state = (n_seq, x.shape[1])
    _dense(chunk_states, (ttt_gated_scan_chunk_states_size(desc) // 4,), torch.float32, dev, "chunk_states")
    for t, name in ((h0, "h0"), (dh_T, "dh_T")):
        if t is not None:
            _dense(t, state, torch.float32, dev, name)
    with _place(dev, stream):
        ws = _space(workspace, lambda: ttt_gated_scan_workspace_size(desc), dev)
        new = torch.empty if cu is None else torch.zeros
        df = new(x.shape, dtype=x.dtype, device=dev) if df is None else df
        dx = new(x.shape, dtype=x.dtype, device=dev) if dx is None else dx
        if dh0 is None and want_dh0:
            dh0 = torch.empty(state, dtype=torch.float32, device=dev)
        if dh0 is not None:
            _dense(dh0, state, torch.float32, dev, "dh0")
        dt, sx = x.dtype, x.shape
        check(lib().ttt_gated_scan_backward(
            desc.ref, _at(cu), f.data_ptr(), _rows(f, sx, dt, dev, "f"), x.data_ptr(), _rows(x, sx, dt, dev, "x"),
            _at(h0), chunk_states.data_ptr(), dy.data_ptr(), _rows(dy, sx, dt, dev, "dy"), _at(dh_T), df.data_ptr(),
            _rows(df, sx, dt, dev, "df"), dx.data_ptr(), _rows(dx, sx, dt, dev, "dx"), _at(dh0), ws.data_ptr(),
            ws.numel(), _stream(stream)), "ttt_gated_scan_backward")
        if check_status:
            check(ttt_mlp_status(ws, stream), "ttt_mlp_status")
    return {"df": df, "dx": dx, "dh0": dh0, "workspace": ws}


def gated_scan_step(f, x, h, *, form: str = "convex", y=None, h_out=None, stream=None):
    """One token of each row: returns (y, h_out) for f, x [B, D] and the state h fp32 [B, D] (h_out may be h)."""
    dev, code = x.get_device(), _dtype_code(x, "x")
    B, D = x.shape
    _ask(B < 2 ** 31 and D < 2 ** 31, "f, x: too many rows or columns")
    _dense(h, (B, D), torch.float32, dev, "h")
    with _place(dev, stream):
        y = torch.empty((B, D), dtype=x.dtype, device=dev) if y is None else y
        h_out = torch.empty_like(h) if h_out is None else _dense(h_out, (B, D), torch.float32, dev, "h_out")
        check(lib().ttt_gated_scan_step(
            B, D, TTT_GATE_FORMS[form], code, f.data_ptr(), _rows(f, x.shape, x.dtype, dev, "f"), x.data_ptr(),
            _rows(x, x.shape, x.dtype, dev, "x"), h.data_ptr(), h_out.data_ptr(), y.data_ptr(),
            _rows(y, x.shape, x.dtype, dev, "y"), _stream(stream)), "ttt_gated_scan_step")
    return y, h_out
