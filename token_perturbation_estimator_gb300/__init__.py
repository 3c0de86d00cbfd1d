"""Python binding of the GB300 Dust estimator library (``include/dust.h``).

Argument marshalling only: each function passes raw device pointers, sizes and
the current CUDA stream to the C ABI of ``lib/libdust_gb300.so``; every step
of the computation runs in that library's CUDA kernels. PyTorch supplies
device memory and streams. There is no fallback: if the library is missing
the import of a function raises.

Functions keep the C names: ``dust_noise``, ``dust_jitter_apply``,
``dust_forward_jitter``,
``dust_credit_scan``, ``dust_error_estimate``, ``dust_estimate_gW``,
``dust_estimate_gW_host``, ``dust_last_error`` (plus the workspace queries);
beside the estimator, ``dust_layer_norm``, ``dust_head_loss`` and
``dust_distill_loss``, each with its ``_grad``; and the rest of a training step,
``dust_gated_up``, ``dust_qk_norm_rope`` and ``dust_policy_loss``, each with its
``_grad``, and ``dust_clip_grads``.
"""
from __future__ import annotations

import ctypes as C
import functools
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "lib", "libdust_gb300.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "dust.h")

# dust_status
OK, ERR_INVALID_ARG, ERR_RANGE, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_WORKSPACE = range(7)
# dust_noise_kind
RADEMACHER, GAUSSIAN, RAW_WORDS, RADEMACHER_PACKED = 0, 1, 2, 3
# dust_dtype
F32, BF16, U32 = 0, 1, 2
# flags
CENTER, ANTITHETIC, ACCUMULATE = 1, 2, 4
FORCE_UNFUSED, FORCE_FUSED, WORD_STREAM1, FORCE_SIMT = 8, 16, 32, 64
# dust_path
PATH_FUSED_TC, PATH_UNFUSED_TC, PATH_SIMT = 1, 2, 3
MAX_TEACHER = 1024  # DUST_MAX_TEACHER
# dust_act, dust_rope_layout, dust_mean
SILU, GELU, RELU2 = 0, 1, 2
ROPE_HALVES, ROPE_PAIRS = 0, 1
MEAN_TOKEN, MEAN_SEQUENCE = 0, 1


class DustError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__("%s: %s" % (where, status_string(status)))


_lib = None


def _signatures():
    i32, i64, u32, u64, f32 = C.c_int32, C.c_int64, C.c_uint32, C.c_uint64, C.c_float
    f64 = C.c_double
    P, SZ, PSZ = C.c_void_p, C.c_size_t, C.POINTER(C.c_size_t)
    return {
        "dust_status_string": (C.c_char_p, [i32]),
        "dust_version": (i32, []),
        "dust_noise": (i32, [P, i32, u64, i32, i64, i64, i64, i64, u32, P]),
        "dust_jitter_apply": (i32, [P, i32, i64, i64, i64, u64, i32, i64, f32, u32, P]),
        "dust_credit_scan_workspace": (i32, [PSZ, i64, i64]),
        "dust_credit_scan": (i32, [P, i64, i64, P, i64, f32, u32, P, P, SZ, P]),
        "dust_error_estimate": (i32, [P, i64, i64, i64, u64, i32, i64, f32, u32, P, i32, P]),
        "dust_contract_workspace": (i32, [PSZ, i64, i64, i64, i32, u32]),
        "dust_contract": (i32, [P, P, i32, i64, i64, i64, f32, u32, P, P, SZ, P]),
        "dust_estimate_gW_workspace": (i32, [PSZ, i64, i64, i64, i64, i32, u32]),
        "dust_estimate_gW": (i32, [P, i32, i64, i64, P, i64, i64, P, i64, u64, i32, i64, f32,
                                   f32, f32, u32, P, P, SZ, P]),
        "dust_estimate_gW_path": (i32, [i64, i64, i64, i64, i32, u32]),
        "dust_estimate_gW_host": (i32, [P, P, i32, i64, i64, P, P, i64, i64, P, P, i64, u64,
                                        i32, i64, f32, f32, f32, u32, P, P, P, SZ, P]),
        "dust_last_error": (i32, [P]),
        "dust_estimate_gW_host_sites": (i32, [P, i64, i32, i32, i64, f32, u32, P]),
        "dust_estimate_gW_sites": (i32, [P, i64, i32, i32, i64, f32, u32, P]),
        "dust_estimate_gW_sites_lanes": (i32, []),
        "dust_credit_scan_noalloc_capacity": (SZ, []),
        "dust_credit_scan_noalloc": (i32, [P, i64, i64, P, i64, f32, u32, P, P]),
        "dust_forward_jitter": (i32, [P, P, i64, i64, i64, u64, i32, i64, i64, f32, u32, i32,
                                      P, P]),
        "dust_local_score": (i32, [P, i32, P, i32, i64, i64, i64, P, P]),
        "dust_scatter_gE_workspace": (i32, [PSZ, i64, i64, i64]),
        "dust_scatter_gE": (i32, [P, i32, P, i64, i64, i64, f32, u32, P, P, SZ, P]),
        "dust_estimate_gE_workspace": (i32, [PSZ, i64, i64, i64, i64]),
        "dust_estimate_gE": (i32, [P, i64, i64, P, i64, i64, P, i64, u64, i32, i64, f32, f32,
                                   f32, u32, P, P, SZ, P]),
        "dust_layer_norm": (i32, [P, i32, i64, i64, i64, P, P, f32, P, i64, P, P, P]),
        "dust_layer_norm_grad_workspace": (i32, [PSZ, i64, i64]),
        "dust_layer_norm_grad": (i32, [P, i64, P, i64, i32, i64, i64, P, P, P, u32, P, i64, P, P,
                                       P, SZ, P]),
        "dust_head_loss_workspace": (i32, [PSZ, i64, i64, i64, i64, i32]),
        "dust_head_loss": (i32, [P, i64, P, i64, i32, i64, i64, i64, i64, P, f32, P, P, P, P, SZ,
                                 P]),
        "dust_head_loss_grad_workspace": (i32, [PSZ, i64, i64, i64, i64, i32]),
        "dust_head_loss_grad": (i32, [P, i64, P, i64, i32, i64, i64, i64, i64, P, f32, P, P, u32,
                                      P, i64, P, i32, P, SZ, P]),
        "dust_distill_loss_workspace": (i32, [PSZ, i64, i64, i64, i64, i64, i32]),
        "dust_distill_loss": (i32, [P, i64, P, i64, i32, i64, i64, i64, i64, P, P, i64, f32, P, P,
                                    P, P, P, SZ, P]),
        "dust_distill_loss_grad_workspace": (i32, [PSZ, i64, i64, i64, i64, i64, i32]),
        "dust_distill_loss_grad": (i32, [P, i64, P, i64, i32, i64, i64, i64, i64, P, P, i64, f32,
                                         P, P, P, u32, P, i64, P, i32, P, SZ, P]),
        "dust_gated_up_workspace": (i32, [PSZ, i64, i64, i64, i32]),
        "dust_gated_up": (i32, [P, i64, P, i64, P, i64, i32, i64, i64, i64, i32, P, i64, P, SZ,
                                P]),
        "dust_gated_up_grad_workspace": (i32, [PSZ, i64, i64, i64, i32]),
        "dust_gated_up_grad": (i32, [P, i64, P, i64, P, i64, P, i64, i32, i64, i64, i64, i32, u32,
                                     P, i64, P, P, i32, P, SZ, P]),
        "dust_qk_norm_rope": (i32, [P, i64, P, i64, i32, i64, i64, P, P, f32, P, P, P, i64, i64,
                                    i32, P, P, P]),
        "dust_qk_norm_rope_grad_workspace": (i32, [PSZ, i64, i64, i64, i64]),
        "dust_qk_norm_rope_grad": (i32, [P, P, P, i64, P, i64, i32, i64, i64, P, P, f32, P, P, P,
                                         i64, i64, i32, u32, P, P, P, P, P, SZ, P]),
        "dust_policy_loss_workspace": (i32, [PSZ, i64, i64, i64]),
        "dust_policy_loss": (i32, [P, P, P, P, i32, P, i64, P, i64, i64, f64, f64, f32, i32, P, P,
                                   P, P, P, P, SZ, P]),
        "dust_policy_loss_grad": (i32, [P, P, P, P, i32, P, i64, P, i64, i64, f64, f64, f32, i32,
                                        P, P, P, SZ, P]),
        "dust_clip_grads_workspace": (i32, [PSZ, i64]),
        "dust_clip_grads": (i32, [P, i64, f32, P, P, SZ, P]),
        "dust_debug_inject_timeout": (i32, [i32]),
        "dust_pipe_probe": (i32, [i32, i64, C.POINTER(C.c_double), P, P]),
        "dust_pipe_probe_threads": (i32, []),
        "dust_profile_enable": (i32, [i32]),
        "dust_profile_read": (i32, [P, i32]),
    }


def lib():
    """The loaded C library. Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libdust_gb300.so is not built (run __graft_entry__.build() or "
                              "python token_perturbation_estimator_gb300/build.py)")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _signatures().items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def header_functions():
    """Names of the functions declared in include/dust.h."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dust_[a-zA-Z0-9_]+)\s*\(", text)))


def status_string(status: int) -> str:
    return lib().dust_status_string(int(status)).decode()


def _check(st, where):
    if st != OK:
        raise DustError(st, where)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t):
    return C.c_void_p(t.data_ptr()) if t is not None else C.c_void_p(0)


def _dtype_code(t):
    import torch
    return {torch.float32: F32, torch.bfloat16: BF16, torch.int32: U32,
            torch.uint32: U32}[t.dtype]


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        if t is not None and not t.is_contiguous():
            raise ValueError("expected a contiguous tensor")


def _expect(t, name, dtypes, shape=None, dim=None):
    """Raise ValueError unless tensor t has one of `dtypes` and, when given,
    exactly `shape` (a tuple) or `dim` dimensions: the C ABI takes raw pointers
    and sizes, so a tensor of another dtype or shape would be misread, or
    written past its end."""
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s"
                         % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if dim is not None and t.dim() != dim:
        raise ValueError("%s must have %d dimensions, got shape %s"
                         % (name, dim, tuple(t.shape)))
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _scan_inputs(delta, seq_offsets):
    import torch
    _expect(delta, "delta", (torch.float32,), dim=2)
    _expect(seq_offsets, "seq_offsets", (torch.int32,), dim=1)


# ------------------------------------------------------------------ calls --

def dust_noise(out, seed, kind, draw_begin, n_draws, T, d_out, flags=0, stream=None):
    _need_cuda(out)
    _check(lib().dust_noise(_ptr(out), _dtype_code(out), seed, kind, draw_begin, n_draws, T,
                            d_out, flags, _stream(stream)), "dust_noise")
    return out


def dust_jitter_apply(y, seed, kind, draw, sigma, flags=0, stream=None):
    """y: CUDA tensor [T, d_out] (row stride may exceed d_out)."""
    if not y.is_cuda or y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be a CUDA [T, d_out] tensor with unit column stride")
    T, d_out = y.shape
    _check(lib().dust_jitter_apply(_ptr(y), _dtype_code(y), y.stride(0), T, d_out, seed, kind,
                                   draw, float(sigma), flags, _stream(stream)),
           "dust_jitter_apply")
    return y


def dust_forward_jitter(X, W, seed, kind, draw_begin, n_draws, sigma, flags=0, clean=False,
                        Y=None, stream=None):
    """X: CUDA bf16 [T, d_in]; W: CUDA bf16 [d_out, d_in]; returns Y bf16
    [clean + n_draws, T, d_out]: X W^T, then X W^T + sigma a^(draw_begin + k)."""
    import torch
    _need_cuda(X, W, Y)
    T, d_in = X.shape
    d_out = W.shape[0]
    if W.dim() != 2 or W.shape[1] != d_in:
        raise ValueError("W must be [d_out, d_in] matching X [T, d_in]")
    c = 1 if clean else 0
    if Y is None:
        Y = torch.empty((c + n_draws, T, d_out), dtype=torch.bfloat16, device=X.device)
    if X.dtype != torch.bfloat16 or W.dtype != torch.bfloat16 or Y.dtype != torch.bfloat16:
        raise ValueError("X, W and Y must be bf16")
    if tuple(Y.shape) != (c + n_draws, T, d_out):
        raise ValueError("Y must be [clean + n_draws, T, d_out]")
    _check(lib().dust_forward_jitter(_ptr(X), _ptr(W), T, d_in, d_out, seed, kind, draw_begin,
                                     n_draws, float(sigma), flags, c, _ptr(Y), _stream(stream)),
           "dust_forward_jitter")
    return Y


def dust_local_score(g, delta_o, out=None, stream=None):
    """g: CUDA [T, d] (f32 or bf16); delta_o: CUDA [K, T, d]; returns the loss
    changes delta f32 [K, T] = <g[t], delta_o[k, t]>."""
    import torch
    _need_cuda(g, delta_o, out)
    K, T, d = delta_o.shape
    if tuple(g.shape) != (T, d):
        raise ValueError("g must be [T, d] matching delta_o [K, T, d]")
    if out is None:
        out = torch.empty((K, T), dtype=torch.float32, device=delta_o.device)
    _check(lib().dust_local_score(_ptr(g), _dtype_code(g), _ptr(delta_o), _dtype_code(delta_o),
                                  K, T, d, _ptr(out), _stream(stream)), "dust_local_score")
    return out


def dust_scatter_gE(g, ids, V, scale=1.0, flags=0, gE=None, workspace=None, stream=None):
    """g: CUDA [T, d] (f32 or bf16); ids: CUDA int32 [T]; returns gE f32 [V, d]."""
    import torch
    _need_cuda(g, ids, gE)
    T, d = g.shape
    if gE is None:
        gE = torch.empty((V, d), dtype=torch.float32, device=g.device)
    n = C.c_size_t(0)
    _check(lib().dust_scatter_gE_workspace(C.byref(n), T, V, d), "dust_scatter_gE_workspace")
    if workspace is None:
        workspace = _workspace(n.value, g.device)
    _check(lib().dust_scatter_gE(_ptr(g), _dtype_code(g), _ptr(ids), T, d, V, float(scale),
                                 flags, _ptr(gE), _ptr(workspace), workspace.numel(),
                                 _stream(stream)), "dust_scatter_gE")
    return gE


def dust_estimate_gE(ids, delta, V, d, seq_offsets, seed, kind, draw_begin, sigma, gamma,
                     scale=1.0, flags=CENTER, gE=None, workspace=None, stream=None):
    """ids: CUDA int32 [T]; delta: f32 [K, T]; returns gE f32 [V, d]."""
    import torch
    _need_cuda(ids, delta, seq_offsets, gE)
    T = ids.numel()
    K = delta.shape[0]
    if gE is None:
        gE = torch.empty((V, d), dtype=torch.float32, device=ids.device)
    n = C.c_size_t(0)
    _check(lib().dust_estimate_gE_workspace(C.byref(n), T, d, V, K), "dust_estimate_gE_workspace")
    if workspace is None:
        workspace = _workspace(n.value, ids.device)
    _check(lib().dust_estimate_gE(_ptr(ids), T, V, _ptr(delta), K, d, _ptr(seq_offsets),
                                  seq_offsets.numel() - 1, seed, kind, draw_begin, float(sigma),
                                  float(gamma), float(scale), flags, _ptr(gE), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "dust_estimate_gE")
    return gE


def dust_credit_scan_workspace(K, T):
    n = C.c_size_t(0)
    _check(lib().dust_credit_scan_workspace(C.byref(n), K, T), "dust_credit_scan_workspace")
    return n.value


def _workspace(nbytes, device):
    import torch
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def dust_credit_scan(delta, seq_offsets, gamma, flags=CENTER, r=None, workspace=None,
                     stream=None):
    """delta: f32 [K, T]; seq_offsets: i32 [n_seq+1]; returns r f32 [T, K]."""
    import torch
    _need_cuda(delta, seq_offsets, r, workspace)
    _scan_inputs(delta, seq_offsets)
    K, T = delta.shape
    if r is None:
        r = torch.empty((T, K), dtype=torch.float32, device=delta.device)
    _expect(r, "r", (torch.float32,), shape=(T, K))
    need = dust_credit_scan_workspace(K, T)
    if workspace is None:
        workspace = _workspace(need, delta.device)
    _check(lib().dust_credit_scan(_ptr(delta), K, T, _ptr(seq_offsets), seq_offsets.numel() - 1,
                                  float(gamma), flags, _ptr(r), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "dust_credit_scan")
    return r


def dust_credit_scan_noalloc(delta, seq_offsets, gamma, flags=CENTER, r=None, stream=None):
    """As dust_credit_scan, with the library's built-in scratch array instead
    of a caller workspace (for callers that cannot allocate device memory).
    r must be passed in by such callers; it is allocated here only for
    convenience when omitted."""
    import torch
    _need_cuda(delta, seq_offsets, r)
    _scan_inputs(delta, seq_offsets)
    K, T = delta.shape
    if r is None:
        r = torch.empty((T, K), dtype=torch.float32, device=delta.device)
    _expect(r, "r", (torch.float32,), shape=(T, K))
    _check(lib().dust_credit_scan_noalloc(_ptr(delta), K, T, _ptr(seq_offsets),
                                          seq_offsets.numel() - 1, float(gamma), flags, _ptr(r),
                                          _stream(stream)), "dust_credit_scan_noalloc")
    return r


def dust_error_estimate(r, d_out, seed, kind, draw_begin, sigma, flags=0, g=None,
                        g_dtype=None, stream=None):
    """r: f32 [T, K]; returns g [T, d_out] (f32 unless g_dtype=torch.bfloat16)."""
    import torch
    _need_cuda(r, g)
    _expect(r, "r", (torch.float32,), dim=2)
    T, K = r.shape
    if g is None:
        g = torch.empty((T, d_out), dtype=g_dtype or torch.float32, device=r.device)
    _expect(g, "g", (torch.float32, torch.bfloat16), shape=(T, d_out))
    _check(lib().dust_error_estimate(_ptr(r), K, T, d_out, seed, kind, draw_begin, float(sigma),
                                     flags, _ptr(g), _dtype_code(g), _stream(stream)),
           "dust_error_estimate")
    return g


def dust_contract(g, X, scale=1.0, flags=0, gW=None, workspace=None, stream=None):
    """g: [T, d_out], X: [T, d_in], same dtype (bf16 or f32); returns
    gW f32 [d_out, d_in] = scale * g^T X."""
    import torch
    _need_cuda(g, X, gW)
    T, d_out = g.shape
    d_in = X.shape[1]
    dt = _dtype_code(X)
    if gW is None:
        gW = torch.empty((d_out, d_in), dtype=torch.float32, device=X.device)
    n = C.c_size_t(0)
    _check(lib().dust_contract_workspace(C.byref(n), T, d_in, d_out, dt, flags),
           "dust_contract_workspace")
    if workspace is None:
        workspace = _workspace(n.value, X.device)
    _check(lib().dust_contract(_ptr(g), _ptr(X), dt, T, d_in, d_out, float(scale), flags,
                               _ptr(gW), _ptr(workspace), workspace.numel(), _stream(stream)),
           "dust_contract")
    return gW


def dust_estimate_gW_workspace(T, d_in, d_out, K, x_dtype, flags=CENTER):
    n = C.c_size_t(0)
    _check(lib().dust_estimate_gW_workspace(C.byref(n), T, d_in, d_out, K, x_dtype, flags),
           "dust_estimate_gW_workspace")
    return n.value


def dust_estimate_gW_path(T, d_in, d_out, K, x_dtype, flags=CENTER):
    p = lib().dust_estimate_gW_path(T, d_in, d_out, K, x_dtype, flags)
    if p < 0:
        raise DustError(-p, "dust_estimate_gW_path")
    return p


def dust_estimate_gW(X, delta, d_out, seq_offsets, seed, kind, draw_begin, sigma, gamma,
                     scale=1.0, flags=CENTER, gW=None, workspace=None, stream=None):
    """X: [T, d_in] bf16 or f32; delta: f32 [K, T]; returns gW f32 [d_out, d_in]."""
    import torch
    _need_cuda(X, delta, seq_offsets, gW, workspace)
    _expect(X, "X", (torch.float32, torch.bfloat16), dim=2)
    _scan_inputs(delta, seq_offsets)
    T, d_in = X.shape
    K = delta.shape[0]
    _expect(delta, "delta", (torch.float32,), shape=(K, T))
    xd = _dtype_code(X)
    if gW is None:
        gW = torch.empty((d_out, d_in), dtype=torch.float32, device=X.device)
    _expect(gW, "gW", (torch.float32,), shape=(d_out, d_in))
    need = dust_estimate_gW_workspace(T, d_in, d_out, K, xd, flags)
    if workspace is None:
        workspace = _workspace(need, X.device)
    _check(lib().dust_estimate_gW(_ptr(X), xd, T, d_in, _ptr(delta), K, d_out,
                                  _ptr(seq_offsets), seq_offsets.numel() - 1, seed, kind,
                                  draw_begin, float(sigma), float(gamma), float(scale), flags,
                                  _ptr(gW), _ptr(workspace), workspace.numel(),
                                  _stream(stream)), "dust_estimate_gW")
    return gW


def dust_estimate_gW_host(X_host, X_dev, delta_host, delta_dev, seq_host, seq_dev, gW_host,
                          gW_dev, d_out, seed, kind, draw_begin, sigma, gamma, scale=1.0,
                          flags=CENTER, workspace=None, stream=None):
    """Host-buffer variant: *_host are CPU tensors (pinned for async copies),
    *_dev are CUDA staging tensors of the same shapes. The caller
    synchronises the stream before reading gW_host."""
    T, d_in = X_host.shape
    K = delta_host.shape[0]
    xd = _dtype_code(X_host)
    need = dust_estimate_gW_workspace(T, d_in, d_out, K, xd, flags)
    if workspace is None:
        workspace = _workspace(need, X_dev.device)
    _check(lib().dust_estimate_gW_host(
        _ptr(X_host), _ptr(X_dev), xd, T, d_in, _ptr(delta_host), _ptr(delta_dev), K, d_out,
        _ptr(seq_host), _ptr(seq_dev), seq_host.numel() - 1, seed, kind, draw_begin,
        float(sigma), float(gamma), float(scale), flags, _ptr(gW_host), _ptr(gW_dev),
        _ptr(workspace), workspace.numel(), _stream(stream)), "dust_estimate_gW_host")
    return gW_host


# ---------------------------------------------- layer norm, head, distillation --
# These calls are short enough on the GPU for the host's part to show (a norm
# of one token takes 3 us there), so each argument is checked in one expression
# and the reason looked for only when that fails.

class _Types:
    def __init__(self):
        import torch
        self.f32, self.bf16 = torch.float32, torch.bfloat16
        self.i32, self.u8 = torch.int32, torch.uint8
        self.code = {torch.float32: F32, torch.bfloat16: BF16}
        self.empty, self.empty_like = torch.empty, torch.empty_like
        self.current_device = torch.cuda.current_device
        # The current stream's handle; the public way builds an object first (5 us).
        self.stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_types_cache = None


def _types():
    global _types_cache
    if _types_cache is None:
        _types_cache = _Types()
    return _types_cache


def _in_stream(fn):
    """Gives fn a keyword `stream`: it then runs with that stream and its device current, so
    that what it allocates (outputs not passed in, workspace) belongs to the
    stream that uses it and is not handed out again while the call runs."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        import torch
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream))
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _dense(t, name, dtype, shape, dev):
    """The address of t (None: NULL). Raises ValueError unless it is a
    contiguous tensor of this dtype and shape on CUDA device `dev`."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == dev):
        _need_cuda(t)
        _expect(t, name, (dtype,), shape=shape)
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    return t.data_ptr()


def _rows(t, name, dtype, shape, dev):
    """The row stride in elements of t, a tensor of this dtype and shape [T, d]
    on CUDA device `dev` with unit column stride and rows that do not overlap;
    raises ValueError for any other."""
    T, d = shape
    if not (t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        _expect(t, name, (dtype,), shape=shape)
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    ld, step = t.stride()
    if T <= 1:
        ld = max(ld, d)
    if (d > 1 and step != 1) or ld < d:
        raise ValueError("%s must have unit column stride and rows that do not overlap" % name)
    return ld


def _values(t, name, dims):
    """The dtype code and CUDA device of t, an f32 or bf16 tensor on the current
    device with one of these numbers of dimensions; raises ValueError for any
    other. (The launch goes to the current device, whatever device its stream
    was asked for: a default stream's handle is 0 on every one.)"""
    ty = _types()
    code = ty.code.get(t.dtype)
    if code is None or not t.is_cuda or t.dim() not in dims:
        if not t.is_cuda:
            raise ValueError("expected a CUDA tensor")
        raise ValueError("%s must be f32 or bf16 with %s dimensions, got %s %s"
                         % (name, " or ".join(map(str, dims)), t.dtype, tuple(t.shape)))
    dev = t.get_device()
    if dev != ty.current_device():
        raise ValueError("%s is on cuda:%d, but the current device (the stream's, where one is "
                         "given) is cuda:%d" % (name, dev, ty.current_device()))
    return code, dev


@functools.lru_cache(maxsize=256)  # a size follows from the other sizes alone
def _query(name, *args):
    n = C.c_size_t(0)
    _check(getattr(lib(), name)(C.byref(n), *args), name)
    return n.value


def _space(workspace, name, ref, dev, *args):
    """The caller's workspace, or a new one of the size that query `name` gives:
    (tensor, address, bytes)."""
    if workspace is None:
        n = _query(name, *args)
        if n == 0:
            return None, None, 0
        workspace = _types().empty(n, dtype=_types().u8, device=ref.device)
        return workspace, workspace.data_ptr(), n
    n = workspace.numel()
    return workspace, _dense(workspace, "workspace", _types().u8, (n,), dev), n


def _output(t, name, dtype, shape, ref, dev):
    """The caller's output, checked, or a new one: (tensor, address)."""
    if t is None:
        t = _types().empty(shape, dtype=dtype, device=ref.device)
        return t, t.data_ptr()
    return t, _dense(t, name, dtype, shape, dev)


def _output_rows(t, name, dtype, shape, ref, dev):
    """The same for rows that may be strided: (tensor, address, row stride)."""
    if t is None:
        t = _types().empty(shape, dtype=dtype, device=ref.device)
        return t, t.data_ptr(), shape[1]
    return t, t.data_ptr(), _rows(t, name, dtype, shape, dev)


@_in_stream
def dust_layer_norm(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None):
    """x: CUDA [T, d] (f32 or bf16, rows may be strided); weight, bias: f32 [d]
    or None; returns (y of x's dtype [T, d], mean f32 [T], rstd f32 [T])."""
    ty = _types()
    code, dev = _values(x, "x", (2,))
    T, d = shape = x.shape
    y, y_at, ld_y = _output_rows(y, "y", x.dtype, shape, x, dev)
    mean, mean_at = _output(mean, "mean", ty.f32, (T,), x, dev)
    rstd, rstd_at = _output(rstd, "rstd", ty.f32, (T,), x, dev)
    st = lib().dust_layer_norm(
        x.data_ptr(), code, _rows(x, "x", x.dtype, shape, dev), T, d,
        _dense(weight, "weight", ty.f32, (d,), dev), _dense(bias, "bias", ty.f32, (d,), dev),
        eps, y_at, ld_y, mean_at, rstd_at, ty.stream_of(dev))
    _check(st, "dust_layer_norm")
    return y, mean, rstd


@_in_stream
def dust_layer_norm_grad(gy, x, mean, rstd, weight=None, flags=0, gx=None, gweight=None,
                         gbias=None, workspace=None):
    """gy, x: CUDA [T, d] (f32 or bf16, one dtype, rows may be strided); mean,
    rstd: f32 [T] of the forward; weight: f32 [d] or None. Returns (gx of x's
    dtype [T, d], gweight f32 [d], gbias f32 [d]); ACCUMULATE adds to the
    gweight and gbias that are passed in."""
    ty = _types()
    code, dev = _values(x, "x", (2,))
    T, d = shape = x.shape
    if flags & ACCUMULATE and (gweight is None or gbias is None):
        raise ValueError("ACCUMULATE needs the gweight and gbias to add to")
    gx, gx_at, ld_gx = _output_rows(gx, "gx", x.dtype, shape, x, dev)
    gweight, gweight_at = _output(gweight, "gweight", ty.f32, (d,), x, dev)
    gbias, gbias_at = _output(gbias, "gbias", ty.f32, (d,), x, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_layer_norm_grad_workspace", x, dev, T, d)
    st = lib().dust_layer_norm_grad(
        gy.data_ptr(), _rows(gy, "gy", x.dtype, shape, dev), x.data_ptr(),
        _rows(x, "x", x.dtype, shape, dev), code, T, d,
        _dense(weight, "weight", ty.f32, (d,), dev), _dense(mean, "mean", ty.f32, (T,), dev),
        _dense(rstd, "rstd", ty.f32, (T,), dev), flags, gx_at, ld_gx, gweight_at, gbias_at,
        ws_at, ws_bytes, ty.stream_of(dev))
    _check(st, "dust_layer_norm_grad")
    return gx, gweight, gbias


def _head_inputs(H, E):
    """dtype code, device, sizes S, T, d, V and the addresses and row strides
    of H [T, d] or [S, T, d] and E [V, d], as the C calls take them."""
    code, dev = _values(H, "H", (2, 3))
    if H.dim() == 3:
        S, T, d = H.shape
        if S == 1:
            rows = H[0]
        elif T == 1:  # the stride between a slice's rows says nothing
            rows = H[:, 0]
        elif T > 0 and H.stride(0) != T * H.stride(1):
            raise ValueError("the slices of H must follow one another")
        else:
            rows = H.as_strided((S * T, d), (H.stride(1), H.stride(2)))
    else:
        S, (T, d), rows = 1, H.shape, H
    ld_h = _rows(rows, "H", H.dtype, (S * T, d), dev)
    if E.dim() != 2 or E.shape[1] != d:
        raise ValueError("E must be [V, d] matching H, got %s" % (tuple(E.shape),))
    V = E.shape[0]
    return code, dev, S, T, d, V, (H.data_ptr(), ld_h, E.data_ptr(),
                                   _rows(E, "E", H.dtype, (V, d), dev), code, S, T, d, V)


def _loss_outputs(H, S, T, dev, loss, lse, delta, changes):
    ty = _types()
    shape = H.shape[:-1]
    loss, loss_at = _output(loss, "loss", ty.f32, shape, H, dev)
    lse, lse_at = _output(lse, "lse", ty.f32, shape, H, dev)
    delta_at = None
    if delta is not None or changes:
        delta, delta_at = _output(delta, "delta", ty.f32, (S - 1, T), H, dev)
    return loss, lse, delta, (loss_at, lse_at), delta_at


def _grad_outputs(H, E, d, dev, flags, gH, gE, gE_dtype):
    ty = _types()
    if flags & ACCUMULATE and gE is None:
        raise ValueError("ACCUMULATE needs the gE to add to")
    ge_type = (gE_dtype or ty.f32) if gE is None else gE.dtype
    gcode = ty.code.get(ge_type)
    if gcode is None:
        raise ValueError("gE must be f32 or bf16, got %s" % ge_type)
    gH, gh_at = _output(gH, "gH", H.dtype, H.shape, H, dev)
    gE, ge_at = _output(gE, "gE", ge_type, E.shape, E, dev)
    return gH, gE, (flags, gh_at, d, ge_at, gcode)


@_in_stream
def dust_head_loss(H, E, targets, scale=1.0, changes=False, loss=None, lse=None, delta=None,
                   workspace=None):
    """H: CUDA [T, d] or [S, T, d] (f32 or bf16); E: [V, d] of H's dtype;
    targets: i32 [T], negative where a token has none. Returns (loss, lse), f32
    of H's leading shape, and with changes=True also delta f32 [S - 1, T], each
    later slice's loss minus the first one's. No logits are kept."""
    ty = _types()
    code, dev, S, T, d, V, operands = _head_inputs(H, E)
    loss, lse, delta, outs, delta_at = _loss_outputs(H, S, T, dev, loss, lse, delta, changes)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_head_loss_workspace", H, dev,
                                        S, T, d, V, code)
    st = lib().dust_head_loss(*operands, _dense(targets, "targets", ty.i32, (T,), dev), scale,
                              *outs, delta_at, ws_at, ws_bytes, ty.stream_of(dev))
    _check(st, "dust_head_loss")
    return (loss, lse) if delta is None else (loss, lse, delta)


@_in_stream
def dust_head_loss_grad(H, E, targets, lse, gloss, scale=1.0, flags=0, gH=None, gE=None,
                        gE_dtype=None, workspace=None):
    """The gradients of dust_head_loss for gloss (f32, the losses' gradient, H's
    leading shape) and the forward's lse: returns (gH of H's shape and dtype,
    gE [V, d], f32 unless gE_dtype is bf16); ACCUMULATE adds to the f32 gE that
    is passed in."""
    ty = _types()
    code, dev, S, T, d, V, operands = _head_inputs(H, E)
    shape = H.shape[:-1]
    gH, gE, outs = _grad_outputs(H, E, d, dev, flags, gH, gE, gE_dtype)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_head_loss_grad_workspace", H, dev,
                                        S, T, d, V, code)
    st = lib().dust_head_loss_grad(*operands, _dense(targets, "targets", ty.i32, (T,), dev),
                                   scale, _dense(lse, "lse", ty.f32, shape, dev),
                                   _dense(gloss, "gloss", ty.f32, shape, dev), *outs,
                                   ws_at, ws_bytes, ty.stream_of(dev))
    _check(st, "dust_head_loss_grad")
    return gH, gE


def _teacher_inputs(ids, teacher, T, dev):
    ty = _types()
    if ids.dim() != 2:
        raise ValueError("ids must be [T, K], got shape %s" % (tuple(ids.shape),))
    K = ids.shape[1]
    return K, (_dense(ids, "ids", ty.i32, (T, K), dev),
               _dense(teacher, "teacher", ty.f32, (T, K), dev), K)


@_in_stream
def dust_distill_loss(H, E, ids, teacher, scale=1.0, changes=False, loss=None, lse=None,
                      student=None, delta=None, workspace=None):
    """Distillation from a teacher's K stored logits a token. H, E as for
    dust_head_loss; ids: i32 [T, K], negative where an entry is absent; teacher:
    f32 [T, K]. Returns (loss, lse, student), student f32 [..., K] the scaled
    logits at ids, and with changes=True also delta f32 [S - 1, T]."""
    ty = _types()
    code, dev, S, T, d, V, operands = _head_inputs(H, E)
    K, entries = _teacher_inputs(ids, teacher, T, dev)
    loss, lse, delta, outs, delta_at = _loss_outputs(H, S, T, dev, loss, lse, delta, changes)
    shape = (*H.shape[:-1], K)
    student, student_at = _output(student, "student", ty.f32, shape, H, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_distill_loss_workspace", H, dev,
                                        S, T, d, V, K, code)
    st = lib().dust_distill_loss(*operands, *entries, scale, *outs, student_at, delta_at,
                                 ws_at, ws_bytes, ty.stream_of(dev))
    _check(st, "dust_distill_loss")
    return (loss, lse, student) if delta is None else (loss, lse, student, delta)


@_in_stream
def dust_distill_loss_grad(H, E, ids, teacher, lse, student, gloss, scale=1.0, flags=0, gH=None,
                           gE=None, gE_dtype=None, workspace=None):
    """The gradients of dust_distill_loss for gloss and the forward's lse and
    student; returns (gH, gE) as dust_head_loss_grad does."""
    ty = _types()
    code, dev, S, T, d, V, operands = _head_inputs(H, E)
    K, entries = _teacher_inputs(ids, teacher, T, dev)
    shape = H.shape[:-1]
    gH, gE, outs = _grad_outputs(H, E, d, dev, flags, gH, gE, gE_dtype)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_distill_loss_grad_workspace", H, dev,
                                        S, T, d, V, K, code)
    st = lib().dust_distill_loss_grad(*operands, *entries, scale,
                                      _dense(lse, "lse", ty.f32, shape, dev),
                                      _dense(student, "student", ty.f32, (*shape, K), dev),
                                      _dense(gloss, "gloss", ty.f32, shape, dev), *outs,
                                      ws_at, ws_bytes, ty.stream_of(dev))
    _check(st, "dust_distill_loss_grad")
    return gH, gE


# ------------------------------------------------ the rest of a training step --

def _gated_inputs(X, Wg, Wu):
    code, dev = _values(X, "X", (2,))
    T, d = X.shape
    if Wg.dim() != 2 or Wg.shape[1] != d:
        raise ValueError("Wg must be [f, d] matching X, got %s" % (tuple(Wg.shape),))
    f = Wg.shape[0]
    return code, dev, T, d, f, (
        X.data_ptr(), _rows(X, "X", X.dtype, (T, d), dev), Wg.data_ptr(),
        _rows(Wg, "Wg", X.dtype, (f, d), dev), Wu.data_ptr(), _rows(Wu, "Wu", X.dtype, (f, d), dev),
        code, T, d, f)


@_in_stream
def dust_gated_up(X, Wg, Wu, act=SILU, h=None, workspace=None):
    """X: CUDA [T, d]; Wg, Wu: [f, d] (all f32 or all bf16, rows may be strided);
    returns h = act(X Wg^T) (X Wu^T), [T, f] of X's dtype."""
    code, dev, T, d, f, operands = _gated_inputs(X, Wg, Wu)
    h, h_at, ld_h = _output_rows(h, "h", X.dtype, (T, f), X, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_gated_up_workspace", X, dev, T, d, f, code)
    st = lib().dust_gated_up(*operands, act, h_at, ld_h, ws_at, ws_bytes, _types().stream_of(dev))
    _check(st, "dust_gated_up")
    return h


@_in_stream
def dust_gated_up_grad(gh, X, Wg, Wu, act=SILU, flags=0, gX=None, gWg=None, gWu=None,
                       gW_dtype=None, workspace=None):
    """The gradients of dust_gated_up for gh ([T, f], X's dtype): returns (gX of
    X's shape and dtype, gWg, gWu [f, d], f32 unless gW_dtype is bf16);
    ACCUMULATE adds to the f32 gWg and gWu that are passed in."""
    ty = _types()
    code, dev, T, d, f, operands = _gated_inputs(X, Wg, Wu)
    if flags & ACCUMULATE and (gWg is None or gWu is None):
        raise ValueError("ACCUMULATE needs the gWg and gWu to add to")
    given = gWg if gWg is not None else gWu
    gw_type = (gW_dtype or ty.f32) if given is None else given.dtype
    gcode = ty.code.get(gw_type)
    if gcode is None:
        raise ValueError("gWg and gWu must be f32 or bf16, got %s" % gw_type)
    gX, gx_at, ld_gx = _output_rows(gX, "gX", X.dtype, (T, d), X, dev)
    gWg, gwg_at = _output(gWg, "gWg", gw_type, (f, d), X, dev)
    gWu, gwu_at = _output(gWu, "gWu", gw_type, (f, d), X, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_gated_up_grad_workspace", X, dev, T, d, f,
                                        code)
    st = lib().dust_gated_up_grad(gh.data_ptr(), _rows(gh, "gh", X.dtype, (T, f), dev), *operands,
                                  act, flags, gx_at, ld_gx, gwg_at, gwu_at, gcode, ws_at, ws_bytes,
                                  ty.stream_of(dev))
    _check(st, "dust_gated_up_grad")
    return gX, gWg, gWu


class _Heads(C.Structure):
    """dust_heads of include/dust.h."""
    _fields_ = [("data", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


def _heads(t, name, dtype, shape, dev):
    """A reference to the dust_heads of t, a tensor of this dtype and shape [T, heads, D] on CUDA
    device `dev` with unit stride inside a head; raises ValueError for any other."""
    if t is None or not (t.dtype is dtype and t.shape == shape and t.get_device() == dev):
        if t is None or not t.is_cuda:
            raise ValueError("%s: expected a CUDA tensor" % name)
        _expect(t, name, (dtype,), shape=shape)
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    token, head, step = t.stride()
    if shape[2] > 1 and step != 1:
        raise ValueError("%s must have unit stride inside a head" % name)
    return C.byref(_Heads(t.data_ptr(), token, head))


def _output_heads(t, name, dtype, shape, ref, dev):
    """The caller's output, or a new one: (tensor, its dust_heads)."""
    if t is None:
        t = _types().empty(shape, dtype=dtype, device=ref.device)
        return t, C.byref(_Heads(t.data_ptr(), shape[1] * shape[2], shape[2]))
    return t, _heads(t, name, dtype, shape, dev)


def _rope_inputs(q, k, wq, wk, positions, cosine, sine, eps, layout):
    ty = _types()
    code, dev = _values(q, "q", (3,))
    T, hq, D = q.shape
    hk = 0 if k is None else k.shape[1]
    if k is not None and (k.dim() != 3 or k.shape[0] != T or k.shape[2] != D):
        raise ValueError("k must be [T, heads, D] matching q, got %s" % (tuple(k.shape),))
    if cosine is None:
        n_pos, rot = 1 << 31, 0  # no table: any position will do
    else:
        if cosine.dim() != 2:
            raise ValueError("cosine must be [positions, rot / 2], got %s" % (tuple(cosine.shape),))
        n_pos, rot = cosine.shape[0], 2 * cosine.shape[1]
    hs_q = _heads(q, "q", q.dtype, (T, hq, D), dev)
    hs_k = None if k is None else _heads(k, "k", q.dtype, (T, hk, D), dev)
    args = (hs_q, hq, hs_k, hk, code, T, D, _dense(wq, "wq", ty.f32, (D,), dev),
            _dense(wk, "wk", ty.f32, (D,), dev), eps, _dense(positions, "positions", ty.i32, (T,), dev),
            _dense(cosine, "cosine", ty.f32, (n_pos, rot // 2), dev),
            _dense(sine, "sine", ty.f32, (n_pos, rot // 2), dev), n_pos, rot, layout)
    return ty, dev, T, hq, hk, D, args


@_in_stream
def dust_qk_norm_rope(q, k, wq, wk, positions, cosine, sine, eps=1e-6, layout=ROPE_HALVES, yq=None,
                      yk=None):
    """q: CUDA [T, hq, D]; k: [T, hk, D] or None (f32 or bf16, tokens and heads
    may be strided, as in a fused projection's row); wq, wk: f32 [D] or None;
    positions: i32 [T], negative for padding; cosine, sine: f32 [positions,
    rot / 2] (None: no rotation). Returns (yq, yk), normed and turned."""
    ty, dev, T, hq, hk, D, args = _rope_inputs(q, k, wq, wk, positions, cosine, sine, eps, layout)
    yq, hs_q = _output_heads(yq, "yq", q.dtype, (T, hq, D), q, dev)
    hs_k = None
    if k is not None:
        yk, hs_k = _output_heads(yk, "yk", q.dtype, (T, hk, D), q, dev)
    st = lib().dust_qk_norm_rope(*args, hs_q, hs_k, ty.stream_of(dev))
    _check(st, "dust_qk_norm_rope")
    return yq, yk


@_in_stream
def dust_qk_norm_rope_grad(gyq, gyk, q, k, wq, wk, positions, cosine, sine, eps=1e-6,
                           layout=ROPE_HALVES, flags=0, gq=None, gk=None, gwq=None, gwk=None,
                           workspace=None):
    """The gradients of dust_qk_norm_rope for gyq and gyk: returns (gq, gk, gwq
    f32 [D], gwk f32 [D]); ACCUMULATE adds to the gwq and gwk that are passed
    in. gyk, gk and gwk are not used where k is None."""
    ty, dev, T, hq, hk, D, args = _rope_inputs(q, k, wq, wk, positions, cosine, sine, eps, layout)
    if flags & ACCUMULATE and (gwq is None or (k is not None and gwk is None)):
        raise ValueError("ACCUMULATE needs the gwq and gwk to add to")
    gy_q, gy_k = _heads(gyq, "gyq", q.dtype, (T, hq, D), dev), None
    gq, hs_q = _output_heads(gq, "gq", q.dtype, (T, hq, D), q, dev)
    gwq, gwq_at = _output(gwq, "gwq", ty.f32, (D,), q, dev)
    hs_k = gwk_at = None
    if k is not None:
        gy_k = _heads(gyk, "gyk", q.dtype, (T, hk, D), dev)
        gk, hs_k = _output_heads(gk, "gk", q.dtype, (T, hk, D), q, dev)
        gwk, gwk_at = _output(gwk, "gwk", ty.f32, (D,), q, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_qk_norm_rope_grad_workspace", q, dev, T, hq,
                                        hk, D)
    st = lib().dust_qk_norm_rope_grad(gy_q, gy_k, *args, flags, hs_q, hs_k, gwq_at, gwk_at, ws_at,
                                      ws_bytes, ty.stream_of(dev))
    _check(st, "dust_qk_norm_rope_grad")
    return gq, gk, gwq, gwk


def _policy_inputs(nll, old, advantages, seq_offsets, ref, targets, clip_low, clip_high, beta, mean,
                   per_token):
    ty = _types()
    if not nll.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if nll.dtype is not ty.f32 or nll.dim() not in (1, 2):
        raise ValueError("nll must be f32 [T] or [S, T], got %s %s" % (nll.dtype, tuple(nll.shape)))
    _, dev = _values(nll, "nll", (1, 2))
    S, T = (1, nll.shape[0]) if nll.dim() == 1 else nll.shape
    n_seq = seq_offsets.numel() - 1
    if n_seq < 0:
        raise ValueError("seq_offsets must have at least one value")
    if per_token is None:
        n = advantages.numel()
        if n == T and n == n_seq and n > 1:
            raise ValueError("as many sequences as tokens: say whether advantages are per_token")
        per_token = n == T
    operands = (_dense(nll, "nll", ty.f32, nll.shape, dev), _dense(old, "old", ty.f32, (T,), dev),
                _dense(ref, "ref", ty.f32, (T,), dev),
                _dense(advantages, "advantages", ty.f32, (T if per_token else n_seq,), dev),
                1 if per_token else 0,
                _dense(seq_offsets, "seq_offsets", ty.i32, (n_seq + 1,), dev), n_seq,
                _dense(targets, "targets", ty.i32, (T,), dev), S, T, clip_low, clip_high, beta, mean)
    return ty, dev, S, T, n_seq, operands


@_in_stream
def dust_policy_loss(nll, old, advantages, seq_offsets, ref=None, targets=None, clip_low=0.2,
                     clip_high=0.2, beta=0.0, mean=MEAN_TOKEN, per_token=None, changes=False,
                     loss=None, total=None, kl=None, clipped=None, delta=None, workspace=None):
    """nll: CUDA f32 [T] or [S, T], dust_head_loss's losses; old, ref: f32 [T], the
    samples' under the policy that drew them and under the reference;
    advantages: f32 [T] or [n_seq] (per_token tells where both fit); targets:
    i32 [T], negative where a token is not scored. Returns (loss of nll's
    shape, total, kl, clipped of nll's leading shape), and with changes=True
    also delta f32 [S - 1, T], each later slice's loss minus the first one's."""
    ty, dev, S, T, n_seq, operands = _policy_inputs(
        nll, old, advantages, seq_offsets, ref, targets, clip_low, clip_high, beta, mean, per_token)
    lead = nll.shape[:-1]
    loss, loss_at = _output(loss, "loss", ty.f32, nll.shape, nll, dev)
    total, total_at = _output(total, "total", ty.f32, lead, nll, dev)
    kl, kl_at = _output(kl, "kl", ty.f32, lead, nll, dev)
    clipped, clipped_at = _output(clipped, "clipped", ty.f32, lead, nll, dev)
    delta_at = None
    if delta is not None or changes:
        delta, delta_at = _output(delta, "delta", ty.f32, (S - 1, T), nll, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_policy_loss_workspace", nll, dev, S, T,
                                        n_seq)
    st = lib().dust_policy_loss(*operands, loss_at, total_at, kl_at, clipped_at, delta_at, ws_at,
                                ws_bytes, ty.stream_of(dev))
    _check(st, "dust_policy_loss")
    return (loss, total, kl, clipped) if delta is None else (loss, total, kl, clipped, delta)


@_in_stream
def dust_policy_loss_grad(nll, old, advantages, seq_offsets, gtotal, ref=None, targets=None,
                          clip_low=0.2, clip_high=0.2, beta=0.0, mean=MEAN_TOKEN, per_token=None,
                          gnll=None, workspace=None):
    """The gradient of dust_policy_loss's total for gtotal (f32, nll's leading
    shape): gnll of nll's shape, which dust_head_loss_grad takes as gloss."""
    ty, dev, S, T, n_seq, operands = _policy_inputs(
        nll, old, advantages, seq_offsets, ref, targets, clip_low, clip_high, beta, mean, per_token)
    gnll, gnll_at = _output(gnll, "gnll", ty.f32, nll.shape, nll, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_policy_loss_workspace", nll, dev, S, T,
                                        n_seq)
    st = lib().dust_policy_loss_grad(*operands,
                                     _dense(gtotal, "gtotal", ty.f32, nll.shape[:-1], dev),
                                     gnll_at, ws_at, ws_bytes, ty.stream_of(dev))
    _check(st, "dust_policy_loss_grad")
    return gnll


class _On:
    """What _output and _space ask of a tensor: where it is."""
    def __init__(self, dev):
        import torch
        self.device = torch.device("cuda", dev)


_on = functools.lru_cache(maxsize=None)(_On)


@_in_stream
def dust_clip_grads(grads, max_norm, out=None, norm=None, workspace=None):
    """grads: a list of contiguous CUDA tensors (f32 or bf16 each), scaled by
    min(1, max_norm / norm) with the norm over all of them: in place, or into
    the tensors `out`. Returns (norm f32 [1], the scaled tensors)."""
    ty = _types()
    dev, codes = ty.current_device(), ty.code
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError("out must have as many tensors as grads")
    flat = []  # dust_grad of include/dust.h, as 64-bit words
    for g, o in zip(grads, out):
        code = codes.get(g.dtype)
        if code is None or not g.is_contiguous() or g.get_device() != dev:
            _values(g, "a gradient", range(65))
            raise ValueError("expected a contiguous tensor")
        to = at = g.data_ptr()
        if o is not g:
            if not (o.dtype is g.dtype and o.shape == g.shape and o.is_contiguous()
                    and o.get_device() == dev):
                _dense(o, "out", g.dtype, g.shape, dev)  # raises
            to = o.data_ptr()
        flat += (at, to, g.numel(), code)
    words = (C.c_int64 * len(flat))(*flat)
    ref = _on(dev)
    norm, norm_at = _output(norm, "norm", ty.f32, (1,), ref, dev)
    workspace, ws_at, ws_bytes = _space(workspace, "dust_clip_grads_workspace", ref, dev, len(grads))
    st = lib().dust_clip_grads(C.addressof(words), len(grads), max_norm, norm_at, ws_at, ws_bytes,
                               ty.stream_of(dev))
    _check(st, "dust_clip_grads")
    return norm, out


PIPE_XU, PIPE_ALU, PIPE_FMA, PIPE_ISSUE = 0, 1, 2, 3


def dust_pipe_probe(pipe, steps, sink, stream=None):
    """Enqueue one pipe-rate probe launch; returns the number of counted
    operations it performs (time it with CUDA events on `stream`). `sink`:
    CUDA float tensor of at least dust_pipe_probe_threads() elements."""
    _need_cuda(sink)
    if sink.numel() < dust_pipe_probe_threads():
        raise ValueError("sink must hold dust_pipe_probe_threads() floats")
    ops = C.c_double(0.0)
    _check(lib().dust_pipe_probe(int(pipe), int(steps), C.byref(ops), _ptr(sink),
                                 _stream(stream)), "dust_pipe_probe")
    return ops.value


def dust_pipe_probe_threads():
    n = lib().dust_pipe_probe_threads()
    if n < 0:
        raise DustError(-n, "dust_pipe_probe_threads")
    return n


class Site(C.Structure):
    """dust_site of include/dust.h: one layer of a multi-site device call."""
    _fields_ = [("X", C.c_void_p), ("T", C.c_int64), ("d_in", C.c_int64),
                ("d_out", C.c_int64), ("delta", C.c_void_p), ("K", C.c_int64),
                ("seq_offsets", C.c_void_p), ("n_seq", C.c_int64), ("seed", C.c_uint64),
                ("sigma", C.c_float), ("gamma", C.c_float), ("gW", C.c_void_p),
                ("workspace", C.c_void_p), ("ws_bytes", C.c_size_t)]


class SiteArray:
    """The marshalled site array of a dust_estimate_gW_sites call, built once
    from a list of dicts (see dust_estimate_gW_sites) and reusable while the
    tensors it points to live (it keeps references to them)."""

    def __init__(self, sites):
        import torch
        self.sites = list(sites)
        self.arr = (Site * max(1, len(self.sites)))()
        self.x_dtype = None
        for i, q in enumerate(self.sites):
            X, delta, so, gW, ws = q["X"], q["delta"], q["seq_offsets"], q["gW"], q["workspace"]
            _need_cuda(X, delta, so, gW, ws)
            _expect(X, "X", (torch.float32, torch.bfloat16), dim=2)
            T, d_in = X.shape
            _expect(delta, "delta", (torch.float32,), dim=2)
            K = delta.shape[0]
            _expect(delta, "delta", (torch.float32,), shape=(K, T))
            _expect(so, "seq_offsets", (torch.int32,), dim=1)
            _expect(gW, "gW", (torch.float32,), dim=2)
            d_out = gW.shape[0]
            _expect(gW, "gW", (torch.float32,), shape=(d_out, d_in))
            _expect(ws, "workspace", (torch.uint8,), dim=1)
            code = _dtype_code(X)
            if self.x_dtype is None:
                self.x_dtype = code
            elif code != self.x_dtype:
                raise ValueError("every site's X must have the same dtype")
            self.arr[i] = Site(_ptr(X), T, d_in, d_out, _ptr(delta), K, _ptr(so), so.numel() - 1,
                               int(q["seed"]), float(q["sigma"]), float(q["gamma"]), _ptr(gW),
                               _ptr(ws), ws.numel())


def dust_estimate_gW_sites(sites, kind, draw_begin, scale=1.0, flags=CENTER, stream=None):
    """Several layers on device buffers in one pass on the library's compute
    lanes (one site's contraction overlaps later sites' weighting).
    `sites`: a SiteArray, or a list of dicts with the CUDA tensors X [T, d_in]
    (bf16 or f32, one dtype for all), delta f32 [K, T], seq_offsets i32
    [n_seq+1], gW f32 [d_out, d_in] (written), a uint8 `workspace` of at least
    dust_estimate_gW_workspace bytes, and the scalars seed, sigma, gamma.
    Returns the gW tensors."""
    a = sites if isinstance(sites, SiteArray) else SiteArray(sites)
    _check(lib().dust_estimate_gW_sites(C.cast(a.arr, C.c_void_p), len(a.sites),
                                        BF16 if a.x_dtype is None else a.x_dtype, kind,
                                        draw_begin, float(scale), flags, _stream(stream)),
           "dust_estimate_gW_sites")
    return [q["gW"] for q in a.sites]


def dust_estimate_gW_sites_lanes():
    return int(lib().dust_estimate_gW_sites_lanes())


class HostSite(C.Structure):
    """dust_host_site of include/dust.h: one layer of a multi-site call."""
    _fields_ = [("X_host", C.c_void_p), ("X_dev", C.c_void_p), ("T", C.c_int64),
                ("d_in", C.c_int64), ("d_out", C.c_int64), ("delta_host", C.c_void_p),
                ("delta_dev", C.c_void_p), ("K", C.c_int64), ("seq_offsets_host", C.c_void_p),
                ("seq_dev", C.c_void_p), ("n_seq", C.c_int64), ("seed", C.c_uint64),
                ("sigma", C.c_float), ("gamma", C.c_float), ("gW_host", C.c_void_p),
                ("gW_dev", C.c_void_p), ("workspace", C.c_void_p), ("ws_bytes", C.c_size_t)]


def dust_estimate_gW_host_sites(sites, kind, draw_begin, scale=1.0, flags=CENTER, stream=None):
    """Several layers from host buffers in one pass (later sites' inputs are
    copied while earlier sites compute). `sites`: list of dicts with the CPU
    tensors X_host [T, d_in], delta_host f32 [K, T], seq_host i32 [n_seq+1],
    gW_host f32 [d_out, d_in] (pinned for overlap), the CUDA staging tensors
    X_dev, delta_dev, seq_dev, gW_dev of the same shapes, a CUDA uint8
    `workspace` and the scalars seed, sigma, gamma. All X share one dtype.
    The caller synchronises the stream before reading the gW_host tensors."""
    import torch
    arr = (HostSite * max(1, len(sites)))()
    xd = None
    for i, q in enumerate(sites):
        Xh, Xd = q["X_host"], q["X_dev"]
        _need_cuda(Xd, q["delta_dev"], q["seq_dev"], q["gW_dev"], q["workspace"])
        _expect(Xh, "X_host", (torch.float32, torch.bfloat16), dim=2)
        T, d_in = Xh.shape
        d_out = q["gW_host"].shape[0]
        K = q["delta_host"].shape[0]
        n_seq = q["seq_host"].numel() - 1
        _expect(Xd, "X_dev", (Xh.dtype,), shape=(T, d_in))
        for nm in ("delta_host", "delta_dev"):
            _expect(q[nm], nm, (torch.float32,), shape=(K, T))
        for nm in ("seq_host", "seq_dev"):
            _expect(q[nm], nm, (torch.int32,), shape=(n_seq + 1,))
        for nm in ("gW_host", "gW_dev"):
            _expect(q[nm], nm, (torch.float32,), shape=(d_out, d_in))
        code = _dtype_code(Xh)
        if xd is None:
            xd = code
        elif code != xd:
            raise ValueError("every site's X must have the same dtype")
        arr[i] = HostSite(_ptr(Xh), _ptr(Xd), T, d_in, d_out, _ptr(q["delta_host"]),
                          _ptr(q["delta_dev"]), K, _ptr(q["seq_host"]), _ptr(q["seq_dev"]),
                          n_seq, int(q["seed"]), float(q["sigma"]), float(q["gamma"]),
                          _ptr(q["gW_host"]), _ptr(q["gW_dev"]), _ptr(q["workspace"]),
                          q["workspace"].numel())
    _check(lib().dust_estimate_gW_host_sites(C.cast(arr, C.c_void_p), len(sites),
                                             BF16 if xd is None else xd, kind, draw_begin,
                                             float(scale), flags, _stream(stream)),
           "dust_estimate_gW_host_sites")
    return [q["gW_host"] for q in sites]


def dust_last_error(stream=None):
    return int(lib().dust_last_error(_stream(stream)))


class _ProfileEntry(C.Structure):
    _fields_ = [("name", C.c_char * 32), ("launches", C.c_int64), ("total_ms", C.c_double)]


def dust_profile_enable(on=True):
    _check(lib().dust_profile_enable(1 if on else 0), "dust_profile_enable")


def dust_profile_read():
    """{kernel family: (launches, total_ms)} since the last read."""
    buf = (_ProfileEntry * 32)()
    n = lib().dust_profile_read(C.cast(buf, C.c_void_p), 32)
    if n < 0:
        raise DustError(-n, "dust_profile_read")
    return {buf[i].name.decode(): (int(buf[i].launches), float(buf[i].total_ms))
            for i in range(n)}
