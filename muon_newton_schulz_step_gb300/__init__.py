"""Python binding of the GB300 Muon optimizer-step library (``libmuon_gb300.so``).

Argument marshalling only: every step of the Muon step runs in the CUDA
kernels of the library, which is loaded with ctypes.  torch supplies device
memory and the stream handle.  There is no CPU or eager fallback: if the
library is not built, every call raises.

The functions mirror the C ABI in ``include/muon.h``:

    muon_ns5_batched(mats, steps=5, coeffs=None, stream=None)
    muon_step(W, G, M, lr, mu, wd, stream=None)
    muon_step_ex(W, G, M, lr, mu, wd, *, steps, coeffs, eps, nesterov, workspace, stream)
    muon_workspace_bytes(shapes)
    muon_device_status(stream=None)
    muon_release_workspace()
    muon_profile_enable(on), muon_profile_read()
    muon_grad_norm(G), muon_grad_clip(G, max_norm, out=None)
    muon_route(logits, top_k, ...), muon_route_backward(d_weights, logits, chosen, ...)
    muon_fp8_quantize(x, ...), muon_fp8_quantize_weight(w), muon_fp8_product(product, a, b, ...)
    muon_fp8_linear(x, w, offsets), muon_fp8_linear_backward(dy, x, w, offsets)
    muon_sort_tokens(chosen, experts, first), muon_dispatch_tokens(x, plan)
    muon_combine_tokens(y, plan, weights), muon_combine_tokens_backward(d, y, plan, weights)
    muon_swiglu(gate, up), muon_swiglu_backward(d, gate, up)
    muon_int4_quantize_weight(w, block), muon_int4_linear(x, w, offsets)

The method: the per-matrix Muon step over whole matrices held on one rank
("How PyTorch Scaled a Near-1T MoE on Europe's Public Supercomputer", section
"Three optimizations that changed the economics", FlexShard bullet).
"""
import contextlib
import ctypes
import functools
import os
from array import array
from typing import NamedTuple

import torch

__all__ = [
    "MuonError", "lib", "LIB_PATH", "EXPORTS", "DEFAULT_COEFFS",
    "muon_ns5_batched", "muon_step", "muon_step_ex", "muon_workspace_bytes",
    "muon_device_status", "muon_release_workspace", "muon_profile_enable",
    "muon_profile_read", "muon_status_string", "MuonStepBatch", "muon_ns5_batched_static",
    "MUON_STATIC_SCRATCH_BYTES", "muon_step_host", "muon_ns_batched_ex", "muon_adamw_step",
    "muon_grad_norm", "muon_grad_clip", "muon_route", "muon_route_backward", "Fp8Matrix", "muon_fp8_quantize",
    "muon_fp8_quantize_weight", "muon_fp8_product", "muon_fp8_padded_rows", "muon_fp8_linear",
    "muon_fp8_linear_backward", "TokenPlan", "muon_sort_tokens", "muon_dispatch_tokens", "muon_combine_tokens",
    "muon_combine_tokens_backward", "muon_swiglu", "muon_swiglu_backward", "Int4Matrix", "muon_int4_quantize_weight",
    "muon_int4_linear",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmuon_gb300.so")
DEFAULT_COEFFS = (3.4445, -4.7750, 2.0315)

# every entry point declared in include/muon.h
EXPORTS = (
    "muon_ns5_batched", "muon_step", "muon_step_opts_init", "muon_step_ex",
    "muon_workspace_bytes", "muon_status_string", "muon_last_error",
    "muon_device_status", "muon_release_workspace", "muon_profile_enable",
    "muon_profile_read", "muon_ns5_batched_static", "muon_step_host", "muon_ns_batched_ex",
    "muon_adamw_step", "muon_grad_norm_workspace_bytes", "muon_grad_norm", "muon_grad_clip", "muon_route_opts_init",
    "muon_route", "muon_route_backward", "muon_fp8_padded_rows", "muon_fp8_quantize", "muon_fp8_quantize_weight",
    "muon_fp8_product", "muon_fp8_linear_workspace_bytes", "muon_fp8_linear", "muon_fp8_linear_backward_workspace_bytes",
    "muon_fp8_linear_backward", "muon_sort_tokens_workspace_bytes", "muon_sort_tokens", "muon_dispatch_tokens",
    "muon_combine_tokens", "muon_combine_tokens_backward", "muon_swiglu", "muon_swiglu_backward",
    "muon_int4_quantize_weight", "muon_int4_linear",
)

MUON_STATIC_SCRATCH_BYTES = 64 << 20

MUON_BF16, MUON_F32 = 0, 1


class MuonError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"status {status}: {detail}")


class _Opts(ctypes.Structure):
    _fields_ = [("w_dtype", ctypes.c_int), ("g_dtype", ctypes.c_int), ("steps", ctypes.c_int),
                ("coeffs", ctypes.POINTER(ctypes.c_float)), ("eps", ctypes.c_float),
                ("nesterov", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("o_out", ctypes.POINTER(ctypes.c_void_p)),
                ("coeffs_per_step", ctypes.c_int), ("g_count", ctypes.c_int), ("ns_fp8_gram", ctypes.c_int)]


class _RouteOpts(ctypes.Structure):
    _fields_ = [("top_k", ctypes.c_int), ("groups", ctypes.c_int), ("top_groups", ctypes.c_int),
                ("score", ctypes.c_int), ("renormalize", ctypes.c_int), ("scale", ctypes.c_float)]


class _KernelStat(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char * 40), ("launches", ctypes.c_int), ("total_ms", ctypes.c_double),
                ("flops", ctypes.c_double), ("bytes", ctypes.c_double)]


_lib = None


def lib():
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built; run `python -m muon_newton_schulz_step_gb300.build` "
            "(nvcc, sm_103a). There is no fallback implementation.")
    L = ctypes.CDLL(LIB_PATH)
    vp, ip, fp = ctypes.c_void_p, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_float)
    vpp = ctypes.POINTER(ctypes.c_void_p)
    L.muon_ns5_batched.argtypes = [vpp, ip, ip, ctypes.c_int, ctypes.c_int, fp, vp]
    L.muon_ns5_batched.restype = ctypes.c_int
    L.muon_ns_batched_ex.argtypes = [vpp, ip, ip, ctypes.c_int, ctypes.c_int, fp, ctypes.c_int, vp]
    L.muon_ns_batched_ex.restype = ctypes.c_int
    L.muon_ns5_batched_static.argtypes = [vpp, ip, ip, ctypes.c_int, ctypes.c_int, fp, vp]
    L.muon_ns5_batched_static.restype = ctypes.c_int
    L.muon_step.argtypes = [vpp, vpp, vpp, ip, ip, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                            ctypes.c_float, vp]
    L.muon_step.restype = ctypes.c_int
    L.muon_step_opts_init.argtypes = [ctypes.POINTER(_Opts)]
    L.muon_step_opts_init.restype = None
    L.muon_step_ex.argtypes = [vpp, vpp, vpp, ip, ip, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                               ctypes.c_float, ctypes.POINTER(_Opts), vp]
    L.muon_step_ex.restype = ctypes.c_int
    L.muon_step_host.argtypes = [vpp, vpp, vpp, ip, ip, ctypes.c_int, ctypes.c_float, ctypes.c_float,
                                 ctypes.c_float, ctypes.POINTER(_Opts), vp]
    L.muon_step_host.restype = ctypes.c_int
    L.muon_adamw_step.argtypes = [vpp, vpp, vpp, vpp, ctypes.POINTER(ctypes.c_longlong), ctypes.c_int,
                                  ctypes.c_int, ctypes.c_int, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                                  ctypes.c_float, ctypes.c_float, ctypes.c_int, vp]
    L.muon_adamw_step.restype = ctypes.c_int
    L.muon_workspace_bytes.argtypes = [ip, ip, ctypes.c_int]
    L.muon_workspace_bytes.restype = ctypes.c_size_t
    L.muon_status_string.argtypes = [ctypes.c_int]
    L.muon_status_string.restype = ctypes.c_char_p
    L.muon_last_error.argtypes = []
    L.muon_last_error.restype = ctypes.c_char_p
    L.muon_device_status.argtypes = [vp, ip]
    L.muon_device_status.restype = ctypes.c_int
    L.muon_release_workspace.argtypes = []
    L.muon_release_workspace.restype = None
    L.muon_profile_enable.argtypes = [ctypes.c_int]
    L.muon_profile_enable.restype = ctypes.c_int
    L.muon_profile_read.argtypes = [ctypes.POINTER(_KernelStat), ctypes.c_int, ip]
    L.muon_profile_read.restype = ctypes.c_int
    ci, ll, sz = ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    rop = ctypes.POINTER(_RouteOpts)
    L.muon_grad_norm_workspace_bytes.argtypes = [vp, ci]
    L.muon_grad_norm_workspace_bytes.restype = sz
    L.muon_grad_norm.argtypes = [vp, vp, vp, ci, vp, sz, vp, vp]
    L.muon_grad_norm.restype = ci
    L.muon_grad_clip.argtypes = [vp, vp, vp, vp, ci, ctypes.c_float, vp, sz, vp, vp]
    L.muon_grad_clip.restype = ci
    L.muon_route_opts_init.argtypes = [rop]
    L.muon_route_opts_init.restype = None
    L.muon_route.argtypes = [vp, ci, ll, ci, ll, vp, rop, vp, vp, vp, vp]
    L.muon_route.restype = ci
    L.muon_route_backward.argtypes = [vp, vp, ci, ll, ci, ll, vp, rop, vp, ll, vp]
    L.muon_route_backward.restype = ci
    L.muon_fp8_padded_rows.argtypes = [ll, ci]
    L.muon_fp8_padded_rows.restype = ll
    L.muon_fp8_quantize.argtypes = [vp, ci, ll, ll, ll, ci, vp, vp, vp, vp, vp, vp]
    L.muon_fp8_quantize.restype = ci
    L.muon_fp8_quantize_weight.argtypes = [vp, ci, ci, ll, ll, vp, vp, vp]
    L.muon_fp8_quantize_weight.restype = ci
    L.muon_fp8_product.argtypes = [ci, vp, vp, vp, vp, ll, ci, ci, ci, vp, vp, ci, ll, vp]
    L.muon_fp8_product.restype = ci
    L.muon_fp8_linear_workspace_bytes.argtypes = [ll, ci, ci, ci]
    L.muon_fp8_linear_workspace_bytes.restype = sz
    L.muon_fp8_linear.argtypes = [vp, ci, ll, ll, vp, vp, ci, ci, ci, vp, vp, sz, vp, ci, ll, vp]
    L.muon_fp8_linear.restype = ci
    L.muon_fp8_linear_backward_workspace_bytes.argtypes = [ll, ci, ci, ci, ci, ci]
    L.muon_fp8_linear_backward_workspace_bytes.restype = sz
    L.muon_fp8_linear_backward.argtypes = [vp, ci, ll, vp, ci, ll, ll, vp, vp, ci, ci, ci, vp, vp, sz, vp, ci, ll, vp, ci, vp]
    L.muon_fp8_linear_backward.restype = ci
    L.muon_sort_tokens_workspace_bytes.argtypes = [ll, ci]
    L.muon_sort_tokens_workspace_bytes.restype = sz
    L.muon_sort_tokens.argtypes = [vp, ll, ci, ci, vp, sz, vp, vp, vp, vp]
    L.muon_sort_tokens.restype = ci
    L.muon_dispatch_tokens.argtypes = [vp, ci, ll, ll, ll, ci, vp, vp, ci, vp, ll, vp]
    L.muon_dispatch_tokens.restype = ci
    L.muon_combine_tokens.argtypes = [vp, ci, ll, ll, ll, ci, vp, vp, ci, vp, vp, ci, ll, vp]
    L.muon_combine_tokens.restype = ci
    L.muon_combine_tokens_backward.argtypes = [vp, ci, ll, vp, ci, ll, ll, ll, ci, vp, vp, ci, vp, vp, ll, vp, vp]
    L.muon_combine_tokens_backward.restype = ci
    L.muon_swiglu.argtypes = [vp, ll, vp, ll, ci, ll, ll, vp, ll, vp]
    L.muon_swiglu.restype = ci
    L.muon_swiglu_backward.argtypes = [vp, ll, vp, ll, vp, ll, ci, ll, ll, vp, ll, vp, ll, vp]
    L.muon_swiglu_backward.restype = ci
    L.muon_int4_quantize_weight.argtypes = [vp, ci, ci, ll, ll, ci, vp, vp, vp]
    L.muon_int4_quantize_weight.restype = ci
    L.muon_int4_linear.argtypes = [vp, ci, ll, ll, vp, vp, ci, ci, ci, ci, vp, vp, ci, ll, vp]
    L.muon_int4_linear.restype = ci
    _lib = L
    return L


def muon_status_string(status: int) -> str:
    return lib().muon_status_string(int(status)).decode()


def _check(rc: int):
    if rc != 0:
        raise MuonError(rc, lib().muon_last_error().decode())


def _stream_handle(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr_array(tensors):
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def _dims(tensors):
    n = len(tensors)
    rows = (ctypes.c_int * n)(*[int(t.shape[0]) for t in tensors])
    cols = (ctypes.c_int * n)(*[int(t.shape[1]) for t in tensors])
    return rows, cols


def _check_mats(name, tensors, dtypes, stacked=False):
    """Every tensor a contiguous CUDA tensor on the current device, 2-D (or
    3-D where ``stacked``), of one of ``dtypes``."""
    device = None
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name}[{i}] must be a tensor")
        ok_dim = t.dim() in (2, 3) if stacked else t.dim() == 2
        if not ok_dim or not t.is_cuda:
            raise ValueError(f"{name}[{i}] must be a {'2-D or 3-D' if stacked else '2-D'} CUDA tensor")
        device = _check_device(f"{name}[{i}]", t, device)
        if not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be contiguous")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}[{i}] has dtype {t.dtype}; expected one of {dtypes}")


def _check_device(what, t, device=None):
    """``t`` must live on the current CUDA device (the library launches there);
    returns that device's index for the next call."""
    if device is None:
        device = torch.cuda.current_device()
    if t.get_device() != device:
        raise ValueError(f"{what} is on cuda:{t.get_device()}; the current device is cuda:{device}")
    return device


def _check_step_shapes(W, G, M, stacked_g):
    """W[i] is 2-D, M[i] has W[i]'s shape and G[i] is W[i]'s shape (or K x that
    shape where ``stacked_g``).  The library reads and writes rows[i] x cols[i]
    elements through each pointer, so a smaller G or M would be overrun."""
    if not (len(W) == len(G) == len(M)):
        raise ValueError("W, G and M must have the same length")
    for i, (w, g, m) in enumerate(zip(W, G, M)):
        for name, t in (("W", w), ("G", g), ("M", m)):
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"{name}[{i}] must be a tensor")
        if w.dim() != 2:
            raise ValueError(f"W[{i}] must be 2-D")
        if tuple(m.shape) != tuple(w.shape):
            raise ValueError(f"M[{i}] has shape {tuple(m.shape)}; W[{i}] has {tuple(w.shape)}")
        if g.dim() not in ((2, 3) if stacked_g else (2,)) or tuple(g.shape[-2:]) != tuple(w.shape):
            raise ValueError(f"G[{i}] has shape {tuple(g.shape)}; expected W[{i}]'s {tuple(w.shape)}"
                             + (" (optionally with a leading stack dimension)" if stacked_g else ""))


def _coeff_array(coeffs):
    if coeffs is None:
        return None
    if len(coeffs) != 3:
        raise ValueError("coeffs must be (a, b, c)")
    return (ctypes.c_float * 3)(*[float(c) for c in coeffs])


def _schedule(coeffs, steps):
    """(array, per_step): one (a, b, c) triple, or a sequence of `steps` triples."""
    if coeffs is None:
        return None, 0
    if len(coeffs) > 0 and hasattr(coeffs[0], "__len__"):
        if len(coeffs) != steps or any(len(t) != 3 for t in coeffs):
            raise ValueError("a coefficient schedule needs one (a, b, c) triple per step")
        flat = [float(v) for t in coeffs for v in t]
        return (ctypes.c_float * max(1, len(flat)))(*flat), 1
    return _coeff_array(coeffs), 0


def muon_ns_batched_ex(mats, steps: int = 5, coeffs=None, stream=None) -> None:
    """muon_ns5_batched where ``coeffs`` may be one (a, b, c) triple or a
    schedule of ``steps`` triples (one per iteration)."""
    mats = list(mats)
    _check_mats("mats", mats, (torch.bfloat16,))
    rows, cols = _dims(mats)
    arr, per_step = _schedule(coeffs, int(steps))
    _check(lib().muon_ns_batched_ex(_ptr_array(mats), rows, cols, len(mats), int(steps), arr, per_step,
                                    _stream_handle(stream)))


def muon_ns5_batched(mats, steps: int = 5, coeffs=None, stream=None) -> None:
    """In-place normalise + Newton-Schulz of a list of bf16 CUDA matrices."""
    mats = list(mats)
    _check_mats("mats", mats, (torch.bfloat16,))
    rows, cols = _dims(mats)
    _check(lib().muon_ns5_batched(_ptr_array(mats), rows, cols, len(mats), int(steps),
                                  _coeff_array(coeffs), _stream_handle(stream)))


def muon_ns5_batched_static(mats, steps: int = 5, coeffs=None, stream=None) -> None:
    """muon_ns5_batched without any device allocation: the library's scratch is a
    fixed MUON_STATIC_SCRATCH_BYTES device array (for callers that cannot call
    cudaMalloc).  Batches needing more scratch raise MuonError; calls that
    overlap on the GPU race on the shared array."""
    mats = list(mats)
    _check_mats("mats", mats, (torch.bfloat16,))
    rows, cols = _dims(mats)
    _check(lib().muon_ns5_batched_static(_ptr_array(mats), rows, cols, len(mats), int(steps),
                                         _coeff_array(coeffs), _stream_handle(stream)))


def _dtype_code(t):
    return MUON_F32 if t.dtype == torch.float32 else MUON_BF16


def muon_step(W, G, M, lr: float, mu: float, wd: float, stream=None) -> None:
    """Muon step with bf16 W and G, fp32 M, defaults for everything else."""
    W, G, M = list(W), list(G), list(M)
    _check_step_shapes(W, G, M, stacked_g=False)
    _check_mats("W", W, (torch.bfloat16,))
    _check_mats("G", G, (torch.bfloat16,))
    _check_mats("M", M, (torch.float32,))
    rows, cols = _dims(W)
    _check(lib().muon_step(_ptr_array(W), _ptr_array(G), _ptr_array(M), rows, cols, len(W),
                           float(lr), float(mu), float(wd), _stream_handle(stream)))


def _g_count(W, G):
    """Gradients per matrix: G[i] is rows x cols, or K x rows x cols (K stacked
    gradients summed in fp32 by the library); every G[i] must use the same K."""
    ks = {1 if g.dim() == 2 else int(g.shape[0]) for g in G}
    if len(ks) > 1:
        raise ValueError("every G[i] must stack the same number of gradients")
    for w, g in zip(W, G):
        if tuple(g.shape[-2:]) != tuple(w.shape):
            raise ValueError("G[i] must match W[i]'s shape (optionally with a leading stack dimension)")
    return ks.pop() if ks else 1


def _opts(W, G, steps, coeffs, eps, nesterov, workspace, o_out=None, fp8_gram=False):
    o = _Opts()
    lib().muon_step_opts_init(ctypes.byref(o))
    o.g_count = _g_count(W, G)
    o.ns_fp8_gram = 1 if fp8_gram else 0
    o.w_dtype = _dtype_code(W[0]) if W else MUON_BF16
    o.g_dtype = _dtype_code(G[0]) if G else MUON_BF16
    o.steps = int(steps)
    o.eps = float(eps)
    o.nesterov = 1 if nesterov else 0
    carr, per_step = _schedule(coeffs, int(steps))
    if carr is not None:
        o.coeffs = ctypes.cast(carr, ctypes.POINTER(ctypes.c_float))
        o.coeffs_per_step = per_step
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
        _check_device("workspace", workspace)
        o.workspace = ctypes.c_void_p(workspace.data_ptr())
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    oarr = None
    if o_out is not None:
        o_out = list(o_out)
        _check_mats("o_out", o_out, (torch.bfloat16,))
        if len(o_out) != len(W) or any(tuple(a.shape) != tuple(b.shape) for a, b in zip(o_out, W)):
            raise ValueError("o_out must match W's shapes")
        oarr = _ptr_array(o_out)
        o.o_out = ctypes.cast(oarr, ctypes.POINTER(ctypes.c_void_p))
    return o, (carr, oarr)


def muon_step_ex(W, G, M, lr: float, mu: float, wd: float, *, steps: int = 5, coeffs=None,
                 eps: float = 1e-7, nesterov: bool = True, workspace=None, o_out=None,
                 fp8_gram: bool = False, stream=None) -> None:
    """Muon step with explicit options; W and G may each be bf16 or fp32.
    ``o_out``: optional list of bf16 CUDA tensors shaped like W receiving O.
    ``fp8_gram``: the FP8 variant (E4M3 operands in the Gram product of the
    tensor-core matrices)."""
    W, G, M = list(W), list(G), list(M)
    _check_step_shapes(W, G, M, stacked_g=True)
    _check_mats("W", W, (torch.bfloat16, torch.float32))
    _check_mats("G", G, (torch.bfloat16, torch.float32), stacked=True)
    _check_mats("M", M, (torch.float32,))
    _check_one_dtype(W, G)
    rows, cols = _dims(W)
    o, _keep = _opts(W, G, steps, coeffs, eps, nesterov, workspace, o_out, fp8_gram)
    _check(lib().muon_step_ex(_ptr_array(W), _ptr_array(G), _ptr_array(M), rows, cols, len(W),
                              float(lr), float(mu), float(wd), ctypes.byref(o),
                              _stream_handle(stream)))


def _check_one_dtype(W, G):
    if W and any(t.dtype != W[0].dtype for t in W):
        raise ValueError("every W must have the same dtype")
    if G and any(t.dtype != G[0].dtype for t in G):
        raise ValueError("every G must have the same dtype")


def _check_host(name, tensors, dtypes):
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or t.is_cuda:
            raise ValueError(f"{name}[{i}] must be a host tensor")
        if not t.is_contiguous() or not t.is_pinned():
            raise ValueError(f"{name}[{i}] must be contiguous pinned host memory")
        if t.dtype not in dtypes:
            raise ValueError(f"{name}[{i}] has dtype {t.dtype}; expected one of {dtypes}")


class MuonHostStep:
    """Pre-marshalled arguments for repeated Muon steps on host-resident
    (pinned) W, G, M; each ``step()`` is one muon_step_host call."""

    def __init__(self, W, G, M, *, steps: int = 5, coeffs=None, eps: float = 1e-7,
                 nesterov: bool = True):
        self.W, self.G, self.M = list(W), list(G), list(M)
        _check_step_shapes(self.W, self.G, self.M, stacked_g=True)
        _check_host("W", self.W, (torch.bfloat16, torch.float32))
        _check_host("G", self.G, (torch.bfloat16, torch.float32))
        _check_host("M", self.M, (torch.float32,))
        _check_one_dtype(self.W, self.G)
        self._w, self._g, self._m = _ptr_array(self.W), _ptr_array(self.G), _ptr_array(self.M)
        self._rows, self._cols = _dims(self.W)
        self._opts, self._keep = _opts(self.W, self.G, steps, coeffs, eps, nesterov, None)

    def step(self, lr: float, mu: float, wd: float, stream=None) -> None:
        _check(lib().muon_step_host(self._w, self._g, self._m, self._rows, self._cols, len(self.W),
                                    float(lr), float(mu), float(wd), ctypes.byref(self._opts),
                                    _stream_handle(stream)))


def muon_step_host(W, G, M, lr: float, mu: float, wd: float, *, steps: int = 5, coeffs=None,
                   eps: float = 1e-7, nesterov: bool = True, stream=None) -> None:
    """Muon step on pinned host tensors (optimizer state kept in host memory)."""
    MuonHostStep(W, G, M, steps=steps, coeffs=coeffs, eps=eps, nesterov=nesterov).step(lr, mu, wd, stream)


def muon_adamw_step(P, G, M, V, *, lr: float, beta1: float = 0.9, beta2: float = 0.95,
                    eps: float = 1e-8, wd: float = 0.0, step: int, stream=None) -> None:
    """AdamW on a list of CUDA tensors (any shape, contiguous; P and G bf16 or
    fp32, M and V fp32); ``step`` is the 1-based step number."""
    P, G, M, V = list(P), list(G), list(M), list(V)
    if not (len(P) == len(G) == len(M) == len(V)):
        raise ValueError("P, G, M and V must have the same length")
    device = None
    for name, L, dts in (("P", P, (torch.bfloat16, torch.float32)), ("G", G, (torch.bfloat16, torch.float32)),
                         ("M", M, (torch.float32,)), ("V", V, (torch.float32,))):
        for i, t in enumerate(L):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.dtype not in dts:
                raise ValueError(f"{name}[{i}] must be a contiguous CUDA tensor of {dts}")
            device = _check_device(f"{name}[{i}]", t, device)
            if t.numel() != P[i].numel():
                raise ValueError(f"{name}[{i}] has {t.numel()} elements; P[{i}] has {P[i].numel()}")
    if P and any(t.dtype != P[0].dtype for t in P) or G and any(t.dtype != G[0].dtype for t in G):
        raise ValueError("every P (and every G) must share one dtype")
    n = len(P)
    numel = (ctypes.c_longlong * max(1, n))(*[t.numel() for t in P])
    pd = _dtype_code(P[0]) if P else MUON_BF16
    gd = _dtype_code(G[0]) if G else MUON_BF16
    _check(lib().muon_adamw_step(_ptr_array(P), _ptr_array(G), _ptr_array(M), _ptr_array(V), numel, n, pd, gd,
                                 float(lr), float(beta1), float(beta2), float(eps), float(wd), int(step),
                                 _stream_handle(stream)))


def muon_workspace_bytes(shapes) -> int:
    shapes = list(shapes)
    n = len(shapes)
    rows = (ctypes.c_int * max(n, 1))(*[int(s[0]) for s in shapes])
    cols = (ctypes.c_int * max(n, 1))(*[int(s[1]) for s in shapes])
    return int(lib().muon_workspace_bytes(rows, cols, n))


def muon_device_status(stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().muon_device_status(_stream_handle(stream), ctypes.byref(st)))
    return st.value


def muon_release_workspace() -> None:
    lib().muon_release_workspace()


def muon_profile_enable(on: bool = True) -> None:
    _check(lib().muon_profile_enable(1 if on else 0))


def muon_profile_read():
    arr = (_KernelStat * 32)()
    n = ctypes.c_int(0)
    _check(lib().muon_profile_read(arr, 32, ctypes.byref(n)))
    return [{"name": arr[i].name.decode(), "launches": arr[i].launches, "total_ms": arr[i].total_ms,
             "flops": arr[i].flops, "bytes": arr[i].bytes} for i in range(n.value)]


class MuonStepBatch:
    """Pre-marshalled arguments for repeated Muon steps on the same tensors.

    Builds the pointer and dimension arrays once; ``step()`` then makes one
    C call per optimizer step.
    """

    def __init__(self, W, G, M, *, steps: int = 5, coeffs=None, eps: float = 1e-7,
                 nesterov: bool = True, workspace=None, fp8_gram: bool = False):
        self.W, self.G, self.M = list(W), list(G), list(M)
        _check_step_shapes(self.W, self.G, self.M, stacked_g=True)
        _check_mats("W", self.W, (torch.bfloat16, torch.float32))
        _check_mats("G", self.G, (torch.bfloat16, torch.float32), stacked=True)
        _check_mats("M", self.M, (torch.float32,))
        _check_one_dtype(self.W, self.G)
        self._w, self._g, self._m = _ptr_array(self.W), _ptr_array(self.G), _ptr_array(self.M)
        self._rows, self._cols = _dims(self.W)
        self._opts, self._keep = _opts(self.W, self.G, steps, coeffs, eps, nesterov, workspace, None, fp8_gram)

    def step(self, lr: float, mu: float, wd: float, stream=None) -> None:
        _check(lib().muon_step_ex(self._w, self._g, self._m, self._rows, self._cols, len(self.W),
                                  float(lr), float(mu), float(wd), ctypes.byref(self._opts),
                                  _stream_handle(stream)))


# ----------------------------------------------- operators around the step --
# These calls run in front of kernels of a few microseconds: their checks read
# each tensor property once, and torch is asked for the current device and
# stream by the cheapest way it has.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(stream):
    """Context in which new tensors belong to ``stream`` (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _handle(stream):
    """The raw handle of ``stream`` (None: the current stream)."""
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _here(name, t):
    """``t`` is a CUDA tensor on the current device (the library launches there)."""
    if t.get_device() != _current_device():
        _check_device(name, t)


_FLOATS = (torch.bfloat16, torch.float32)


_FLOAT_CODE = {torch.bfloat16: MUON_BF16, torch.float32: MUON_F32}


def _refuse_flat(name, tensors):
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in _FLOATS or not t.is_contiguous():
            raise ValueError(f"{name}[{i}] must be a contiguous CUDA tensor of {_FLOATS}")
        _check_device(f"{name}[{i}]", t)


def _flat_list(name, tensors):
    """Contiguous CUDA tensors on the current device as C arrays: (pointers,
    elements, element type codes).  One pass per property: half the time of a
    loop over the tensors."""
    try:
        codes = [_FLOAT_CODE[t.dtype] for t in tensors]
        whole = [t.is_contiguous() for t in tensors]
        where = [t.get_device() for t in tensors]
        if False in whole or -1 in where or (where and where.count(_current_device()) != len(where)):
            _refuse_flat(name, tensors)
        return (array("Q", [t.data_ptr() for t in tensors]), array("q", [t.numel() for t in tensors]),
                array("i", codes))
    except (AttributeError, KeyError, TypeError):
        _refuse_flat(name, tensors)
        raise


def _at(a):
    """Address of a C array."""
    return a.buffer_info()[0]


def muon_grad_norm(G, stream=None) -> torch.Tensor:
    """Global 2-norm of a list of contiguous CUDA gradients (bf16 and fp32 may
    be mixed), as a 0-dim fp32 CUDA tensor."""
    G = list(G)
    ptrs, numel, dtypes = _flat_list("G", G)
    L = lib()
    need = L.muon_grad_norm_workspace_bytes(_at(numel), len(G))
    with _on(stream):
        buf = torch.empty(need // 4 + 4, dtype=torch.float32, device="cuda")   # the norm, partial sums from byte 16 on
        at = buf.data_ptr()
        _check(L.muon_grad_norm(_at(ptrs), _at(numel), _at(dtypes), len(G), at + 16, need, at, _handle(stream)))
    return buf[0]


def muon_grad_clip(G, max_norm: float, out=None, stream=None) -> torch.Tensor:
    """Scale every gradient by min(1, max_norm / (norm + 1e-6)), in place or
    into ``out`` (tensors like G); returns the norm before clipping (0-dim
    fp32 CUDA tensor).  Nothing is read back to the host."""
    G = list(G)
    ptrs, numel, dtypes = _flat_list("G", G)
    optrs = None
    if out is not None:
        out = list(out)
        if len(out) != len(G):
            raise ValueError("out must have one tensor for each of G")
        optrs, onumel, odtypes = _flat_list("out", out)
        if onumel != numel or odtypes != dtypes:
            raise ValueError("out must have the dtype and number of elements of G, tensor by tensor")
    L = lib()
    need = L.muon_grad_norm_workspace_bytes(_at(numel), len(G))
    with _on(stream):
        buf = torch.empty(need // 4 + 4, dtype=torch.float32, device="cuda")
        at = buf.data_ptr()
        _check(L.muon_grad_clip(_at(ptrs), None if optrs is None else _at(optrs), _at(numel), _at(dtypes), len(G),
                                float(max_norm), at + 16, need, at, _handle(stream)))
    return buf[0]


def _check_rows(name, t, dtypes, rows=None, cols=None):
    """A 2-D CUDA tensor whose rows are contiguous (any row stride that does not
    overlap them): (rows, cols, row stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype not in dtypes or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor of {dtypes}")
    _here(name, t)
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} has shape {(r, c)}; expected ({rows}, {cols})")
    ld, inner = t.stride()
    if r <= 1 or c == 0:
        ld = max(ld, c)
    if r * c and ((c > 1 and inner != 1) or ld < c):
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
    return r, c, max(ld, c)


def _check_vector(name, t, dtype, n):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or tuple(t.shape) != (n,) \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} {dtype}")
    _here(name, t)


_SCORES = {"softmax": 0, "sigmoid": 1}


@functools.lru_cache(maxsize=256)
def _kept_route_opts(top_k, score, groups, top_groups, renormalize, scale):
    o = _RouteOpts(top_k, groups, top_groups, score, renormalize, scale)
    return o, ctypes.byref(o)


def _route_opts(top_k, score, groups, top_groups, renormalize, scale):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {tuple(_SCORES)}")
    # kept by value: a tensor among the arguments may change in place
    return _kept_route_opts(int(top_k), _SCORES[score], int(groups), int(groups if top_groups is None else top_groups),
                            1 if renormalize else 0, float(scale))


def muon_route(logits, top_k: int, *, bias=None, score: str = "softmax", groups: int = 1, top_groups=None,
               renormalize: bool = True, scale: float = 1.0, stream=None):
    """Choose ``top_k`` experts for each row of ``logits`` (tokens x experts,
    bf16 or fp32): (weights fp32 tokens x top_k, experts int32 tokens x top_k,
    tokens of each expert int32).  ``bias`` (fp32, one per expert) steers the
    choice only; ``groups`` / ``top_groups`` limit it to the best groups of
    consecutive experts.  Experts masked by a logit of -inf are not chosen;
    places left over get expert -1 and weight 0."""
    tokens, experts, ld = _check_rows("logits", logits, _FLOATS)
    if bias is not None:
        _check_vector("bias", bias, torch.float32, experts)
    o, ref = _route_opts(top_k, score, groups, top_groups, renormalize, scale)
    with _on(stream):
        weights = torch.empty((tokens, o.top_k), dtype=torch.float32, device="cuda")
        chosen = torch.empty((tokens, o.top_k), dtype=torch.int32, device="cuda")
        counts = torch.empty(experts, dtype=torch.int32, device="cuda")
        _check(lib().muon_route(logits.data_ptr(), _dtype_code(logits), tokens, experts, ld,
                                None if bias is None else bias.data_ptr(), ref, weights.data_ptr(),
                                chosen.data_ptr(), counts.data_ptr(), _handle(stream)))
    return weights, chosen, counts


def muon_route_backward(d_weights, logits, chosen, *, score: str = "softmax", renormalize: bool = True,
                        scale: float = 1.0, stream=None) -> torch.Tensor:
    """Gradient of the logits (their dtype) from that of ``muon_route``'s
    weights, for the experts it chose."""
    tokens, experts, ld = _check_rows("logits", logits, _FLOATS)
    _, top_k, _ = _check_rows("chosen", chosen, (torch.int32,), tokens)
    _check_rows("d_weights", d_weights, (torch.float32,), tokens, top_k)
    if not chosen.is_contiguous() or not d_weights.is_contiguous():
        raise ValueError("chosen and d_weights must be contiguous")
    _, ref = _route_opts(top_k, score, 1, 1, renormalize, scale)
    with _on(stream):
        d = torch.empty((tokens, experts), dtype=logits.dtype, device="cuda")
        _check(lib().muon_route_backward(d_weights.data_ptr(), logits.data_ptr(), _dtype_code(logits), tokens, experts,
                                         ld, chosen.data_ptr(), ref, d.data_ptr(), experts, _handle(stream)))
    return d


class Fp8Matrix(NamedTuple):
    """E4M3 codes with one E8M0 scale byte (exponent + 127) for each block of 128.

    ``kind`` "row" (128 columns of one row), "col" (128 rows of one column,
    groups padded to multiples of 128 rows) or "block" (128 x 128).
    ``codes``: float8_e4m3fn, rows x cols rounded up to 128, zero past ``cols``
    ("block": optionally stacked, experts x rows x ...).  ``scale``: uint8 --
    "row" (column blocks, rows), "col" (row blocks, codes' columns), "block"
    (..., row blocks, column blocks)."""
    codes: torch.Tensor
    scale: torch.Tensor
    kind: str
    cols: int


def _up128(n):
    return (n + 127) // 128 * 128


def _check_offsets(offsets, groups=None):
    """(groups, device pointer or None) of the row offsets of tokens sorted by expert."""
    if offsets is None:
        return 1, None
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be a 1-D int32 CUDA tensor of groups + 1 entries")
    _check_vector("offsets", offsets, torch.int32, offsets.numel() if groups is None else groups + 1)
    return offsets.numel() - 1, offsets.data_ptr()


def muon_fp8_padded_rows(rows: int, groups: int = 1) -> int:
    """Rows of the "col" codes of ``rows`` rows in ``groups`` groups."""
    return int(lib().muon_fp8_padded_rows(int(rows), int(groups)))


def muon_fp8_quantize(x, *, row: bool = True, col: bool = False, offsets=None, stream=None):
    """``x`` (2-D, bf16 or fp32) as E4M3 with scales for blocks of 128 along its
    rows (``row``), along its columns (``col``; blocks start anew at each group
    of ``offsets``), or both from one read: (row Fp8Matrix or None, col
    Fp8Matrix or None).  With ``col`` and ``offsets`` the codes of rows of no
    group are not set."""
    rows, cols, ld = _check_rows("x", x, _FLOATS)
    groups, optr = _check_offsets(offsets)
    ldq = _up128(cols)
    with _on(stream):
        r = c = None
        if row:
            r = Fp8Matrix(torch.empty((rows, ldq), dtype=torch.float8_e4m3fn, device="cuda"),
                          torch.empty((ldq // 128, rows), dtype=torch.uint8, device="cuda"), "row", cols)
        if col:
            padded = muon_fp8_padded_rows(rows, groups)
            c = Fp8Matrix(torch.empty((padded, ldq), dtype=torch.float8_e4m3fn, device="cuda"),
                          torch.empty((padded // 128, ldq), dtype=torch.uint8, device="cuda"), "col", cols)
        _check(lib().muon_fp8_quantize(x.data_ptr(), _dtype_code(x), rows, cols, ld, groups, optr,
                                       r.codes.data_ptr() if row else None, r.scale.data_ptr() if row else None,
                                       c.codes.data_ptr() if col else None, c.scale.data_ptr() if col else None,
                                       _handle(stream)))
    return r, c


def muon_fp8_quantize_weight(w, stream=None) -> Fp8Matrix:
    """A weight (rows x cols, or stacked experts x rows x cols; bf16 or fp32,
    contiguous) as E4M3 with a scale for each 128 x 128 block."""
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3) or not w.is_cuda or w.dtype not in _FLOATS \
            or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous 2-D or 3-D CUDA tensor of {_FLOATS}")
    _check_device("w", w)
    rows, cols = w.shape[-2:]
    with _on(stream):
        m = Fp8Matrix(torch.empty((*w.shape[:-1], _up128(cols)), dtype=torch.float8_e4m3fn, device="cuda"),
                      torch.empty((*w.shape[:-2], _up128(rows) // 128, _up128(cols) // 128), dtype=torch.uint8,
                                  device="cuda"), "block", cols)
        _check(lib().muon_fp8_quantize_weight(w.data_ptr(), _dtype_code(w), w.shape[0] if w.dim() == 3 else 1, rows, cols,
                                              m.codes.data_ptr(), m.scale.data_ptr(), _handle(stream)))
    return m


def _check_fp8(name, m, kind, codes_shape, scale_shape):
    if not isinstance(m, Fp8Matrix) or m.kind != kind:
        raise ValueError(f'{name} must be an Fp8Matrix of kind "{kind}"')
    for what, t, dt, shape in (("codes", m.codes, torch.float8_e4m3fn, codes_shape),
                               ("scale", m.scale, torch.uint8, scale_shape)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dt or not t.is_contiguous() \
                or tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name}.{what} must be a contiguous CUDA tensor of {dt} with shape {tuple(shape)}")
        _check_device(f"{name}.{what}", t)


def _check_weight(w, offsets):
    """(n, k, groups, offsets' pointer) of a "block" weight that goes with ``offsets``."""
    if not isinstance(w, Fp8Matrix) or not isinstance(w.codes, torch.Tensor) or not isinstance(w.scale, torch.Tensor):
        raise ValueError('the weight must be an Fp8Matrix of kind "block", as muon_fp8_quantize_weight makes it')
    codes, scale = w.codes, w.scale
    shape, k = codes.shape, int(w.cols)
    stacked = len(shape) == 3
    if w.kind != "block" or len(shape) not in (2, 3):
        raise ValueError('the weight must be an Fp8Matrix of kind "block" with 2-D or 3-D codes')
    if stacked != (offsets is not None):
        raise ValueError("a stacked weight goes with offsets, a single one without")
    n = shape[-2]
    kb, nb = (k + 127) // 128, (n + 127) // 128
    if codes.dtype != torch.float8_e4m3fn or shape[-1] != 128 * kb or not codes.is_cuda or not codes.is_contiguous():
        raise ValueError(f"the weight's codes must be a contiguous CUDA tensor of {torch.float8_e4m3fn} with rows of {128 * kb}")
    if scale.dtype != torch.uint8 or tuple(scale.shape) != (*shape[:-2], nb, kb) or not scale.is_cuda \
            or not scale.is_contiguous():
        raise ValueError(f"the weight's scale must be a contiguous CUDA tensor of {torch.uint8} with shape "
                         f"{(*shape[:-2], nb, kb)}")
    _here("the weight's codes", codes)
    _here("the weight's scale", scale)
    groups, optr = _check_offsets(offsets, shape[0] if stacked else 1)
    return n, k, groups, optr


def _product(code, a, b, tokens, n, k, groups, optr, out, ld, stream):
    _check(lib().muon_fp8_product(code, a.codes.data_ptr(), a.scale.data_ptr(), b.codes.data_ptr(), b.scale.data_ptr(),
                                  tokens, n, k, groups, optr, out.data_ptr(), _dtype_code(out), ld,
                                  _handle(stream)))


def muon_fp8_product(product: str, a, b, *, offsets=None, tokens=None, out=None, out_dtype=torch.bfloat16,
                     stream=None):
    """One product of a linear layer on E4M3 operands (``Fp8Matrix``):

    "forward"      out[t, n] = sum_k a[t, k] b[g, n, k]     a "row", b "block"
    "grad_input"   out[t, k] = sum_n a[t, n] b[g, n, k]     a "row", b "block"
    "grad_weight"  out[g, n, k] = sum_t a[t, n] b[t, k]     a "col", b "col"

    With ``offsets`` (int32, experts + 1, on the device) rows offsets[g] to
    offsets[g + 1] are expert g's and b (or out) is stacked over experts.
    ``tokens`` (grad_weight): the rows that the operands were made from.
    ``out``: optional preallocated result, bf16 or fp32 (rows contiguous).  Rows of
    no expert are left as they are in ``out``, and not set in a new result
    (``muon_fp8_linear`` makes them zero)."""
    if product in ("forward", "grad_input"):
        n, k, groups, optr = _check_weight(b, offsets)
        inner, red = (n, k) if product == "forward" else (k, n)
        if not isinstance(a, Fp8Matrix) or not isinstance(a.codes, torch.Tensor) or a.codes.dim() != 2 or a.cols != red:
            raise ValueError(f'a must be an Fp8Matrix of kind "row" with {red} columns')
        tokens = a.codes.shape[0]
        _check_fp8("a", a, "row", (tokens, _up128(red)), (_up128(red) // 128, tokens))
        with _on(stream):
            if out is None:
                out = torch.empty((tokens, inner), dtype=out_dtype, device="cuda")
            _, _, ld = _check_rows("out", out, _FLOATS, tokens, inner)
            _product(0 if product == "forward" else 1, a, b, tokens, n, k, groups, optr, out, ld, stream)
        return out
    if product != "grad_weight":
        raise ValueError('product must be "forward", "grad_input" or "grad_weight"')
    groups, optr = _check_offsets(offsets)
    if tokens is None:
        raise ValueError('"grad_weight" needs tokens, the number of rows that the operands were made from')
    tokens = int(tokens)
    padded = muon_fp8_padded_rows(tokens, groups)
    for name, m in (("a", a), ("b", b)):
        if not isinstance(m, Fp8Matrix):
            raise ValueError(f'{name} must be an Fp8Matrix of kind "col"')
        _check_fp8(name, m, "col", (padded, _up128(m.cols)), (padded // 128, _up128(m.cols)))
    n, k = int(a.cols), int(b.cols)
    shape = (n, k) if offsets is None else (groups, n, k)
    with _on(stream):
        if out is None:
            out = torch.empty(shape, dtype=out_dtype, device="cuda")
        elif not isinstance(out, torch.Tensor) or not out.is_cuda or out.dtype not in _FLOATS \
                or tuple(out.shape) != shape or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous CUDA tensor of {_FLOATS} with shape {shape}")
        _check_device("out", out)
        _product(2, a, b, tokens, n, k, groups, optr, out, k, stream)
    return out


def muon_fp8_linear(x, w, *, offsets=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x W^T in 8 bits: ``x`` (tokens x k, bf16 or fp32) is rounded to E4M3 by
    row blocks and multiplied with ``w`` (``muon_fp8_quantize_weight``).  With
    ``offsets``, tokens are sorted by expert and ``w`` is stacked over experts;
    rows of no expert give zero."""
    n, k, groups, optr = _check_weight(w, offsets)
    tokens, _, ld = _check_rows("x", x, _FLOATS, None, k)
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be one of {_FLOATS}")
    L = lib()
    need = L.muon_fp8_linear_workspace_bytes(tokens, n, k, offsets is not None)
    with _on(stream):
        out = torch.empty((tokens, n), dtype=out_dtype, device="cuda")
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        _check(L.muon_fp8_linear(x.data_ptr(), _dtype_code(x), tokens, ld, w.codes.data_ptr(), w.scale.data_ptr(), n, k,
                                 groups, optr, None if ws is None else ws.data_ptr(), need, out.data_ptr(), _dtype_code(out), n, _handle(stream)))
    return out


def muon_fp8_linear_backward(dy, x, w, *, offsets=None, need_dx: bool = True, need_dw: bool = True,
                             dx_dtype=torch.bfloat16, dw_dtype=torch.bfloat16, stream=None):
    """(dx, dW) of ``muon_fp8_linear`` from dy (tokens x n): dx = dy W with dy by
    row blocks, dW = dy^T x with both by col blocks; either may be left out
    (None).  dy is read once for both; rows of no expert give a zero dx."""
    n, k, groups, optr = _check_weight(w, offsets)
    tokens, _, ld_dy = _check_rows("dy", dy, _FLOATS, None, n)
    _, _, ld_x = _check_rows("x", x, _FLOATS, tokens, k)
    if dx_dtype not in _FLOATS or dw_dtype not in _FLOATS:
        raise ValueError(f"dx_dtype and dw_dtype must be of {_FLOATS}")
    dx = dw = None
    with _on(stream):
        if need_dx:
            dx = torch.empty((tokens, k), dtype=dx_dtype, device="cuda")
        if need_dw:
            dw = torch.empty((n, k) if offsets is None else (groups, n, k), dtype=dw_dtype, device="cuda")
        need = lib().muon_fp8_linear_backward_workspace_bytes(tokens, n, k, groups, int(need_dx), int(need_dw))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        _check(lib().muon_fp8_linear_backward(
            dy.data_ptr(), _dtype_code(dy), ld_dy, x.data_ptr(), _dtype_code(x), ld_x, tokens, w.codes.data_ptr(),
            w.scale.data_ptr(), n, k, groups, optr, ws.data_ptr() if need else None, need, dx.data_ptr() if need_dx and tokens else None,
            MUON_F32 if dx_dtype == torch.float32 else MUON_BF16, k, dw.data_ptr() if need_dw else None,
            MUON_F32 if dw_dtype == torch.float32 else MUON_BF16, _handle(stream)))
    return dx, dw


# ----------------------------------- between an expert layer's routing and its result --
# torch.empty costs a call of a few microseconds as much again (4 us of 9, measured on a
# GB300's host between launches); the allocation alone, on the current device, 0.9.  It is
# not of torch's public interface: the first use tries it, and where it is not there or
# gives anything else, results come from torch.empty.  (They are written whole, so that
# what torch.empty may fill them with never shows.)
_empty_strided = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _allocates(f):
    """Whether ``f(sizes, strides, dtype)`` makes such a tensor on the current device."""
    try:
        t = f((2, 3), (3, 1), torch.bfloat16)
        return t.is_cuda and t.get_device() == _current_device() and t.dtype is torch.bfloat16 \
            and tuple(t.shape) == (2, 3) and t.stride() == (3, 1)
    except Exception:
        return False


def _first_allocation(sizes, strides, dtype):
    global _allocate
    _allocate = _empty_strided if _allocates(_empty_strided) else None
    return torch.empty(sizes, dtype=dtype, device="cuda") if _allocate is None else _allocate(sizes, strides, dtype)


_allocate = _first_allocation


def _new_rows(rows, cols, dtype):
    """A new tensor, rows x cols, on the current device and stream."""
    if _allocate is None:
        return torch.empty((rows, cols), dtype=dtype, device="cuda")
    return _allocate((rows, cols), (cols or 1, 1), dtype)


def _new_vector(n, dtype):
    if _allocate is None:
        return torch.empty(n, dtype=dtype, device="cuda")
    return _allocate((n,), (1,), dtype)


def _matrix(name, t, rows=None, cols=None):
    """(rows, cols, row stride, type code) of a 2-D bf16 or fp32 CUDA tensor with contiguous rows."""
    try:
        code, (r, c), (ld, inner) = _FLOAT_CODE[t.dtype], t.shape, t.stride()
        if inner == 1 and ld >= c and (rows is None or r == rows) and (cols is None or c == cols) \
                and t.is_cuda and t.get_device() == _current_device():
            return r, c, ld, code
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    r, c, ld = _check_rows(name, t, _FLOATS, rows, cols)    # says what is wrong, or takes a form seldom met
    return r, c, ld, _FLOAT_CODE[t.dtype]


class TokenPlan(NamedTuple):
    """Where the rows of routed tokens lie, sorted by expert (``muon_sort_tokens``;
    int32).  ``order`` (tokens * top_k): the entry (token * top_k + j) at each place;
    ``place`` (tokens x top_k): the place of each entry; ``offsets`` (experts + 1): the
    places of each expert, as the experts' products take them.  Entries without an
    expert here lie before ``offsets[0]``."""
    order: torch.Tensor
    place: torch.Tensor
    offsets: torch.Tensor


def muon_sort_tokens(chosen, experts: int, *, first: int = 0, stream=None) -> TokenPlan:
    """The entries of ``chosen`` (tokens x top_k, int32, contiguous, as ``muon_route``
    gives them) sorted by expert, for the ``experts`` experts from number ``first`` on
    (those that this rank holds).  Entries of other experts, or of none, come first;
    equal ones keep their order."""
    if stream is not None:
        with _on(stream):
            return muon_sort_tokens(chosen, experts, first=first)
    try:
        fine, (tokens, top_k) = _plain(chosen, torch.int32), chosen.shape
    except (AttributeError, TypeError, ValueError):
        fine = False
    if not fine:
        tokens, top_k, _ = _check_rows("chosen", chosen, (torch.int32,))        # says what is wrong
        if not chosen.is_contiguous():
            raise ValueError("chosen must be contiguous")
    experts, first, n = int(experts), int(first), tokens * top_k
    if experts < 1:
        raise ValueError(f"experts is {experts}")
    L = lib()
    need = L.muon_sort_tokens_workspace_bytes(n, experts)
    order, place, offsets = _new_vector(n, torch.int32), _new_rows(tokens, top_k, torch.int32), \
        _new_vector(experts + 1, torch.int32)
    ws = _new_vector(need, torch.uint8) if need else None
    _check(L.muon_sort_tokens(chosen.data_ptr(), n, first, experts, None if ws is None else ws.data_ptr(), need,
                              order.data_ptr(), place.data_ptr(), offsets.data_ptr(), _handle(None)))
    return TokenPlan(order, place, offsets)


def _plain(t, dtype):
    """Whether ``t`` is a contiguous tensor of ``dtype`` on the current device."""
    return t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.get_device() == _current_device()


def _check_plan(plan):
    """(tokens, top_k, experts, addresses of places and offsets) of a plan, whose tensors are checked."""
    if not isinstance(plan, TokenPlan):
        raise ValueError("plan must be a TokenPlan, as muon_sort_tokens makes it")
    _, place, offsets = plan
    tokens, top_k, _ = _check_rows("plan.place", place, (torch.int32,))
    if not place.is_contiguous():
        raise ValueError("plan.place must be contiguous")
    if top_k < 1:
        raise ValueError("plan.place has no columns")
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("plan.offsets must be a 1-D int32 CUDA tensor of experts + 1 entries")
    n = offsets.numel()
    _check_vector("plan.offsets", offsets, torch.int32, n)
    return tokens, top_k, n - 1, place.data_ptr(), offsets.data_ptr()


def _check_weights(weights, tokens, top_k):
    if weights is None:
        return None
    _check_rows("weights", weights, (torch.float32,), tokens, top_k)
    if not weights.is_contiguous():
        raise ValueError("weights must be contiguous")
    return weights.data_ptr()


def _planned(plan, name, t, sorted_rows, weights=None):
    """(tokens, top_k, cols, row stride, type code, experts, addresses of places, offsets and weights)
    of a plan with the tokens' rows ``t``, or their entries' (``sorted_rows``), and weights."""
    try:
        _, place, offsets = plan
        (tokens, top_k), (n,), (rows, cols), (ld, inner) = place.shape, offsets.shape, t.shape, t.stride()
        here = t.get_device()
        if type(plan) is TokenPlan and inner == 1 and ld >= cols and rows == (tokens * top_k if sorted_rows else tokens) \
                and n >= 2 and top_k >= 1 and place.dtype is torch.int32 and offsets.dtype is torch.int32 \
                and place.is_contiguous() and offsets.is_contiguous() and here >= 0 and place.get_device() == here \
                and offsets.get_device() == here == _current_device() \
                and (weights is None or (weights.dtype is torch.float32 and weights.shape == place.shape
                                         and weights.is_contiguous() and weights.get_device() == here)):
            return (tokens, top_k, cols, ld, _FLOAT_CODE[t.dtype], n - 1, place.data_ptr(), offsets.data_ptr(),
                    None if weights is None else weights.data_ptr())
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    # one by one: says what is wrong, or takes a form seldom met
    tokens, top_k, experts, at_place, at_offsets = _check_plan(plan)
    _, cols, ld, code = _matrix(name, t, tokens * top_k if sorted_rows else tokens)
    return tokens, top_k, cols, ld, code, experts, at_place, at_offsets, _check_weights(weights, tokens, top_k)


def muon_dispatch_tokens(x, plan: TokenPlan, stream=None) -> torch.Tensor:
    """``x``'s rows (tokens x cols, bf16 or fp32) sorted by expert: tokens * top_k
    rows, row plan.place[t, j] a copy of x[t]; rows of no expert are zero.  Its gradient
    is ``muon_combine_tokens`` without weights."""
    if stream is not None:
        with _on(stream):
            return muon_dispatch_tokens(x, plan)
    tokens, top_k, cols, ld, code, experts, place, offsets, _ = _planned(plan, "x", x, False)
    out = _new_rows(tokens * top_k, cols, x.dtype)
    if cols:
        _check(lib().muon_dispatch_tokens(x.data_ptr(), code, tokens, cols, ld, top_k, place, offsets, experts,
                                          out.data_ptr(), cols, _handle(None)))
    return out


def muon_combine_tokens(y, plan: TokenPlan, weights=None, *, out_dtype=None, stream=None) -> torch.Tensor:
    """The way back: out[t] = sum over j of weights[t, j] * y[plan.place[t, j]], summed in
    fp32 in the order of j.  ``y``: tokens * top_k rows, bf16 or fp32; ``weights``: fp32,
    tokens x top_k (None: 1); ``out_dtype``: y's unless given.  Entries without an expert
    here take no part, whatever their rows and weights hold."""
    if stream is not None:
        with _on(stream):
            return muon_combine_tokens(y, plan, weights, out_dtype=out_dtype)
    tokens, top_k, cols, ld, code, experts, place, offsets, wptr = _planned(plan, "y", y, True, weights)
    if out_dtype is None:
        out_dtype = y.dtype
    elif out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be one of {_FLOATS}")
    out = _new_rows(tokens, cols, out_dtype)
    if cols:
        _check(lib().muon_combine_tokens(y.data_ptr(), code, ld, tokens, cols, top_k, place, offsets, experts, wptr,
                                         out.data_ptr(), _FLOAT_CODE[out_dtype], cols, _handle(None)))
    return out


def muon_combine_tokens_backward(d, y, plan: TokenPlan, weights=None, *, need_dy: bool = True, need_dw: bool = True,
                                 stream=None):
    """(dy, d_weights) of ``muon_combine_tokens`` from ``d`` (tokens x cols, bf16 or fp32):
    dy[plan.place[t, j]] = weights[t, j] * d[t] (y's dtype), d_weights[t, j] = <d[t],
    y[plan.place[t, j]]> (fp32), both zero for entries without an expert here.  Either may be
    left out (None); without weights there is no d_weights."""
    if stream is not None:
        with _on(stream):
            return muon_combine_tokens_backward(d, y, plan, weights, need_dy=need_dy, need_dw=need_dw)
    tokens, top_k, cols, ld_y, code, experts, place, offsets, wptr = _planned(plan, "y", y, True, weights)
    _, _, ld_d, d_code = _matrix("d", d, tokens, cols)
    dy = _new_rows(tokens * top_k, cols, y.dtype) if need_dy else None
    dw = _new_rows(tokens, top_k, torch.float32) if need_dw and weights is not None else None
    if cols:
        _check(lib().muon_combine_tokens_backward(
            d.data_ptr(), d_code, ld_d, y.data_ptr(), code, ld_y, tokens, cols, top_k, place, offsets, experts, wptr,
            None if dy is None else dy.data_ptr(), cols, None if dw is None else dw.data_ptr(), _handle(None)))
    elif dw is not None:
        dw.zero_()
    return dy, dw


def _check_gated(gate, up):
    try:
        code, here, (rows, cols), (ld_gate, inner), (ld_up, inner_up) = \
            _FLOAT_CODE[gate.dtype], gate.get_device(), gate.shape, gate.stride(), up.stride()
        if up.dtype is gate.dtype and up.shape == gate.shape and inner == inner_up == 1 and ld_gate >= cols \
                and ld_up >= cols and here >= 0 and up.get_device() == here == _current_device():
            return rows, cols, ld_gate, ld_up, code
    except (AttributeError, KeyError, TypeError, ValueError):
        pass
    rows, cols, ld_gate, code = _matrix("gate", gate)
    _, _, ld_up, up_code = _matrix("up", up, rows, cols)
    if up_code != code:
        raise ValueError("gate and up must share one dtype")
    return rows, cols, ld_gate, ld_up, code


def muon_swiglu(gate, up, stream=None) -> torch.Tensor:
    """gate / (1 + exp(-gate)) * up, in fp32 and rounded once (rows x cols, bf16 or fp32,
    both of one dtype; views such as the halves of one product are read in place)."""
    if stream is not None:
        with _on(stream):
            return muon_swiglu(gate, up)
    rows, cols, ld_gate, ld_up, code = _check_gated(gate, up)
    out = _new_rows(rows, cols, gate.dtype)
    if cols:
        _check(lib().muon_swiglu(gate.data_ptr(), ld_gate, up.data_ptr(), ld_up, code, rows, cols, out.data_ptr(), cols,
                                 _handle(None)))
    return out


def muon_swiglu_backward(d, gate, up, *, joined: bool = False, stream=None):
    """(d_gate, d_up) of ``muon_swiglu`` from ``d``, in its dtype.  ``joined``: one tensor,
    rows x 2 cols, d_gate before d_up, as the gradient of one product that made gate and up
    wants them."""
    if stream is not None:
        with _on(stream):
            return muon_swiglu_backward(d, gate, up, joined=joined)
    rows, cols, ld_gate, ld_up, code = _check_gated(gate, up)
    _, _, ld_d, d_code = _matrix("d", d, rows, cols)
    if d_code != code:
        raise ValueError("d must be of gate's dtype")
    if joined:
        d_gate = d_up = _new_rows(rows, 2 * cols, gate.dtype)
        ld, on = 2 * cols, cols * gate.element_size()
    else:
        d_gate, d_up, ld, on = _new_rows(rows, cols, gate.dtype), _new_rows(rows, cols, gate.dtype), cols, 0
    if cols:
        _check(lib().muon_swiglu_backward(d.data_ptr(), ld_d, gate.data_ptr(), ld_gate, up.data_ptr(), ld_up, code, rows,
                                          cols, d_gate.data_ptr(), ld, d_up.data_ptr() + on, ld, _handle(None)))
    return d_gate if joined else (d_gate, d_up)


class Int4Matrix(NamedTuple):
    """A weight of 4 bits: w[n, k] = code[n, k] * scale[k // block, n], codes from -8 to 7.

    ``codes``: uint8, rows x (cols rounded up to 128) / 2, the even column in the low
    half, zero past ``cols``; ``scale``: bf16, (cols rounded up to 128) / block x rows, zero
    for blocks past ``cols``; both optionally stacked over experts.  ``block``: 32, 64 or 128 columns."""
    codes: torch.Tensor
    scale: torch.Tensor
    block: int
    cols: int


def muon_int4_quantize_weight(w, block: int = 128, stream=None) -> Int4Matrix:
    """A weight (rows x cols, or stacked experts x rows x cols; bf16 or fp32, contiguous) in
    4 bits, with a scale (max|w| / 7 in bf16) for each ``block`` columns of a row."""
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3) or not w.is_cuda or w.dtype not in _FLOATS \
            or not w.is_contiguous():
        raise ValueError(f"w must be a contiguous 2-D or 3-D CUDA tensor of {_FLOATS}")
    _here("w", w)
    block = int(block)
    if block not in (32, 64, 128):
        raise ValueError("block must be 32, 64 or 128")
    rows, cols = w.shape[-2:]
    up = _up128(cols)
    with _on(stream):
        m = Int4Matrix(torch.empty((*w.shape[:-1], up // 2), dtype=torch.uint8, device="cuda"),
                       torch.empty((*w.shape[:-2], up // block, rows), dtype=torch.bfloat16, device="cuda"), block, cols)
        _check(lib().muon_int4_quantize_weight(w.data_ptr(), _dtype_code(w), w.shape[0] if w.dim() == 3 else 1, rows, cols,
                                               block, m.codes.data_ptr(), m.scale.data_ptr(), _handle(stream)))
    return m


def _check_int4(w, offsets):
    """(n, k, groups, offsets' pointer) of a weight of 4 bits that goes with ``offsets``."""
    if not isinstance(w, Int4Matrix) or not isinstance(w.codes, torch.Tensor) or not isinstance(w.scale, torch.Tensor):
        raise ValueError("the weight must be an Int4Matrix, as muon_int4_quantize_weight makes it")
    codes, scale, block, k = w
    shape, k = codes.shape, int(k)
    if len(shape) not in (2, 3) or block not in (32, 64, 128):
        raise ValueError("the weight must be an Int4Matrix with 2-D or 3-D codes and a block of 32, 64 or 128")
    stacked = len(shape) == 3
    if stacked != (offsets is not None):
        raise ValueError("a stacked weight goes with offsets, a single one without")
    n, up = shape[-2], _up128(k)
    here, want = codes.get_device(), ((shape[0], up // block, n) if stacked else (up // block, n))
    if shape[-1] == up // 2 and scale.shape == want and codes.dtype is torch.uint8 and scale.dtype is torch.bfloat16 \
            and codes.is_contiguous() and scale.is_contiguous() and here >= 0 \
            and scale.get_device() == here == _current_device():
        if not stacked:
            return n, k, 1, None
        return n, k, *_check_offsets(offsets, shape[0])
    # one by one: says what is wrong
    if shape[-1] != up // 2 or codes.dtype != torch.uint8 or not codes.is_cuda or not codes.is_contiguous():
        raise ValueError(f"the weight's codes must be a contiguous CUDA tensor of {torch.uint8} with rows of {up // 2}")
    if scale.shape != want or scale.dtype != torch.bfloat16 or not scale.is_cuda or not scale.is_contiguous():
        raise ValueError(f"the weight's scale must be a contiguous CUDA tensor of {torch.bfloat16} with shape {want}")
    _here("the weight's codes", codes)
    _here("the weight's scale", scale)
    if not stacked:
        return n, k, 1, None
    groups, optr = _check_offsets(offsets, shape[0])
    return n, k, groups, optr


def muon_int4_linear(x, w: Int4Matrix, *, offsets=None, out_dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """y = x W^T with a weight of 4 bits (``muon_int4_quantize_weight``), for serving: ``x``
    (tokens x k, bf16 or fp32) is not rounded.  With ``offsets``, tokens are sorted by expert
    and ``w`` is stacked over experts; rows of no expert give zero.  The weight has no gradient.
    Made for few tokens: past 16 of one weight, or about 8 of each expert, ``muon_fp8_linear``, which
    rounds x to 8 bits, is the faster one."""
    if stream is not None:
        with _on(stream):
            return muon_int4_linear(x, w, offsets=offsets, out_dtype=out_dtype)
    n, k, groups, optr = _check_int4(w, offsets)
    tokens, _, ld, code = _matrix("x", x, None, k)
    if out_dtype not in _FLOATS:
        raise ValueError(f"out_dtype must be one of {_FLOATS}")
    out = _new_rows(tokens, n, out_dtype)
    _check(lib().muon_int4_linear(x.data_ptr(), code, tokens, ld, w.codes.data_ptr(), w.scale.data_ptr(), int(w.block), n,
                                  k, groups, optr, out.data_ptr(), _FLOAT_CODE[out_dtype], n, _handle(None)))
    return out
