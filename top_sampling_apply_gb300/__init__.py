"""Per-row vocabulary selection on GB300, the training step on the rows it
sampled, and the norm, scores and loss at the vocabulary head: thin Python binding of libtsa.so.

The calls mirror the C ABI in include/tsa.h (logits-processor, "API";
lm-head-topk, "API").  This module only marshals arguments: it checks torch
tensors' device, dtype and contiguity, passes raw pointers and the current
CUDA stream, and maps status codes to exceptions.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import os
import threading
from typing import NamedTuple, Optional, Union

import torch

from . import _build

__all__ = ["apply_token_bitmask", "sample", "topk", "policy_loss", "preference_loss", "PolicyLoss",
           "PreferenceLoss", "lm_head_logprob", "AdamWPlan", "adamw_state", "adamw_plan", "adamw_step",
           "adamw_state_values", "rms_norm", "RMSNorm", "rms_norm_backward", "quantize_rows", "lm_head_int8",
           "lm_head_cross_entropy", "CrossEntropy", "device_status", "max_vocab", "load_library", "TSAError"]

_DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_lock = threading.Lock()
_lib = None
_workspaces = {}  # device index -> uint8 scratch tensor


class TSAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s (status %d)" % (msg, status))
        self.status = status


def load_library(path: Optional[str] = None):
    """Load libtsa.so (built by ``__graft_entry__.build()`` or
    ``python -m top_sampling_apply_gb300._build``).  Raises if it is missing:
    the product has no CPU path."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.LIB
        if not os.path.exists(p):
            raise RuntimeError("libtsa.so not built: run __graft_entry__.build() (nvcc, sm_103a)")
        lib = ctypes.CDLL(p)
        P, i64, i32, u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint64
        f32, sz, ci = ctypes.c_float, ctypes.c_size_t, ctypes.c_int
        lib.tsa_apply_token_bitmask.argtypes = [P, ci, i64, i64, i64, P, i64, P]
        lib.tsa_sample.argtypes = [P, ci, i64, i64, i64, P, i64, P, f32, P, i32, P, f32, P, f32,
                                   u64, u64, P, P, P, sz, P]
        lib.tsa_sample_noalloc.argtypes = [P, ci, i64, i64, i64, P, i64, P, f32, P, i32, P, f32,
                                           P, f32, u64, u64, P, P, P]
        lib.tsa_topk.argtypes = [P, ci, i64, i64, i64, i32, P, P, P, sz, P]
        lib.tsa_sample_icdf.argtypes = [P, ci, i64, i64, i64, P, i64, P, f32, P, i32, P, f32, P,
                                        f32, P, P, P, P, sz, P]
        lib.tsa_bitmask_from_allowed.argtypes = [P, i64, i64, i64, P, i64, P]
        lib.tsa_sample_sequential.argtypes = [P, ci, i64, i64, i64, P, i64, P, f32, P, i32, P, f32,
                                              P, f32, u64, u64, P, P, P, sz, P]
        lib.tsa_sample_sequential_workspace_bytes.argtypes = [i64, i64, ci]
        lib.tsa_sample_sequential_workspace_bytes.restype = sz
        lib.tsa_lm_head_topk.argtypes = [P, i64, i64, i64, P, i64, i64, P, i32, P, P, P, sz, P]
        lib.tsa_lm_head_topk_workspace_bytes.argtypes = [i64, i64, i32]
        lib.tsa_lm_head_topk_workspace_bytes.restype = sz
        lib.tsa_selective_log_softmax.argtypes = [P, ci, i64, i64, i64, P, i64, P, f32, P, P, P]
        lib.tsa_policy_loss.argtypes = [P, ci, i64, i64, i64, P, i64, P, f32, P, P, P, P, P, f32, f32, f32,
                                        f32, P, P, P, P, P, i64, P, sz, P]
        lib.tsa_policy_loss_workspace_bytes.argtypes = [i64, i64, ci]
        lib.tsa_policy_loss_workspace_bytes.restype = sz
        lib.tsa_preference_loss.argtypes = [P, ci, i64, i64, i64, f32, P, P, i64, P, P, f32, f32, f32, ci,
                                            P, P, P, P, P, i64, P, sz, P]
        lib.tsa_preference_loss_workspace_bytes.argtypes = [i64]
        lib.tsa_preference_loss_workspace_bytes.restype = sz
        lib.tsa_lm_head_logprob.argtypes = [P, i64, i64, i64, P, i64, i64, P, f32, P, i64, P, f32, P, P, P, sz, P]
        lib.tsa_lm_head_logprob_workspace_bytes.argtypes = [i64, i64]
        lib.tsa_lm_head_logprob_workspace_bytes.restype = sz
        lib.tsa_lm_head_cross_entropy.argtypes = [P, i64, i64, i64, P, i64, i64, P, f32, P, P, f32, P, P, P, P, i64,
                                                  P, i64, P, P, sz, P]
        lib.tsa_lm_head_cross_entropy_workspace_bytes.argtypes = [i64, i64, i64, ci, ci]
        lib.tsa_lm_head_cross_entropy_workspace_bytes.restype = sz
        lib.tsa_rms_norm.argtypes = [P, ci, i64, i64, i64, P, ci, P, i64, f32, ci, P, i64, P, P, i64, P, P]
        lib.tsa_rms_norm_backward.argtypes = [P, i64, P, ci, i64, i64, i64, P, ci, P, P, i64, P, i64, P, P, sz, P]
        lib.tsa_rms_norm_backward_workspace_bytes.argtypes = [i64, i64]
        lib.tsa_rms_norm_backward_workspace_bytes.restype = sz
        lib.tsa_quantize_rows.argtypes = [P, ci, i64, i64, i64, P, i64, P, P]
        lib.tsa_lm_head_int8.argtypes = [P, i64, i64, i64, P, P, i64, i64, P, P, P, ci, i64, P, sz, P]
        lib.tsa_lm_head_int8_workspace_bytes.argtypes = [i64, i64]
        lib.tsa_lm_head_int8_workspace_bytes.restype = sz
        f64 = ctypes.c_double
        lib.tsa_adamw_step.argtypes = [P, i64, ci, ci, i32, f64, f64, f64, f64, f64, i64, P, u64, u64, P]
        lib.tsa_adamw_state_values.argtypes = [P, i64, P, P, P]
        lib.tsa_sample_workspace_bytes.argtypes = [i64, i64, ci]
        lib.tsa_sample_workspace_bytes.restype = sz
        lib.tsa_topk_workspace_bytes.argtypes = [i64, i64, i32, ci]
        lib.tsa_topk_workspace_bytes.restype = sz
        lib.tsa_status_string.argtypes = [ci]
        lib.tsa_status_string.restype = ctypes.c_char_p
        lib.tsa_device_status.argtypes = [ci]
        lib.tsa_selftest_wait_timeout.argtypes = [ctypes.c_uint32, P]
        lib.tsa_max_vocab.argtypes = [ci]
        lib.tsa_max_vocab.restype = i64
        for fn in ("tsa_apply_token_bitmask", "tsa_sample", "tsa_sample_noalloc", "tsa_topk",
                   "tsa_sample_icdf", "tsa_bitmask_from_allowed", "tsa_sample_sequential", "tsa_lm_head_topk",
                   "tsa_policy_loss", "tsa_preference_loss", "tsa_lm_head_logprob", "tsa_adamw_step",
                   "tsa_adamw_state_values", "tsa_lm_head_cross_entropy", "tsa_rms_norm", "tsa_rms_norm_backward",
                   "tsa_quantize_rows", "tsa_lm_head_int8",
                   "tsa_device_status", "tsa_selftest_wait_timeout"):
            getattr(lib, fn).restype = ci
        _lib = lib
        return lib


def _check(status: int):
    if status != 0:
        lib = load_library()
        raise TSAError(status, lib.tsa_status_string(status).decode())


_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _call(index: int, fn, *args):
    """A call of the library for tensors on CUDA device ``index``: a launch goes to the current
    device, so that one is made current if another is."""
    if _current_device() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        _check(status)


def _written(tensors) -> None:
    """Raises the versions of tensors written in place, as torch's own operations do: autograd then
    refuses a backward pass that needs what they held.  Inference tensors have none."""
    torch.autograd.graph.increment_version(tensors)


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


def _rows(logits: torch.Tensor):
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dtype not in _DT:
        raise ValueError("logits dtype must be float32, float16 or bfloat16")
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D [B, V] with unit stride along V")
    return logits.shape[0], logits.shape[1], logits.stride(0)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _workspace(nbytes: int, device: torch.device) -> torch.Tensor:
    """A device workspace of at least ``nbytes``, cached per device (calls on
    different streams must not run concurrently on the same workspace)."""
    idx = device.index if device.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(idx)
    if ws is None or ws.numel() < nbytes:
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        _workspaces[idx] = ws
    return ws


def max_vocab(dtype: torch.dtype) -> int:
    return int(load_library().tsa_max_vocab(_DT[dtype]))


def apply_token_bitmask(logits: torch.Tensor, bitmask: torch.Tensor) -> torch.Tensor:
    """logits-processor, "API": set logits to -inf, in place, where the packed
    bit is 0 (bit 1 = allowed).  bitmask: int32 [B, >= ceil(V / 32)]."""
    lib = load_library()
    B, V, stride = _rows(logits)
    if bitmask.dtype != torch.int32 or not bitmask.is_cuda or bitmask.dim() != 2:
        raise ValueError("bitmask must be a CUDA int32 [B, W] tensor")
    if bitmask.shape[0] != B or bitmask.stride(1) != 1:
        raise ValueError("bitmask must have B rows and unit stride along W")
    if bitmask.shape[1] < (V + 31) // 32:
        raise ValueError("bitmask needs ceil(V / 32) words per row")
    _call(logits.get_device(), lib.tsa_apply_token_bitmask, _ptr(logits), _DT[logits.dtype], B, V, stride,
          _ptr(bitmask), bitmask.stride(0), _stream(logits))
    return logits


Param = Union[float, int, torch.Tensor]


def _param(x: Param, B: int, dtype: torch.dtype, device):
    """(device pointer or None, scalar) for a per-row parameter."""
    if isinstance(x, torch.Tensor):
        if x.dim() == 0:
            return None, x.item()
        if x.shape != (B,) or x.dtype != dtype or x.device != device or not x.is_contiguous():
            raise ValueError("per-row parameter must be a contiguous %s [B] tensor on %s"
                             % (dtype, device))
        return x, 0
    return None, x


def sample(logits: torch.Tensor, temperature: Param = 1.0, top_k: Param = 0, top_p: Param = 1.0,
           min_p: Param = 0.0, seed: int = 0, offset: int = 0,
           bitmask: Optional[torch.Tensor] = None, return_min_kept: bool = False,
           out: Optional[torch.Tensor] = None, sequential: bool = False):
    """logits-processor, "API": one int64 token per row (-1 for a row with no
    allowed finite logit).  Each sampling parameter is a scalar or a [B]
    tensor (float32 for temperature / top_p / min_p, int32 for top_k).  With
    ``bitmask`` the mask is applied on load; the logits are not modified.
    ``sequential`` takes top-p over the softmax renormalised over the top-k
    survivors (the transformers processor chain) instead of the full one."""
    lib = load_library()
    B, V, stride = _rows(logits)
    dev = logits.device
    T, Ts = _param(temperature, B, torch.float32, dev)
    K, Ks = _param(top_k, B, torch.int32, dev)
    Pp, Ps = _param(top_p, B, torch.float32, dev)
    M, Ms = _param(min_p, B, torch.float32, dev)
    if bitmask is not None:
        if bitmask.dtype != torch.int32 or bitmask.device != dev or bitmask.dim() != 2:
            raise ValueError("bitmask must be an int32 [B, W] tensor on the logits' device")
        if bitmask.shape[0] != B or bitmask.stride(1) != 1 or bitmask.shape[1] < (V + 31) // 32:
            raise ValueError("bitmask must be [B, >= ceil(V / 32)] with unit stride along W")
        mstride = bitmask.stride(0)
    else:
        mstride = 0
    tokens = out if out is not None else torch.empty(B, dtype=torch.int64, device=dev)
    vstar = torch.empty(B, dtype=torch.float32, device=dev) if return_min_kept else None
    if sequential:
        nws = int(lib.tsa_sample_sequential_workspace_bytes(B, V, _DT[logits.dtype]))
        ws = _workspace(nws, dev) if nws > 0 else None
        call = lib.tsa_sample_sequential
    else:
        nws = int(lib.tsa_sample_workspace_bytes(B, V, _DT[logits.dtype]))
        ws = _workspace(nws, dev) if nws > 0 else None
        call = lib.tsa_sample
    _call(logits.get_device(), call, _ptr(logits), _DT[logits.dtype], B, V, stride, _ptr(bitmask), mstride, _ptr(T),
          float(Ts), _ptr(K), int(Ks), _ptr(Pp), float(Ps), _ptr(M), float(Ms), int(seed) & 0xFFFFFFFFFFFFFFFF,
          int(offset) & 0xFFFFFFFFFFFFFFFF, _ptr(tokens), _ptr(vstar), _ptr(ws), nws, _stream(logits))
    return (tokens, vstar) if return_min_kept else tokens


def sample_icdf(logits: torch.Tensor, uniform: torch.Tensor, temperature: Param = 1.0, top_k: Param = 0,
                top_p: Param = 1.0, min_p: Param = 0.0, bitmask: Optional[torch.Tensor] = None,
                return_min_kept: bool = False, out: Optional[torch.Tensor] = None):
    """logits-mask-xpu, "Usage" / "Method": the inverse-CDF draw from the caller's
    ``uniform`` (float32 [B] in [0, 1) on the logits' device) over the keep set of
    ``sample``: the first kept token, in index order, whose running weight passes
    u W.  Parameters as ``sample`` (no seed: the draw is the uniform's)."""
    lib = load_library()
    B, V, stride = _rows(logits)
    dev = logits.device
    if uniform.dtype != torch.float32 or uniform.device != dev or uniform.shape != (B,) \
            or not uniform.is_contiguous():
        raise ValueError("uniform must be a contiguous float32 [B] tensor on the logits' device")
    T, Ts = _param(temperature, B, torch.float32, dev)
    K, Ks = _param(top_k, B, torch.int32, dev)
    Pp, Ps = _param(top_p, B, torch.float32, dev)
    M, Ms = _param(min_p, B, torch.float32, dev)
    mstride = _mask_stride(bitmask, B, V, dev)
    tokens = out if out is not None else torch.empty(B, dtype=torch.int64, device=dev)
    vstar = torch.empty(B, dtype=torch.float32, device=dev)
    nws = int(lib.tsa_sample_workspace_bytes(B, V, _DT[logits.dtype]))
    ws = _workspace(nws, dev) if nws > 0 else None
    _call(logits.get_device(), lib.tsa_sample_icdf, _ptr(logits), _DT[logits.dtype], B, V, stride, _ptr(bitmask),
          mstride, _ptr(T), float(Ts), _ptr(K), int(Ks), _ptr(Pp), float(Ps), _ptr(M), float(Ms), _ptr(uniform),
          _ptr(tokens), _ptr(vstar), _ptr(ws), nws, _stream(logits))
    return (tokens, vstar) if return_min_kept else tokens


def bitmask_from_allowed(allowed: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """logits-mask-xpu, "Usage": a CUDA bool [B, V] allow-set packed into int32
    [B, ceil(V / 32)] words (token i at bit i % 32 of word i // 32)."""
    lib = load_library()
    if allowed.dtype != torch.bool or not allowed.is_cuda or allowed.dim() != 2 or allowed.stride(1) != 1:
        raise ValueError("allowed must be a CUDA bool [B, V] tensor with unit stride along V")
    B, V = allowed.shape
    W = (V + 31) // 32
    bits = out if out is not None else torch.empty(B, W, dtype=torch.int32, device=allowed.device)
    if bits.dtype != torch.int32 or bits.device != allowed.device or bits.shape[0] != B \
            or bits.shape[1] < W or bits.stride(1) != 1:
        raise ValueError("out must be an int32 [B, >= ceil(V / 32)] tensor on the same device")
    _call(allowed.get_device(), lib.tsa_bitmask_from_allowed, _ptr(allowed), B, V, allowed.stride(0), _ptr(bits),
          bits.stride(0), _stream(allowed))
    return bits


def _mask_stride(bitmask: Optional[torch.Tensor], B: int, V: int, dev) -> int:
    if bitmask is None:
        return 0
    if bitmask.dtype != torch.int32 or bitmask.device != dev or bitmask.dim() != 2:
        raise ValueError("bitmask must be an int32 [B, W] tensor on the logits' device")
    if bitmask.shape[0] != B or bitmask.stride(1) != 1 or bitmask.shape[1] < (V + 31) // 32:
        raise ValueError("bitmask must be [B, >= ceil(V / 32)] with unit stride along W")
    return bitmask.stride(0)


def selective_log_softmax(logits: torch.Tensor, index: torch.Tensor, temperature: Param = 1.0,
                          bitmask: Optional[torch.Tensor] = None,
                          out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """selective_log_softmax, "Selective Log Softmax": one float per row, the
    log-softmax of the allowed, temperature-scaled row at ``index`` (int64
    [B]); T <= 0 uses T = 1.  -inf for a disallowed index, NaN for an index
    outside [0, V) or a row with no allowed finite logit.  Called with
    ``sample``'s tokens it gives their log-probabilities before filtering."""
    lib = load_library()
    B, V, stride = _rows(logits)
    dev = logits.device
    if index.dtype != torch.int64 or index.device != dev or index.shape != (B,) or not index.is_contiguous():
        raise ValueError("index must be a contiguous int64 [B] tensor on the logits' device")
    T, Ts = _param(temperature, B, torch.float32, dev)
    if bitmask is not None:
        if bitmask.dtype != torch.int32 or bitmask.device != dev or bitmask.dim() != 2:
            raise ValueError("bitmask must be an int32 [B, W] tensor on the logits' device")
        if bitmask.shape[0] != B or bitmask.stride(1) != 1 or bitmask.shape[1] < (V + 31) // 32:
            raise ValueError("bitmask must be [B, >= ceil(V / 32)] with unit stride along W")
        mstride = bitmask.stride(0)
    else:
        mstride = 0
    res = out if out is not None else torch.empty(B, dtype=torch.float32, device=dev)
    _call(logits.get_device(), lib.tsa_selective_log_softmax, _ptr(logits), _DT[logits.dtype], B, V, stride,
          _ptr(bitmask), mstride, _ptr(T), float(Ts), _ptr(index), _ptr(res), _stream(logits))
    return res


def sample_noalloc(logits: torch.Tensor, tokens_out: torch.Tensor, temperature: Param = 1.0,
                   top_k: Param = 0, top_p: Param = 1.0, min_p: Param = 0.0, seed: int = 0,
                   offset: int = 0, bitmask: Optional[torch.Tensor] = None,
                   min_kept_out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``sample`` for callers that cannot allocate device memory: the library
    uses its own fixed device scratch (at most
    ``sample_noalloc_max_bytes()`` of workspace), so nothing is allocated
    here; the caller passes the int64 [B] ``tokens_out`` (and optionally the
    float32 [B] ``min_kept_out``).  Calls overlapping on the GPU share that
    scratch and must not run concurrently."""
    lib = load_library()
    B, V, stride = _rows(logits)
    dev = logits.device
    T, Ts = _param(temperature, B, torch.float32, dev)
    K, Ks = _param(top_k, B, torch.int32, dev)
    Pp, Ps = _param(top_p, B, torch.float32, dev)
    M, Ms = _param(min_p, B, torch.float32, dev)
    if tokens_out is None:
        raise ValueError("tokens_out is required")
    for t, dt, name in ((tokens_out, torch.int64, "tokens_out"), (min_kept_out, torch.float32, "min_kept_out")):
        if t is not None and (t.shape != (B,) or t.dtype != dt or t.device != dev or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous %s [B] tensor on %s" % (name, dt, dev))
    if bitmask is not None:
        if bitmask.dtype != torch.int32 or bitmask.device != dev or bitmask.dim() != 2:
            raise ValueError("bitmask must be an int32 [B, W] tensor on the logits' device")
        if bitmask.shape[0] != B or bitmask.stride(1) != 1 or bitmask.shape[1] < (V + 31) // 32:
            raise ValueError("bitmask must be [B, >= ceil(V / 32)] with unit stride along W")
        mstride = bitmask.stride(0)
    else:
        mstride = 0
    _call(logits.get_device(), lib.tsa_sample_noalloc, _ptr(logits), _DT[logits.dtype], B, V, stride, _ptr(bitmask),
          mstride, _ptr(T), float(Ts), _ptr(K), int(Ks), _ptr(Pp), float(Ps), _ptr(M), float(Ms),
          int(seed) & 0xFFFFFFFFFFFFFFFF, int(offset) & 0xFFFFFFFFFFFFFFFF, _ptr(tokens_out), _ptr(min_kept_out),
          _stream(logits))
    return tokens_out


def sample_noalloc_max_bytes() -> int:
    """Size of the fixed scratch behind ``sample_noalloc``: a (B, V, dtype)
    whose ``tsa_sample_workspace_bytes`` exceeds it is rejected."""
    return 16 * 1024 * 1024


def lm_head_topk(hidden: torch.Tensor, weight: torch.Tensor, k: int, bias: Optional[torch.Tensor] = None):
    """lm-head-topk, "API" (the dense head): (values float32 [M, k], indices
    int64 [M, k]) of the exact top-k of hidden @ weight^T (+ bias), sorted
    descending, ties to the lower index; the score matrix is never written.
    hidden bf16 [M <= 4, H], weight bf16 [V, H] (unit stride along H)."""
    lib = load_library()
    for t, name in ((hidden, "hidden"), (weight, "weight")):
        if t.dtype != torch.bfloat16 or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("%s must be a CUDA bfloat16 2-D tensor with unit stride along H" % name)
    M, H = hidden.shape
    V = weight.shape[0]
    if weight.shape[1] != H or weight.device != hidden.device:
        raise ValueError("weight must be [V, H] on the hidden rows' device")
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (V,) or bias.device != hidden.device
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 [V] tensor on the same device")
    dev = hidden.device
    values = torch.empty(M, k, dtype=torch.float32, device=dev)
    indices = torch.empty(M, k, dtype=torch.int64, device=dev)
    nws = int(lib.tsa_lm_head_topk_workspace_bytes(M, V, k))
    ws = _workspace(nws, dev) if nws > 0 else None
    _call(hidden.get_device(), lib.tsa_lm_head_topk, _ptr(hidden), M, H, hidden.stride(0), _ptr(weight), V,
          weight.stride(0), _ptr(bias), int(k), _ptr(values), _ptr(indices), _ptr(ws), nws, _stream(hidden))
    return values, indices


def topk(logits: torch.Tensor, k: int):
    """lm-head-topk, "API": (values float32 [B, k], indices int64 [B, k]),
    sorted by value descending, ties to the lower index; k <= 2048."""
    lib = load_library()
    B, V, stride = _rows(logits)
    values = torch.empty(B, k, dtype=torch.float32, device=logits.device)
    indices = torch.empty(B, k, dtype=torch.int64, device=logits.device)
    _call(logits.get_device(), lib.tsa_topk, _ptr(logits), _DT[logits.dtype], B, V, stride, int(k), _ptr(values),
          _ptr(indices), None, 0, _stream(logits))
    return values, indices


def _vec(t: Optional[torch.Tensor], n: int, dtype: torch.dtype, index: int, name: str):
    """Checks an optional contiguous [n] tensor on CUDA device ``index``; its address, or None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != index or t.dim() != 1 or t.size(0) != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s [%d] tensor on cuda:%d" % (name, dtype, n, index))
    return t.data_ptr()


def _temperature(x: Param, n: int, index: int):
    """(address or None, scalar) of a temperature."""
    if isinstance(x, torch.Tensor) and x.dim() > 0:
        return _vec(x, n, torch.float32, index, "temperature"), 0.0
    return None, float(x)


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _grad_rows(grad, logits: torch.Tensor) -> Optional[torch.Tensor]:
    """The tensor a call writes its gradient to: none, the caller's, or a new
    one whose rows start at the logits' alignment (the fast path)."""
    if isinstance(grad, torch.Tensor):
        if grad.shape != logits.shape or grad.dtype != logits.dtype or grad.device != logits.device \
                or (grad.shape[0] > 0 and grad.stride(1) != 1):
            raise ValueError("grad must have the logits' shape, dtype and device and unit stride along V")
        return grad
    if not grad:
        return None
    B, V = logits.shape
    first = logits.data_ptr() % 16
    if first == 0 and logits.stride(0) == V or B == 0:
        return torch.empty((B, V), dtype=logits.dtype, device=logits.device)
    es = logits.element_size()
    first //= es
    stride = V + (logits.stride(0) - V) % (16 // es)
    buf = torch.empty(B * stride + first, dtype=logits.dtype, device=logits.device)
    return buf[first:].as_strided((B, V), (stride, 1))


class PolicyLoss(NamedTuple):
    """What ``policy_loss`` returns."""
    loss: torch.Tensor  # float32 scalar: the weighted sum over rows
    row_loss: torch.Tensor  # float32 [B]
    logprob: torch.Tensor  # float32 [B]: ln p of each row's token
    entropy: Optional[torch.Tensor]  # float32 [B]
    grad: Optional[torch.Tensor]  # [B, V] of the logits' dtype: d loss / d logits


def policy_loss(logits: torch.Tensor, tokens: torch.Tensor, old_logprob: torch.Tensor, advantage: torch.Tensor,
                ref_logprob: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                clip_low: float = 0.2, clip_high: float = 0.2, kl_coef: float = 0.0, entropy_coef: float = 0.0,
                temperature: Param = 1.0, bitmask: Optional[torch.Tensor] = None, return_entropy: bool = False,
                grad: Union[bool, torch.Tensor] = True) -> PolicyLoss:
    """The clipped policy loss of sampled tokens, with a KL term against
    ``ref_logprob`` and an entropy bonus, and its gradient on the logits.

    A row's loss is -min(r A, clip(r, 1 - clip_low, 1 + clip_high) A) + kl_coef
    (exp(ref - lp) - (ref - lp) - 1) - entropy_coef H, with lp the row's
    ``selective_log_softmax`` at its token and r = exp(lp - old_logprob); the loss is the
    sum of ``weight`` times it (None: the mean).  ``tokens`` as ``sample`` gives them: a
    token of -1 skips its row, as a weight of 0 does, and skipped rows' logits are not read.
    ``grad``: True for a new tensor, a tensor to write (``logits`` itself for in place), or
    False for the loss alone.  There is no autograd graph: the gradient is returned, and
    ``logits.backward(r.grad)`` carries it further (in place only where what made the logits
    does not need them again: autograd refuses otherwise)."""
    lib = _lib or load_library()
    B, V, stride = _rows(logits)
    dev = logits.get_device()
    tok = _vec(tokens, B, torch.int64, dev, "tokens")
    old = _vec(old_logprob, B, torch.float32, dev, "old_logprob")
    adv = _vec(advantage, B, torch.float32, dev, "advantage")
    ref = _vec(ref_logprob, B, torch.float32, dev, "ref_logprob")
    wgt = _vec(weight, B, torch.float32, dev, "weight")
    T, Ts = _temperature(temperature, B, dev)
    device, dt = logits.device, _DT[logits.dtype]
    mstride = 0 if bitmask is None else _mask_stride(bitmask, B, V, device)
    g = _grad_rows(grad, logits)
    # an allocation each: on the host that is cheaper than views of one
    empty, f32 = torch.empty, torch.float32
    loss, row, lp = empty((), dtype=f32, device=device), empty(B, dtype=f32, device=device), \
        empty(B, dtype=f32, device=device)
    ent = empty(B, dtype=f32, device=device) if return_entropy else None
    nws, ws = 0, None
    if g is not None and V > 131072:  # shorter rows need none
        nws = lib.tsa_policy_loss_workspace_bytes(B, V, dt)
        ws = empty(nws, dtype=torch.uint8, device=device) if nws else None
    _call(dev, lib.tsa_policy_loss, logits.data_ptr(), dt, B, V, stride,
          None if bitmask is None else bitmask.data_ptr(), mstride, T, Ts, tok, old, adv, ref, wgt, clip_low,
          clip_high, kl_coef, entropy_coef, loss.data_ptr(), row.data_ptr(), lp.data_ptr(),
          None if ent is None else ent.data_ptr(), None if g is None else g.data_ptr(),
          0 if g is None else g.stride(0), None if ws is None else ws.data_ptr(), nws, _raw_stream(dev))
    if g is not None and g is grad:
        _written(g)
    return PolicyLoss(loss, row, lp, ent, g)


class PreferenceLoss(NamedTuple):
    """What ``preference_loss`` returns."""
    loss: torch.Tensor  # float32 scalar: the mean over pairs
    pair_loss: torch.Tensor  # float32 [P]
    reward: torch.Tensor  # float32 [2 P]: beta times each sequence's log-ratio
    logprob: torch.Tensor  # float32 [N]
    grad: Optional[torch.Tensor]  # [N, V] of the logits' dtype


def preference_loss(logits: torch.Tensor, tokens: torch.Tensor, seq_start: torch.Tensor,
                    weight: Optional[torch.Tensor] = None, ref_logprob: Optional[torch.Tensor] = None,
                    beta: float = 0.1, label_smoothing: float = 0.0, margin: float = 0.0, average: bool = False,
                    temperature: float = 1.0, grad: Union[bool, torch.Tensor] = True) -> PreferenceLoss:
    """The loss of preferred over rejected answers from paired log-ratios, and its
    gradient on the logits.

    The rows are the tokens of 2 P sequences one after another, the preferred answers first:
    sequence s is rows ``seq_start[s]`` to ``seq_start[s + 1]`` (int64 [2 P + 1] on the logits'
    device), pair p is sequences p and P + p.  A sequence's log-ratio is the sum of
    ``weight`` times (log-probability - ``ref_logprob``) over its rows, divided by the sum of
    the weights with ``average``.  A weight of 0 skips a row (its logits are not read)."""
    lib = _lib or load_library()
    N, V, stride = _rows(logits)
    dev = logits.get_device()
    if seq_start.dim() != 1 or seq_start.numel() % 2 == 0:
        raise ValueError("seq_start must have 2 P + 1 entries")
    P = seq_start.numel() // 2
    start = _vec(seq_start, 2 * P + 1, torch.int64, dev, "seq_start")
    tok = _vec(tokens, N, torch.int64, dev, "tokens")
    wgt = _vec(weight, N, torch.float32, dev, "weight")
    ref = _vec(ref_logprob, N, torch.float32, dev, "ref_logprob")
    g = _grad_rows(grad, logits)
    device, empty, f32 = logits.device, torch.empty, torch.float32
    loss, pair, reward, lp = empty((), dtype=f32, device=device), empty(P, dtype=f32, device=device), \
        empty(2 * P, dtype=f32, device=device), empty(N, dtype=f32, device=device)
    nws = lib.tsa_preference_loss_workspace_bytes(N)
    ws = empty(nws, dtype=torch.uint8, device=device) if nws else None
    _call(dev, lib.tsa_preference_loss, logits.data_ptr(), _DT[logits.dtype], N, V, stride, temperature, tok, start,
          P, wgt, ref, beta, label_smoothing, margin, 1 if average else 0, loss.data_ptr(), pair.data_ptr(),
          reward.data_ptr(), lp.data_ptr(), None if g is None else g.data_ptr(), 0 if g is None else g.stride(0),
          None if ws is None else ws.data_ptr(), nws, _raw_stream(dev))
    if g is not None and g is grad:
        _written(g)
    return PreferenceLoss(loss, pair, reward, lp, g)


def lm_head_logprob(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, softcap: float = 0.0, temperature: Param = 1.0,
                    bitmask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``selective_log_softmax`` of hidden @ weight^T (+ bias, capped to softcap tanh(z /
    softcap) where softcap > 0) at ``tokens``, float32 [M], without writing the scores.
    hidden bf16 [M, H], weight bf16 [V, H] (unit stride along H); temperature and bitmask as
    there.  The log-probabilities under a rollout or reference policy that ``policy_loss`` and
    ``preference_loss`` take."""
    lib = _lib or load_library()
    for t, name in ((hidden, "hidden"), (weight, "weight")):
        if t.dtype is not torch.bfloat16 or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("%s must be a CUDA bfloat16 2-D tensor with unit stride along H" % name)
    M, H = hidden.shape
    V = weight.size(0)
    dev = hidden.get_device()
    if weight.size(1) != H or weight.get_device() != dev:
        raise ValueError("weight must be [V, H] on the hidden rows' device")
    tok = _vec(tokens, M, torch.int64, dev, "tokens")
    b = _vec(bias, V, torch.float32, dev, "bias")
    res = torch.empty(M, dtype=torch.float32, device=hidden.device) if out is None else out
    to = _vec(res, M, torch.float32, dev, "out")
    T, Ts = _temperature(temperature, M, dev)
    mstride = 0 if bitmask is None else _mask_stride(bitmask, M, V, hidden.device)
    nws = lib.tsa_lm_head_logprob_workspace_bytes(M, V)
    ws = torch.empty(nws, dtype=torch.uint8, device=hidden.device) if nws else None
    _call(dev, lib.tsa_lm_head_logprob, hidden.data_ptr(), M, H, hidden.stride(0), weight.data_ptr(), V,
          weight.stride(0), b, softcap, None if bitmask is None else bitmask.data_ptr(), mstride, T, Ts, tok, to,
          None if ws is None else ws.data_ptr(), nws, _raw_stream(dev))
    if out is not None:
        _written(out)
    return res


class _AdamTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_exp", ctypes.c_void_p),
                ("exp_avg_sq_exp", ctypes.c_void_p), ("n", ctypes.c_int64)]


class AdamWPlan:
    """A list of parameters with their gradients and states, checked and laid out once for
    ``adamw_step``.  It holds the tensors and the memory they have when it is made: a gradient
    that becomes another tensor (``zero_grad(set_to_none=True)``), or a parameter whose ``data``
    is assigned anew, needs a new plan."""

    def __init__(self, params, grads, exp_avg, exp_avg_sq, exp_avg_exp=None, exp_avg_sq_exp=None):
        params, grads, exp_avg, exp_avg_sq = list(params), list(grads), list(exp_avg), list(exp_avg_sq)
        n = len(params)
        bits = 8 if exp_avg and exp_avg[0].dtype == torch.uint8 else 32
        lists = [("params", params), ("grads", grads), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq)]
        if bits == 8:
            if exp_avg_exp is None or exp_avg_sq_exp is None:
                raise ValueError("8-bit states need exp_avg_exp and exp_avg_sq_exp")
            exp_avg_exp, exp_avg_sq_exp = list(exp_avg_exp), list(exp_avg_sq_exp)
            lists += [("exp_avg_exp", exp_avg_exp), ("exp_avg_sq_exp", exp_avg_sq_exp)]
        elif exp_avg_exp is not None or exp_avg_sq_exp is not None:
            raise ValueError("32-bit states have no exponents")
        for name, seq in lists:
            if len(seq) != n:
                raise ValueError("%s must have as many tensors as params" % name)
        if n:
            dev = params[0].device
            dts = {"params": params[0].dtype, "grads": grads[0].dtype}
            state = torch.uint8 if bits == 8 else torch.float32
            if not params[0].is_cuda:
                raise ValueError("params must be CUDA tensors")
            if dts["params"] not in (torch.float32, torch.bfloat16) or dts["grads"] not in _DT:
                raise ValueError("params must be float32 or bfloat16, grads float32, float16 or bfloat16")
            for name, seq in lists:
                dt = dts.get(name, state)
                for i, t in enumerate(seq):
                    want = (params[i].numel() + 255) // 256 if name.endswith("_exp") else params[i].numel()
                    if t.device != dev or t.dtype != dt or not t.is_contiguous() or t.numel() != want:
                        raise ValueError("%s[%d] must be a contiguous %s tensor of %d elements on %s"
                                         % (name, i, dt, want, dev))
        self.params, self.grads = params, grads
        self.exp_avg, self.exp_avg_sq = exp_avg, exp_avg_sq
        self.exp_avg_exp, self.exp_avg_sq_exp = exp_avg_exp, exp_avg_sq_exp
        self.bits = bits
        self.sizes = [p.numel() for p in params]
        self.index = params[0].get_device() if params else torch.cuda.current_device()
        self._dts = (_DT[params[0].dtype], _DT[grads[0].dtype]) if params else (0, 0)
        # the tensors whose versions a step raises: views share their base's
        bases = [p if p._base is None else p._base for p in params]
        self._versions = list({id(t): t for t in bases}.values())
        # the table's addresses stay the plan's own, whatever becomes of the tensors
        self._memory = [t.untyped_storage() for _, seq in lists for t in seq]
        self._table = (_AdamTensor * max(1, len(params)))()
        for i, p in enumerate(params):
            t = self._table[i]
            t.param, t.grad, t.n = p.data_ptr(), grads[i].data_ptr(), p.numel()
            t.exp_avg, t.exp_avg_sq = exp_avg[i].data_ptr(), exp_avg_sq[i].data_ptr()
            if bits == 8:
                t.exp_avg_exp, t.exp_avg_sq_exp = exp_avg_exp[i].data_ptr(), exp_avg_sq_exp[i].data_ptr()


def adamw_state(params, bits: int = 32):
    """Zero states for ``adamw_plan``: lists (exp_avg, exp_avg_sq, exp_avg_exp, exp_avg_sq_exp);
    float32 and None, None for 32 bits, uint8 codes and a uint8 exponent a block of 256 for 8."""
    if bits not in (8, 32):
        raise ValueError("bits must be 8 or 32")
    dt = torch.float32 if bits == 32 else torch.uint8
    m, v = ([torch.zeros(p.shape, dtype=dt, device=p.device) for p in params] for _ in range(2))
    if bits == 32:
        return m, v, None, None
    me, ve = ([torch.zeros((p.numel() + 255) // 256, dtype=torch.uint8, device=p.device) for p in params]
              for _ in range(2))
    return m, v, me, ve


def adamw_plan(params, grads, exp_avg, exp_avg_sq, exp_avg_exp=None, exp_avg_sq_exp=None) -> AdamWPlan:
    """Checks and lays out the tensors of ``adamw_step``: contiguous CUDA tensors, parameters
    float32 or bfloat16, gradients float32, float16 or bfloat16, states float32 or uint8 with a
    uint8 exponent a block of 256 (see ``adamw_state``)."""
    return AdamWPlan(params, grads, exp_avg, exp_avg_sq, exp_avg_exp, exp_avg_sq_exp)


def adamw_step(plan: AdamWPlan, step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01, grad_scale: Optional[torch.Tensor] = None, seed: int = 0,
               offset: int = 0) -> None:
    """One AdamW step over every tensor of the plan, in place.

    ``step`` counts from 1 (bias correction).  ``grad_scale``: a float32 [1] tensor that
    multiplies the gradients; a value that is not finite skips the step.  ``seed``, ``offset``
    key the random rounding of bf16 parameters and 8-bit second moments; advance ``offset``
    every step, and use another seed than ``sample``'s, whose words come from the same function."""
    lib = _lib or load_library()
    scale = _vec(grad_scale, 1, torch.float32, plan.index, "grad_scale")
    _call(plan.index, lib.tsa_adamw_step, plan._table, len(plan.params), plan._dts[0], plan._dts[1], plan.bits, lr,
          beta1, beta2, eps, weight_decay, step, scale, int(seed) & 0xFFFFFFFFFFFFFFFF,
          int(offset) & 0xFFFFFFFFFFFFFFFF, _raw_stream(plan.index))
    _written(plan._versions)


def adamw_state_values(plan: AdamWPlan, exp_avg_out=None, exp_avg_sq_out=None):
    """The values that a plan's 8-bit states stand for, as lists of bfloat16 tensors (which hold
    them exactly): (exp_avg, exp_avg_sq), for checkpoints and inspection."""
    lib = load_library()
    if plan.bits != 8:
        raise ValueError("32-bit states are their own values")
    T, sizes, outs, ptrs = torch.Tensor, plan.sizes, [], []
    for given, like in ((exp_avg_out, plan.exp_avg), (exp_avg_sq_out, plan.exp_avg_sq)):
        given = [torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) for t in like] if given is None \
            else given if isinstance(given, list) else list(given)
        if list(map(T.numel, given)) != sizes or any(t.dtype is not torch.bfloat16 for t in given) \
                or any(d != plan.index for d in map(T.get_device, given)) or not all(map(T.is_contiguous, given)):
            raise ValueError("outputs must be contiguous bfloat16 tensors of the states' sizes")
        outs.append(given)
        ptrs.append(array.array("Q", list(map(T.data_ptr, given))))
    _call(plan.index, lib.tsa_adamw_state_values, plan._table, len(sizes), ptrs[0].buffer_info()[0],
          ptrs[1].buffer_info()[0], _raw_stream(plan.index))
    for given, mine in zip((exp_avg_out, exp_avg_sq_out), outs):
        if given is not None:
            _written(mine)
    return outs[0], outs[1]


def _matrix(t: torch.Tensor, index: int, shape, dtype: torch.dtype, name: str, unit: str = "H") -> torch.Tensor:
    """Checks a [rows, columns] tensor of unit stride along its columns on CUDA device ``index``."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or \
            (t.stride(1) != 1 and shape[1] > 1 and shape[0] > 0):
        raise ValueError("%s must be a %s %s tensor on cuda:%d with unit stride along %s"
                         % (name, dtype, list(shape), index, unit))
    return t


def _hidden_rows(t: torch.Tensor, name: str):
    if not t.is_cuda or t.dtype not in _DT or t.dim() != 2 or (t.stride(1) != 1 and t.size(1) > 1):
        raise ValueError("%s must be a CUDA float32, float16 or bfloat16 2-D tensor with unit stride along H" % name)
    N, H = t.shape
    return N, H, t.get_device()


def _norm_weight(weight: torch.Tensor, x: torch.Tensor) -> None:
    dt = weight.dtype
    if (dt is not x.dtype and dt is not torch.float32) or weight.get_device() != x.get_device() or weight.dim() != 1 \
            or weight.size(0) != x.size(1) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous [H] tensor of the rows' dtype or float32 on their device")


class RMSNorm(NamedTuple):
    """What ``rms_norm`` returns."""
    out: torch.Tensor  # [N, H] of the rows' dtype, or int8
    scale: Optional[torch.Tensor]  # float32 [N]: what an int8 row's codes are multiplied by
    residual: Optional[torch.Tensor]  # [N, H]: the rows with the residual added, rounded to their dtype
    rstd: torch.Tensor  # float32 [N]: what ``rms_norm_backward`` takes


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None, eps: float = 1e-6,
             quantize: bool = False, out: Optional[torch.Tensor] = None,
             residual_out: Optional[torch.Tensor] = None) -> RMSNorm:
    """The root-mean-square norm that makes the hidden rows of the ``lm_head_*`` calls.

    With s = x, or x + ``residual`` rounded to their dtype, out = s / sqrt(mean(s^2) + eps) *
    ``weight``.  ``quantize`` gives the rows in 8 bits, as ``lm_head_int8`` takes them: scale = max|y| / 127 of the
    unrounded row y, and codes round(y / scale), ties to even.  x [N, H <= 16384] float32,
    float16 or bfloat16, weight [H] of that dtype or float32.  ``out`` may be x or residual (not if
    ``quantize``), and ``residual_out`` too: x, residual or a tensor of its own."""
    lib = _lib or load_library()
    N, H, dev = _hidden_rows(x, "x")
    _norm_weight(weight, x)
    dt, device, empty = x.dtype, x.device, torch.empty
    # an allocation each: on the host that is cheaper than views of one
    if out is not None:
        y = _matrix(out, dev, (N, H), torch.int8 if quantize else dt, "out")
    elif quantize:
        y = empty((N, H), dtype=torch.int8, device=device)
    else:
        y = empty((N, H), dtype=dt, device=device)
    total = r = to = scale = None
    rs = ts = 0
    if residual is not None:
        _matrix(residual, dev, (N, H), dt, "residual")
        total = empty((N, H), dtype=dt, device=device) if residual_out is None else \
            _matrix(residual_out, dev, (N, H), dt, "residual_out")
        r, rs, to, ts = residual.data_ptr(), residual.stride(0), total.data_ptr(), total.stride(0)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if quantize:
        scale = empty(N, dtype=torch.float32, device=device)
    rstd = empty(N, dtype=torch.float32, device=device)
    _call(dev, lib.tsa_rms_norm, x.data_ptr(), _DT[dt], N, H, x.stride(0), weight.data_ptr(), _DT[weight.dtype], r, rs,
          eps, 1 if quantize else 0, y.data_ptr(), y.stride(0), None if scale is None else scale.data_ptr(), to, ts,
          rstd.data_ptr(), _raw_stream(dev))
    if out is not None:
        _written(out)
    if residual_out is not None:
        _written(residual_out)
    return RMSNorm(y, scale, total, rstd)


def rms_norm_backward(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, rstd: torch.Tensor,
                      grad_residual: Optional[torch.Tensor] = None, grad_x: Optional[torch.Tensor] = None,
                      grad_weight: Optional[torch.Tensor] = None):
    """The gradients (grad_x, grad_weight) of ``rms_norm`` for the gradient ``grad`` of its
    (unquantised) result.  ``x``: the rows that were normalised (its ``residual`` where one was added), ``rstd`` as it
    gave it.  ``grad_residual``, the gradient that arrives along the residual stream, is added to grad_x, which
    is then that of x and of the residual alike.  ``grad_x`` may be ``grad``, ``grad_residual`` or a tensor of its
    own; ``grad_weight`` has the weight's dtype.  Sums in float32, over rows in a fixed order."""
    lib = _lib or load_library()
    N, H, dev = _hidden_rows(x, "x")
    _norm_weight(weight, x)
    _matrix(grad, dev, (N, H), x.dtype, "grad")
    if grad_residual is not None:
        _matrix(grad_residual, dev, (N, H), x.dtype, "grad_residual")
    r = _vec(rstd, N, torch.float32, dev, "rstd")
    dx = torch.empty((N, H), dtype=x.dtype, device=x.device) if grad_x is None else \
        _matrix(grad_x, dev, (N, H), x.dtype, "grad_x")
    dw = torch.empty(H, dtype=weight.dtype, device=x.device) if grad_weight is None else grad_weight
    to = _vec(dw, H, weight.dtype, dev, "grad_weight")
    nws = lib.tsa_rms_norm_backward_workspace_bytes(N, H)
    ws = torch.empty(nws, dtype=torch.uint8, device=x.device) if nws else None
    _call(dev, lib.tsa_rms_norm_backward, grad.data_ptr(), grad.stride(0), x.data_ptr(), _DT[x.dtype], N, H,
          x.stride(0), weight.data_ptr(), _DT[weight.dtype], r,
          None if grad_residual is None else grad_residual.data_ptr(),
          0 if grad_residual is None else grad_residual.stride(0), dx.data_ptr(), dx.stride(0), to,
          None if ws is None else ws.data_ptr(), nws, _raw_stream(dev))
    for t in (grad_x, grad_weight):
        if t is not None:
            _written(t)
    return dx, dw


def quantize_rows(x: torch.Tensor, out: Optional[torch.Tensor] = None):
    """Rows in 8 bits: (codes int8 [N, H], scale float32 [N]) with scale = max|x| / 127 of each row and codes
    round(x / scale), ties to even.  A row of zeros has scale 0; a row that is not finite codes 0 and a scale of
    NaN.  Lays out the weight of ``lm_head_int8``, whose rows are vocabulary entries."""
    lib = _lib or load_library()
    N, H, dev = _hidden_rows(x, "x")
    q = torch.empty((N, H), dtype=torch.int8, device=x.device) if out is None else \
        _matrix(out, dev, (N, H), torch.int8, "out")
    scale = torch.empty(N, dtype=torch.float32, device=x.device)
    _call(dev, lib.tsa_quantize_rows, x.data_ptr(), _DT[x.dtype], N, H, x.stride(0), q.data_ptr(), q.stride(0),
          scale.data_ptr(), _raw_stream(dev))
    if out is not None:
        _written(out)
    return q, scale


def lm_head_int8(hidden: torch.Tensor, hidden_scale: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
                 bias: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The scores [M, V] of a head in 8-bit integers, for ``sample``, ``topk`` and the losses: hidden_scale[m]
    weight_scale[v] times the exact integer product of int8 hidden [M, H] and int8 weight [V, H], plus ``bias`` (float32
    [V]), rounded once to ``dtype``.  ``rms_norm(quantize=True)`` makes the hidden rows, ``quantize_rows`` the weight."""
    lib = _lib or load_library()
    for t, name in ((hidden, "hidden"), (weight, "weight")):
        if t.dtype is not torch.int8 or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("%s must be a CUDA int8 2-D tensor with unit stride along H" % name)
    M, H = hidden.shape
    V = weight.size(0)
    dev = hidden.get_device()
    if weight.size(1) != H or weight.get_device() != dev:
        raise ValueError("weight must be [V, H] on the hidden rows' device")
    hs = _vec(hidden_scale, M, torch.float32, dev, "hidden_scale")
    ws = _vec(weight_scale, V, torch.float32, dev, "weight_scale")
    b = _vec(bias, V, torch.float32, dev, "bias")
    if dtype not in _DT:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    z = torch.empty((M, V), dtype=dtype, device=hidden.device) if out is None else \
        _matrix(out, dev, (M, V), dtype, "out", "V")
    nws = lib.tsa_lm_head_int8_workspace_bytes(M, H)
    work = torch.empty(nws, dtype=torch.uint8, device=hidden.device) if nws else None
    _call(dev, lib.tsa_lm_head_int8, hidden.data_ptr(), M, H, hidden.stride(0), hs, weight.data_ptr(), V,
          weight.stride(0), ws, b, z.data_ptr(), _DT[dtype], z.stride(0), None if work is None else work.data_ptr(),
          nws, _raw_stream(dev))
    if out is not None:
        _written(out)
    return z


class CrossEntropy(NamedTuple):
    """What ``lm_head_cross_entropy`` returns."""
    loss: torch.Tensor  # float32 scalar: the weighted sum over rows
    row_loss: torch.Tensor  # float32 [M]
    lse: torch.Tensor  # float32 [M]: the log-sum-exp of each row's scores
    grad_hidden: Optional[torch.Tensor]  # bfloat16 [M, H]
    grad_weight: Optional[torch.Tensor]  # bfloat16 [V, H]
    grad_bias: Optional[torch.Tensor]  # float32 [V]


def lm_head_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                          bias: Optional[torch.Tensor] = None, softcap: float = 0.0,
                          row_weight: Optional[torch.Tensor] = None, z_loss: float = 0.0,
                          grad_hidden: Union[bool, torch.Tensor] = True,
                          grad_weight: Union[bool, torch.Tensor] = True,
                          grad_bias: Union[bool, torch.Tensor] = True) -> CrossEntropy:
    """The cross entropy of the scores hidden @ weight^T (+ bias, capped to softcap tanh(z /
    softcap) where softcap > 0) against ``targets``, and its gradients, without the scores: they are
    formed a piece of the vocabulary at a time.

    A row's loss is lse - z[target] + z_loss lse^2 with lse = ln sum exp(z); the loss is the sum of
    ``row_weight`` times it (None: the mean over the rows that count).  A target outside [0, V) or a weight of
    0 skips a row: its hidden row is not used and its outputs are 0.  hidden bf16 [M, H], weight
    bf16 [V, H], targets int64 [M], bias and row_weight float32.  Each gradient: True for a new tensor, a
    tensor to write (an ``adamw_plan``'s, say), or False for none; with all False the loss alone."""
    lib = _lib or load_library()
    for t, name in ((hidden, "hidden"), (weight, "weight")):
        if t.dtype is not torch.bfloat16 or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
            raise ValueError("%s must be a CUDA bfloat16 2-D tensor with unit stride along H" % name)
    M, H = hidden.shape
    V = weight.size(0)
    dev = hidden.get_device()
    if weight.size(1) != H or weight.get_device() != dev:
        raise ValueError("weight must be [V, H] on the hidden rows' device")
    t = _vec(targets, M, torch.int64, dev, "targets")
    b = _vec(bias, V, torch.float32, dev, "bias")
    w = _vec(row_weight, M, torch.float32, dev, "row_weight")
    empty, device, bf16, f32 = torch.empty, hidden.device, torch.bfloat16, torch.float32
    given = [g for g in (grad_hidden, grad_weight, grad_bias) if isinstance(g, torch.Tensor)]
    dh = _matrix(grad_hidden, dev, (M, H), bf16, "grad_hidden") if isinstance(grad_hidden, torch.Tensor) else \
        empty((M, H), dtype=bf16, device=device) if grad_hidden else None
    dw = _matrix(grad_weight, dev, (V, H), bf16, "grad_weight") if isinstance(grad_weight, torch.Tensor) else \
        empty((V, H), dtype=bf16, device=device) if grad_weight else None
    db = None
    if isinstance(grad_bias, torch.Tensor):
        if bias is None:
            raise ValueError("grad_bias needs a bias")
        db = grad_bias
    elif grad_bias and bias is not None:
        db = empty(V, dtype=f32, device=device)
    to_b = _vec(db, V, f32, dev, "grad_bias")
    loss, row, lse = empty((), dtype=f32, device=device), empty(M, dtype=f32, device=device), \
        empty(M, dtype=f32, device=device)
    grads = dh is not None or dw is not None or db is not None
    nws = lib.tsa_lm_head_cross_entropy_workspace_bytes(M, H, V, 1 if grads else 0, 0 if db is None else 1)
    ws = empty(nws, dtype=torch.uint8, device=device) if nws else None
    _call(dev, lib.tsa_lm_head_cross_entropy, hidden.data_ptr(), M, H, hidden.stride(0), weight.data_ptr(), V,
          weight.stride(0), b, softcap, t, w, z_loss, loss.data_ptr(), row.data_ptr(), lse.data_ptr(),
          None if dh is None else dh.data_ptr(), 0 if dh is None else dh.stride(0),
          None if dw is None else dw.data_ptr(), 0 if dw is None else dw.stride(0), to_b,
          None if ws is None else ws.data_ptr(), nws, _raw_stream(dev))
    if given:
        _written(given)
    return CrossEntropy(loss, row, lse, dh, dw, db)


def device_status(clear: bool = True) -> int:
    """0, or TSA_ERR_DEVICE_TIMEOUT (-8) if a kernel's bounded wait ran out."""
    return int(load_library().tsa_device_status(1 if clear else 0))
