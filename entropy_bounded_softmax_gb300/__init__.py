"""Entropy-bounded softmax (``constrained_softmax``) for GB300 (sm_103a).

For each row of a [batch, num_classes] fp32 logit matrix: softmax and its
entropy; if the entropy exceeds ``entropy_bound`` the temperature is bisected
on [t_min, min(1, t_max)] for ``max_iter`` steps and softmax(l / T) is
written ("BURT-IMMA CUDA Kernel API Reference", section 2.1);
:func:`attention_softmax` is section 2.6's masked, optionally causal row
softmax of attention scores.  The backward
(section 6.3, with the 1/T of softmax(l / T) restored) gives the gradient
with respect to the logits; :class:`ConstrainedSoftmaxFunction` joins the two
for autograd.

Attention of language models: :func:`fused_attention` (softmax(scale q k^T) v
without the scores in memory), :func:`fused_attention_backward`, joined for
autograd by :class:`FusedAttentionFunction`, and :func:`paged_attention` (one
new token per sequence over a key-value cache in pages).

PyTorch supplies device memory and the current stream; the computation runs
in the hand-written CUDA kernels of ``libcsoftmax.so`` behind a C ABI
(``include/entropy_bounded_softmax.h``).  There is no CPU path: the calls
raise if the library is missing or the tensors are not on a CUDA device.
"""
from __future__ import annotations

import contextlib

from . import _lib
from ._lib import (CONSTANTS, cs_attention_softmax, cs_attention_softmax_ex,
                   cs_attention_shape, cs_biencoder_attention,
                   cs_biencoder_attention_ex,
                   cs_check_fused_attention_args,
                   cs_check_fused_attention_backward_args,
                   cs_fused_attention, cs_fused_attention_backward,
                   cs_fused_attention_backward_workspace,
                   cs_check_paged_attention_args, cs_paged_attention,
                   cs_paged_attention_workspace,
                   cs_paged_shape,
                   cs_check_biencoder_args, cs_plan_biencoder_host,
                   cs_check_args, cs_check_attention_args,
                   cs_check_backward_args, cs_constrained_softmax,
                   cs_constrained_softmax_backward,
                   cs_constrained_softmax_backward_ex,
                   cs_constrained_softmax_ex, cs_get_error,
                   cs_constrained_softmax_bf16, cs_constrained_softmax_bf16_ex,
                   cs_check_args_bf16,
                   cs_plan_attention_host, cs_plan_attention_launch,
                   cs_plan_backward_host, cs_plan_backward_launch,
                   cs_plan_host, cs_plan_launch, cs_probe_ex2,
                   cs_probe_ex2_sink_floats, cs_status_string,
                   cs_test_wait_timeout, cs_version, options)

__all__ = [
    "constrained_softmax", "constrained_softmax_backward",
    "ConstrainedSoftmaxFunction", "get_error", "plan", "plan_backward",
    "version", "CsError", "ERROR_BITS", "VARIANTS", "options",
    "cs_constrained_softmax", "cs_constrained_softmax_ex",
    "cs_constrained_softmax_bf16", "cs_constrained_softmax_bf16_ex",
    "cs_check_args_bf16",
    "cs_constrained_softmax_backward", "cs_constrained_softmax_backward_ex",
    "cs_get_error", "cs_plan_launch", "cs_plan_host",
    "cs_plan_backward_launch", "cs_plan_backward_host", "cs_check_args",
    "cs_check_backward_args", "cs_probe_ex2", "cs_probe_ex2_sink_floats",
    "cs_test_wait_timeout", "cs_version", "cs_status_string",
    "attention_softmax", "plan_attention", "cs_attention_softmax",
    "cs_attention_softmax_ex", "cs_plan_attention_launch",
    "cs_plan_attention_host", "cs_check_attention_args",
    "biencoder_attention", "cs_biencoder_attention",
    "cs_biencoder_attention_ex", "cs_plan_biencoder_host",
    "cs_check_biencoder_args",
    "fused_attention", "fused_attention_backward", "FusedAttentionFunction",
    "cs_attention_shape", "cs_fused_attention", "cs_fused_attention_backward",
    "cs_fused_attention_backward_workspace", "cs_check_fused_attention_args",
    "cs_check_fused_attention_backward_args",
    "paged_attention", "cs_paged_shape", "cs_paged_attention",
    "cs_paged_attention_workspace",
    "cs_check_paged_attention_args",
]

# Defaults of section 2.1's signature.
DEFAULT_ENTROPY_BOUND = 0.20
DEFAULT_T_MIN = 0.01
DEFAULT_T_MAX = 10.0
DEFAULT_MAX_ITER = 20

VARIANTS = {"auto": CONSTANTS["CS_VARIANT_AUTO"],
            "rowgroup": CONSTANTS["CS_VARIANT_ROWGROUP"],
            "cluster": CONSTANTS["CS_VARIANT_CLUSTER"]}
ERROR_BITS = {name: 1 << CONSTANTS[f"CS_ERR_{name}"]
              for name in ("NAN_INPUT", "INF_INPUT", "ENTROPY_OVERFLOW",
                           "TIMEOUT", "BAD_PAGE")}


_STAY = contextlib.nullcontext()


class CsError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: status {status} "
                         f"({_lib.cs_status_string(status)})")


def _stream_handle(device) -> int:
    """The raw cudaStream_t of the current stream of a CUDA device."""
    import torch
    idx = device.index if device.index is not None else torch.cuda.current_device()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(idx)
    return torch.cuda.current_stream(device).cuda_stream


def _on_device(device):
    """A context that makes `device` current: none when it already is (the
    common case, and the cheapest: the call is on every step's path)."""
    import torch
    if device.index is None or device.index == torch.cuda.current_device():
        return _STAY
    return torch.cuda.device(device)


def constrained_softmax(logits, entropy_bound: float = DEFAULT_ENTROPY_BOUND,
                        t_min: float = DEFAULT_T_MIN,
                        t_max: float = DEFAULT_T_MAX,
                        max_iter: int = DEFAULT_MAX_ITER,
                        return_t: bool = False, out=None, t_out=None,
                        variant: str = "auto", param: int = 0,
                        threads: int = 0, strict: bool = False,
                        evals_out=None):
    """Entropy-bounded softmax of a CUDA [batch, num_classes] tensor of fp32
    logits, or of bf16 logits (``cs_constrained_softmax_bf16``: promoted
    exactly to fp32 on load; the probabilities are fp32 either way).

    Returns the probabilities (and the per-row temperature if ``return_t``).
    ``out``/``t_out`` may be given to write into existing tensors.  The call
    is asynchronous on the current stream; per-row conditions (NaN/Inf rows,
    unsatisfiable bounds) are read with :func:`get_error`.
    ``variant``/``param``/``threads``/``strict`` are the launch options
    of ``cs_constrained_softmax_ex`` (defaults: automatic); ``evals_out``, an
    int32 [batch] tensor on the same device, receives how many temperatures
    each row's exponentials were evaluated at.
    """
    import torch
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.device.type != "cuda":
        raise ValueError("logits must be on a CUDA device")
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("logits must be float32 or bfloat16")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [batch, num_classes]")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    batch, num_classes = logits.shape
    if out is None:
        out = torch.empty(logits.shape, dtype=torch.float32,
                          device=logits.device)
    elif (out.shape != logits.shape or out.dtype != torch.float32
          or out.device != logits.device or not out.is_contiguous()):
        raise ValueError("out must be a contiguous float32 tensor shaped like "
                         "logits on the same device")
    t_ptr = None
    if return_t or t_out is not None:
        if t_out is None:
            t_out = torch.empty(batch, dtype=torch.float32,
                                device=logits.device)
        elif (t_out.shape != (batch,) or t_out.dtype != torch.float32
              or t_out.device != logits.device or not t_out.is_contiguous()):
            raise ValueError("t_out must be a contiguous float32 [batch] "
                             "tensor on the logits' device")
        t_ptr = t_out.data_ptr()
    e_ptr = None
    if evals_out is not None:
        if (not isinstance(evals_out, torch.Tensor)
                or evals_out.shape != (batch,)
                or evals_out.dtype != torch.int32
                or evals_out.device != logits.device
                or not evals_out.is_contiguous()):
            raise ValueError("evals_out must be a contiguous int32 [batch] "
                             "tensor on the logits' device")
        e_ptr = evals_out.data_ptr()
    entry = (cs_constrained_softmax_bf16_ex
             if logits.dtype == torch.bfloat16 else cs_constrained_softmax_ex)
    with _on_device(logits.device):
        st = entry(
            logits.data_ptr(), out.data_ptr(), batch, num_classes,
            float(entropy_bound), float(t_min), float(t_max), int(max_iter),
            t_ptr, options(VARIANTS[variant], param, threads, int(strict),
                           e_ptr),
            _stream_handle(logits.device))
    if st != 0:
        raise CsError(st, "cs_constrained_softmax")
    return (out, t_out) if return_t else out


def _check_like(name, x, ref) -> None:
    import torch
    if (not isinstance(x, torch.Tensor) or x.shape != ref.shape
            or x.dtype != torch.float32 or x.device != ref.device
            or not x.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 tensor shaped "
                         "like probs on the same device")


def constrained_softmax_backward(probs, grad_output, t, out=None,
                                 variant: str = "auto", param: int = 0,
                                 threads: int = 0):
    """Gradient with respect to the logits: (1/T) p (g - <g, p>) per row.

    ``probs`` and ``t`` are the forward's output and temperatures
    (``constrained_softmax(..., return_t=True)``), ``grad_output`` the
    upstream gradient; all on one CUDA device, fp32, contiguous.  Rows whose
    T is NaN (rows the forward zeroed) get zeros.  ``out`` may be given, and
    may be ``probs`` or ``grad_output`` itself (in place).  Asynchronous on
    the current stream.
    """
    import torch
    if not isinstance(probs, torch.Tensor) or probs.device.type != "cuda":
        raise ValueError("probs must be a CUDA tensor")
    if probs.dim() != 2:
        raise ValueError("probs must be 2-D [batch, num_classes]")
    _check_like("probs", probs, probs)
    _check_like("grad_output", grad_output, probs)
    batch, num_classes = probs.shape
    if (not isinstance(t, torch.Tensor) or t.shape != (batch,)
            or t.dtype != torch.float32 or t.device != probs.device
            or not t.is_contiguous()):
        raise ValueError("t must be a contiguous float32 [batch] tensor on "
                         "probs' device")
    if out is None:
        out = torch.empty_like(probs)
    else:
        _check_like("out", out, probs)
    with _on_device(probs.device):
        st = cs_constrained_softmax_backward_ex(
            probs.data_ptr(), grad_output.data_ptr(), t.data_ptr(),
            out.data_ptr(), batch, num_classes,
            options(VARIANTS[variant], param, threads, 0),
            _stream_handle(probs.device))
    if st != 0:
        raise CsError(st, "cs_constrained_softmax_backward")
    return out


def attention_softmax(scores, mask=None, causal: bool = False, out=None,
                      variant: str = "auto", param: int = 0,
                      threads: int = 0):
    """Section 2.6 attention_softmax of CUDA fp32 scores [B, H, S, S].

    ``mask`` is None or an additive fp32 mask of shape [B, S] or
    [B, 1, 1, S] (0 attends; -inf, or the page's -1e9, masks); ``causal``
    removes keys j > i from row i.  ``out`` may be given, ``scores`` itself
    included (in place).  Asynchronous on the current stream; rows with
    NaN/Inf inputs are zeroed and reported by :func:`get_error`.
    """
    import torch
    if not isinstance(scores, torch.Tensor) or scores.device.type != "cuda":
        raise ValueError("scores must be a CUDA tensor")
    if (scores.dtype != torch.float32 or scores.dim() != 4
            or scores.shape[2] != scores.shape[3] or not scores.is_contiguous()):
        raise ValueError("scores must be a contiguous float32 [B, H, S, S] "
                         "tensor")
    B, H, S, _ = scores.shape
    m_ptr = None
    if mask is not None:
        if (not isinstance(mask, torch.Tensor) or mask.dtype != torch.float32
                or mask.device != scores.device or not mask.is_contiguous()
                or mask.numel() != B * S
                or tuple(mask.shape) not in ((B, S), (B, 1, 1, S))):
            raise ValueError("mask must be a contiguous float32 [B, S] or "
                             "[B, 1, 1, S] tensor on the scores' device")
        m_ptr = mask.data_ptr()
    if out is None:
        out = torch.empty_like(scores)
    elif (out.shape != scores.shape or out.dtype != torch.float32
          or out.device != scores.device or not out.is_contiguous()):
        raise ValueError("out must be a contiguous float32 tensor shaped like "
                         "scores on the same device")
    with _on_device(scores.device):
        st = cs_attention_softmax_ex(
            scores.data_ptr(), out.data_ptr(), m_ptr, B, H, S,
            int(bool(causal)), options(VARIANTS[variant], param, threads, 0),
            _stream_handle(scores.device))
    if st != 0:
        raise CsError(st, "cs_attention_softmax")
    return out


def biencoder_attention(query, keys, values, scale=None,
                        entropy_bound: float = DEFAULT_ENTROPY_BOUND,
                        t_min: float = DEFAULT_T_MIN,
                        t_max: float = DEFAULT_T_MAX,
                        max_iter: int = DEFAULT_MAX_ITER, out=None,
                        return_attn: bool = False, return_t: bool = False,
                        lanes: int = 0, fused: bool = False):
    """Section 2.5 biencoder_attention: scores = query @ keys^T * scale
    (default 1/sqrt(d_head)), the constrained softmax of every score row,
    then attn @ values (on the tensor cores for d_head <= 64 and
    context_len <= d_head unless ``fused``, which runs all three steps in
    one kernel on the FMA pipes).  query [B, H, Q, D], keys and values
    [B, H, K, D], CUDA fp32 contiguous.  Returns the output [B, H, Q, D]
    (and the weights [B, H, Q, K] and temperatures [B, H, Q] when asked).
    Asynchronous on the current stream."""
    import math
    import torch
    for name, x in (("query", query), ("keys", keys), ("values", values)):
        if (not isinstance(x, torch.Tensor) or x.device.type != "cuda"
                or x.dtype != torch.float32 or x.dim() != 4
                or not x.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA float32 "
                             "4-D tensor")
    B, H, Q, D = query.shape
    K = keys.shape[2]
    if keys.shape != (B, H, K, D) or values.shape != (B, H, K, D):
        raise ValueError("keys and values must be [B, H, K, D]")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = torch.empty_like(query)
    attn = t = None
    if return_attn:
        attn = torch.empty((B, H, Q, K), dtype=torch.float32,
                           device=query.device)
    if return_t:
        t = torch.empty((B, H, Q), dtype=torch.float32, device=query.device)
    variant = (CONSTANTS["CS_VARIANT_FUSED"] if fused
               else VARIANTS["rowgroup"] if lanes else 0)
    opt = options(variant, lanes, 0, 0)
    with _on_device(query.device):
        st = cs_biencoder_attention_ex(
            query.data_ptr(), keys.data_ptr(), values.data_ptr(),
            out.data_ptr(), B, Q, K, D, H, float(scale), float(entropy_bound),
            float(t_min), float(t_max), int(max_iter),
            attn.data_ptr() if attn is not None else None,
            t.data_ptr() if t is not None else None, opt,
            _stream_handle(query.device))
    if st != 0:
        raise CsError(st, "cs_biencoder_attention")
    res = (out,) + ((attn,) if return_attn else ()) + ((t,) if return_t else ())
    return res if len(res) > 1 else out


def _check_heads(name, x, shape, device) -> None:
    """Raises what is wrong with a [batch, heads, length, d_head] bf16
    tensor of fused attention."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if x.dim() != 4:
        raise ValueError(f"{name} must be 4-D [batch, heads, length, d_head]")
    if x.get_device() != device:
        raise ValueError(f"{name} must be on the query's device")
    if tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}")
    if not x.numel():
        return
    st = x.stride()
    if st[3] != 1:
        raise ValueError(f"{name}'s head dimension must be contiguous")
    if x.data_ptr() & 15 or any(n > 1 and (s <= 0 or s % 8)
                                for n, s in zip(shape[:3], st)):
        raise ValueError(f"{name}'s base must be 16-byte aligned and its "
                         "batch, head and position strides positive "
                         "multiples of 8 elements")


def _check_attention(query, keys, values, mask, scale, lse, same) -> None:
    """Raises what is wrong with the arguments of fused attention, if
    anything is; `same`: the tensors that have to be shaped like query, by
    name.  The calls look at the properties that they need themselves, and
    leave strides, addresses and ranges to the library; only what either
    refuses comes here for its message."""
    import torch
    for name, x in (("query", query), ("keys", keys)):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if x.dim() != 4:
            raise ValueError(f"{name} must be 4-D [batch, heads, length, "
                             "d_head]")
    dev = query.get_device()
    B, H, Sq, D = query.shape
    Hk, Sk = keys.shape[1], keys.shape[2]
    if keys.shape[0] != B or keys.shape[3] != D:
        raise ValueError("keys must be [batch, kv_heads, key_len, d_head] "
                         "with the query's batch and d_head")
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError("the query's heads must be a multiple of the keys'")
    if D < 8 or D > 128 or D % 8:
        raise ValueError("d_head must be a multiple of 8 in 8..128")
    _check_heads("query", query, query.shape, dev)
    _check_heads("keys", keys, keys.shape, dev)
    _check_heads("values", values, keys.shape, dev)
    for name, x in same.items():
        _check_heads(name, x, query.shape, dev)
    if scale is not None and not 0.0 < scale <= 2.0 ** 127:
        raise ValueError("scale must be positive and at most 2^127")
    if mask is not None:
        if (not isinstance(mask, torch.Tensor) or mask.dtype != torch.bool
                or mask.device != query.device
                or tuple(mask.shape) != (B, Sk)):
            raise ValueError("mask must be a bool [batch, key_len] tensor on "
                             "the query's device")
        if ((Sk > 1 and mask.stride(1) != 1)
                or (B > 1 and mask.stride(0) < Sk)):
            raise ValueError("mask's rows must be contiguous and not overlap")
    if lse is not None and (
            not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32
            or lse.shape != query.shape[:3] or lse.get_device() != dev
            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [batch, heads, "
                         "query_len] tensor on the query's device")


def _attention_ok(torch, query, keys, values, mask, lse, same):
    """Whether the properties that the library cannot see are right: types,
    devices, shapes and contiguous last dimensions."""
    t = torch.Tensor
    if not (isinstance(query, t) and isinstance(keys, t)
            and isinstance(values, t)):
        return False
    bf16, dev = torch.bfloat16, query.get_device()
    shape, ks = query.shape, keys.shape
    if (query.dtype is not bf16 or keys.dtype is not bf16
            or values.dtype is not bf16 or dev < 0
            or keys.get_device() != dev or values.get_device() != dev
            or len(shape) != 4 or len(ks) != 4 or values.shape != ks
            or ks[0] != shape[0] or ks[3] != shape[3] or shape[3] < 2
            or query.stride(3) != 1 or keys.stride(3) != 1
            or values.stride(3) != 1):
        return False
    for x in same:
        if (not isinstance(x, t) or x.dtype is not bf16
                or x.get_device() != dev or x.shape != shape
                or x.stride(3) != 1):
            return False
    if mask is not None and (
            not isinstance(mask, t) or mask.dtype is not torch.bool
            or mask.get_device() != dev or mask.shape != (ks[0], ks[2])
            or mask.stride(1) != 1):
        return False
    return lse is None or (
        isinstance(lse, t) and lse.dtype is torch.float32
        and lse.get_device() == dev and lse.shape == shape[:3]
        and lse.is_contiguous())


def fused_attention(query, keys, values, mask=None, causal: bool = False,
                    scale=None, out=None, return_lse: bool = False):
    """softmax(scale query keys^T) values over CUDA bf16 tensors, without the
    scores in memory: query [B, H, Sq, D], keys and values [B, Hk, Sk, D],
    H a multiple of Hk (head h reads key head h // (H // Hk)), D a multiple
    of 8 up to 128.

    ``mask`` is None or a bool [B, Sk] tensor, False for keys that no query
    attends (padding; what they hold has no effect); ``causal`` keeps keys
    j <= i + Sk - Sq for query i; ``scale`` defaults to 1/sqrt(D).  A query
    without keys gets zeros.  Any strides that are multiples of 8 elements
    over a contiguous head dimension are taken, [B, S, H, D] storage seen as
    [B, H, S, D] among them.  Returns the output [B, H, Sq, D] in bf16, in
    the query's memory order (or ``out``), and with ``return_lse`` the log of
    the softmax's sums [B, H, Sq] in fp32 (-inf without keys), which
    :func:`fused_attention_backward` takes.  Asynchronous on the current
    stream; NaN or infinite scores propagate and are reported by
    :func:`get_error`.

    Where autograd records and query, keys or values require a gradient, the
    call goes through :class:`FusedAttentionFunction`: the output carries the
    gradient, the log of the sums does not, and ``out`` is refused.  (Tangents
    of forward mode are not seen here; the class refuses them.)
    """
    import torch
    same = () if out is None else (out,)
    if not _attention_ok(torch, query, keys, values, mask, None, same):
        _check_attention(query, keys, values, mask, scale, None,
                         {} if out is None else {"out": out})
    if ((query.requires_grad or keys.requires_grad or values.requires_grad)
            and torch.is_grad_enabled()):
        if out is not None:
            raise ValueError("out takes no gradient: call under "
                             "torch.no_grad(), or without it")
        # What autograd's function would copy is refused here as ever.
        _check_attention(query, keys, values, mask, scale, None, {})
        return _autograd_class("FusedAttentionFunction").apply(
            query, keys, values, mask, causal, scale, return_lse)
    B, H, Sq, D = query.shape
    _, Hk, Sk, _ = keys.shape
    if out is None:
        out = torch.empty_like(query)
    lse = None
    if return_lse:
        lse = torch.empty((B, H, Sq), dtype=torch.float32,
                          device=query.device)
    shape = _lib.pack_attention_shape(
        B, H, Hk, Sq, Sk, D, 1 if causal else 0,
        D ** -0.5 if scale is None else scale, query.stride(), keys.stride(),
        values.stride(), out.stride(), Sk if mask is None else mask.stride(0))
    with _on_device(query.device):
        st = cs_fused_attention(
            query.data_ptr(), keys.data_ptr(), values.data_ptr(),
            out.data_ptr(), lse.data_ptr() if return_lse else None,
            None if mask is None else mask.data_ptr(), shape,
            _stream_handle(query.device))
    if st != 0:
        _check_attention(query, keys, values, mask, scale, lse, {"out": out})
        raise CsError(st, "cs_fused_attention")
    return (out, lse) if return_lse else out


def fused_attention_backward(query, keys, values, out, lse, grad_output,
                             mask=None, causal: bool = False, scale=None):
    """Gradients of :func:`fused_attention` with respect to query, keys and
    values, given ``grad_output``, that of its output, and its ``out`` and
    ``lse`` (``return_lse=True``).  The probabilities are recomputed; every
    sum has a fixed order, so repeated calls give the same bits.  Returns
    bf16 gradients in the memory order of their tensors; removed keys get
    zeros.  The gradients are not themselves differentiable.  Asynchronous on
    the current stream.
    """
    import torch
    same = {"out": out, "grad_output": grad_output}
    if lse is None or not _attention_ok(torch, query, keys, values, mask, lse,
                                        (out, grad_output)):
        _check_attention(query, keys, values, mask, scale,
                         False if lse is None else lse, same)
    B, H, Sq, D = query.shape
    _, Hk, Sk, _ = keys.shape
    dq, dk, dv = (torch.empty_like(query), torch.empty_like(keys),
                  torch.empty_like(values))
    shape = _lib.pack_attention_backward_shape(
        B, H, Hk, Sq, Sk, D, 1 if causal else 0,
        D ** -0.5 if scale is None else scale, query.stride(), keys.stride(),
        values.stride(), out.stride(), grad_output.stride(), dq.stride(),
        dk.stride(), dv.stride(), Sk if mask is None else mask.stride(0))
    size = max(cs_fused_attention_backward_workspace(shape), 0)
    work = torch.empty(size, dtype=torch.uint8, device=query.device)
    with _on_device(query.device):
        st = cs_fused_attention_backward(
            query.data_ptr(), keys.data_ptr(), values.data_ptr(),
            out.data_ptr(), lse.data_ptr(), grad_output.data_ptr(),
            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
            None if mask is None else mask.data_ptr(), shape, work.data_ptr(),
            size, _stream_handle(query.device))
    if st != 0:
        _check_attention(query, keys, values, mask, scale, lse, same)
        raise CsError(st, "cs_fused_attention_backward")
    return dq, dk, dv


def _check_paged(query, key_pages, value_pages, page_table, lengths, scale,
                 out) -> None:
    """Raises what is wrong with the arguments of paged attention, if
    anything is (as _check_attention)."""
    import torch
    for name, x, dim in (("query", query, 3), ("key_pages", key_pages, 4)):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if x.dim() != dim:
            raise ValueError(f"{name} must have {dim} dimensions")
    dev = query.device
    if query.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("query must be a bfloat16 or float16 tensor")
    B, H, D = query.shape
    _, page_size, Hk, _ = key_pages.shape
    if key_pages.shape[3] != D:
        raise ValueError("key_pages must be [pages, page_size, kv_heads, "
                         "d_head] with the query's d_head")
    if H < 1 or Hk < 1 or H % Hk or page_size < 1:
        raise ValueError("the query's heads must be a multiple of the "
                         "pages', and page_size positive")
    if D < 8 or D > 256 or D % 8:
        raise ValueError("d_head must be a multiple of 8 in 8..256")
    for name, x, shape in (("query", query, query.shape),
                           ("key_pages", key_pages, key_pages.shape),
                           ("value_pages", value_pages, key_pages.shape),
                           ("out", out, query.shape)):
        if name == "out" and x is None:
            continue
        if not isinstance(x, torch.Tensor) or x.device != dev:
            raise ValueError(f"{name} must be a CUDA tensor on the query's "
                             "device")
        if x.dtype != query.dtype:
            raise TypeError(f"{name} must be {query.dtype}")
        if x.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}")
        if x.numel() and (
                x.stride(-1) != 1 or x.data_ptr() & 15
                or any(n > 1 and s % 8
                       for n, s in zip(shape[:-1], x.stride()))):
            raise ValueError(f"{name}'s last dimension must be contiguous, "
                             "its base 16-byte aligned and its other strides "
                             "multiples of 8 elements")
    for name, x, dim in (("page_table", page_table, 2),
                         ("lengths", lengths, 1)):
        if (not isinstance(x, torch.Tensor) or x.dtype != torch.int32
                or x.device != dev or x.dim() != dim or x.shape[0] != B
                or (x.shape[-1] > 1 and x.stride(-1) != 1)):
            raise ValueError(f"{name} must be an int32 tensor of the batch's "
                             "rows, contiguous along its last dimension, on "
                             "the query's device")
    if B > 1 and page_table.stride(0) < page_table.shape[1]:
        raise ValueError("page_table's rows must not overlap")
    if scale is not None and not 0.0 < scale <= 2.0 ** 127:
        raise ValueError("scale must be positive and at most 2^127")


def _paged_ok(torch, query, key_pages, value_pages, page_table, lengths, out):
    """Whether the properties that the library cannot see are right."""
    t = torch.Tensor
    if not (isinstance(query, t) and isinstance(key_pages, t)
            and isinstance(value_pages, t) and isinstance(page_table, t)
            and isinstance(lengths, t)):
        return False
    dtype, dev = query.dtype, query.get_device()
    qs, ps = query.shape, key_pages.shape
    i32 = torch.int32
    return ((dtype is torch.bfloat16 or dtype is torch.float16) and dev >= 0
            and key_pages.dtype is dtype and value_pages.dtype is dtype
            and page_table.dtype is i32 and lengths.dtype is i32
            and key_pages.get_device() == dev
            and value_pages.get_device() == dev
            and page_table.get_device() == dev and lengths.get_device() == dev
            and len(qs) == 3 and len(ps) == 4 and value_pages.shape == ps
            and ps[3] == qs[2] and qs[2] > 1
            and page_table.dim() == 2 and page_table.shape[0] == qs[0]
            and lengths.shape == qs[:1]
            and query.stride(2) == 1 and key_pages.stride(3) == 1
            and value_pages.stride(3) == 1 and page_table.stride(1) == 1
            and lengths.stride(0) == 1
            and (out is None or (
                isinstance(out, t) and out.dtype is dtype
                and out.get_device() == dev and out.shape == qs
                and out.stride(2) == 1)))


def paged_attention(query, key_pages, value_pages, page_table, lengths,
                    scale=None, out=None, return_lse: bool = False):
    """Attention of one new token per sequence over a paged key-value cache:
    softmax(scale query keys^T) values over the sequence's tokens.

    ``query`` [B, H, D]; ``key_pages`` and ``value_pages``
    [pages, page_size, Hk, D], H a multiple of Hk, D a multiple of 8 up to
    256, all bf16 or all fp16 on one CUDA device; ``page_table`` int32
    [B, n]: token j of sequence b is in slot j % page_size of page
    ``page_table[b, j // page_size]``; ``lengths`` int32 [B].  Table entries
    and slots past a length are not read.  ``scale`` defaults to 1/sqrt(D).
    Returns [B, H, D] (or ``out``), zeros for a length of 0, and with
    ``return_lse`` the log of the softmax's sums [B, H] in fp32.
    Asynchronous on the current stream; lengths and page numbers out of
    range are left out and reported by :func:`get_error`, and so are NaN or
    infinite scores, which propagate.  For serving: there is no backward pass,
    and the result carries no gradient.
    """
    import torch
    given = (query, key_pages, value_pages, page_table, lengths)
    if not _paged_ok(torch, *given, out):
        _check_paged(*given, scale, out)
    dtype = query.dtype
    B, H, D = query.shape
    pages, page_size, Hk, _ = key_pages.shape
    if out is None:
        out = torch.empty((B, H, D), dtype=dtype, device=query.device)
    lse = None
    if return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=query.device)
    shape = _lib.pack_paged_shape(
        B, H, Hk, D, page_size, pages, page_table.shape[1],
        1 if dtype is torch.float16 else 0,
        D ** -0.5 if scale is None else scale, query.stride(), out.stride(),
        key_pages.stride(), value_pages.stride(), page_table.stride(0))
    size = max(cs_paged_attention_workspace(shape), 0)
    work = None
    if size:
        work = torch.empty(size, dtype=torch.uint8, device=query.device)
    with _on_device(query.device):
        st = cs_paged_attention(
            query.data_ptr(), key_pages.data_ptr(), value_pages.data_ptr(),
            page_table.data_ptr(), lengths.data_ptr(), out.data_ptr(),
            lse.data_ptr() if return_lse else None, shape,
            work.data_ptr() if size else None, size,
            _stream_handle(query.device))
    if st != 0:
        _check_paged(*given, scale, out)
        raise CsError(st, "cs_paged_attention")
    return (out, lse) if return_lse else out


def plan_attention(batch: int, heads: int, seq_len: int, aligned: bool = True,
                   variant: str = "auto", param: int = 0,
                   threads: int = 0) -> dict:
    """The attention_softmax launch plan on the current device."""
    st, p = cs_plan_attention_launch(batch, heads, seq_len, int(aligned),
                                     options(VARIANTS[variant], param,
                                             threads, 0))
    if st != 0:
        raise CsError(st, "cs_plan_attention_launch")
    return p.as_dict()


def _autograd_function():
    import torch

    class ConstrainedSoftmaxFunction(torch.autograd.Function):
        """Autograd wrapper of section 6.3: forward = constrained_softmax,
        backward = constrained_softmax_backward at the forward's
        temperatures.  ``apply(logits, entropy_bound, t_min, t_max,
        max_iter)``; only the logits receive a gradient."""

        @staticmethod
        def forward(ctx, logits, entropy_bound=DEFAULT_ENTROPY_BOUND,
                    t_min=DEFAULT_T_MIN, t_max=DEFAULT_T_MAX,
                    max_iter=DEFAULT_MAX_ITER):
            out, t = constrained_softmax(logits.contiguous(), entropy_bound,
                                         t_min, t_max, max_iter,
                                         return_t=True)
            ctx.save_for_backward(out, t)
            return out

        @staticmethod
        def backward(ctx, grad_output):
            out, t = ctx.saved_tensors
            grad = constrained_softmax_backward(out, grad_output.contiguous(),
                                                t)
            return grad, None, None, None, None

    return ConstrainedSoftmaxFunction


def _fused_attention_function():
    import torch

    def strided(x):
        """x itself where the kernels take its strides, else a copy."""
        ok = (x.dim() == 4 and x.stride(3) == 1 and x.data_ptr() % 16 == 0
              and all(n <= 1 or (s > 0 and s % 8 == 0)
                      for n, s in zip(x.shape[:3], x.stride()[:3])))
        return x if ok else x.clone(memory_format=torch.contiguous_format)

    class FusedAttentionFunction(torch.autograd.Function):
        """Autograd wrapper of :func:`fused_attention`: ``apply(query, keys,
        values, mask, causal, scale, return_lse)``; query, keys and values
        receive gradients, once (there is no second derivative, forward mode
        or vmap rule: torch refuses them).  Inputs and masks whose strides
        the kernels do not take (expanded ones, for example) are copied.  The
        backward pass computes the three gradients together, and hands on
        those that are needed.  It can be captured into a CUDA graph after a
        warm-up on a side stream, as any of torch's; let no eager graph of
        the same leaves live then, whose accumulation is tied to the stream
        of its first use."""

        @staticmethod
        def forward(ctx, query, keys, values, mask=None, causal=False,
                    scale=None, return_lse=False):
            query, keys, values = (strided(x) for x in (query, keys, values))
            if (isinstance(mask, torch.Tensor) and mask.dim() == 2
                    and (mask.stride(1) != 1
                         or mask.stride(0) < mask.shape[1])):
                mask = mask.contiguous()
            out, lse = fused_attention(query, keys, values, mask, causal,
                                       scale, return_lse=True)
            ctx.save_for_backward(query, keys, values, out, lse, mask)
            ctx.causal, ctx.scale = causal, scale
            ctx.set_materialize_grads(False)
            if not return_lse:
                return out
            ctx.mark_non_differentiable(lse)
            return out, lse

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, grad_output, _=None):
            if grad_output is None:
                return (None,) * 7
            query, keys, values, out, lse, mask = ctx.saved_tensors
            grads = fused_attention_backward(
                query, keys, values, out, lse, strided(grad_output), mask,
                ctx.causal, ctx.scale)
            return (*(x if needed else None
                      for x, needed in zip(grads, ctx.needs_input_grad)),
                    None, None, None, None)

    return FusedAttentionFunction


def _autograd_class(name):
    """An autograd class of the package.  They need torch, and are built on
    first use so that the package imports without torch (the C ABI tests run
    without it)."""
    cls = globals().get(name)
    if cls is None:
        cls = {"ConstrainedSoftmaxFunction": _autograd_function,
               "FusedAttentionFunction": _fused_attention_function}[name]()
        globals()[name] = cls
    return cls


def __getattr__(name):
    if name in ("ConstrainedSoftmaxFunction", "FusedAttentionFunction"):
        return _autograd_class(name)
    raise AttributeError(name)


def get_error(device=None) -> set[str]:
    """Synchronise the current stream, read and clear the device error word;
    returns the names of the conditions seen since the last call."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None \
        else torch.device(device)
    with _on_device(dev):
        st, mask = cs_get_error(_stream_handle(dev))
    if st != 0:
        raise CsError(st, "cs_get_error")
    return {name for name, bit in ERROR_BITS.items() if mask & bit}


def plan(batch: int, num_classes: int, variant: str = "auto",
         param: int = 0, threads: int = 0, strict: bool = False) -> dict:
    """The launch plan for this shape on the current device."""
    st, p = cs_plan_launch(batch, num_classes,
                           options(VARIANTS[variant], param, threads,
                                   int(strict)))
    if st != 0:
        raise CsError(st, "cs_plan_launch")
    return p.as_dict()


def plan_backward(batch: int, num_classes: int, variant: str = "auto",
                  param: int = 0, threads: int = 0) -> dict:
    """The backward's launch plan for this shape on the current device."""
    st, p = cs_plan_backward_launch(batch, num_classes,
                                    options(VARIANTS[variant], param,
                                            threads, 0))
    if st != 0:
        raise CsError(st, "cs_plan_backward_launch")
    return p.as_dict()


def version() -> str:
    return cs_version()
