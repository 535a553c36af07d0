"""The sequence operators on tensors: token embedding, layer norm, cross attention.

What reads and trains the rows a table gathers.  Each function checks its
tensors, allocates what it returns and its workspace from torch's caching
allocator, and makes one call of the C ABI (``include/recis.h`` states the
formulas); the arithmetic is in the library's HIP kernels, and there is no
fallback.  Forward and backward are separate calls, as the table's are: no
graph is recorded, and a forward call whose inputs require a gradient warns.

Tensors are float32 or bfloat16 on the current GPU.  Rows (the last axis) are
contiguous, the other axes may be strided; a tensor whose last axis is strided
is copied first.  Work is queued on `stream` (default: torch's current
stream); with another stream than the one the inputs were made on, order the
two first, as for any torch call.

`error`, where a call has it: an int32 tensor of one element, zero at first,
in which the GPU records tokens, lengths and offsets out of range; ``check``
raises for what it holds.
"""
from __future__ import annotations

import contextlib
import warnings
from typing import Optional

import torch

from . import recis
from .recis import RECIS_DTYPE_BF16, RECIS_DTYPE_F32

_DTYPES = {torch.float32: RECIS_DTYPE_F32, torch.bfloat16: RECIS_DTYPE_BF16}


def _dtype(name: str, t) -> int:
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32 or bfloat16, not {t.dtype}")
    return d


def _on_gpu(*tensors):
    """Every tensor given is on the current GPU."""
    here = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"every tensor must be on the current GPU (cuda:{here}); {list(t.shape)} is on {t.device}")


def _forward_of(name: str, *tensors):
    """The same for a forward call; says so where a gradient would get lost."""
    _on_gpu(*tensors)
    for t in tensors:
        if t is not None and t.requires_grad and torch.is_grad_enabled():
            warnings.warn(f"sequence.{name} records no graph, so its inputs get no gradient through it: call "
                          f"{name}_backward, and pass detached tensors or work under torch.no_grad()", stacklevel=3)
            return


def _index(name: str, t, dtype, shape):
    """A contiguous integer tensor of one shape."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    return t.contiguous()


def _error_word(error):
    if error is not None and (error.dtype != torch.int32 or error.numel() != 1):
        raise ValueError("error must be an int32 tensor of one element")
    return error


def _rows(t):
    """t [..., dim] as rows one stride apart, and that stride."""
    dim = t.shape[-1]
    if t.is_contiguous():
        return t, dim
    if t.dim() == 2 and (t.stride(1) == 1 or dim == 1) and t.stride(0) >= dim:
        return t, t.stride(0)
    return t.contiguous(), dim


def _like(t):
    """A new contiguous tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty_like(t, memory_format=torch.contiguous_format)


def _written(name: str, t, shape, dtype):
    """An output given by the caller: rows one stride apart, written in place."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    rows, stride = _rows(t)
    if rows is not t:
        raise ValueError(f"{name} must have rows that are contiguous and one stride apart")
    return stride


@contextlib.contextmanager
def _on(stream, *tensors):
    """Allocations belong to `stream`, and the tensors it reads stay until it has."""
    with torch.cuda.stream(stream):
        yield
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def check(error, stream=None):
    """Raises RecisError for what the GPU recorded in an error word.  Waits for
    `stream`, which has to be the one of every call that was given the word; by
    default for all the GPU's streams."""
    if stream is None:
        torch.cuda.synchronize(error.device)
        stream = torch.cuda.current_stream(error.device)
    with torch.cuda.stream(stream):
        bits = int(error.item())
    for status in (recis.RECIS_ERR_KEY_RANGE, recis.RECIS_ERR_INVALID_ARG):
        if bits >> status & 1:
            raise recis.RecisError(status, "device error")


# --------------------------------------------------------------- embedding
def embed(tokens, weight, scale: float = 1.0, out=None, error=None, stream=None):
    """scale * weight[tokens]: tokens int64 of any shape, weight [rows, dim];
    a negative token is padding and gives zeros.  Returns [*tokens.shape, dim]."""
    if stream is not None:
        with _on(stream, tokens, weight, out, error):
            return embed(tokens, weight, scale, out, error)
    _forward_of("embed", tokens, weight, out, _error_word(error))
    if tokens.dtype != torch.int64 or weight.dim() != 2:
        raise ValueError("tokens must be int64 and weight [rows, dim]")
    dtype = _dtype("weight", weight)
    rows, dim = weight.shape
    tokens = tokens.contiguous()
    weight, w_stride = _rows(weight)
    if out is None:
        out = weight.new_empty((*tokens.shape, dim))
        stride = dim
    else:
        stride = _written("out", out, (*tokens.shape, dim), weight.dtype)
    recis.recis_embed_fwd(tokens, tokens.numel(), weight, dtype, rows, dim, w_stride, scale, out, stride, error)
    return out


def embed_backward(tokens, grad_out, rows: int, scale: float = 1.0, dtype=None, out=None, error=None, stream=None):
    """The gradient [rows, dim] of embed's weight: scale times the sum of
    grad_out's rows of equal tokens, the rows no token names zero.  dtype:
    float32 or bfloat16 (default: grad_out's)."""
    if stream is not None:
        with _on(stream, tokens, grad_out, out, error):
            return embed_backward(tokens, grad_out, rows, scale, dtype, out, error)
    _on_gpu(tokens, grad_out, out, _error_word(error))
    dim = grad_out.shape[-1] if grad_out.dim() else 0
    if tokens.dtype != torch.int64 or tuple(grad_out.shape) != (*tokens.shape, dim):
        raise ValueError("tokens must be int64 [...] and grad_out [..., dim] over the same places")
    g_dtype = _dtype("grad_out", grad_out)
    n = tokens.numel()
    tokens = tokens.contiguous()
    grad_out, g_stride = _rows(grad_out)
    if out is None:
        out = grad_out.new_empty((rows, dim), dtype=dtype or grad_out.dtype)
        stride = dim
    else:
        stride = _written("out", out, (rows, dim), dtype or out.dtype)
    nbytes = recis.recis_embed_bwd_workspace_bytes(n, rows, dim)
    workspace = grad_out.new_empty(max(nbytes, 0), dtype=torch.uint8)
    recis.recis_embed_bwd(tokens, n, grad_out, g_dtype, g_stride, rows, dim, scale, out, _dtype("out", out), stride,
                          workspace, nbytes, error)
    return out


# --------------------------------------------------------------- layer norm
def _norm_weights(weight, bias, dim: int) -> int:
    one = weight if weight is not None else bias
    if one is None:
        return RECIS_DTYPE_F32
    for t in (weight, bias):
        if t is not None and (t.shape != (dim,) or t.dtype != one.dtype or not t.is_contiguous()):
            raise ValueError(f"weight and bias must be contiguous [{dim}] of one type")
    return _dtype("weight", one)


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, stats: bool = True, out=None, stream=None):
    """Layer norm over x's last axis.  Returns (y, mean, rstd), the statistics
    float32 over the other axes; with stats False only y."""
    if stream is not None:
        with _on(stream, x, weight, bias, out):
            return layer_norm(x, weight, bias, eps, stats, out)
    _forward_of("layer_norm", x, weight, bias, out)
    if x.dim() < 1:
        raise ValueError("x must be [..., dim]")
    dtype, dim = _dtype("x", x), x.shape[-1]
    w_dtype = _norm_weights(weight, bias, dim)
    m = x.numel() // dim if dim else 0
    x, x_stride = _rows(x)
    if out is None:
        y, y_stride = _like(x), dim
    else:
        y, y_stride = out, _written("out", out, x.shape, x.dtype)
    mean = rstd = None
    if stats:
        mean, rstd = x.new_empty((2, *x.shape[:-1]), dtype=torch.float32).unbind(0)
    recis.recis_layernorm_fwd(x, dtype, x_stride, m, dim, weight, bias, w_dtype, eps, y, y_stride, mean, rstd)
    return (y, mean, rstd) if stats else y


def layer_norm_backward(grad_y, x, mean, rstd, weight=None, need_weight: bool = True, weight_dtype=None, stream=None):
    """Gradients (grad_x, grad_weight, grad_bias) of layer_norm from its mean
    and rstd.  The last two are float32, or weight's type, or weight_dtype;
    None with need_weight False."""
    if stream is not None:
        with _on(stream, grad_y, x, mean, rstd, weight):
            return layer_norm_backward(grad_y, x, mean, rstd, weight, need_weight, weight_dtype)
    _on_gpu(grad_y, x, mean, rstd, weight)
    if x.dim() < 1 or grad_y.shape != x.shape or grad_y.dtype != x.dtype:
        raise ValueError("grad_y and x must have one shape [..., dim] and type")
    dtype, dim = _dtype("x", x), x.shape[-1]
    m = x.numel() // dim if dim else 0
    for name, t in (("mean", mean), ("rstd", rstd)):
        if t.dtype != torch.float32 or t.numel() != m or not t.is_contiguous():
            raise ValueError(f"{name} must be layer_norm's, contiguous float32 over x's leading axes")
    _norm_weights(weight, None, dim)
    wt = weight_dtype or (weight.dtype if weight is not None else torch.float32)
    if wt not in _DTYPES or (weight is not None and weight.dtype != wt):
        raise ValueError("weight_dtype must be float32 or bfloat16, and weight's own type where there is one")
    x, x_stride = _rows(x)
    grad_y, g_stride = _rows(grad_y)
    dx = _like(x)
    dw = db = workspace = None
    nbytes = 0
    if need_weight:
        dw, db = x.new_empty((2, dim), dtype=wt).unbind(0)
        nbytes = recis.recis_layernorm_bwd_workspace_bytes(m, dim)
        workspace = x.new_empty(max(nbytes, 0), dtype=torch.uint8)
    recis.recis_layernorm_bwd(grad_y, g_stride, x, x_stride, dtype, m, dim, mean, rstd, weight, _DTYPES[wt], dx, dim,
                              dw, db, workspace, nbytes)
    return dx, dw, db


# ---------------------------------------------------------- cross attention
def _heads(t):
    """Head vectors contiguous; the other axes as they are."""
    return t if t.stride(-1) == 1 or t.shape[-1] == 1 else t.contiguous()


def _strides(t):
    """(batch, position, head) strides; packed tensors have no batch stride."""
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


def _attn_desc(q, k, v, kv_lens, kv_offsets, kv_mask, max_kv_len, scale, error):
    if q.dim() != 4 or k.dim() != (4 if kv_offsets is None else 3) or v.shape != k.shape:
        raise ValueError("q must be [batch, q_len, q_heads, head_dim], k and v both [batch, kv_len, kv_heads, "
                         "head_dim], or [kv_rows, kv_heads, head_dim] with kv_offsets")
    if not q.dtype == k.dtype == v.dtype:
        raise ValueError("q, k and v must be of one type")
    b, q_len, q_heads, head_dim = q.shape
    if k.shape[-1] != head_dim or (kv_offsets is None and k.shape[0] != b):
        raise ValueError("k and v must have q's head_dim and batch")
    kv_len = k.shape[1] if kv_offsets is None else max_kv_len or 0
    d = recis.recis_attn_desc()
    d.dtype = _dtype("q", q)
    d.batch, d.q_len, d.kv_len, d.q_heads, d.kv_heads, d.head_dim = map(
        recis.int32, (b, q_len, kv_len, q_heads, k.shape[-2], head_dim))
    d.scale = max(head_dim, 1) ** -0.5 if scale is None else scale  # (the call refuses 0)
    keep = []
    if kv_offsets is not None:
        if kv_lens is not None or max_kv_len is None:
            raise ValueError("packed keys (kv_offsets) take max_kv_len, and no kv_lens")
        keep.append(_index("kv_offsets", kv_offsets, torch.int32, (b + 1,)))
        d.kv_offsets, d.kv_rows = keep[-1].data_ptr(), k.shape[0]
    else:
        if max_kv_len is not None and max_kv_len != kv_len:
            raise ValueError("max_kv_len goes with kv_offsets")
        if kv_lens is not None:
            keep.append(_index("kv_lens", kv_lens, torch.int32, (b,)))
            d.kv_lens = keep[-1].data_ptr()
    if kv_mask is not None:
        if kv_mask.dtype not in (torch.bool, torch.uint8) or tuple(kv_mask.shape) != tuple(k.shape[:-2]):
            raise ValueError(f"kv_mask must be bool or uint8 {list(k.shape[:-2])}")
        keep.append(kv_mask if kv_mask.stride(-1) == 1 else kv_mask.contiguous())
        d.kv_mask, d.mask_stride = keep[-1].data_ptr(), keep[-1].stride(0) if kv_offsets is None else 0
    if error is not None:
        d.error = _error_word(error).data_ptr()
    d.q_strides[:], d.k_strides[:], d.v_strides[:] = _strides(q), _strides(k), _strides(v)
    return d, keep


def cross_attention(q, k, v, kv_lens=None, kv_offsets=None, kv_mask=None, max_kv_len: Optional[int] = None,
                    scale: Optional[float] = None, return_lse: bool = False, error=None, stream=None):
    """softmax(scale q k^T) v for q [batch, q_len, q_heads, head_dim] over keys

    * padded, k and v [batch, kv_len, kv_heads, head_dim], entry b having its
      first kv_lens[b] (int32, default: all), or
    * packed, k and v [kv_rows, kv_heads, head_dim], entry b having rows
      kv_offsets[b] .. kv_offsets[b + 1] - 1 (int32 [batch + 1], as the lookup's
      bag offsets), none more than max_kv_len;

    kv_mask (bool or uint8, [batch, kv_len] or [kv_rows]) leaves further keys
    out where it is zero.  q_heads is a multiple of kv_heads; scale defaults to
    head_dim ** -0.5.  Returns out as q's shape and, with return_lse, the
    float32 [batch, q_len, q_heads] that the backward pass takes.  An entry
    without keys gives zeros, and lse -inf."""
    if stream is not None:
        with _on(stream, q, k, v, kv_lens, kv_offsets, kv_mask, error):
            return cross_attention(q, k, v, kv_lens, kv_offsets, kv_mask, max_kv_len, scale, return_lse, error)
    _forward_of("cross_attention", q, k, v, kv_lens, kv_offsets, kv_mask, error)
    q, k, v = _heads(q), _heads(k), _heads(v)
    d, keep = _attn_desc(q, k, v, kv_lens, kv_offsets, kv_mask, max_kv_len, scale, error)
    out = _like(q)
    d.o_strides[:] = _strides(out)
    lse = q.new_empty(q.shape[:3], dtype=torch.float32) if return_lse else None
    nbytes = recis.recis_cross_attn_workspace_bytes(d, False)
    workspace = q.new_empty(nbytes, dtype=torch.uint8) if nbytes > 0 else None
    recis.recis_cross_attn_fwd(d, q, k, v, out, lse, workspace, nbytes)
    return (out, lse) if return_lse else out


def cross_attention_backward(grad_out, q, k, v, out, lse, kv_lens=None, kv_offsets=None, kv_mask=None,
                             max_kv_len: Optional[int] = None, scale: Optional[float] = None, error=None,
                             stream=None):
    """Gradients (grad_q, grad_k, grad_v) of cross_attention from its out and
    lse; the other arguments as there.  Keys that do not count get zeros."""
    if stream is not None:
        with _on(stream, grad_out, q, k, v, out, lse, kv_lens, kv_offsets, kv_mask, error):
            return cross_attention_backward(grad_out, q, k, v, out, lse, kv_lens, kv_offsets, kv_mask, max_kv_len,
                                            scale, error)
    _on_gpu(grad_out, q, k, v, out, lse, kv_lens, kv_offsets, kv_mask, error)
    if not grad_out.shape == out.shape == q.shape or not grad_out.dtype == out.dtype == q.dtype:
        raise ValueError("grad_out and out must have q's shape and type")
    if lse.dtype != torch.float32 or lse.shape != q.shape[:3] or not lse.is_contiguous():
        raise ValueError("lse must be cross_attention's, contiguous float32 [batch, q_len, q_heads]")
    q, k, v, out, grad_out = _heads(q), _heads(k), _heads(v), _heads(out), _heads(grad_out)
    d, keep = _attn_desc(q, k, v, kv_lens, kv_offsets, kv_mask, max_kv_len, scale, error)
    dq = _like(q)
    dk, dv = _like(k), _like(v)
    if not q.shape[0]:  # without a batch entry nothing is written
        dk.zero_(), dv.zero_()
    d.o_strides[:], d.do_strides[:], d.dq_strides[:] = _strides(out), _strides(grad_out), _strides(dq)
    d.dk_strides[:], d.dv_strides[:] = _strides(dk), _strides(dv)
    nbytes = recis.recis_cross_attn_workspace_bytes(d, True)
    workspace = q.new_empty(max(nbytes, 0), dtype=torch.uint8)
    recis.recis_cross_attn_bwd(d, grad_out, q, k, v, out, lse, dq, dk, dv, workspace, nbytes)
    return dq, dk, dv
