"""The sequence operators on tensors: token embedding, layer norm, cross attention,
and those of a growing history: rotary positions, causal self attention, and a
paged cache of keys and values with its append and the attention that reads it.

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
import math
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


# --------------------------------------------------------- rotary positions
# (These calls are made for a few microseconds of work, and a tensor's shape, taken from it, costs a quarter of one:
# each is taken once.)
def _st(t):
    """Strides of (batch entry, position, head) or (page, slot, head)."""
    s = t.stride()
    return s[:3] if len(s) == 4 else (0, s[0], s[1])


def _heads_st(t, head_dim):
    """t with its head vectors contiguous, and those strides."""
    s = t.stride()
    if s[-1] != 1 and head_dim != 1:
        t = t.contiguous()
        s = t.stride()
    return t, (s[:3] if len(s) == 4 else (0, s[0], s[1]))


def _serves(name: str, *tensors):
    """Checks of a call that serves only: it has no backward pass."""
    _on_gpu(*tensors)
    if not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            warnings.warn(f"sequence.{name} is for serving and has no backward pass: pass detached tensors or work "
                          "under torch.no_grad()", stacklevel=3)
            return


def _head_tensor(name: str, t, shape, dtype):
    """An output or a cache given by the caller: head vectors contiguous, no element twice."""
    if t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {dtype} {list(shape)}, not {t.dtype} {list(t.shape)}")
    if not t.is_contiguous() and ((t.shape[-1] > 1 and t.stride(-1) != 1) or any(
            st == 0 and n > 1 for st, n in zip(t.stride(), t.shape))):
        raise ValueError(f"{name} is written in place: its head vectors must be contiguous and no axis expanded")


def _freqs(freqs, head_dim: int) -> int:
    """Elements of a head that turn."""
    if freqs.dtype != torch.float64 or freqs.dim() != 1 or not freqs.is_contiguous():
        raise ValueError("freqs must be contiguous float64 [rotated elements / 2]")
    rot_dim = 2 * freqs.numel()
    if rot_dim > head_dim:
        raise ValueError(f"{rot_dim // 2} pairs are more than a head of {head_dim} has")
    return rot_dim


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_len: Optional[int] = None, slow: float = 1.0, fast: float = 4.0, device=None):
    """Radians a position for the pairs of the first rot_dim elements of a head: f[i] = base ** (-2 i / rot_dim), as
    a float64 tensor on the GPU that is made once and given to ``rotary`` and ``cache_append``.  For histories
    longer than a model was trained on, scaling

    * "linear": every f / factor;
    * "base": base * factor ** (rot_dim / (rot_dim - 2)) in place of base, so that the first pair turns as before and
      the last 1 / factor as fast;
    * "parts": a pair that turns n = original_len * f / 2 pi times over the original length keeps its f where n >=
      fast, gets f / factor where n <= slow, and in between the mean of the two with weights (n - slow) / (fast -
      slow) and the rest."""
    if rot_dim < 0 or rot_dim % 2:
        raise ValueError("rot_dim must be even")
    if scaling not in ("none", "linear", "base", "parts") or not factor > 0 or not base > 0:
        raise ValueError("scaling is 'none', 'linear', 'base' or 'parts', factor and base are above 0")
    if scaling == "base":
        if rot_dim <= 2:
            raise ValueError("scaling the base takes more than one pair")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = torch.tensor([base ** (-2 * i / rot_dim) for i in range(rot_dim // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if original_len is None or not fast > slow:
            raise ValueError("scaling by parts takes original_len, and fast above slow")
        keep = ((original_len * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * (keep + (1 - keep) / factor)
    return f.to("cuda" if device is None else device)


def _rotary(x, freqs, positions, interleaved, amplitude, out, backward):
    shape, dtype = tuple(x.shape), _dtype("x", x)
    if len(shape) not in (3, 4):
        raise ValueError("x must be [seq, heads, head_dim] or [batch, seq, heads, head_dim]")
    batch, seq, heads, head_dim = shape if len(shape) == 4 else (1, *shape)
    rot_dim = _freqs(freqs, head_dim)
    x, x_st = _heads_st(x, head_dim)
    if out is None:
        out = _like(x)
    else:
        _head_tensor("out", out, shape, x.dtype)
    at, at_strides = 0, (0, 0)
    if positions is not None:
        if positions.dtype != torch.int64 or tuple(positions.shape) not in (shape[:-2], (seq,)):
            raise ValueError(f"positions must be int64 {list(shape[:-2])} or [{seq}]")
        at, at_strides = positions.data_ptr(), positions.stride()
        if len(at_strides) == 1:
            at_strides = (0, *at_strides)
    if batch and seq and heads:
        int32 = recis.int32
        desc = recis.pack_rotary_desc(dtype, int32(heads), int32(head_dim), rot_dim, 1 if interleaved else 0, amplitude,
                                      batch, seq, freqs.data_ptr() if rot_dim else 0, at, *at_strides, *x_st, *_st(out))
        recis.recis_rotary(desc, backward, x, out)
    return out


def rotary(x, freqs, positions=None, interleaved: bool = False, amplitude: float = 1.0, out=None, stream=None):
    """Rotary positions of heads x [seq, heads, head_dim] or [batch, seq, heads, head_dim]: pair i of each head turned
    by positions * freqs[i], the elements past 2 * len(freqs) copied.  Pairs are (i, i + len(freqs)), or (2i, 2i + 1)
    interleaved.  positions: int64 over x's leading axes or [seq] (default: 0 .. seq - 1); freqs: float64, as
    ``rotary_frequencies`` makes them; amplitude multiplies what is turned.  out may be x, or shares no element
    with it."""
    if stream is not None:
        with _on(stream, x, freqs, positions, out):
            return rotary(x, freqs, positions, interleaved, amplitude, out)
    _forward_of("rotary", x, freqs, positions, out)
    return _rotary(x, freqs, positions, interleaved, amplitude, out, False)


def rotary_backward(grad_out, freqs, positions=None, interleaved: bool = False, amplitude: float = 1.0, out=None,
                    stream=None):
    """The gradient of rotary's x: grad_out turned back.  Arguments as there; out may be grad_out, or shares no element
    with it."""
    if stream is not None:
        with _on(stream, grad_out, freqs, positions, out):
            return rotary_backward(grad_out, freqs, positions, interleaved, amplitude, out)
    _on_gpu(grad_out, freqs, positions, out)
    return _rotary(grad_out, freqs, positions, interleaved, amplitude, out, True)


# -------------------------------------------------------------- paged cache
def _paged(page_table, kv_lens, q_offsets, batch, error):
    """What both calls on a cache check alike: (page_table, its width and stride, pointers of it, kv_lens, q_offsets and
    error), and what of it has to stay."""
    width = tuple(page_table.shape)
    if page_table.dtype != torch.int32 or len(width) != 2 or width[0] != batch:
        raise ValueError(f"page_table must be int32 [{batch}, pages an entry may have]")
    stride = page_table.stride()
    if (width[1] > 1 and stride[1] != 1) or (batch > 1 and stride[0] < width[1]):  # (one row expanded among them)
        page_table = page_table.contiguous()
        stride = page_table.stride()
    if kv_lens.dtype != torch.int32 or tuple(kv_lens.shape) != (batch,):
        raise ValueError(f"kv_lens must be torch.int32 [{batch}], not {kv_lens.dtype} {list(kv_lens.shape)}")
    kv_lens, at = kv_lens.contiguous(), 0
    if q_offsets is not None:
        if q_offsets.dtype != torch.int32 or q_offsets.dim() != 1:
            raise ValueError("q_offsets must be int32 [batch + 1]")
        q_offsets = q_offsets.contiguous()
        at = q_offsets.data_ptr()
    return (recis.int32(width[1]), stride[0] if batch > 1 else width[1],
            (at, kv_lens.data_ptr(), page_table.data_ptr(), 0 if error is None else _error_word(error).data_ptr()),
            (page_table, kv_lens, q_offsets))


def cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q=None, q_offsets=None, freqs=None,
                 interleaved: bool = False, amplitude: float = 1.0, error=None, stream=None):
    """Stores the keys and values of new events in a paged cache, in place, in one launch.

    k and v [batch, new, kv_heads, head_dim], or packed [rows, kv_heads, head_dim] with q_offsets (int32 [batch + 1]:
    entry b has rows q_offsets[b] .. q_offsets[b + 1] - 1).  k_cache and v_cache [pages, page_size, kv_heads,
    head_dim]; page_table int32 [batch, width]: key j of entry b lies in slot j % page_size of page page_table[b, j //
    page_size].  kv_lens int32 [batch] counts each entry's keys with the new ones, whose last is at position kv_lens[b]
    - 1; rows that fall at negative positions are padding and are not stored (an entry of kv_lens 0 is idle).

    With freqs the keys are turned by their positions on the way (``rotary``), and with q [.., q_heads, head_dim], the
    queries of the same rows, the call returns those turned (rows of no entry zero); without q it returns None."""
    if stream is not None:
        with _on(stream, k, v, k_cache, v_cache, page_table, kv_lens, q, q_offsets, freqs, error):
            return cache_append(k, v, k_cache, v_cache, page_table, kv_lens, q, q_offsets, freqs, interleaved,
                                amplitude, error)
    _serves("cache_append", k, v, k_cache, v_cache, page_table, kv_lens, q, q_offsets, freqs, error)
    shape, packed = tuple(k.shape), q_offsets is not None
    if len(shape) != (3 if packed else 4) or tuple(v.shape) != shape:
        raise ValueError("k and v must both be [batch, new, kv_heads, head_dim], or [rows, kv_heads, head_dim] with "
                         "q_offsets")
    kv_heads, head_dim = shape[-2:]
    kind, dtype = k.dtype, _dtype("k", k)
    if v.dtype != kind or k_cache.dtype != kind or (q is not None and q.dtype != kind):
        raise ValueError("q, k, v and the caches must be of one type")
    batch = q_offsets.numel() - 1 if packed else shape[0]
    cache = tuple(k_cache.shape)
    if len(cache) != 4:
        raise ValueError("k_cache and v_cache must both be [pages, page_size, kv_heads, head_dim] of one type")
    _head_tensor("k_cache", k_cache, (cache[0], cache[1], kv_heads, head_dim), kind)
    _head_tensor("v_cache", v_cache, cache, kind)
    width, table_st, at, keep = _paged(page_table, kv_lens, q_offsets, batch, error)
    k, k_st = _heads_st(k, head_dim)
    v, v_st = _heads_st(v, head_dim)
    out, q_heads, q_st, out_st = None, 0, (0, 0, 0), (0, 0, 0)
    if q is not None:
        if freqs is None:
            raise ValueError("q is turned by its positions: it takes freqs")
        q_shape = tuple(q.shape)
        if len(q_shape) != len(shape) or q_shape[:-2] != shape[:-2] or q_shape[-1] != head_dim:
            raise ValueError("q must have k's rows and head_dim")
        q, q_st = _heads_st(q, head_dim)
        out = _like(q) if batch else torch.zeros_like(q)
        q_heads, out_st = q_shape[-2], _st(out)
    rot_dim = 0 if freqs is None else _freqs(freqs, head_dim)
    int32 = recis.int32
    desc = recis.pack_append_desc(
        dtype, int32(batch), 0 if packed else int32(shape[1]), int32(q_heads), int32(kv_heads), int32(head_dim), rot_dim,
        1 if interleaved else 0, amplitude, int32(cache[1]), width, cache[0], table_st, shape[0] if packed else 0, *q_st,
        *out_st, *k_st, *v_st, *_st(k_cache), *_st(v_cache), freqs.data_ptr() if rot_dim else 0, *at)
    recis.recis_cache_append(desc, q, k, v, out, k_cache, v_cache)
    return out


def _band(window, sinks: int):
    """(window, sinks) as the C ABI has them."""
    if window is not None and window < 1:
        raise ValueError("window counts the positions a row sees, itself among them: at least 1")
    if sinks < 0:
        raise ValueError("sinks must not be negative")
    return 0 if window is None else recis.int32(window), recis.int32(sinks)


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, q_offsets=None, max_q_len: Optional[int] = None,
                    causal: bool = True, window: Optional[int] = None, sinks: int = 0, scale: Optional[float] = None,
                    return_lse: bool = False, out=None, error=None, stream=None):
    """Attention of new events to the paged cache that ``cache_append`` fills, their own keys among it.

    q [batch, new, q_heads, head_dim], or packed [rows, q_heads, head_dim] with q_offsets (int32 [batch + 1]), no entry
    having more than max_q_len rows; q_heads is a multiple of the cache's kv_heads.  Causal, the last row of entry b is
    at position kv_lens[b] - 1 and each row sees the keys up to its position: with window the latest `window` of them,
    itself among them, and the first `sinks` ones.  Not causal (candidates reading a history), every row sees all
    kv_lens[b] keys.  Returns q's shape (in out, if given, which shares no element with the others) and with return_lse
    the float32 log of the sums of exponentials [.., q_heads].  Rows that see no key, at negative positions or of an
    entry without keys, give zeros and -inf.  Packed rows of no entry are not written: in a result that the call allocates they are zeros and -inf.
    Keys before the window that no new row sees are not read, nor their pages' numbers: such pages may be given away.
    Keys of another page whose number is out of range do not count (and are recorded in error).  A cache whose heads
    are not contiguous is copied whole first, with a warning."""
    if stream is not None:
        with _on(stream, q, k_cache, v_cache, page_table, kv_lens, q_offsets, out, error):
            return paged_attention(q, k_cache, v_cache, page_table, kv_lens, q_offsets, max_q_len, causal, window,
                                   sinks, scale, return_lse, out, error)
    _serves("paged_attention", q, k_cache, v_cache, page_table, kv_lens, q_offsets, out, error)
    shape, packed = tuple(q.shape), q_offsets is not None
    if len(shape) != (3 if packed else 4) or packed != (max_q_len is not None):
        raise ValueError("q must be [batch, new, q_heads, head_dim], or [rows, q_heads, head_dim] with q_offsets and "
                         "max_q_len")
    cache, kind, head_dim = tuple(k_cache.shape), q.dtype, shape[-1]
    if len(cache) != 4 or tuple(v_cache.shape) != cache or cache[3] != head_dim or k_cache.dtype != kind \
            or v_cache.dtype != kind:
        raise ValueError("k_cache and v_cache must both be [pages, page_size, kv_heads, head_dim], of q's type and "
                         "head_dim")
    if not causal and (window is not None or sinks):
        raise ValueError("a window takes causal rows")
    dtype = _dtype("q", q)
    batch = q_offsets.numel() - 1 if packed else shape[0]
    width, table_st, at, keep = _paged(page_table, kv_lens, q_offsets, batch, error)
    q, q_st = _heads_st(q, head_dim)
    given = k_cache, v_cache
    k_cache, k_st = _heads_st(k_cache, head_dim)
    v_cache, v_st = _heads_st(v_cache, head_dim)
    if k_cache is not given[0] or v_cache is not given[1]:
        warnings.warn("a cache whose heads are not contiguous is copied whole, in every call of paged_attention",
                      stacklevel=2)
    if out is None:
        out = q.new_zeros(shape) if packed else _like(q)
    else:
        _head_tensor("out", out, shape, kind)
    lse = q.new_full(shape[:-1], -math.inf, dtype=torch.float32) if return_lse else None
    int32 = recis.int32
    desc = recis.pack_paged_attn_desc(
        dtype, int32(batch), int32(max_q_len if packed else shape[1]), int32(shape[-2]), int32(cache[2]),
        int32(head_dim), 1 if causal else 0, *_band(window, sinks), int32(cache[1]), width,
        max(head_dim, 1) ** -0.5 if scale is None else scale, cache[0], table_st, shape[0] if packed else 0, *q_st,
        *_st(out), *k_st, *v_st, *at)
    nbytes = recis.recis_paged_attn_workspace_bytes(desc)
    workspace = q.new_empty(nbytes, dtype=torch.uint8) if nbytes > 0 else None
    recis.recis_paged_attn_fwd(desc, q, k_cache, v_cache, out, lse, workspace, nbytes)
    return (out, lse) if return_lse else out


# ----------------------------------------------------------- self attention
def _self_desc(q, k, v, lens, offsets, kv_mask, max_len, window, sinks, scale, error):
    packed = offsets is not None
    if q.dim() != (3 if packed else 4) or k.dim() != q.dim() or v.shape != k.shape or q.shape[:-2] != k.shape[:-2] \
            or q.shape[-1] != k.shape[-1]:
        raise ValueError("q must be [batch, len, q_heads, head_dim], or [rows, q_heads, head_dim] with offsets, and k "
                         "and v the same with kv_heads")
    if not q.dtype == k.dtype == v.dtype:
        raise ValueError("q, k and v must be of one type")
    if packed != (max_len is not None) or (packed and lens is not None):
        raise ValueError("packed histories (offsets) take max_len, and no lens; padded ones no max_len")
    dtype = _dtype("q", q)
    batch, length = (offsets.numel() - 1, max_len) if packed else q.shape[:2]
    keep, mask, mask_stride = None, 0, 0
    if packed:
        keep = _index("offsets", offsets, torch.int32, (batch + 1,))
    elif lens is not None:
        keep = _index("lens", lens, torch.int32, (batch,))
    if kv_mask is not None:
        if kv_mask.dtype not in (torch.bool, torch.uint8) or kv_mask.shape != k.shape[:-2]:
            raise ValueError(f"kv_mask must be bool or uint8 {list(k.shape[:-2])}")
        kv_mask = kv_mask if kv_mask.stride(-1) == 1 else kv_mask.contiguous()
        mask, mask_stride = kv_mask.data_ptr(), 0 if packed else kv_mask.stride(0)
    int32, head_dim = recis.int32, q.shape[-1]
    head = (dtype, int32(batch), int32(length), int32(q.shape[-2]), int32(k.shape[-2]), int32(head_dim),
            *_band(window, sinks), max(head_dim, 1) ** -0.5 if scale is None else scale, q.shape[0] if packed else 0,
            *_st(q), *_st(k), *_st(v))
    at = keep.data_ptr() if keep is not None else 0
    tail = (0 if packed else at, at if packed else 0, mask, mask_stride,
            0 if error is None else _error_word(error).data_ptr())
    return head, tail, batch > 0 and length > 0, (keep, kv_mask)


def self_attention(q, k, v, lens=None, offsets=None, kv_mask=None, max_len: Optional[int] = None,
                   window: Optional[int] = None, sinks: int = 0, scale: Optional[float] = None,
                   return_lse: bool = False, error=None, stream=None):
    """Causal attention of histories to themselves: position p sees the positions up to p, with window the latest
    `window` of them, itself among them, and the first `sinks` ones.

    q [batch, len, q_heads, head_dim], k and v [batch, len, kv_heads, head_dim], entry b having its first lens[b]
    positions (int32, default: all); or packed, [rows, heads, head_dim], entry b having rows offsets[b] .. offsets[b +
    1] - 1 (int32 [batch + 1], as the lookup's bag offsets), none more than max_len.  kv_mask (bool or uint8, [batch,
    len] or [rows]) leaves further positions out as keys where it is zero.  q_heads is a multiple of kv_heads.  Returns
    q's shape and, with return_lse, the float32 [.., q_heads] that the backward pass takes.  Rows that see no key, past
    the length among them, give zeros and -inf; packed rows of no entry too."""
    if stream is not None:
        with _on(stream, q, k, v, lens, offsets, kv_mask, error):
            return self_attention(q, k, v, lens, offsets, kv_mask, max_len, window, sinks, scale, return_lse, error)
    _forward_of("self_attention", q, k, v, lens, offsets, kv_mask, error)
    q, k, v = _heads(q), _heads(k), _heads(v)
    head, tail, some, keep = _self_desc(q, k, v, lens, offsets, kv_mask, max_len, window, sinks, scale, error)
    out = _like(q) if some else q.new_zeros(q.shape)
    lse = None
    if return_lse:
        lse = q.new_empty(q.shape[:-1], dtype=torch.float32)
        if offsets is not None:
            lse.fill_(-math.inf)
    desc = recis.pack_self_attn_desc(*head, *_st(out), *[0] * 12, *tail)
    nbytes = recis.recis_self_attn_workspace_bytes(desc, False)
    workspace = q.new_empty(nbytes, dtype=torch.uint8) if nbytes > 0 else None
    recis.recis_self_attn_fwd(desc, q, k, v, out, lse, workspace, nbytes)
    return (out, lse) if return_lse else out


def self_attention_backward(grad_out, q, k, v, out, lse, lens=None, offsets=None, kv_mask=None,
                            max_len: Optional[int] = None, window: Optional[int] = None, sinks: int = 0,
                            scale: Optional[float] = None, error=None, stream=None):
    """Gradients (grad_q, grad_k, grad_v) of self_attention from its out and lse; the other arguments as there.  Rows
    that see no key and positions that do not count get zeros."""
    if stream is not None:
        with _on(stream, grad_out, q, k, v, out, lse, lens, offsets, kv_mask, error):
            return self_attention_backward(grad_out, q, k, v, out, lse, lens, offsets, kv_mask, max_len, window, sinks,
                                           scale, error)
    _on_gpu(grad_out, q, k, v, out, lse, lens, offsets, kv_mask, error)
    if not grad_out.shape == out.shape == q.shape or not grad_out.dtype == out.dtype == q.dtype:
        raise ValueError("grad_out and out must have q's shape and type")
    if lse.dtype != torch.float32 or lse.shape != q.shape[:-1] or not lse.is_contiguous():
        raise ValueError("lse must be self_attention's, contiguous float32 over q's leading axes and heads")
    q, k, v, out, grad_out = _heads(q), _heads(k), _heads(v), _heads(out), _heads(grad_out)
    head, tail, some, keep = _self_desc(q, k, v, lens, offsets, kv_mask, max_len, window, sinks, scale, error)
    dq, dk, dv = _like(q), _like(k), _like(v)
    if not some:  # without an entry nothing is written
        dq.zero_(), dk.zero_(), dv.zero_()
    desc = recis.pack_self_attn_desc(*head, *_st(out), *_st(grad_out), *_st(dq), *_st(dk), *_st(dv), *tail)
    nbytes = recis.recis_self_attn_workspace_bytes(desc, True)
    workspace = q.new_empty(max(nbytes, 0), dtype=torch.uint8)
    recis.recis_self_attn_bwd(desc, grad_out, q, k, v, out, lse, dq, dk, dv, workspace, nbytes)
    return dq, dk, dv
