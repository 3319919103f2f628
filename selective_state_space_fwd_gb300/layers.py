"""The operators around the scan: short causal convolution, norm of the residual
stream, softmax cross entropy over the vocabulary, distillation from a teacher's top
logits, the gated linear recurrence, and the embedding lookup.

Argument marshalling only, like ``_binding``: dtypes, shapes, devices and
strides are checked, outputs and workspaces are allocated when the caller
passes none, and the library's kernels do the work.  Weights, biases,
statistics and weight gradients are fp32; activations are fp32 or bf16.  Every
function takes ``stream=`` (a stream or its handle) and runs on the current
PyTorch stream without it.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from ._binding import (ConvShapes, DistillShapes, DType, EmbedShapes, NormShapes, RecurShapes,
                       SsmError, XentShapes, _check, load)

_F32 = torch.float32
_CODES = {_F32: int(DType.F32), torch.bfloat16: int(DType.BF16)}

# The current stream's handle by device index, and the current device: a tenth of
# the cost of torch.cuda.current_stream and current_device, which are a good part
# of a short call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


# The sizes as the library takes them: equal sizes share one structure, which the
# library only reads, and the workspace bytes that follow from them.
@functools.lru_cache(maxsize=512)
def _conv_sizes(*sizes):
    return ctypes.byref(ConvShapes(*sizes))


@functools.lru_cache(maxsize=512)
def _norm_sizes(*sizes):
    return ctypes.byref(NormShapes(*sizes))


@functools.lru_cache(maxsize=512)
def _xent_sizes(*sizes):
    return ctypes.byref(XentShapes(*sizes))


@functools.lru_cache(maxsize=512)
def _distill_sizes(*sizes):
    return ctypes.byref(DistillShapes(*sizes))


@functools.lru_cache(maxsize=512)
def _recur_sizes(*sizes):
    return ctypes.byref(RecurShapes(*sizes))


@functools.lru_cache(maxsize=512)
def _embed_sizes(*sizes):
    return ctypes.byref(EmbedShapes(*sizes))


@functools.lru_cache(maxsize=512)
def _conv_workspace(sizes):
    return load().ssm_conv_bwd_workspace_bytes(sizes)


@functools.lru_cache(maxsize=512)
def _norm_workspace(sizes):
    return load().ssm_norm_bwd_workspace_bytes(sizes)


@functools.lru_cache(maxsize=512)
def _xent_workspace(sizes, backward):
    return load().ssm_xent_workspace_bytes(sizes, backward)


@functools.lru_cache(maxsize=512)
def _distill_workspace(sizes, backward):
    return load().ssm_distill_workspace_bytes(sizes, backward)


@functools.lru_cache(maxsize=512)
def _recur_workspace(sizes):
    return load().ssm_recur_bwd_workspace_bytes(sizes)


@functools.lru_cache(maxsize=512)
def _embed_workspace(sizes):
    return load().ssm_embed_bwd_workspace_bytes(sizes)


def _code(dtype) -> int:
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _dense(t, name, shape, dtype, dev):
    """The contiguous tensor `t`, checked (the common case without the cost of
    building messages)."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev or not t.is_contiguous():
        _check(t, name, shape, dtype, dev)
    return t


def _new(out, name, shape, dtype, dev):
    return (torch.empty(shape, dtype=dtype, device=dev) if out is None
            else _dense(out, name, shape, dtype, dev))


def _like(out, name, t, shape, dev):
    """`out`, checked, or a new contiguous tensor of t's type."""
    if out is not None:
        return _dense(out, name, shape, t.dtype, dev)
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(shape, dtype=t.dtype, device=dev)


def _addr(t):
    return None if t is None else t.data_ptr()


def _on_stream(stream, f, t, *args, **kw):
    """f(t, *args, **kw) with `stream` (or its handle) as PyTorch's current
    stream: the call's outputs and workspaces are then allocated where they are
    used, and take no memory that another stream may still be using."""
    dev = _cuda(t, "the first argument")
    if not hasattr(stream, "cuda_stream"):
        stream = (torch.cuda.ExternalStream(int(stream), device=dev) if int(stream)
                  else torch.cuda.default_stream(dev))
    if stream.device != dev:
        raise ValueError(f"stream: on {stream.device}, expected {dev}")
    with torch.cuda.stream(stream):
        return f(t, *args, **kw)


def _call(fn, dev, *args):
    """fn(*args, the current stream of `dev`) on `dev`, raising SsmError on a bad
    status."""
    index = dev.index
    handle = _raw_stream(index)
    if _device() == index:
        st = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, handle)
    if st != 0:
        raise SsmError(st, fn.__name__)


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _conv_args(x, weight, bias, silu, rank):
    """Checked (device, dtype code, batch, seqlen, dim, width, ConvShapes) of a
    convolution whose x has `rank` dimensions, the last of them contiguous."""
    dev = _cuda(x, "x")
    code = _code(x.dtype)
    size, stride = x.shape, x.stride()
    if len(size) != rank:
        raise ValueError(f"x: {len(size)} dimensions, expected {rank}")
    if weight.dim() != 2:
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected [dim, width]")
    width = weight.shape[1]
    if rank == 3:
        batch, seqlen, dim = size
        step = stride[1] if seqlen > 1 else dim
    else:
        batch, dim = size
        seqlen, step = 1, dim
    if stride[-1] != 1 and dim > 1:
        raise ValueError("x: the channels must be contiguous")
    _dense(weight, "weight", (dim, width), _F32, dev)
    if bias is not None:
        _dense(bias, "bias", (dim,), _F32, dev)
    # the stride of an axis of one element is never used; the row's own length
    # keeps it from deciding the alignment rule
    return dev, code, batch, seqlen, dim, width, _conv_sizes(
        batch, seqlen, dim, width, stride[0] if batch > 1 else dim, step, 1 if silu else 0)


def conv_fwd(x, weight, bias=None, valid_len=None, *, state0=None, silu: bool = True,
             want_final: bool = False, out=None, out_final=None, stream=None):
    """The short causal convolution of every channel along time.

    x: [batch, L, dim], fp32 or bf16, channels contiguous; rows may be strided
    (columns of a wider projection).  weight: fp32 [dim, width], width 2 to 4,
    the last tap on the current step; bias: fp32 [dim]; valid_len: int32
    [batch], steps past it give 0 whatever x holds there.  state0: like x, [batch,
    width - 1, dim], the steps before the first (zeros when None).  With
    ``silu`` the result is silu(pre).  Returns y [batch, L, dim], or
    ``(y, final)`` with ``want_final``, final [batch, width - 1, dim] being the
    last valid steps, from which a next call or ``conv_step`` continues."""
    if stream is not None:
        return _on_stream(stream, conv_fwd, x, weight, bias, valid_len, state0=state0, silu=silu,
                          want_final=want_final, out=out, out_final=out_final)
    dev, code, batch, L, dim, width, sizes = _conv_args(x, weight, bias, silu, 3)
    if valid_len is not None:
        _dense(valid_len, "valid_len", (batch,), torch.int32, dev)
    if state0 is not None:
        _dense(state0, "state0", (batch, width - 1, dim), x.dtype, dev)
    y = _like(out, "out", x, (batch, L, dim), dev)
    final = None
    if want_final or out_final is not None:
        final = _new(out_final, "out_final", (batch, width - 1, dim), x.dtype, dev)
    _call(load().ssm_conv_fwd, dev, x.data_ptr(), weight.data_ptr(), _addr(bias),
          _addr(valid_len), _addr(state0), y.data_ptr(), _addr(final), sizes, code)
    return y if final is None else (y, final)


def conv_bwd(x, weight, bias=None, valid_len=None, *, dy, state0=None, silu: bool = True,
             want_dbias: bool | None = None, want_dstate0: bool = False, workspace=None,
             stream=None) -> dict:
    """Every gradient of sum(dy * y) for ``conv_fwd`` on the same inputs: a dict
    of dx (like x, contiguous), dweight and dbias (fp32; dbias None without a
    bias, or as ``want_dbias`` says) and dstate0 (when wanted).  ``workspace``,
    a CUDA uint8 tensor, is allocated here when None."""
    if stream is not None:
        return _on_stream(stream, conv_bwd, x, weight, bias, valid_len, dy=dy, state0=state0,
                          silu=silu, want_dbias=want_dbias, want_dstate0=want_dstate0,
                          workspace=workspace)
    dev, code, batch, L, dim, width, sizes = _conv_args(x, weight, bias, silu, 3)
    if valid_len is not None:
        _dense(valid_len, "valid_len", (batch,), torch.int32, dev)
    if state0 is not None:
        _dense(state0, "state0", (batch, width - 1, dim), x.dtype, dev)
    _dense(dy, "dy", (batch, L, dim), x.dtype, dev)
    lib = load()
    ws = _workspace(workspace, _conv_workspace(sizes), dev)
    if want_dbias is None:
        want_dbias = bias is not None
    g = {"dx": torch.empty_like(dy), "dweight": torch.empty_like(weight),
         "dbias": torch.empty((dim,), dtype=_F32, device=dev) if want_dbias else None,
         "dstate0": torch.empty((batch, width - 1, dim), dtype=x.dtype, device=dev)
         if want_dstate0 else None}
    _call(lib.ssm_conv_bwd, dev, x.data_ptr(), weight.data_ptr(), _addr(bias),
          _addr(valid_len), _addr(state0), dy.data_ptr(), g["dx"].data_ptr(),
          g["dweight"].data_ptr(), _addr(g["dbias"]), _addr(g["dstate0"]), ws.data_ptr(),
          ws.numel(), sizes, code)
    return g


def conv_step(x, weight, bias=None, *, state, silu: bool = True, out=None, stream=None):
    """One step of the convolution on a carried state, in place (decode).

    x: [batch, dim] (rows may be strided); state: like x, [batch, width - 1,
    dim], the last steps, oldest first (``conv_fwd``'s final state): the oldest
    leaves and x becomes the newest.  Returns y [batch, dim]."""
    if stream is not None:
        return _on_stream(stream, conv_step, x, weight, bias, state=state, silu=silu, out=out)
    dev, code, batch, _, dim, width, sizes = _conv_args(x, weight, bias, silu, 2)
    _dense(state, "state", (batch, width - 1, dim), x.dtype, dev)
    y = _like(out, "out", x, (batch, dim), dev)
    _call(load().ssm_conv_step, dev, x.data_ptr(), weight.data_ptr(), _addr(bias),
          state.data_ptr(), y.data_ptr(), sizes, code)
    return y


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor on x's device")
    return workspace


def _rows(t, dim):
    return t.numel() // dim if dim else 0


def norm_fwd(x, weight, bias=None, *, residual=None, rms: bool = False, eps: float = 1e-5,
             want_stats: bool = False, out=None, out_r=None, stream=None):
    """The norm of the residual stream, with the addition that precedes it.

    x: [..., dim], fp32 or bf16, contiguous, dim up to 8192.  With ``residual``
    (like x, or fp32) the sum r = x + residual, stored in the residual's type,
    is what is normalised; without it, x is.  weight, bias: fp32 [dim].
    ``rms`` takes the mean as 0 (root-mean-square norm).  Returns
    ``(y, r, stats)``: y like x, r the sum (None without a residual; ``out_r``
    may be ``residual`` itself), stats fp32 [2, rows] with the means and the
    reciprocal standard deviations (None unless ``want_stats``)."""
    if stream is not None:
        return _on_stream(stream, norm_fwd, x, weight, bias, residual=residual, rms=rms, eps=eps,
                          want_stats=want_stats, out=out, out_r=out_r)
    dev = _cuda(x, "x")
    code = _code(x.dtype)
    shape = x.shape
    dim = shape[-1] if shape else 0
    rows = _rows(x, dim)
    if not x.is_contiguous():
        raise ValueError("x: must be contiguous")
    _dense(weight, "weight", (dim,), _F32, dev)
    if bias is not None:
        _dense(bias, "bias", (dim,), _F32, dev)
    rcode, r = code, None
    if residual is not None:
        rcode = _code(residual.dtype)
        _dense(residual, "residual", shape, residual.dtype, dev)
        r = _like(out_r, "out_r", residual, shape, dev)
    elif out_r is not None:
        raise ValueError("out_r needs a residual")
    y = _like(out, "out", x, shape, dev)
    stats = torch.empty((2, rows), dtype=_F32, device=dev) if want_stats else None
    sizes = _norm_sizes(rows, dim, 1 if rms else 0, eps, code, rcode)
    _call(load().ssm_norm_fwd, dev, x.data_ptr(), _addr(residual), weight.data_ptr(),
          _addr(bias), y.data_ptr(), _addr(r), _addr(stats), sizes)
    return y, r, stats


def norm_bwd(r, weight, *, stats, dy, dr=None, rms: bool = False, want_dbias: bool = False,
             workspace=None, stream=None) -> dict:
    """Every gradient of sum(dy * y) + sum(dr * r) for ``norm_fwd``.

    r: what was normalised (the forward's r, or x without a residual); stats:
    the forward's; dy like y; dr like r, the gradient that arrives along the
    residual stream (None for none).  Returns a dict: dx (dy's type), dresidual
    (r's type; the same tensor as dx when the types are equal), dweight and
    dbias (fp32; dbias None unless wanted)."""
    if stream is not None:
        return _on_stream(stream, norm_bwd, r, weight, stats=stats, dy=dy, dr=dr, rms=rms,
                          want_dbias=want_dbias, workspace=workspace)
    dev = _cuda(r, "r")
    code, rcode = _code(dy.dtype), _code(r.dtype)
    shape = r.shape
    dim = shape[-1] if shape else 0
    rows = _rows(r, dim)
    if not r.is_contiguous():
        raise ValueError("r: must be contiguous")
    _dense(dy, "dy", shape, dy.dtype, dev)
    _dense(weight, "weight", (dim,), _F32, dev)
    _dense(stats, "stats", (2, rows), _F32, dev)
    if dr is not None:
        _dense(dr, "dr", shape, r.dtype, dev)
    lib = load()
    sizes = _norm_sizes(rows, dim, 1 if rms else 0, 0.0, code, rcode)
    ws = _workspace(workspace, _norm_workspace(sizes), dev)
    dx = torch.empty_like(dy)
    dres = torch.empty_like(r) if rcode != code else None
    dweight = torch.empty_like(weight)
    dbias = torch.empty_like(weight) if want_dbias else None
    _call(lib.ssm_norm_bwd, dev, r.data_ptr(), weight.data_ptr(), stats.data_ptr(),
          dy.data_ptr(), _addr(dr), dx.data_ptr(), _addr(dres), dweight.data_ptr(), _addr(dbias),
          ws.data_ptr(), ws.numel(), sizes)
    return {"dx": dx, "dresidual": dx if dres is None else dres, "dweight": dweight,
            "dbias": dbias}


def _xent_args(h, weight, targets, ignore_index):
    """Checked (device, dtype code, tokens, XentShapes) of a cross entropy."""
    dev = _cuda(h, "h")
    code = _code(h.dtype)
    if h.dim() != 2:
        raise ValueError(f"h: shape {tuple(h.shape)}, expected [tokens, dim]")
    if weight.dim() != 2:
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected [vocab, dim]")
    tokens, dim = h.shape
    vocab = weight.shape[0]
    _dense(h, "h", (tokens, dim), h.dtype, dev)
    _dense(weight, "weight", (vocab, dim), h.dtype, dev)
    _dense(targets, "targets", (tokens,), torch.int64, dev)
    return dev, code, tokens, _xent_sizes(tokens, vocab, dim, int(ignore_index))


def xent_fwd(h, weight, targets, *, ignore_index: int = -100, workspace=None, stream=None):
    """Softmax cross entropy of every token over the vocabulary, from the hidden
    states, without keeping the logits h weight^T.

    h: bf16 [tokens, dim]; weight: bf16 [vocab, dim] (the output embedding), dim
    a multiple of 8; targets: int64 [tokens].  Returns ``(loss, lse)``, fp32
    [tokens]: the losses and the logs of the softmax's denominators, which
    ``xent_bwd`` needs.  Tokens whose target is ``ignore_index`` get 0 in both
    and their rows of h are not used; a target outside the vocabulary gives
    NaN."""
    if stream is not None:
        return _on_stream(stream, xent_fwd, h, weight, targets, ignore_index=ignore_index,
                          workspace=workspace)
    dev, code, tokens, sizes = _xent_args(h, weight, targets, ignore_index)
    lib = load()
    ws = _workspace(workspace, _xent_workspace(sizes, 0), dev)
    loss = torch.empty((tokens,), dtype=_F32, device=dev)
    lse = torch.empty((tokens,), dtype=_F32, device=dev)
    _call(lib.ssm_xent_fwd, dev, h.data_ptr(), weight.data_ptr(), targets.data_ptr(),
          loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), sizes, code)
    return loss, lse


def xent_bwd(h, weight, targets, *, lse, dloss, ignore_index: int = -100, workspace=None,
             stream=None) -> dict:
    """The gradients of sum(dloss * loss) for ``xent_fwd``: a dict of dh (like h;
    0 for ignored tokens) and dweight (like weight).  lse: the forward's; dloss:
    fp32 [tokens]."""
    if stream is not None:
        return _on_stream(stream, xent_bwd, h, weight, targets, lse=lse, dloss=dloss,
                          ignore_index=ignore_index, workspace=workspace)
    dev, code, tokens, sizes = _xent_args(h, weight, targets, ignore_index)
    _dense(lse, "lse", (tokens,), _F32, dev)
    _dense(dloss, "dloss", (tokens,), _F32, dev)
    lib = load()
    ws = _workspace(workspace, _xent_workspace(sizes, 1), dev)
    dh, dweight = torch.empty_like(h), torch.empty_like(weight)
    _call(lib.ssm_xent_bwd, dev, h.data_ptr(), weight.data_ptr(), targets.data_ptr(),
          lse.data_ptr(), dloss.data_ptr(), dh.data_ptr(), dweight.data_ptr(), ws.data_ptr(),
          ws.numel(), sizes, code)
    return {"dh": dh, "dweight": dweight}


def _distill_args(h, weight, ids, logits, temperature, ignore_index):
    """Checked (device, dtype code, tokens, DistillShapes) of a distillation."""
    dev = _cuda(h, "h")
    code = _code(h.dtype)
    if h.dim() != 2:
        raise ValueError(f"h: shape {tuple(h.shape)}, expected [tokens, dim]")
    if weight.dim() != 2:
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected [vocab, dim]")
    if ids.dim() != 2:
        raise ValueError(f"ids: shape {tuple(ids.shape)}, expected [tokens, top]")
    tokens, dim = h.shape
    vocab, top = weight.shape[0], ids.shape[1]
    _dense(h, "h", (tokens, dim), h.dtype, dev)
    _dense(weight, "weight", (vocab, dim), h.dtype, dev)
    _dense(ids, "ids", (tokens, top), torch.int64, dev)
    teacher = _code(logits.dtype)
    _dense(logits, "logits", (tokens, top), logits.dtype, dev)
    return dev, code, tokens, _distill_sizes(tokens, vocab, dim, top, int(ignore_index),
                                             float(temperature), teacher)


def distill_fwd(h, weight, ids, logits, *, temperature: float = 1.0, ignore_index: int = -100,
                workspace=None, stream=None):
    """The divergence of a student's next-token distribution from a teacher's, of
    which the top logits are known, without keeping the student's logits
    h weight^T:

        loss = sum_k q_k (log q_k - log p[ids_k]),
        q = softmax(logits / temperature) over the token's entries,
        p = softmax(h weight^T / temperature) over the vocabulary.

    h: bf16 [tokens, dim]; weight: bf16 [vocab, dim], dim a multiple of 8; ids:
    int64 [tokens, top] and logits: fp32 or bf16 [tokens, top], the teacher's
    entries in any order, top up to 1024.  Entries of ``ignore_index``, or with a
    logit of -infinity, take no part; an id that comes twice counts twice.  Returns
    ``(loss, lse)``, fp32 [tokens]; lse, the log of p's denominator, is what
    ``distill_bwd`` needs.  Tokens without entries get 0 in both and their rows of
    h are not used; any other id outside the vocabulary gives NaN."""
    if stream is not None:
        return _on_stream(stream, distill_fwd, h, weight, ids, logits, temperature=temperature,
                          ignore_index=ignore_index, workspace=workspace)
    dev, code, tokens, sizes = _distill_args(h, weight, ids, logits, temperature, ignore_index)
    lib = load()
    ws = _workspace(workspace, _distill_workspace(sizes, 0), dev)
    loss = torch.empty((tokens,), dtype=_F32, device=dev)
    lse = torch.empty((tokens,), dtype=_F32, device=dev)
    _call(lib.ssm_distill_fwd, dev, h.data_ptr(), weight.data_ptr(), ids.data_ptr(),
          logits.data_ptr(), loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), sizes,
          code)
    return loss, lse


def distill_bwd(h, weight, ids, logits, *, lse, dloss, temperature: float = 1.0,
                ignore_index: int = -100, workspace=None, stream=None) -> dict:
    """The gradients of sum(dloss * loss) for ``distill_fwd`` in the student: a dict
    of dh (like h; 0 for tokens without entries) and dweight (like weight).  lse:
    the forward's; dloss: fp32 [tokens]."""
    if stream is not None:
        return _on_stream(stream, distill_bwd, h, weight, ids, logits, lse=lse, dloss=dloss,
                          temperature=temperature, ignore_index=ignore_index, workspace=workspace)
    dev, code, tokens, sizes = _distill_args(h, weight, ids, logits, temperature, ignore_index)
    _dense(lse, "lse", (tokens,), _F32, dev)
    _dense(dloss, "dloss", (tokens,), _F32, dev)
    lib = load()
    ws = _workspace(workspace, _distill_workspace(sizes, 1), dev)
    dh, dweight = torch.empty_like(h), torch.empty_like(weight)
    _call(lib.ssm_distill_bwd, dev, h.data_ptr(), weight.data_ptr(), ids.data_ptr(),
          logits.data_ptr(), lse.data_ptr(), dloss.data_ptr(), dh.data_ptr(), dweight.data_ptr(),
          ws.data_ptr(), ws.numel(), sizes, code)
    return {"dh": dh, "dweight": dweight}


def _recur_args(gate, value, floor, rank):
    """Checked (device, dtype code, batch, seqlen, dim, RecurShapes) of a
    recurrence whose gate and value have `rank` dimensions, the last of them
    contiguous."""
    dev = _cuda(gate, "gate")
    dtype, size = gate.dtype, gate.shape
    code = _code(dtype)
    if len(size) != rank:
        raise ValueError(f"gate: {len(size)} dimensions, expected {rank}")
    if value.dtype is not dtype:
        raise TypeError(f"value: dtype {value.dtype}, expected {dtype}")
    if value.shape != size or value.device != dev:
        raise ValueError(f"value: shape {tuple(value.shape)} on {value.device}, "
                         f"expected {tuple(size)} on {dev}")
    gs, vs = gate.stride(), value.stride()
    if rank == 3:
        batch, seqlen, dim = size
        if seqlen > 1:
            g_step, v_step = gs[1], vs[1]
        else:
            g_step = v_step = dim
    else:
        batch, dim = size
        seqlen, g_step, v_step = 1, dim, dim
    if dim > 1 and (gs[-1] != 1 or vs[-1] != 1):
        raise ValueError("gate and value: the channels must be contiguous")
    if floor is not None:
        _dense(floor, "floor", (dim,), _F32, dev)
    # the stride of an axis of one element is never used; the row's own length
    # keeps it from deciding the alignment rule
    if batch > 1:
        sizes = _recur_sizes(batch, seqlen, dim, gs[0], g_step, vs[0], v_step)
    else:
        sizes = _recur_sizes(batch, seqlen, dim, dim, g_step, dim, v_step)
    return dev, code, batch, seqlen, dim, sizes


def recur_fwd(gate, value, floor=None, valid_len=None, *, state0=None, want_final: bool = False,
              want_states: bool = False, out=None, out_final=None, stream=None):
    """The gated linear recurrence of every channel along time,

        h[t] = a[t] h[t-1] + (1 - a[t]) value[t],
        a[t] = floor + (1 - floor) sigmoid(gate[t]).

    gate, value: [batch, L, dim], fp32 or bf16, channels contiguous; rows may be
    strided (halves of the columns of one projection).  floor: fp32 [dim], in
    [0, 1], 0 when None; valid_len: int32 [batch], steps past it give 0 and leave
    the state, whatever gate and value hold there.  state0: fp32 [batch, dim], h
    before the first step (zeros when None).  Returns ``(y, final, states)``: y
    [batch, L, dim] like gate, h of every step; final fp32 [batch, dim], from
    which a next call or ``recur_step`` continues (None unless ``want_final`` or
    ``out_final``, which may be ``state0`` itself: a state carried in place);
    states fp32 [batch, chunks, dim], which ``recur_bwd`` needs (None unless
    ``want_states``)."""
    if stream is not None:
        return _on_stream(stream, recur_fwd, gate, value, floor, valid_len, state0=state0,
                          want_final=want_final, want_states=want_states, out=out,
                          out_final=out_final)
    dev, code, batch, L, dim, sizes = _recur_args(gate, value, floor, 3)
    if valid_len is not None:
        _dense(valid_len, "valid_len", (batch,), torch.int32, dev)
    if state0 is not None:
        _dense(state0, "state0", (batch, dim), _F32, dev)
    lib = load()
    y = _like(out, "out", gate, (batch, L, dim), dev)
    final = states = None
    if want_final or out_final is not None:
        final = _new(out_final, "out_final", (batch, dim), _F32, dev)
    if want_states:
        states = torch.empty((batch, lib.ssm_recur_chunks(sizes), dim), dtype=_F32, device=dev)
    _call(lib.ssm_recur_fwd, dev, gate.data_ptr(), value.data_ptr(), _addr(floor),
          _addr(valid_len), _addr(state0), y.data_ptr(), _addr(final), _addr(states), sizes, code)
    return y, final, states


def recur_bwd(gate, value, floor=None, valid_len=None, *, states, dy, dfinal=None,
              want_dstate0: bool = False, workspace=None, stream=None) -> dict:
    """Every gradient of sum(dy * y) + sum(dfinal * final) for ``recur_fwd`` on
    the same inputs: a dict of dgate and dvalue (like gate, contiguous), dfloor
    (fp32; None without a floor) and dstate0 (fp32, when wanted).  states: the
    forward's; dfinal: fp32 [batch, dim] or None.  ``workspace``, a CUDA uint8
    tensor, is only used with a floor and is allocated here when None."""
    if stream is not None:
        return _on_stream(stream, recur_bwd, gate, value, floor, valid_len, states=states, dy=dy,
                          dfinal=dfinal, want_dstate0=want_dstate0, workspace=workspace)
    dev, code, batch, L, dim, sizes = _recur_args(gate, value, floor, 3)
    lib = load()
    if valid_len is not None:
        _dense(valid_len, "valid_len", (batch,), torch.int32, dev)
    _dense(states, "states", (batch, lib.ssm_recur_chunks(sizes), dim), _F32, dev)
    _dense(dy, "dy", (batch, L, dim), gate.dtype, dev)
    if dfinal is not None:
        _dense(dfinal, "dfinal", (batch, dim), _F32, dev)
    g = {"dgate": torch.empty_like(dy), "dvalue": torch.empty_like(dy), "dfloor": None,
         "dstate0": torch.empty((batch, dim), dtype=_F32, device=dev) if want_dstate0 else None}
    ws = None
    if floor is not None:
        g["dfloor"] = torch.empty_like(floor)
        ws = _workspace(workspace, _recur_workspace(sizes), dev)
    _call(lib.ssm_recur_bwd, dev, gate.data_ptr(), value.data_ptr(), _addr(floor),
          _addr(valid_len), states.data_ptr(), dy.data_ptr(), _addr(dfinal),
          g["dgate"].data_ptr(), g["dvalue"].data_ptr(), _addr(g["dfloor"]), _addr(g["dstate0"]),
          _addr(ws), 0 if ws is None else ws.numel(), sizes, code)
    return g


def recur_step(gate, value, floor=None, *, state, out=None, stream=None):
    """One step of the recurrence on a carried state, in place (decode).

    gate, value: [batch, dim] (rows may be strided); state: fp32 [batch, dim], h
    (``recur_fwd``'s final state), advanced by the step.  Returns y [batch, dim]
    like gate."""
    if stream is not None:
        return _on_stream(stream, recur_step, gate, value, floor, state=state, out=out)
    dev, code, batch, _, dim, sizes = _recur_args(gate, value, floor, 2)
    _dense(state, "state", (batch, dim), _F32, dev)
    y = _like(out, "out", gate, (batch, dim), dev)
    _call(load().ssm_recur_step, dev, gate.data_ptr(), value.data_ptr(), _addr(floor),
          state.data_ptr(), y.data_ptr(), sizes, code)
    return y


def embed_fwd(ids, weight, *, scale: float = 1.0, ignore_index: int = -100, dtype=None, out=None,
              stream=None):
    """The embedding lookup y = scale weight[ids].

    ids: int64 [...], contiguous; weight: [vocab, dim], fp32 or bf16.  Returns y
    [..., dim] in the weight's type, or in fp32 with ``dtype`` (a residual stream
    kept in 32 bits); it is rounded once.  Tokens of ``ignore_index`` (padding) get
    rows of zeros, any other id outside the vocabulary a row of NaN."""
    if stream is not None:
        return _on_stream(stream, embed_fwd, ids, weight, scale=scale, ignore_index=ignore_index,
                          dtype=dtype, out=out)
    dev = _cuda(ids, "ids")
    if weight.dim() != 2:
        raise ValueError(f"weight: shape {tuple(weight.shape)}, expected [vocab, dim]")
    code = _code(weight.dtype)
    vocab, dim = weight.shape
    shape = ids.shape
    _dense(ids, "ids", shape, torch.int64, dev)
    _dense(weight, "weight", (vocab, dim), weight.dtype, dev)
    dtype = weight.dtype if dtype is None else dtype
    y = _new(out, "out", (*shape, dim), dtype, dev)
    _call(load().ssm_embed_fwd, dev, ids.data_ptr(), weight.data_ptr(), y.data_ptr(),
          _embed_sizes(ids.numel(), vocab, dim, int(ignore_index), float(scale), code,
                       _code(dtype)))
    return y


def embed_bwd(ids, dy, *, vocab: int | None = None, scale: float = 1.0, ignore_index: int = -100,
              dtype=None, add_to=None, workspace=None, stream=None):
    """The gradient of sum(dy * y) in the weight of ``embed_fwd``, summed in fp32
    in an order that the ids fix and rounded once.

    dy: [..., dim] for ids [...].  Returns dweight [vocab, dim] in ``dtype`` (dy's
    when None; dy may be fp32 for a bf16 weight).  With ``add_to``, [vocab, dim],
    the sums are added to it instead (the gradient of a tied output embedding,
    say) and it is returned; rows that no token names stay as they are.  Tokens of
    ``ignore_index``, and ids outside the vocabulary, take no part."""
    if stream is not None:
        return _on_stream(stream, embed_bwd, ids, dy, vocab=vocab, scale=scale,
                          ignore_index=ignore_index, dtype=dtype, add_to=add_to,
                          workspace=workspace)
    dev = _cuda(ids, "ids")
    shape = ids.shape
    _dense(ids, "ids", shape, torch.int64, dev)
    if dy.dim() < 1:
        raise ValueError("dy: no dimensions, expected [..., dim]")
    dim = dy.shape[-1]
    io = _code(dy.dtype)
    _dense(dy, "dy", (*shape, dim), dy.dtype, dev)
    if add_to is not None:
        if dtype is not None and dtype != add_to.dtype:
            raise TypeError(f"dtype: {dtype}, but add_to is {add_to.dtype}")
        if vocab is not None and add_to.shape[:1] != (vocab,):
            raise ValueError(f"vocab: {vocab}, but add_to is {tuple(add_to.shape)}")
        vocab = add_to.shape[0] if add_to.dim() else 0
        dweight = _dense(add_to, "add_to", (vocab, dim), add_to.dtype, dev)
    else:
        if vocab is None:
            raise ValueError("vocab: needed without add_to")
        dweight = torch.empty((vocab, dim), dtype=dy.dtype if dtype is None else dtype, device=dev)
    sizes = _embed_sizes(ids.numel(), vocab, dim, int(ignore_index), float(scale),
                         _code(dweight.dtype), io)
    ws = _workspace(workspace, _embed_workspace(sizes), dev)
    _call(load().ssm_embed_bwd, dev, ids.data_ptr(), dy.data_ptr(), dweight.data_ptr(),
          0 if add_to is None else 1, ws.data_ptr(), ws.numel(), sizes)
    return dweight
