"""The operators around the scan: short causal convolution, norm of the residual
stream, and softmax cross entropy over the vocabulary.

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

from ._binding import ConvShapes, DType, NormShapes, SsmError, XentShapes, _check, load

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
def _conv_workspace(sizes):
    return load().ssm_conv_bwd_workspace_bytes(sizes)


@functools.lru_cache(maxsize=512)
def _norm_workspace(sizes):
    return load().ssm_norm_bwd_workspace_bytes(sizes)


@functools.lru_cache(maxsize=512)
def _xent_workspace(sizes, backward):
    return load().ssm_xent_workspace_bytes(sizes, backward)


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
