"""The selective scan and the operators around it as differentiable PyTorch
functions.

``selective_scan`` runs the library's forward (``scan_fwd``), keeping the
chunk boundary states the backward replays from, and its backward
(``scan_bwd``) when autograd asks for gradients: the recompute scheme of [P1]
s3.4 (only the chunk states are stored between the two passes).  This module
only passes tensors between PyTorch and the C ABI; every step of both passes
runs in the library's kernels.  The gradients themselves have no derivatives:
differentiating them again (after create_graph=True) raises a RuntimeError.
"""
import functools

import torch

from ._binding import scan_bwd, scan_fwd
from .layers import conv_bwd, conv_fwd, norm_bwd, norm_fwd, xent_bwd, xent_fwd


class _Final(torch.autograd.Function):
    """Passes gradients on, tied to the tensors they were computed from, and refuses
    to be differentiated."""

    @staticmethod
    def forward(ctx, name, count, *tensors):
        ctx.name = name
        return tuple(None if t is None else t.detach() for t in tensors[count:])

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name}: its gradients cannot be differentiated again")


def _once(name):
    """Marks the backward of the function that users call `name`.  With
    create_graph=True its results depend on the incoming gradients and on what the
    forward saved, which PyTorch cannot see inside a kernel: without the mark a
    second derivative would take them for constants, silently."""
    def mark(backward):
        @functools.wraps(backward)
        def marked(ctx, *grads):
            if not torch.is_grad_enabled():
                return backward(ctx, *grads)
            with torch.no_grad():
                out = backward(ctx, *grads)
            tied = [t for t in (*grads, *ctx.saved_tensors) if t is not None and t.requires_grad]
            return _Final.apply(name, len(tied), *tied, *out) if tied else out
        return marked
    return mark


class _SelectiveScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, delta, A, B, C, D, z, valid_len, h0, chunk_len):
        y, states = scan_fwd(x, delta, A, B, C, D, z, valid_len, chunk_len=chunk_len, h0=h0)
        ctx.save_for_backward(x, delta, A, B, C, D, z, valid_len, h0, states)
        ctx.chunk_len = chunk_len
        return y

    @staticmethod
    @_once("selective_scan")
    def backward(ctx, dy):
        x, delta, A, B, C, D, z, valid_len, h0, states = ctx.saved_tensors
        want_dh0 = h0 is not None and ctx.needs_input_grad[8]
        g = scan_bwd(x, delta, A, B, C, D, z, valid_len, chunk_states=states,
                     chunk_len=ctx.chunk_len, dy=dy.contiguous(), h0=h0, want_dh0=want_dh0)
        # B and C share the I/O dtype; their gradients are summed in fp32
        dB = g["dB"].to(B.dtype)
        dC = g["dC"].to(C.dtype)
        return (g["dx"], g["ddelta"], g["dA"], dB, dC, g["dD"], g["dz"], None,
                g["dh0"] if want_dh0 else None, None)


def selective_scan(x, delta, A, B, C, D=None, z=None, valid_len=None, *, h0=None,
                   chunk_len: int = 256):
    """y = the selective scan of the inputs (as ``scan_fwd``), differentiable in
    x, delta, A, B, C, D, z and h0.  ``chunk_len`` (1 .. 512) is the spacing of
    the boundary states kept for the backward: a multiple of 16 lets the
    backward take its tiled kernel."""
    return _SelectiveScan.apply(x, delta, A, B, C, D, z, valid_len, h0, int(chunk_len))


class _CausalConv(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, valid_len, state0, silu):
        ctx.save_for_backward(x, weight, bias, valid_len, state0)
        ctx.silu = silu
        return conv_fwd(x, weight, bias, valid_len, state0=state0, silu=silu)

    @staticmethod
    @_once("causal_conv")
    def backward(ctx, dy):
        x, weight, bias, valid_len, state0 = ctx.saved_tensors
        g = conv_bwd(x, weight, bias, valid_len, dy=dy.contiguous(), state0=state0, silu=ctx.silu,
                     want_dstate0=state0 is not None and ctx.needs_input_grad[4])
        return g["dx"], g["dweight"], g["dbias"], None, g["dstate0"], None


def causal_conv(x, weight, bias=None, valid_len=None, *, state0=None, silu: bool = True):
    """y = the short causal convolution of x (as ``conv_fwd``), differentiable in
    x, weight, bias and state0."""
    return _CausalConv.apply(x, weight, bias, valid_len, state0, bool(silu))


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, residual, rms, eps):
        y, r, stats = norm_fwd(x, weight, bias, residual=residual, rms=rms, eps=eps,
                               want_stats=True)
        ctx.save_for_backward(x if r is None else r, weight, stats)
        ctx.rms, ctx.bias, ctx.x_dtype = rms, bias is not None, x.dtype
        ctx.set_materialize_grads(False)
        return y, r

    @staticmethod
    @_once("layer_norm")
    def backward(ctx, dy, dr):
        r, weight, stats = ctx.saved_tensors
        dy = torch.zeros(r.shape, dtype=ctx.x_dtype, device=r.device) if dy is None else dy
        g = norm_bwd(r, weight, stats=stats, dy=dy.contiguous(),
                     dr=None if dr is None else dr.contiguous(), rms=ctx.rms, want_dbias=ctx.bias)
        return (g["dx"], g["dweight"], g["dbias"],
                g["dresidual"] if ctx.needs_input_grad[3] else None, None, None)


def layer_norm(x, weight, bias=None, *, residual=None, rms: bool = False, eps: float = 1e-5):
    """The norm of x (as ``norm_fwd``), differentiable in x, weight, bias and
    residual.  Returns y, or ``(y, r)`` with a residual, r = x + residual being
    the stream that the next layer adds to."""
    y, r = _LayerNorm.apply(x, weight, bias, residual, bool(rms), float(eps))
    return y if residual is None else (y, r)


class _CrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, weight, targets, ignore_index):
        loss, lse = xent_fwd(h, weight, targets, ignore_index=ignore_index)
        ctx.save_for_backward(h, weight, targets, lse)
        ctx.ignore_index = ignore_index
        return loss

    @staticmethod
    @_once("linear_cross_entropy")
    def backward(ctx, dloss):
        h, weight, targets, lse = ctx.saved_tensors
        g = xent_bwd(h, weight, targets, lse=lse, dloss=dloss.contiguous(),
                     ignore_index=ctx.ignore_index)
        return g["dh"], g["dweight"], None, None


def linear_cross_entropy(h, weight, targets, *, ignore_index: int = -100, reduction: str = "mean"):
    """Softmax cross entropy over the vocabulary of the logits h weight^T, which
    are never kept (as ``xent_fwd``), differentiable in h and weight.  h: bf16
    [..., dim], targets: int64 [...] or flat, [tokens].  ``reduction``: "mean" over the tokens that
    are not ignored (0 when all are), "sum", or "none" for the losses like
    targets."""
    if reduction not in ("mean", "sum", "none"):
        raise ValueError(f"reduction: {reduction!r}, expected 'mean', 'sum' or 'none'")
    if targets.dim() != 1 and targets.shape != h.shape[:-1]:
        raise ValueError(f"targets: shape {tuple(targets.shape)}, expected {tuple(h.shape[:-1])}")
    loss = _CrossEntropy.apply(h.reshape(-1, h.shape[-1]), weight, targets.reshape(-1),
                               int(ignore_index))
    if reduction == "none":
        return loss.view(targets.shape)
    total = loss.sum()
    return total if reduction == "sum" else total / (targets != ignore_index).sum().clamp(min=1)
