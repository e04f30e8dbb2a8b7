"""Differentiable layer norm and embedding for models trained with SignMuon,
forward and backward run by the HIP library (include/signmuon_layers.h).

Of a transformer's parameters these are the ones whose gradients are not
matrix products.  Both gradients are sums in a fixed order (no
floating-point atomics), so replicas that vote on the signs of the same
gradient see the same bits.  ``layer_norm`` and ``embedding`` are functions of
tensors; ``LayerNorm`` and ``Embedding`` are modules over them.

Under an optimizer made with ``SignMuon(..., direct_grads=True)`` the backward
passes write the parameter gradients in float32 straight into the flat array
that the step reads (see ``optim``); ``p.grad`` stays None then.  Otherwise, in
``torch.autograd.grad`` and while a HIP graph is being captured, they return
them in the parameter's dtype as any other operator does.  The gradients cannot
be differentiated again, and there are no forward-mode derivatives.
"""
from __future__ import annotations

from typing import Optional

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import binding as B


def _dense_rows(t):
    """t itself where the library takes its strides, else a contiguous copy."""
    try:
        B._rows(t, "t")
    except TypeError:
        return t.contiguous()
    return t


def _followed(*inputs) -> bool:
    """Whether a gradient, a tangent or a trace follows a call on these inputs.
    The kernels are hidden from all three, so it goes through the autograd
    function: that gives the gradient, refuses the tangent and is what a trace
    records."""
    if torch.jit.is_tracing():
        return True
    grad = torch.is_grad_enabled()
    return any(t is not None and (grad and t.requires_grad
                                  or forward_ad.unpack_dual(t).tangent is not None)
               for t in inputs)


def _slot(p):
    return None if p is None else p.__dict__.get("_signmuon_slot")


def _accumulates(ctx, i) -> bool:
    """Whether this backward pass adds to the grad of tensor input i (inputs
    that are None or no tensors are not counted), a leaf: not where
    backward(inputs=...) leaves it out, nor in torch.autograd.grad, which hands
    the gradient to its caller (or drops it)."""
    try:
        return torch._C._will_engine_execute_node(ctx.next_functions[i][0])
    except RuntimeError:      # the engine's answer where grad() asks for the leaf
        return False


def _direct(ctx, i, slot):
    """The owner of the slot that the gradient of tensor input i goes to, to be
    held until it is written; None where it does not: once the optimizer is
    gone, or in a graph, whose replays would not tell the optimizer what they
    wrote."""
    owner = None if slot is None else slot.owner()
    if owner is None or not _accumulates(ctx, i) or torch.cuda.is_current_stream_capturing():
        return None
    return owner


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, slots):
        x = _dense_rows(x)
        y, mean, rstd = B.layer_norm(x, weight, bias, eps, want_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias_dtype = None if bias is None else bias.dtype
        ctx.slots = slots
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        want_x, want_w, want_b = ctx.needs_input_grad[:3]
        dw = db = dtype = None
        add = False
        owners = [_direct(ctx, i, s) if want else None
                  for i, s, want in zip((1, 1 + (weight is not None)), ctx.slots,
                                        (want_w, want_b))]
        direct = [None if o is None else s for o, s in zip(owners, ctx.slots)]
        if direct[0] is direct[1]:      # one parameter as weight and bias
            direct = [None, None]
        if any(direct):
            dtype = torch.float32
            add = any(s is not None and s.filled for s in direct)
            out = []
            for s, want in zip(direct, (want_w, want_b)):
                if s is not None:
                    out.append(s.open(add))
                elif want:
                    out.append(torch.zeros(x.shape[-1], dtype=dtype, device=x.device))
                else:
                    out.append(None)
            dw, db = out
        elif want_w or want_b:
            dtype = weight.dtype if want_w else ctx.bias_dtype
        dx, dw, db = B.layer_norm_backward(
            _dense_rows(dy), x, weight, mean, rstd, want_x, want_w, want_b, dweight=dw, dbias=db,
            dtype=dtype, accumulate=add)
        grads = []
        for g, s, like in ((dw, direct[0], None if weight is None else weight.dtype),
                           (db, direct[1], ctx.bias_dtype)):
            if s is not None:
                s.close()
                g = None
            grads.append(g if g is None else g.to(like))
        return dx, grads[0], grads[1], None, None


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5):
    """Layer norm over x's last dimension, times weight plus bias (vectors of
    one dtype, or None).  x: float32 or bfloat16, of any leading shape."""
    if _followed(x, weight, bias):
        return _LayerNorm.apply(x, weight, bias, eps, (_slot(weight), _slot(bias)))
    return B.layer_norm(_dense_rows(x), weight, bias, eps)


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, padding_idx, slot):
        ctx.save_for_backward(tokens)
        ctx.table = (weight.shape[0], weight.dtype, scale, padding_idx, slot)
        return B.embedding(tokens, weight, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        tokens, = ctx.saved_tensors
        vocab, dtype, scale, padding, slot = ctx.table
        dy = _dense_rows(dy)
        owner = _direct(ctx, 1, slot)
        if owner is not None:
            add = slot.filled
            B.embedding_backward(dy, tokens, vocab, scale, padding, dW=slot.open(add),
                                 accumulate=add)
            slot.close()
            return None, None, None, None, None
        dw = B.embedding_backward(dy, tokens, vocab, scale, padding, dtype=dtype)
        return None, dw, None, None, None


def embedding(tokens, weight, scale: float = 1.0, padding_idx: Optional[int] = None):
    """scale * weight[tokens] for integer tokens of any shape.  Rows of
    padding_idx are looked up but get no gradient.  A token outside the table
    makes its row NaN and adds nothing to the gradient."""
    if padding_idx is not None and not 0 <= padding_idx < weight.shape[0]:
        raise ValueError("padding_idx must lie in the table")
    tokens = tokens.contiguous()
    if _followed(weight):
        return _Embedding.apply(tokens, weight.contiguous(), float(scale), padding_idx,
                                _slot(weight))
    return B.embedding(tokens, weight.contiguous(), scale)


class LayerNorm(torch.nn.Module):
    """layer_norm with weight (ones at first) and, unless bias is False, bias
    (zeros) of the given width."""

    def __init__(self, width: int, eps: float = 1e-5, bias: bool = True, device=None,
                 dtype=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        self.bias = (torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype))
                     if bias else None)

    def forward(self, x):
        return layer_norm(x, self.weight, self.bias, self.eps)


class Embedding(torch.nn.Module):
    """embedding with a table of vocab x dim, drawn from N(0, 0.02^2)."""

    def __init__(self, vocab: int, dim: int, scale: float = 1.0,
                 padding_idx: Optional[int] = None, device=None, dtype=None):
        super().__init__()
        self.scale = scale
        self.padding_idx = padding_idx
        self.weight = torch.nn.Parameter(
            torch.empty(vocab, dim, device=device, dtype=dtype).normal_(std=0.02))

    def forward(self, tokens):
        return embedding(tokens, self.weight, self.scale, self.padding_idx)
