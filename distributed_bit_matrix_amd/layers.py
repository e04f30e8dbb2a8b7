"""Differentiable layers for models trained with SignMuon, forward and backward
run by the HIP library (include/signmuon_layers.h).

``layer_norm`` and ``embedding`` have the parameters of a transformer whose
gradients are not matrix products; ``rms_norm`` (with the residual's addition),
``gated_mlp`` and ``linear_cross_entropy`` (which keeps no logits) are what comes
after them in a gated one.  All gradients are sums in a fixed order (no
floating-point atomics), so replicas that vote on the signs of the same gradient
see the same bits.  They are functions of tensors; ``LayerNorm``, ``Embedding``,
``RMSNorm``, ``GatedMLP`` and ``LinearCrossEntropy`` are modules over them.

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


def _grad_arrays(ctx, slots, wants, first, likes):
    """What a backward pass writes its weights' gradients to: (arrays, None for a
    new one; direct slots; the owners that have to live until they are written;
    add; dtype).  The weights are tensor inputs `first` and on."""
    owners = [_direct(ctx, first + i, s) if want else None
              for i, (s, want) in enumerate(zip(slots, wants))]
    direct = [None if o is None else s for o, s in zip(owners, slots)]
    held = [s for s in direct if s is not None]
    if len(set(map(id, held))) < len(held):      # one parameter in two places
        direct = [None] * len(direct)
        held = []
    if not held:
        return [None] * len(direct), direct, owners, False, likes[0][1]
    add = any(s.filled for s in held)
    arrays = []
    for s, want, (shape, _, device) in zip(direct, wants, likes):
        if s is not None:
            arrays.append(s.open(add).view(shape))
        elif want and add:
            arrays.append(torch.zeros(shape, dtype=torch.float32, device=device))
        else:
            arrays.append(None)
    return arrays, direct, owners, add, torch.float32


def _grads_out(direct, grads, likes):
    """The gradients to return: None for those that went to their slots."""
    out = []
    for s, g, (_, dtype, _) in zip(direct, grads, likes):
        if s is not None:
            s.close()
            g = None
        out.append(g if g is None else g.to(dtype))
    return out


def _like(t):
    return (t.shape, t.dtype, t.device)


class _RMSNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps, slot):
        x = _dense_rows(x)
        if residual is not None:
            residual = _dense_rows(residual)
        y, h, rstd = B.rms_norm(x, weight, residual, eps, want_stats=True)
        ctx.save_for_backward(h, weight, rstd)
        ctx.slot = slot
        ctx.set_materialize_grads(False)
        return y if residual is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight, rstd = ctx.saved_tensors
        want_w = ctx.needs_input_grad[1]
        want_x = ctx.needs_input_grad[0] or ctx.needs_input_grad[2]
        if dy is None:               # the sum alone was used
            return (dh if ctx.needs_input_grad[0] else None, None,
                    dh if ctx.needs_input_grad[2] else None, None, None)
        dh = None if dh is None else _dense_rows(dh)
        dw, direct, owners, add, dtype = [None], [None], None, False, None
        if want_w:
            dw, direct, owners, add, dtype = _grad_arrays(ctx, [ctx.slot], [True], 1,
                                                          [_like(weight)])
        dx, g = B.rms_norm_backward(_dense_rows(dy), h, weight, rstd, dh, want_x, want_w,
                                    dweight=dw[0], dtype=dtype, accumulate=add)
        if want_w:
            g, = _grads_out(direct, [g], [_like(weight)])
        return (dx if ctx.needs_input_grad[0] else None, g,
                dx if ctx.needs_input_grad[2] else None, None, None)


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6):
    """Root-mean-square norm over x's last dimension, times weight: y.  With a
    residual (of x's shape and dtype) the norm is taken of h = x + residual, and
    (y, h) returned: h is the residual of the next layer.  x: float32 or bfloat16,
    of any leading shape."""
    if _followed(x, weight, residual):
        return _RMSNorm.apply(x, weight, residual, eps, _slot(weight))
    return B.rms_norm(_dense_rows(x), weight, None if residual is None else _dense_rows(residual),
                      eps)


class _GatedMLP(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, slots):
        x = _dense_rows(x)
        y, pre = B.gated_mlp(x, w_gate, w_up, w_down, activation, want_pre=True)
        ctx.save_for_backward(x, w_gate, w_up, w_down, pre)
        ctx.activation, ctx.slots = activation, slots
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, pre = ctx.saved_tensors
        wants = ctx.needs_input_grad[1:4]
        likes = [_like(w) for w in (w_gate, w_up, w_down)]
        dw, direct, owners, add, dtype = _grad_arrays(ctx, ctx.slots, wants, 1, likes)
        dx, *grads = B.gated_mlp_backward(
            _dense_rows(dy), x, w_gate, w_up, w_down, pre, ctx.activation,
            want=(ctx.needs_input_grad[0], *wants), dw_gate=dw[0], dw_up=dw[1], dw_down=dw[2],
            dtype=dtype, accumulate=add)
        return (dx, *_grads_out(direct, grads, likes), None, None)


def gated_mlp(x, w_gate, w_up, w_down, activation: str = "silu"):
    """(act(x w_gate^T) * (x w_up^T)) w_down^T over x's last dimension; activation
    "silu" or "gelu".  x: float32 or bfloat16, of any leading shape; the weights are
    of its dtype: (hidden, dim) twice and (dim, hidden).  A pass with gradients keeps
    the two pre-activations in float32."""
    w_gate, w_up, w_down = w_gate.contiguous(), w_up.contiguous(), w_down.contiguous()
    if _followed(x, w_gate, w_up, w_down):
        return _GatedMLP.apply(x, w_gate, w_up, w_down, activation,
                               (_slot(w_gate), _slot(w_up), _slot(w_down)))
    return B.gated_mlp(_dense_rows(x), w_gate, w_up, w_down, activation)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, targets, ignore_index, reduction, slot):
        x = _dense_rows(x)
        loss, lse = B.linear_cross_entropy(x, weight, targets, ignore_index, reduction,
                                           want_lse=True)
        ctx.save_for_backward(x, weight, targets, lse)
        ctx.call = (ignore_index, reduction, slot)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        x, weight, targets, lse = ctx.saved_tensors
        ignore_index, reduction, slot = ctx.call
        want_x, want_w = ctx.needs_input_grad[:2]
        dw, direct, owners, add, dtype = _grad_arrays(ctx, [slot], [want_w], 1, [_like(weight)])
        dx, g = B.linear_cross_entropy_backward(
            dloss.contiguous(), x, weight, targets, lse, ignore_index, reduction, want_x, want_w,
            dweight=dw[0], dtype=dtype, accumulate=add)
        return (dx, *_grads_out(direct, [g], [_like(weight)]), None, None, None, None)


def linear_cross_entropy(x, weight, targets, ignore_index: int = -100, reduction: str = "mean"):
    """Softmax cross entropy of the logits x weight^T against integer targets of x's
    leading shape, in float32; the logits are not kept, in either pass.  Rows whose
    target is ignore_index count nowhere, whatever they hold.  reduction: "mean" (0
    where no row counts), "sum" or "none".  weight: (vocab, dim) of x's dtype, for
    instance an embedding's table.  A target outside the table makes its row's loss
    and gradients NaN."""
    weight, targets = weight.contiguous(), targets.contiguous()
    if _followed(x, weight):
        return _LinearCrossEntropy.apply(x, weight, targets, int(ignore_index), reduction,
                                         _slot(weight))
    return B.linear_cross_entropy(_dense_rows(x), weight, targets, ignore_index, reduction)


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


class RMSNorm(torch.nn.Module):
    """rms_norm with a weight (ones at first) of the given width."""

    def __init__(self, width: int, eps: float = 1e-6, device=None, dtype=None):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))

    def forward(self, x, residual=None):
        return rms_norm(x, self.weight, residual, self.eps)


class GatedMLP(torch.nn.Module):
    """gated_mlp with weights drawn from N(0, 1 / columns)."""

    def __init__(self, dim: int, hidden: int, activation: str = "silu", device=None, dtype=None):
        super().__init__()
        self.activation = activation

        def weight(rows, cols):
            return torch.nn.Parameter(
                torch.empty(rows, cols, device=device, dtype=dtype).normal_(std=cols ** -0.5))

        self.w_gate, self.w_up = weight(hidden, dim), weight(hidden, dim)
        self.w_down = weight(dim, hidden)

    def forward(self, x):
        return gated_mlp(x, self.w_gate, self.w_up, self.w_down, self.activation)


class LinearCrossEntropy(torch.nn.Module):
    """linear_cross_entropy with a weight of vocab x dim, drawn from N(0, 0.02^2), or
    with the one given (an embedding's, to share it)."""

    def __init__(self, vocab: int, dim: int, ignore_index: int = -100, reduction: str = "mean",
                 weight: Optional[torch.nn.Parameter] = None, device=None, dtype=None):
        super().__init__()
        if weight is not None and tuple(weight.shape) != (vocab, dim):
            raise ValueError("weight must be vocab x dim")
        self.ignore_index, self.reduction = ignore_index, reduction
        self.weight = torch.nn.Parameter(
            torch.empty(vocab, dim, device=device, dtype=dtype).normal_(std=0.02)
        ) if weight is None else weight

    def forward(self, x, targets):
        return linear_cross_entropy(x, self.weight, targets, self.ignore_index, self.reduction)
