"""The residual norm, the gated feed-forward block and the linear cross entropy in
64 bits, with error bounds for the library's float32 evaluation (not a test
module; torch in float64 on the inputs' device, shares nothing with the library).

Bounds are built as in tests/layer_reference.py: u = 2^-24; a float32 sum of n
terms, in any order, is off by at most chain(n) = 2 n u times the sum of their
absolute values; a stored value by half a step.  Products of bfloat16 operands
are exact in float32.  A float32 product is summed from three bfloat16 planes of
either operand: a plane is at most 2^-8 of the one before it, so what the planes
leave and the three pairs that are left out come to 2^-24 of |a b| each, five in
all with what is of higher order, and there are six times as many terms.
"""
import torch

U32 = 2.0 ** -24
TINY = 2.0 ** -126
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def chain(n):
    return 2.0 * n * U32


def stored(v, err, dtype):
    """Bound of a value v, computed within err, once it is stored in dtype."""
    return err + HALF_STEP[dtype] * (v.abs() + err) + TINY


def product_error(k, dtype):
    """Relative to the product of absolute values."""
    return chain(k) if dtype == torch.bfloat16 else chain(6 * k) + 5 * U32


def kept(err, v, dtype):
    """Bound of an operand v of a second product, computed within err, once it is
    rounded to the operands' type."""
    return stored(v, err, dtype)


# --- linear cross entropy -------------------------------------------------

def loss(x, w, targets, ignore):
    """(loss of every row, lse) in float64."""
    x, w = x.double(), w.double()
    keep = targets != ignore
    ok = keep & (targets >= 0) & (targets < w.shape[0])
    z = x @ w.T
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    picked = z.gather(1, torch.where(ok, targets, 0)[:, None])[:, 0]
    each = torch.where(ok, lse - picked, torch.nan)
    zero = torch.zeros_like(lse)
    return torch.where(keep, each, zero), torch.where(keep, lse, zero)


def loss_bounds(x, w, targets, ignore):
    """Bounds of the errors of (loss of every row, lse).  A logit is off by e; a
    term of the sum, exp(z - top), by e of z and three roundings of its argument
    (both factors of it and the power of two's), 4 u more from the power itself.
    The sum has 32 terms a lane, 2 steps over lanes, then strips of 64 or 128
    logits by 64 lanes, two roundings a step, and 6 steps over those.  lse adds
    a logarithm and a sum."""
    dtype = x.dtype
    x, w = x.double(), w.double()
    dim, vocab = x.shape[1], w.shape[0]
    z = x @ w.T
    e = product_error(dim, dtype) * (x.abs() @ w.abs().T)
    top = z.amax(1, keepdim=True)
    p = torch.softmax(z, 1)
    terms = chain(32 + 2 + 4 * (vocab / 64 / 64 + 1) + 6 + 4)
    e_lse = (p * (e + 3 * U32 * (z - top).abs())).sum(1) * 1.1 + terms
    e_lse = e_lse + e.amax(1) * 2 ** -6
    top = top[:, 0].abs()
    ln = torch.log(torch.exp(z - z.amax(1, keepdim=True)).sum(1)).abs()
    e_lse = e_lse + 4 * U32 * (top + ln + 1)
    at = targets.clamp(0, vocab - 1)[:, None]
    e_each = e_lse + e.gather(1, at)[:, 0] + 4 * U32 * z.gather(1, at)[:, 0].abs()
    keep = targets != ignore
    zero = torch.zeros_like(e_lse)
    return torch.where(keep, e_each, zero) + TINY, torch.where(keep, e_lse, zero) + TINY


def reduce_loss(each, targets, ignore, reduction):
    if reduction == "none":
        return each
    total = each.sum()
    if reduction == "mean":
        total = total / max(1, int((targets != ignore).sum()))
    return total


def _loss_g(dloss, x, w, targets, lse, ignore, reduction):
    """(G, its error before it is rounded) of the rows that count."""
    keep = targets != ignore
    live = int(keep.sum())
    z = x.double() @ w.double().T
    e = product_error(x.shape[1], x.dtype) * (x.double().abs() @ w.double().abs().T)
    arg = z - lse.double()[:, None]
    p = torch.exp(arg)
    hot = torch.zeros_like(p)
    hot.scatter_(1, targets.clamp(0, w.shape[0] - 1)[:, None], 1.0)
    scale = dloss.double().expand(targets.shape)
    if reduction == "mean":
        scale = scale / max(1, live)
    scale = torch.where(keep, scale, 0.0)[:, None]
    g = torch.where(keep[:, None], (p - hot) * scale, 0.0)
    # the argument's three roundings, the power, the difference and two more
    e_g = torch.where(keep[:, None],
                      scale.abs() * (p * (1.1 * e + 3 * U32 * arg.abs() + 6 * U32)
                                     + 4 * U32 * (p - hot).abs()), 0.0)
    return g, e_g


def loss_grad(dloss, x, w, targets, lse, ignore, reduction):
    """(dx, dw) in float64; rows that do not count add nothing, whatever they hold."""
    keep = (targets != ignore)[:, None]
    x = torch.where(keep, x, torch.zeros_like(x))
    g, _ = _loss_g(dloss, x, w, targets, lse, ignore, reduction)
    return g @ w.double(), g.T.contiguous() @ x.double()


def loss_grad_bounds(dloss, x, w, targets, lse, ignore, reduction, dw_dtype):
    """Bounds of (dx, dw): G is rounded to the operands' type."""
    dtype = x.dtype
    keep = (targets != ignore)[:, None]
    x = torch.where(keep, x, torch.zeros_like(x))
    g, e_g = _loss_g(dloss, x, w, targets, lse, ignore, reduction)
    e_g = torch.where(keep, kept(e_g, g, dtype), 0.0)
    ax, aw, ag = x.double().abs(), w.double().abs(), g.abs() + e_g
    rows, vocab = g.shape
    # splits and pieces are joined: a few more terms
    e_x = e_g @ aw + product_error(vocab + 64, dtype) * (ag @ aw)
    e_w = e_g.T.contiguous() @ ax + product_error(rows + 64, dtype) * (ag.T.contiguous() @ ax)
    return (stored(g @ w.double(), e_x, dtype),
            stored(g.T.contiguous() @ x.double(), e_w, dw_dtype))
