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


def likely_loss(x, w, targets):
    """(loss, its bound) of rows whose target's logit is among the largest, where the loss,
    log(1 + s) of the others' sum s, is far smaller than the logits that it comes from.  A
    term of s is off by its two logits' errors, three roundings of their distance and 4 u of
    the power; the sum by one rounding of at most 1 + s for each of 32 terms and 2 steps over
    lanes, two for each strip that a lane joins (or, of few rows, for each group of 16 that a
    wave has: at most vocab / 1024 + 4), and 6 more steps over lanes; 6 for the target's
    own power, the logarithm and the sum."""
    dtype = x.dtype
    x, w = x.double(), w.double()
    dim, vocab = x.shape[1], w.shape[0]
    z = x @ w.T
    gap = z.gather(1, targets[:, None]) - z
    e = product_error(dim, dtype) * (x.abs() @ w.abs().T).amax(1, keepdim=True)
    terms = torch.exp(-gap).scatter(1, targets[:, None], 0.0)
    s = terms.sum(1)
    e_s = (terms * 1.1 * (2 * e + 3 * U32 * gap.abs() + 4 * U32)).sum(1)
    n = 32 + 2 + 2 * (vocab / 1024 + 4) + 6 + 6
    want = torch.log1p(s)
    return want, e_s / (1 + s) + n * U32 * (1 + want)


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


# --- residual root-mean-square norm ---------------------------------------

def rms_sum(x, r):
    """The sum as it is stored: one float32 addition, rounded to the stream's type."""
    return x if r is None else (x.float() + r.float()).to(x.dtype)


def rms(h, w, eps):
    """(y, rstd) in float64 of the stored sum."""
    h = h.double()
    rstd = 1 / torch.sqrt((h * h).mean(-1) + eps)
    y = h * rstd[..., None]
    return (y if w is None else y * w.double()), rstd


def rms_bounds(h, w, eps):
    """Bounds of (y before it is stored, rstd): the squares' mean is off by the sum
    and two roundings a term, rstd by half of that and 4 roundings (sum with eps,
    root, reciprocal, division by the width), y by 3 more."""
    y, rstd = rms(h, w, eps)
    rel = 0.5 * (chain(h.shape[-1]) + 2 * U32) + 5 * U32
    return y.abs() * (rel + 3 * U32) + TINY, rstd * rel


def e4m3_half_step(v):
    """Half the distance of the e4m3 values around v (|v| <= 448): 3 fraction bits
    down to 2^-6, steps of 2^-9 below."""
    e = torch.where(v == 0, -5, torch.frexp(v).exponent.clamp(min=-5))
    return torch.exp2(e.double() - 5)


def e4m3_nearest(v):
    """The e4m3 value nearest to float64 v, |v| <= 448, halves to the even one."""
    step = 2 * e4m3_half_step(v)
    return torch.round(v / step) * step        # (torch.round: halves to even)


def rows_with_ties(device=None):
    """(x, v): 128 rows whose largest values are the integers of 8 bits, one in front of
    every 128 columns, among them all values of 8 bits down to 2^-20 of it; and v = 448 x /
    max.  Many of v are middles between two e4m3 values, also where the maximum's
    reciprocal is inexact (odd multiples of 7)."""
    most = torch.arange(128, 256, device=device, dtype=torch.float64)
    h = (most * torch.exp2(-torch.arange(20, device=device, dtype=torch.float64))[:, None]).ravel()
    h[1::2] *= -1
    x = torch.where(h.abs() <= most[:, None], h, 0.0)
    x = torch.nn.functional.pad(x, (0, 21 * 127 - x.shape[1])).view(128, 21, 127)
    x = torch.cat([most[:, None, None].expand(128, 21, 1), x], 2).reshape(128, 21 * 128)
    return x, 448 * x / most[:, None]


def e4m3_scales(y, block):
    """max |y| / 448 of a row's blocks, at least 2^-126."""
    parts = [y] if block is None else y.split(block, -1)
    s = torch.stack([p.abs().amax(-1) for p in parts], -1) / 448.0
    return s.clamp(min=2.0 ** -126)


def rms_grad(dy, h, w, rstd, dh):
    """(dx, dw) in float64 from the saved statistics."""
    dy, h, rs = dy.double(), h.double(), rstd.double()[..., None]
    xh = h * rs
    g = dy if w is None else dy * w.double()
    dx = rs * (g - xh * (g * xh).mean(-1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * xh).sum(0)


def rms_grad_bounds(dy, h, w, rstd, dh, dw_dtype):
    """Bounds of (dx, dw).  xhat is off by one rounding, g by one, a term of the
    mean by three, the mean by its sum and two; dx by four more.  dw: a term's two
    roundings and a sum over rows, in parts."""
    dtype, rows, cols = dy.dtype, dy.shape[0], dy.shape[1]
    dx, dw = rms_grad(dy, h, w, rstd, dh)
    dy, h, rs = dy.double(), h.double(), rstd.double()[..., None]
    xh = h * rs
    g = dy if w is None else dy * w.double()
    c2 = (g * xh).mean(-1, keepdim=True)
    e_c2 = (chain(cols) + 4 * U32) * (g * xh).abs().mean(-1, keepdim=True) + 2 * U32 * c2.abs()
    e_dx = rs * (6 * U32 * (g.abs() + (xh * c2).abs()) + xh.abs() * e_c2) + 2 * U32 * dx.abs()
    if dh is not None:
        e_dx = e_dx + 2 * U32 * dh.double().abs()
    e_dw = (chain(rows + 64) + 3 * U32) * (dy * xh).abs().sum(0)
    return stored(dx, e_dx, dtype), stored(dw, e_dw, dw_dtype)


# --- gated feed-forward block ----------------------------------------------

def _act(kind, g):
    """(activation, slope) in float64."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    p = 0.5 * torch.erfc(-g * 0.5 ** 0.5)
    return g * p, p + g * torch.exp(-0.5 * g * g) * (2 * torch.pi) ** -0.5


def mlp(x, wg, wu, wd, kind):
    """(y, pre) in float64."""
    x = x.double()
    g, u = x @ wg.double().T, x @ wu.double().T
    return (_act(kind, g)[0] * u) @ wd.double().T, torch.cat([g, u], 1)


def _act_error(kind, g):
    """Of the activation, for an exact argument: the exponential's argument is off
    by three roundings of it (times its own slope: at most the activation and half
    its argument), the error function by two steps of one; some products."""
    a = _act(kind, g)[0].abs()
    return 8 * U32 * (g.abs() + a) + 4 * U32 * g.abs() * a


def mlp_bounds(x, wg, wu, wd, kind):
    """Bounds of (y, pre).  Both slopes are below 1.13; h is rounded to the operands'
    type before its product."""
    dtype = x.dtype
    ax, dim, hidden = x.double().abs(), x.shape[1], wg.shape[0]
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    e = product_error(dim, dtype)
    e_g, e_u = e * (ax @ wg.double().abs().T), e * (ax @ wu.double().abs().T)
    a = _act(kind, g)[0]
    e_a = 1.13 * e_g + _act_error(kind, g)
    h = a * u
    e_h = kept(e_a * (u.abs() + e_u) + a.abs() * e_u + 2 * U32 * h.abs(), h, dtype)
    awd = wd.double().abs().T.contiguous()
    e_y = e_h @ awd + product_error(hidden + 64, dtype) * ((h.abs() + e_h) @ awd)
    e_pre = torch.cat([e_g, e_u], 1)
    return (stored(h @ wd.double().T, e_y, dtype),
            stored(torch.cat([g, u], 1), e_pre, torch.float32))


def mlp_grad(dy, x, wg, wu, wd, pre, kind):
    """(dx, dwg, dwu, dwd) in float64 from the saved pre-activations."""
    dy, x = dy.double(), x.double()
    g, u = pre.double().chunk(2, 1)
    a, slope = _act(kind, g)
    dh = dy @ wd.double()
    dg, du = dh * u * slope, dh * a
    return (dg @ wg.double() + du @ wu.double(), dg.T.contiguous() @ x, du.T.contiguous() @ x,
            dy.T.contiguous() @ (a * u))


def mlp_grad_bounds(dy, x, wg, wu, wd, pre, kind, dw_dtype):
    """Bounds of (dx, dwg, dwu, dwd): dg, du and h are rounded to the operands'
    type before their products."""
    dtype = x.dtype
    want = mlp_grad(dy, x, wg, wu, wd, pre, kind)
    rows, dim, hidden = x.shape[0], x.shape[1], wg.shape[0]
    g, u = pre.double().chunk(2, 1)
    a, slope = _act(kind, g)
    ady, ax = dy.double().abs(), x.double().abs()
    dh = dy.double() @ wd.double()
    e_dh = product_error(dim, dtype) * (ady @ wd.double().abs())
    e_a, e_s = _act_error(kind, g), 16 * U32 * (1 + g.abs())
    s = slope.abs()
    dg, du, h = dh * u * slope, dh * a, a * u
    e_dg = kept(u.abs() * (e_dh * (s + e_s) + dh.abs() * e_s) + 3 * U32 * dg.abs(), dg, dtype)
    e_du = kept(e_dh * (a.abs() + e_a) + dh.abs() * e_a + 2 * U32 * du.abs(), du, dtype)
    e_h = kept(e_a * u.abs() + 2 * U32 * h.abs(), h, dtype)
    adg, adu, ah = dg.abs() + e_dg, du.abs() + e_du, h.abs() + e_h
    awg, awu = wg.double().abs(), wu.double().abs()
    e_x = (e_dg @ awg + e_du @ awu
           + product_error(2 * hidden + 64, dtype) * (adg @ awg + adu @ awu))
    p = product_error(rows + 64, dtype)
    t = lambda m: m.T.contiguous()  # noqa: E731
    errors = (e_x, t(e_dg) @ ax + p * (t(adg) @ ax), t(e_du) @ ax + p * (t(adu) @ ax),
              t(ady) @ e_h + p * (t(ady) @ ah))
    return tuple(stored(v, e, dt) for v, e, dt in zip(want, errors,
                                                      (dtype, dw_dtype, dw_dtype, dw_dtype)))
