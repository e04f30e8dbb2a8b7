"""Layer norm and embedding in 64 bits, with error bounds for a float32
evaluation (not a test module; NumPy only, shares nothing with the library).

u = 2^-24 is float32's unit roundoff.  A sum of n float32 terms, in any order
and with any rounding of its partial sums, is off by at most n u sum|term| to
first order (n - 1 additions, each off by u times a partial sum of absolute
values); 2 n u covers the higher orders for n < 2^22.  A result stored in a
dtype is off by at most half a step: u |v| in float32, 2^-8 |v| in bfloat16.
"""
import numpy as np

U32 = 2.0 ** -24
TINY = 2.0 ** -126       # results below the normal range are off by less
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def chain(n):
    """Relative error of a float32 sum of n terms against sum|term|."""
    return 2.0 * n * U32


def bf16_values(x):
    """float32 values rounded to bfloat16, nearest even (finite input)."""
    b = np.ascontiguousarray(np.asarray(x, np.float32)).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)).astype(np.uint32).view(
        np.float32)


def stored(v, err, dtype):
    """Bound of a value v, computed within err, once it is stored in dtype."""
    return err + HALF_STEP[dtype] * (np.abs(v) + err) + TINY


def norm(x, gamma, beta, eps):
    """(y, mean, rstd) in float64; gamma and beta may be None."""
    x = np.asarray(x, np.float64)
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = 1.0 / np.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[..., None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def norm_bounds(x, gamma, beta, eps, dtype):
    """Bounds of |y|, |mean| and |rstd| errors.  mean: a sum of cols terms and
    a division.  The deviations inherit mean's error e and one rounding; the
    squares' mean is off by e^2 (the deviations themselves sum to zero), two
    roundings a term and the sum.  rstd: half of that, relatively, and 4
    roundings (sum with eps, root, reciprocal).  y: 4 more."""
    y, mean, rstd = norm(x, gamma, beta, eps)
    x = np.asarray(x, np.float64)
    n = x.shape[-1]
    e_mean = chain(n) * np.abs(x).mean(-1) + 2 * U32 * np.abs(mean)
    d = np.abs(x - mean[..., None])
    var = (d * d).mean(-1)
    e_var = 2 * e_mean ** 2 + (chain(n) + 8 * U32) * var
    r = 0.5 * e_var / (var + eps) * 2 + 8 * U32
    g = 1.0 if gamma is None else np.abs(np.asarray(gamma, np.float64))
    e_y = g * rstd[..., None] * ((1 + r[..., None]) * e_mean[..., None]
                                 + d * (r[..., None] + 8 * U32))
    e_y = e_y + 4 * U32 * np.abs(y)
    if beta is not None:
        e_y = e_y + 4 * U32 * np.abs(np.asarray(beta, np.float64))
    return stored(y, e_y, dtype), e_mean + TINY, r * rstd


def norm_grad(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta) in float64 from the saved statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rs = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * rs
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    n = x.shape[1]
    dx = rs * (g - g.sum(1, keepdims=True) / n - xh * ((g * xh).sum(1, keepdims=True) / n))
    return dx, (dy * xh).sum(0), dy.sum(0)


def norm_grad_bounds(dy, x, gamma, mean, rstd, dtype, dw_dtype, before=(0.0, 0.0)):
    """Bounds of the errors of dx, dgamma and dbeta.  xhat carries two
    roundings and g one; the two row means are sums of cols terms; dx is put
    together with at most 6 more.  dgamma's terms carry three."""
    dx, dg, db = norm_grad(dy, x, gamma, mean, rstd)
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    rs = np.asarray(rstd, np.float64)[:, None]
    xh = np.abs((x - np.asarray(mean, np.float64)[:, None]) * rs)
    g = np.abs(dy if gamma is None else dy * np.asarray(gamma, np.float64))
    n, rows = x.shape[1], x.shape[0]
    m1, m2 = g.mean(1, keepdims=True), (g * xh).mean(1, keepdims=True)
    e = rs * ((chain(n) + 8 * U32) * (m1 + xh * m2) + 8 * U32 * g)
    e_g = (chain(rows) + 8 * U32) * (np.abs(dy) * xh).sum(0) + U32 * np.abs(before[0])
    e_b = chain(rows) * np.abs(dy).sum(0) + U32 * np.abs(before[1])
    return (stored(dx, e, dtype), stored(dg + before[0], e_g, dw_dtype),
            stored(db + before[1], e_b, dw_dtype))


def embed(w, tokens, scale):
    """scale * w[tokens]; rows of tokens outside the table are NaN."""
    w, tokens = np.asarray(w, np.float64), np.asarray(tokens)
    ok = (tokens >= 0) & (tokens < len(w))
    out = scale * w[np.where(ok, tokens, 0)]
    out[~ok] = np.nan
    return out


def embed_grad(dy, tokens, vocab, scale, padding=None):
    """(dW, sum of |terms|, terms) of every row of the table, in float64."""
    dy, tokens = np.asarray(dy, np.float64), np.asarray(tokens).reshape(-1)
    ok = (tokens >= 0) & (tokens < vocab)
    if padding is not None:
        ok &= tokens != padding
    dw = np.zeros((vocab, dy.shape[1]))
    mag = np.zeros_like(dw)
    np.add.at(dw, tokens[ok], dy[ok])
    np.add.at(mag, tokens[ok], np.abs(dy[ok]))
    return scale * dw, abs(scale) * mag, np.bincount(tokens[ok], minlength=vocab)


def embed_grad_bounds(dw, mag, counts, dtype, before=0.0):
    """A sum of `counts` terms, the scale's rounding, and the addition to what
    was there."""
    err = (chain(counts)[:, None] + 2 * U32) * mag + U32 * np.abs(before)
    return stored(dw + before, err, dtype)


# --------------------------------------------------------------------------
# Inputs whose sums are exact: small integers times powers of two, so that every
# partial sum is an integer below 2^24 in units of its row or column, in
# whatever order it is taken.  What is lost from a sum shows then, however
# many terms the sum has, where a bound for inexact ones grows with their
# number.
# --------------------------------------------------------------------------
def pattern(cols):
    """1, -1, 1, -1, ..., and a last 0 if cols is odd: it and its products with
    constants sum to 0, also over any run of pairs."""
    p = np.where(np.arange(cols) % 2 == 0, 1.0, -1.0)
    if cols % 2:
        p[-1] = 0.0
    return p


def exact_norm(rows, cols, eps, dtype):
    """x, (y, mean, rstd) and their bounds, without weights.  Row r is 2^k (2 +
    pattern), k = r mod 8: the mean is 2^(k+1) exactly, the deviations and
    their squares are exact, and the sum of squares is 4^k times the number of
    nonzero entries.  The variance then takes up to 2 roundings (times the
    rounded reciprocal of cols; or one, divided by cols), eps one, the root
    halves these 3, and the root and the reciprocal add one each: 3.5.  y
    adds one."""
    p = pattern(cols)
    k = 2.0 ** (np.arange(rows) % 8)[:, None]
    x = (k * (2 + p)).astype(np.float32)
    rstd = 1 / np.sqrt(k[:, 0] ** 2 * ((p != 0).sum() / cols) + eps)
    y = k * p * rstd[:, None]
    return x, (y, 2 * k[:, 0], rstd), (stored(y, 5 * U32 * np.abs(y), dtype),
                                       0 * rstd, 4 * U32 * rstd)


def exact_norm_grad(rows, cols, dtype):
    """dy, x, (dx, dgamma, dbeta) and dx's bound, for mean 0, rstd 1 and no
    gamma; dgamma and dbeta are exact.  xhat is the pattern p; dy is 2, 3 p and
    1 + 2 p in turn, times 2^(r mod 4).  Both row sums are exact; their means
    take 2 roundings at most (times the rounded reciprocal of cols), and dx is
    put together with 3 more."""
    assert rows * 8 * 3 < 2 ** 24 and cols * 8 * 3 <= 3 * 2 ** 23
    p = pattern(cols)
    r = np.arange(rows)
    kinds = np.stack([0 * p + 2, 3 * p, 1 + 2 * p])
    dy = kinds[r % 3] * 2.0 ** (r % 4)[:, None]
    x = np.broadcast_to(p, (rows, cols))
    c1, c2 = dy.mean(1, keepdims=True), (dy * x).mean(1, keepdims=True)
    dx = dy - c1 - x * c2
    e = 6 * U32 * (np.abs(dy) + np.abs(c1) + np.abs(x * c2))
    return (dy.astype(np.float32), x.astype(np.float32), (dx, (dy * x).sum(0), dy.sum(0)),
            stored(dx, e, dtype))


def exact_embed_grad(dy, tokens, vocab):
    """Sums of integer rows by token, one column at a time."""
    dy = np.asarray(dy, np.float64)
    dw = np.stack([np.bincount(tokens, dy[:, c], minlength=vocab) for c in range(dy.shape[1])], 1)
    assert np.abs(dw).max() < 2 ** 24
    return dw
