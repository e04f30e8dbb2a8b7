"""Layer norm and embedding on the GPU, forward and backward, against their
definitions in 64 bits (tests/layer_reference.py holds those and the error
bounds), through the C ABI, the torch functions and the optimizer."""
import numpy as np
import pytest

from distributed_bit_matrix_amd import binding as B
from tests import layer_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = float(np.float32(1e-5))


def dev(a, dtype="f32"):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(DT[dtype])


def host(t):
    torch.cuda.synchronize()
    return t.detach().float().cpu().numpy().astype(np.float64)


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


def values(rng, shape, dtype, std=1.0, mean=0.0):
    v = (std * rng.standard_normal(shape) + mean).astype(np.float32)
    return R.bf16_values(v) if dtype == "bf16" else v


def within(got, want, bound, what):
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), off[bad][:4], bound[bad][:4])


# every boundary of the kernels' row widths, odd ones, one column and many
SHAPES = [(1, 1), (3, 1), (5, 2), (7, 3), (257, 4), (33, 7), (65, 8), (64, 9), (100, 31),
          (9, 32), (130, 33), (77, 63), (41, 64), (19, 65), (50, 127), (23, 128), (31, 255),
          (12, 256), (37, 257), (5, 511), (6, 512), (29, 513), (200, 768), (17, 1000),
          (18, 1001), (11, 1024), (10, 1025), (6, 2047), (7, 2048), (5, 2049), (3, 4095),
          (4, 4096), (3, 4097), (2, 8191), (3, 8192), (2, 8193), (3, 16384), (2, 16385),
          (2, 32768), (2, 32769), (1, 100003), (1500, 24), (1100, 96), (4100, 5), (2000, 1)]


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_forward(rows, cols, x_dtype):
    w_dtype = "bf16" if (rows + cols) % 2 else "f32"
    print(f"norm {rows}x{cols} {x_dtype} weights {w_dtype}", flush=True)
    rng = np.random.default_rng(rows * 131071 + cols)
    x = values(rng, (rows, cols), x_dtype, 1.5, 0.4)
    g, b = values(rng, cols, w_dtype, 0.3, 1.0), values(rng, cols, w_dtype, 0.3)
    for gamma, beta in ((g, b), (g, None), (None, b), (None, None)):
        y, mean, rstd = B.layer_norm(
            dev(x, x_dtype), None if gamma is None else dev(gamma, w_dtype),
            None if beta is None else dev(beta, w_dtype), EPS, want_stats=True)
        wy, wm, wr = R.norm(x, gamma, beta, EPS)
        by, bm, br = R.norm_bounds(x, gamma, beta, EPS, x_dtype)
        within(host(mean), wm, bm, "mean")
        within(host(rstd), wr, br, "rstd")
        within(host(y), wy, by, "y")
    # without statistics, and in place: the same bits
    t = dev(x, x_dtype)
    assert torch.equal(bits(B.layer_norm(t, None, None, EPS)), bits(y))
    B.layer_norm(t, None, None, EPS, Y=t)
    assert torch.equal(bits(t), bits(y))


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_backward(rows, cols, x_dtype):
    w_dtype = "f32" if (rows + cols) % 2 else "bf16"
    print(f"norm grad {rows}x{cols} {x_dtype} weights {w_dtype}", flush=True)
    rng = np.random.default_rng(rows * 131071 + cols + 1)
    x = values(rng, (rows, cols), x_dtype, 1.5, 0.4)
    dy = values(rng, (rows, cols), x_dtype)
    g = values(rng, cols, w_dtype, 0.3, 1.0)
    _, m, r = R.norm(x, None, None, EPS)
    m, r = m.astype(np.float32), r.astype(np.float32)
    X, DY, M_, R_ = dev(x, x_dtype), dev(dy, x_dtype), dev(m), dev(r)
    for gamma in (g, None):
        W = None if gamma is None else dev(gamma, w_dtype)
        want = R.norm_grad(dy, x, gamma, m, r)
        for dw_dtype in ("f32", "bf16"):
            got = B.layer_norm_backward(DY, X, W, M_, R_, dtype=DT[dw_dtype])
            bound = R.norm_grad_bounds(dy, x, gamma, m, r, x_dtype, dw_dtype)
            for a, w, e, name in zip(got, want, bound, ("dx", "dgamma", "dbeta")):
                within(host(a), w, e, name)
    # accumulation adds to what is there; dX may be dY; each result by itself
    old = [values(rng, cols, "f32"), values(rng, cols, "f32")]
    acc = [dev(v) for v in old]
    d2 = DY.clone()
    dx, dg, db = B.layer_norm_backward(d2, X, W, M_, R_, dX=d2, dweight=acc[0], dbias=acc[1],
                                       accumulate=True)
    bound = R.norm_grad_bounds(dy, x, gamma, m, r, x_dtype, "f32", old)
    assert torch.equal(bits(dx), bits(got[0])) and dx is d2
    within(host(dg), want[1] + old[0], bound[1], "dgamma +=")
    within(host(db), want[2] + old[1], bound[2], "dbeta +=")
    both = B.layer_norm_backward(DY, X, W, M_, R_)
    for k in range(3):
        one = B.layer_norm_backward(DY, X, W, M_, R_, want_x=k == 0, want_weight=k == 1,
                                    want_bias=k == 2)
        assert [v is not None for v in one] == [k == j for j in range(3)]
        assert torch.equal(bits(one[k]), bits(both[k]))


# many rows at the boundaries of the kernels' row widths (up to 2048 rows and
# 2^22 entries still go in one launch)
LARGE = [(1030, c) for c in (1, 3, 4, 7, 8, 31, 33, 63, 65, 127, 129, 255, 257, 511, 513, 767,
                             1001, 1023, 1025, 2047, 2049, 4071)] + \
    [(1025, 4097), (513, 8191), (512, 8193), (350, 12287), (340, 12289), (257, 16383),
     (70, 16385)]


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", LARGE)
def test_norm_backward_large(rows, cols, x_dtype):
    print(f"norm grad large {rows}x{cols} {x_dtype}", flush=True)
    rng = np.random.default_rng(rows + cols)
    x, dy = values(rng, (rows, cols), x_dtype, 1.5, 0.4), values(rng, (rows, cols), x_dtype)
    g = values(rng, cols, "f32", 0.3, 1.0)
    _, m, r = R.norm(x, None, None, EPS)
    m, r = m.astype(np.float32), r.astype(np.float32)
    d2 = dev(dy, x_dtype)
    got = B.layer_norm_backward(d2, dev(x, x_dtype), dev(g), dev(m), dev(r))
    for a, w, e, name in zip(got, R.norm_grad(dy, x, g, m, r),
                             R.norm_grad_bounds(dy, x, g, m, r, x_dtype, "f32"),
                             ("dx", "dgamma", "dbeta")):
        within(host(a), w, e, name)
    inplace = B.layer_norm_backward(d2, dev(x, x_dtype), dev(g), dev(m), dev(r), dX=d2)
    for a, b in zip(got, inplace):
        assert torch.equal(bits(a), bits(b))
    assert B.layer_norm_backward_workspace(rows, cols) > 0 or rows * cols <= 1 << 22


@pytest.mark.parametrize("rows,cols", [(12289, 768), (70000, 24), (3001, 4096), (300, 16384),
                                       (140000, 3)])
def test_norm_many_rows(rows, cols):
    print(f"norm many rows {rows}x{cols}", flush=True)
    rng = np.random.default_rng(rows)
    x, dy = values(rng, (rows, cols), "bf16", 2.0, 1.0), values(rng, (rows, cols), "bf16")
    g, b = values(rng, cols, "f32", 0.3, 1.0), values(rng, cols, "f32", 0.3)
    X, DY = dev(x, "bf16"), dev(dy, "bf16")
    y, m, r = B.layer_norm(X, dev(g), dev(b), EPS, want_stats=True)
    within(host(y), R.norm(x, g, b, EPS)[0], R.norm_bounds(x, g, b, EPS, "bf16")[0], "y")
    got = B.layer_norm_backward(DY, X, dev(g), m, r)
    m, r = host(m), host(r)
    for a, w, e, name in zip(got, R.norm_grad(dy, x, g, m, r),
                             R.norm_grad_bounds(dy, x, g, m, r, "bf16", "f32"),
                             ("dx", "dgamma", "dbeta")):
        within(host(a), w, e, name)
    again = B.layer_norm_backward(DY, X, dev(g), dev(m.astype(np.float32)),
                                  dev(r.astype(np.float32)))
    for a, c in zip(got, again):
        assert torch.equal(bits(a), bits(c))


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [5, 64, 257, 768, 5000])
def test_norm_strided_and_misaligned(cols, x_dtype):
    """Rows inside a wider matrix that start anywhere; what lies between and
    around the rows stays as it was."""
    print(f"norm strided {cols} {x_dtype}", flush=True)
    rng = np.random.default_rng(cols)
    rows, pad = 13, 3
    wide = values(rng, (2, rows, cols + pad), x_dtype)
    x, dy = wide[0, :, 1:1 + cols], wide[1, :, 2:2 + cols]
    T = dev(wide, x_dtype)
    X, DY = T[0, :, 1:1 + cols], T[1, :, 2:2 + cols]
    G = dev(np.concatenate([[9.0], values(rng, cols, "f32")]).astype(np.float32))[1:]
    out = torch.full((rows * cols + 2,), 7.0, device="cuda", dtype=DT[x_dtype])
    Y = out[1:-1].view(rows, cols)
    y, m, r = B.layer_norm(X, G, None, EPS, want_stats=True, Y=Y)
    g = host(G)
    within(host(Y), R.norm(x, g, None, EPS)[0], R.norm_bounds(x, g, None, EPS, x_dtype)[0], "y")
    assert float(out[0]) == 7.0 and float(out[-1]) == 7.0
    m0, r0 = host(m), host(r)
    sums = torch.full((2 * cols + 3,), 7.0, device="cuda")
    B.layer_norm_backward(DY, X, G, m, r, dX=Y, dweight=sums[1:1 + cols],
                          dbias=sums[2 + cols:2 + 2 * cols])
    want = R.norm_grad(dy, x, g, m0, r0)
    bound = R.norm_grad_bounds(dy, x, g, m0, r0, x_dtype, "f32")
    within(host(Y), want[0], bound[0], "dx")
    within(host(sums[1:1 + cols]), want[1], bound[1], "dgamma")
    within(host(sums[2 + cols:2 + 2 * cols]), want[2], bound[2], "dbeta")
    assert [float(out[0]), float(out[-1]), float(sums[0]), float(sums[1 + cols]),
            float(sums[-1])] == [7.0] * 5
    assert torch.equal(T, dev(wide, x_dtype))


@pytest.mark.parametrize("cols", [1, 8, 100, 768, 3000, 20000, 40000])
def test_norm_special_rows(cols):
    """Constant rows give beta; a NaN or an infinity stays in its row."""
    print(f"norm special rows {cols}", flush=True)
    rng = np.random.default_rng(cols)
    x = values(rng, (9, cols), "f32")
    x[1] = 3.0
    x[2] = 0.0
    x[4, cols // 2] = np.nan
    x[6, cols - 1] = np.inf
    x[7, 0] = -np.inf
    b = values(rng, cols, "f32")
    y, m, r = B.layer_norm(dev(x), None, dev(b), EPS, want_stats=True)
    y = host(y)
    fine = [0, 1, 2, 3, 5, 8]
    within(y[fine], R.norm(x[fine], None, b, EPS)[0],
           R.norm_bounds(x[fine], None, b, EPS, "f32")[0], "y")
    assert np.array_equal(y[2], b.astype(np.float64))
    assert np.isnan(y[[4, 6, 7]]).all()
    dy = values(rng, (9, cols), "f32")
    dx = host(B.layer_norm_backward(dev(dy), dev(x), None, m, r)[0])
    assert np.isnan(dx[[4, 6, 7]]).all() and np.isfinite(dx[fine]).all()


def test_norm_large_mean():
    """A mean of 1000 deviations: the deviations are taken from the mean
    before they are squared."""
    rng = np.random.default_rng(5)
    for cols in (768, 5000, 40000):
        x = values(rng, (6, cols), "f32", 1.0, 1000.0)
        y, m, r = B.layer_norm(dev(x), None, None, EPS, want_stats=True)
        within(host(y), R.norm(x, None, None, EPS)[0],
               R.norm_bounds(x, None, None, EPS, "f32")[0], "y")
        # a difference of squares would be off by u mean^2 = 6% of the variance
        assert np.abs(host(r) - R.norm(x, None, None, EPS)[2]).max() < 1e-3


def test_norm_no_rows():
    X = torch.empty((0, 40), device="cuda")
    y, m, r = B.layer_norm(X, None, None, EPS, want_stats=True)
    assert y.shape == (0, 40) and m.shape == (0,)
    _, dg, db = B.layer_norm_backward(X, X, None, m, r)
    assert host(dg).tolist() == [0.0] * 40 and host(db).tolist() == [0.0] * 40
    old = dev(np.arange(40, dtype=np.float32))
    B.layer_norm_backward(X, X, None, m, r, dweight=old, dbias=old.clone(), accumulate=True)
    assert host(old).tolist() == list(range(40))


def test_norm_gradient_against_differences():
    """dx, dgamma, dbeta against central differences of the definition, whose
    own error at step 1e-5 is about 1e-10."""
    rng = np.random.default_rng(11)
    rows, cols, h = 6, 37, 1e-5
    x, dy = values(rng, (rows, cols), "f32"), values(rng, (rows, cols), "f32")
    g, b = values(rng, cols, "f32", 0.3, 1.0), values(rng, cols, "f32")
    y, m, r = B.layer_norm(dev(x), dev(g), dev(b), EPS, want_stats=True)
    got = [host(t) for t in B.layer_norm_backward(dev(dy), dev(x), dev(g), m, r)]

    def loss(x, g, b):
        return float((np.asarray(dy, np.float64) * R.norm(x, g, b, EPS)[0]).sum())

    args = [x.astype(np.float64), g.astype(np.float64), b.astype(np.float64)]
    bound = R.norm_grad_bounds(dy, x, g, host(m), host(r), "f32", "f32")
    # the saved statistics are themselves rounded: both gradients of x move by
    # the statistics' relative error times their terms' magnitude
    slack = 64 * R.U32 * np.abs(dy).max() * np.abs(g).max() * host(r).max() * cols
    for k in range(3):
        for i in np.ndindex(args[k].shape):
            if k == 0 and (i[0] * cols + i[1]) % 5:
                continue
            hi, lo = [a.copy() for a in args], [a.copy() for a in args]
            hi[k][i] += h
            lo[k][i] -= h
            d = (loss(*hi) - loss(*lo)) / (2 * h)
            assert abs(got[k][i] - d) <= bound[k][i] + slack + 1e-7, (k, i, got[k][i], d)


# --------------------------------------------------------------------------
# Embedding
# --------------------------------------------------------------------------
@pytest.mark.parametrize("w_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("y_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (8, 5, 1), (3, 100, 2), (70, 11, 3),
                                         (1000, 50, 7), (33, 1000, 8), (5, 9, 63), (100, 64, 64),
                                         (9, 300, 257), (129, 33, 768), (4, 7, 1001),
                                         (6, 20, 4096), (2, 3, 70001), (5000, 17, 4)])
def test_embedding_forward(n, vocab, dim, y_dtype, w_dtype):
    print(f"embed n={n} {vocab}x{dim} {w_dtype}->{y_dtype}", flush=True)
    rng = np.random.default_rng(n + vocab + dim)
    w = values(rng, (vocab, dim), w_dtype)
    t = rng.integers(0, vocab, n)
    t[0], t[-1] = 0, vocab - 1
    W = dev(w, w_dtype)
    for token_type in (torch.int64, torch.int32):
        T = torch.from_numpy(t).cuda().to(token_type)
        for scale in (1.0, -0.37):
            want = R.embed(w, t, float(np.float32(scale)))
            got = B.embedding(T, W, scale, out_dtype=DT[y_dtype])
            within(host(got), want, R.stored(want, R.U32 * np.abs(want), y_dtype), "y")
            if scale == 1.0 and y_dtype == w_dtype:
                assert torch.equal(bits(got), bits(W[T.long()]))


def test_embedding_tokens_outside_the_table():
    w = np.arange(12, dtype=np.float32).reshape(4, 3)
    t = np.array([0, -1, 3, 4, 2, 2 ** 40, -2 ** 40])
    got = host(B.embedding(torch.from_numpy(t).cuda(), dev(w)))
    assert np.array_equal(got, R.embed(w, t, 1.0), equal_nan=True)
    dy = np.ones((7, 3), np.float32)
    dw = host(B.embedding_backward(dev(dy), torch.from_numpy(t).cuda(), 4))
    assert np.array_equal(dw, R.embed_grad(dy, t, 4, 1.0)[0])
    assert dw[:, 0].tolist() == [1, 0, 1, 1]


def _tokens(rng, kind, n, vocab):
    if kind == "same":
        return np.full(n, rng.integers(0, vocab))
    if kind == "last":
        return np.full(n, vocab - 1)
    if kind == "positions":
        return np.arange(n) % vocab
    if kind == "falling":
        return (vocab - 1 - np.arange(n) % vocab)
    if kind == "skew":                  # many tokens of one residue
        return 5 + 256 * rng.integers(0, vocab // 256, n)
    if kind == "zipf":
        return np.minimum((vocab ** rng.random(n)).astype(np.int64) - 1, vocab - 1)
    return rng.integers(0, vocab, n)


GRADS = [(1, 1, 1, "uniform"), (2, 3, 5, "same"), (63, 7, 4, "uniform"), (64, 64, 8, "positions"),
         (65, 1000, 3, "uniform"), (777, 1000, 257, "zipf"), (1000, 1, 33, "same"),
         (3000, 2, 9, "uniform"), (4097, 300, 64, "zipf"), (2500, 40000, 17, "zipf"),
         (5000, 131073, 4, "uniform"), (6000, 257, 100, "falling"), (1025, 5000, 768, "zipf"),
         (900, 1024, 1001, "same"), (300, 600000, 2, "last"), (20000, 513, 12, "zipf"),
         (50000, 4096, 3, "zipf"), (70000, 100, 1, "uniform"), (33000, 70000, 2, "zipf"),
         (150000, 30000, 2, "zipf"), (131073, 3, 5, "same"), (4000, 64, 2048, "zipf"),
         (20000, 70000, 8, "skew"), (800, 70000, 40, "skew"), (896, 300, 30, "zipf"),
         (897, 300, 30, "zipf"), (896, 513, 5, "same"), (40000, 200000, 3, "skew"),
         (65536, 2000, 3, "zipf"), (65537, 2000, 3, "zipf"), (131072, 131072, 2, "zipf"),
         (100001, 300000, 2, "skew"), (262145, 17, 2, "uniform"), (70001, 1, 3, "same"),
         (600001, 1048576, 1, "uniform"), (2048, 300, 70, "same"), (2047, 5000, 260, "zipf"),
         (2048, 1000, 5, "skew"), (1793, 2, 9, "uniform"), (2049, 1000, 7, "skew"),
         (2048, 600, 3, "skew"), (1500, 131072, 4, "skew")]


@pytest.mark.parametrize("dy_dtype,dw_dtype", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"),
                                               ("bf16", "bf16")])
@pytest.mark.parametrize("n,vocab,dim,kind", GRADS)
def test_embedding_backward(n, vocab, dim, kind, dy_dtype, dw_dtype):
    print(f"embed grad n={n} {vocab}x{dim} {kind} {dy_dtype}->{dw_dtype}", flush=True)
    rng = np.random.default_rng(n * 7 + vocab + dim)
    dy = values(rng, (n, dim), dy_dtype)
    t = _tokens(rng, kind, n, vocab)
    scale = float(np.float32(0.7))
    T, DY = torch.from_numpy(t).cuda(), dev(dy, dy_dtype)
    want, mag, counts = R.embed_grad(dy, t, vocab, scale)
    got = B.embedding_backward(DY, T, vocab, scale, dtype=DT[dw_dtype])
    within(host(got), want, R.embed_grad_bounds(want, mag, counts, dw_dtype), "dW")
    again = B.embedding_backward(DY, T.int(), vocab, scale, dtype=DT[dw_dtype])
    assert torch.equal(bits(got), bits(again))      # fixed order; either token type
    if dw_dtype == "f32":
        old = values(rng, (vocab, dim), "f32")
        acc = dev(old)
        B.embedding_backward(DY, T, vocab, scale, dW=acc, accumulate=True)
        within(host(acc), want + old, R.embed_grad_bounds(want, mag, counts, "f32", old), "dW +=")
        untouched = counts == 0
        assert np.array_equal(host(acc)[untouched], old[untouched].astype(np.float64))


@pytest.mark.parametrize("n,vocab,dim", [(500, 40, 12), (5000, 700, 33)])
def test_embedding_backward_padding_and_strides(n, vocab, dim):
    """Padding and foreign tokens add nothing, not even infinities or NaN;
    rows of dY inside a wider matrix; the memory around dW stays."""
    print(f"embed grad padding n={n} {vocab}x{dim}", flush=True)
    rng = np.random.default_rng(n)
    t = rng.integers(0, vocab, n)
    t[rng.random(n) < 0.3] = 5
    t[rng.random(n) < 0.05] = -100
    t[rng.random(n) < 0.05] = vocab
    wide = values(rng, (n, dim + 3), "bf16")
    wide[t == 5] = np.nan
    wide[(t < 0) | (t >= vocab)] = np.inf
    dy = wide[:, 1:1 + dim].copy()
    dy[~np.isfinite(dy)] = 0.0
    out = torch.full((vocab * dim + 2,), 7.0, device="cuda")
    dW = out[1:-1].view(vocab, dim)
    B.embedding_backward(dev(wide, "bf16")[:, 1:1 + dim], torch.from_numpy(t).cuda(), vocab,
                         padding=5, dW=dW)
    want, mag, counts = R.embed_grad(dy, t, vocab, 1.0, padding=5)
    assert counts[5] == 0
    within(host(dW), want, R.embed_grad_bounds(want, mag, counts, "f32"), "dW")
    assert float(out[0]) == 7.0 and float(out[-1]) == 7.0


def test_embedding_backward_special_values():
    """An infinity or NaN reaches its own token's row and column only."""
    dy = np.ones((400, 6), np.float32)
    t = np.arange(400) % 10
    dy[13, 2], dy[27, 4] = np.nan, np.inf
    dw = host(B.embedding_backward(dev(dy), torch.from_numpy(t).cuda(), 12))
    want = np.full((12, 6), 40.0)
    want[10:] = 0.0
    want[3, 2], want[7, 4] = np.nan, np.inf
    assert np.array_equal(dw, want, equal_nan=True)


def test_embedding_no_tokens():
    T = torch.empty(0, dtype=torch.int64, device="cuda")
    W = torch.ones((5, 3), device="cuda")
    assert B.embedding(T, W).shape == (0, 3)
    dw = B.embedding_backward(torch.empty((0, 3), device="cuda"), T, 5)
    assert host(dw).tolist() == [[0.0] * 3] * 5
    B.embedding_backward(torch.empty((0, 3), device="cuda"), T, 5, dW=W, accumulate=True)
    assert host(W).tolist() == [[1.0] * 3] * 5


def test_rows_past_32_bits():
    """A batch of 2^31 + 1024 entries: offsets past 32 bits on every array."""
    dim = 1024
    n = (1 << 21) + 1
    print(f"rows past 32 bits: {n} x {dim}", flush=True)
    T = torch.arange(n, device="cuda") % 3
    W = torch.tensor([[1.0], [2.0], [4.0]], device="cuda").repeat(1, dim).bfloat16()
    W[:, 5] = 8.0
    Y = B.embedding(T, W)
    assert torch.equal(Y[-1], W[(n - 1) % 3]) and torch.equal(Y[n // 2], W[(n // 2) % 3])
    dW = B.embedding_backward(Y, T, 3)
    counts = np.bincount(np.arange(n) % 3, minlength=3).astype(np.float64)
    want = counts[:, None] * host(W)
    # terms of equal sign, powers of two: each partial sum is rounded once
    within(host(dW), want, R.embed_grad_bounds(want, want, counts, "f32"), "dW")
    Z, m, r = B.layer_norm(Y, None, None, EPS, want_stats=True)
    wy, wm, wr = R.norm(host(Y[-3:]), None, None, EPS)
    by, bm, br = R.norm_bounds(host(Y[-3:]), None, None, EPS, "bf16")
    within(host(Z[-3:]), wy, by, "y")
    dx, dg, db = B.layer_norm_backward(Y, Y, None, m, r, dX=Z)
    want = R.norm_grad(host(Y[-3:]), host(Y[-3:]), None, host(m[-3:]), host(r[-3:]))[0]
    bound = R.norm_grad_bounds(host(Y[-3:]), host(Y[-3:]), None, host(m[-3:]), host(r[-3:]),
                               "bf16", "f32")[0]
    within(host(dx[-3:]), want, bound, "dx")
    total = (counts[:, None] * host(W)).sum(0)
    within(host(db), total, R.stored(total, R.chain(n) * total, "f32"), "dbeta")


# --------------------------------------------------------------------------
# Streams, graphs, autograd, the optimizer
# --------------------------------------------------------------------------
def _batch(seed, n=700, vocab=90, dim=160):
    rng = np.random.default_rng(seed)
    return (torch.from_numpy(rng.integers(0, vocab, n)).cuda(), dev(values(rng, (n, dim), "f32")),
            dev(values(rng, (vocab, dim), "f32")), dev(values(rng, dim, "f32", 0.3, 1.0)),
            dev(values(rng, dim, "f32")))


def _all(T, DY, W, G, Bi, out=None, ws=(None, None), stream=None):
    o = out or {}
    Y = B.embedding(T, W, 0.5, out=o.get("Y"), stream=stream)
    Z, m, r = B.layer_norm(Y, G, Bi, EPS, True, o.get("Z"), o.get("m"), o.get("r"),
                           stream=stream)
    dx, dg, db = B.layer_norm_backward(DY, Y, G, m, r, dX=o.get("dx"), dweight=o.get("dg"),
                                       dbias=o.get("db"), ws=ws[0], stream=stream)
    dW = B.embedding_backward(dx, T, W.shape[0], 0.5, dW=o.get("dW"), ws=ws[1], stream=stream)
    return dict(Y=Y, Z=Z, m=m, r=r, dx=dx, dg=dg, db=db, dW=dW)


def test_two_streams_at_once():
    sets = [_batch(s) for s in (1, 2)]
    want = [_all(*b) for b in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(20):
        for k in (0, 1):
            got[k].append(_all(*sets[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for o in got[k]:
            for name in o:
                assert torch.equal(o[name], want[k][name]), (k, name)


def test_graph_replays_match_eager():
    """Two captured runs with workspaces of their own, replayed in turn, with
    eager work and changed inputs between the replays."""
    sets = [_batch(s) for s in (3, 4)]
    graphs, outs, keep = [], [], []
    side = torch.cuda.Stream()
    for b in sets:
        o = _all(*b)
        n, dim = b[1].shape
        ws = (torch.empty(B.layer_norm_backward_workspace(n, dim), dtype=torch.uint8,
                          device="cuda"),
              torch.empty(B.embedding_backward_workspace(n, b[2].shape[0], dim),
                          dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            _all(*b, out=o, ws=ws)
        graphs.append(g)
        outs.append(o)
        keep.append(ws)
    for rep in range(4):
        for k in (0, 1):
            fresh = _batch(10 * rep + k)
            for old, new in zip(sets[k], fresh):
                old.copy_(new)
            for t in outs[k].values():
                t.fill_(float("nan"))
            graphs[k].replay()
            want = _all(*fresh)
            torch.cuda.synchronize()
            for name in want:
                assert torch.equal(outs[k][name], want[name]), (rep, k, name)
    del keep


def test_autograd_matches_the_definition():
    from distributed_bit_matrix_amd import layers as L
    rng = np.random.default_rng(21)
    for p_dtype in ("f32", "bf16"):
        vocab, dim = 50, 96
        w, g, b = (values(rng, s, p_dtype, sd, mu) for s, sd, mu in
                   (((vocab, dim), 1.0, 0.0), (dim, 0.3, 1.0), (dim, 0.3, 0.0)))
        t = rng.integers(0, vocab, (4, 33))
        t[0, :5] = 7
        W, G, Bi = (dev(v, p_dtype).requires_grad_() for v in (w, g, b))
        h = L.embedding(torch.from_numpy(t).cuda(), W, scale=2.0, padding_idx=7)
        h.retain_grad()
        y = L.layer_norm(h, G, Bi, EPS)
        assert y.shape == (4, 33, dim) and y.dtype == DT[p_dtype]
        dy = values(rng, y.shape, p_dtype)
        y.backward(dev(dy, p_dtype))
        hx = host(h).reshape(-1, dim)
        _, m, r = R.norm(hx, None, None, EPS)
        m, r = m.astype(np.float32), r.astype(np.float32)
        want = R.norm_grad(dy.reshape(-1, dim), hx, g, m, r)
        bound = R.norm_grad_bounds(dy.reshape(-1, dim), hx, g, m, r, p_dtype, p_dtype)
        # the kernel's own statistics differ from these by a few roundings
        bound = [e + 64 * R.U32 * np.abs(dy).max() * np.abs(g).max() * r.max() * dim
                 for e in bound]
        within(host(h.grad).reshape(-1, dim), want[0], bound[0], "dx")
        within(host(G.grad), want[1], bound[1], "dgamma")
        within(host(Bi.grad), want[2], bound[2], "dbeta")
        dw, mag, counts = R.embed_grad(host(h.grad).reshape(-1, dim), t, vocab, 2.0, padding=7)
        assert counts[7] == 0 and W.grad.dtype == DT[p_dtype]
        within(host(W.grad), dw, R.embed_grad_bounds(dw, mag, counts, p_dtype), "dW")


def test_autograd_strided_expanded_and_frozen():
    from distributed_bit_matrix_amd import layers as L
    x = torch.randn(6, 5, 32, device="cuda").transpose(0, 1).requires_grad_()
    w = torch.randn(32, device="cuda").requires_grad_()
    y = L.layer_norm(x, w, None, EPS)
    y.sum().backward()                      # the gradient of y is an expanded scalar
    xd = x.detach().double().requires_grad_()
    wd = w.detach().double().requires_grad_()
    torch.nn.functional.layer_norm(xd, (32,), wd, None, EPS).sum().backward()
    assert torch.allclose(x.grad.double(), xd.grad, atol=2e-5)
    assert torch.allclose(w.grad.double(), wd.grad, atol=2e-5)
    v = torch.randn(32, device="cuda")      # frozen weight: only x gets a gradient
    x2 = torch.randn(7, 32, device="cuda", requires_grad=True)
    L.layer_norm(x2, v, v, EPS).square().sum().backward()
    assert x2.grad is not None and v.grad is None
    with pytest.raises(RuntimeError):       # once differentiable
        g, = torch.autograd.grad(L.layer_norm(x2, v, v, EPS).square().sum(), x2,
                                 create_graph=True)
        g.sum().backward()


def _model(dtype, vocab=61, dim=48):
    from distributed_bit_matrix_amd import layers as L

    class Model(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.tokens = L.Embedding(vocab, dim, device="cuda", dtype=dtype)
            self.positions = L.Embedding(16, dim, device="cuda", dtype=dtype)
            self.norm = L.LayerNorm(dim, device="cuda", dtype=dtype)
            self.mix = torch.nn.Linear(dim, dim, device="cuda", dtype=dtype)
            self.last = L.LayerNorm(dim, bias=False, device="cuda", dtype=dtype)

        def forward(self, t):
            h = self.tokens(t) + self.positions(torch.arange(t.shape[1], device="cuda").expand(
                t.shape).contiguous())
            h = h + self.mix(self.norm(h))
            return torch.nn.functional.linear(self.last(h), self.tokens.weight)   # shared table

    torch.manual_seed(0)
    return Model()


def _loss(model, t):
    return torch.nn.functional.cross_entropy(model(t[:, :-1]).float().flatten(0, 1),
                                             t[:, 1:].flatten())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_direct_gradients_reach_the_step(dtype):
    """The flat array of the step holds, for every parameter, the gradient
    that the ordinary path gives, summed over two backward passes, also of the
    table that the output product shares; the step then moves the weights."""
    from distributed_bit_matrix_amd import optim as SO
    t = torch.randint(61, (2, 3, 17), device="cuda",
                      generator=torch.Generator(device="cuda").manual_seed(3))
    plain, direct = _model(DT[dtype]), _model(DT[dtype])
    o1 = SO.SignMuon(plain.parameters(), scale="fro")
    o2 = SO.SignMuon(direct.parameters(), scale="fro", direct_grads=True)
    for step in range(2):
        for o, m in ((o1, plain), (o2, direct)):
            o.zero_grad()
            for k in range(2):
                _loss(m, t[k]).backward()
        names = [n for n, _ in direct.named_parameters()]
        for n, p in direct.named_parameters():
            assert (p.grad is None) == (n not in ("tokens.weight", "mix.weight", "mix.bias")), n
        o1.step()
        o2.step()
        torch.cuda.synchronize()
        assert not o1.nonfinite() and not o2.nonfinite()
        a, b = o1._groups[0], o2._groups[0]
        for n, (r, c, off, _) in zip(names, b.layout):
            ga, gb = host(a.G[off:off + r * c]), host(b.G[off:off + r * c])
            # ordinary gradients: each backward pass and each sum rounded to the dtype;
            # at most 4 roundings of magnitudes up to the largest entry
            tol = 4 * (R.HALF_STEP[dtype] + 4 * R.U32) * 2 * np.abs(gb).max() + R.TINY
            assert np.abs(ga - gb).max() <= tol, (step, n)
            assert np.abs(gb).max() > 0, n
        # the same weights for the next round
        with torch.no_grad():
            for p, q in zip(plain.parameters(), direct.parameters()):
                p.copy_(q)
    # nothing since the last step: the gradient is zero, not the old one
    o2.zero_grad()
    o2.step()
    assert float(b.G.abs().max()) == 0.0


def test_direct_gradients_on_another_stream():
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    w = torch.nn.Parameter(torch.zeros(3000, 512, device="cuda"))
    opt = SO.SignMuon([w], scale="fro", K=1, direct_grads=True)
    t = torch.arange(3000, device="cuda")
    side = torch.cuda.Stream()
    for step in range(5):
        opt.zero_grad()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for k in range(3):
                (L.embedding(t, w) * float(step + 1)).sum().backward()
        opt.step()      # ordered after the writes by the optimizer itself
        torch.cuda.synchronize()
        assert w.grad is None
        assert torch.equal(opt._groups[0].G, torch.full_like(opt._groups[0].G, 3.0 * (step + 1)))


def test_direct_gradients_end_with_their_optimizer():
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    w = torch.nn.Parameter(torch.randn(32, device="cuda"))
    opt = SO.SignMuon([w], scale="fro", K=1, direct_grads=True)
    x = torch.randn(4, 32, device="cuda")
    L.layer_norm(x, w).sum().backward()
    assert w.grad is None
    y = L.layer_norm(x, w).sum()
    del opt
    y.backward()
    assert w.grad is not None
    SO.SignMuon([w], scale="fro", K=1).step()      # and an ordinary one takes over
    w.grad = None
    L.layer_norm(x, w).sum().backward()
    assert w.grad is not None


@pytest.mark.parametrize("direct", [False, True])
def test_sparse_gradients_are_summed_in_order(direct):
    """torch.nn.Embedding(sparse=True): tokens and rows go straight into the
    step's flat array, bit for bit what the library's own gradient is."""
    from distributed_bit_matrix_amd import optim as SO
    rng = np.random.default_rng(8)
    table = torch.nn.Embedding(40, 24, sparse=True, device="cuda")
    other = torch.nn.Parameter(torch.randn(8, 24, device="cuda"))
    opt = SO.SignMuon([table.weight, other], scale="fro", K=2, direct_grads=direct)
    T = torch.from_numpy(rng.integers(0, 40, (30, 20))).cuda()
    C = dev(values(rng, (30, 20, 24), "f32"))
    for step in range(3):
        opt.zero_grad()
        ((table(T) * C).sum() + other.sum()).backward()
        assert table.weight.grad.is_sparse
        want = B.embedding_backward(C, T, 40)
        opt.step()
        torch.cuda.synchronize()
        assert torch.equal(opt._groups[0].G[:40 * 24].view(40, 24), want)
    assert not opt.nonfinite()


def test_foreign_token_is_reported_by_the_step():
    from distributed_bit_matrix_amd import optim as SO
    model = _model(torch.float32)
    opt = SO.SignMuon(model.parameters(), scale="fro", direct_grads=True)
    before = [p.detach().clone() for p in model.parameters()]
    t = torch.randint(61, (3, 17), device="cuda")
    t[1, 4] = 61
    h = model.tokens(t)
    (model.last(model.norm(h))).sum().backward()
    opt.step()
    assert opt.nonfinite()
    for p, b in zip(model.parameters(), before):
        assert torch.equal(p, b)


def _filled(p):
    return p._signmuon_slot.filled


def test_direct_gradients_only_where_a_pass_adds_to_the_parameter():
    """torch.autograd.grad returns its gradients and leaves the step's alone,
    backward(inputs=...) writes those it names, and the next plain backward
    pass writes all."""
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    rng = np.random.default_rng(12)
    t = torch.arange(24, device="cuda") % 7
    table = torch.nn.Parameter(dev(values(rng, (7, 40), "f32")))
    w = torch.nn.Parameter(dev(values(rng, (40,), "f32")))
    b = torch.nn.Parameter(dev(values(rng, (40,), "f32")))
    c = dev(values(rng, (24, 40), "f32"))
    params = [table, w, b]

    def loss():
        return (L.layer_norm(L.embedding(t, table), w, b, EPS) * c).sum()

    want = torch.autograd.grad(loss(), params)
    opt = SO.SignMuon(params, scale="fro", K=1, direct_grads=True)
    got = torch.autograd.grad(loss(), params)
    assert not any(_filled(p) for p in params)
    for g, q in zip(got, want):
        assert torch.equal(g, q)
    got = torch.autograd.grad(loss(), [w])
    assert torch.equal(got[0], want[1]) and not any(_filled(p) for p in params)
    loss().backward(inputs=[w])
    assert [_filled(p) for p in params] == [False, True, False]
    opt.zero_grad()
    loss().backward()
    assert all(_filled(p) and p.grad is None for p in params)
    for p, q in zip(params, want):
        assert torch.equal(p._signmuon_slot.grad, q)


def test_direct_gradients_of_one_parameter_in_both_places():
    """weight and bias the same parameter: its gradient is the sum of both."""
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    rng = np.random.default_rng(13)
    x = dev(values(rng, (50, 24), "f32"))
    c = dev(values(rng, (50, 24), "f32"))
    w = torch.nn.Parameter(dev(values(rng, (24,), "f32")))
    want, = torch.autograd.grad((L.layer_norm(x, w, w, EPS) * c).sum(), [w])
    opt = SO.SignMuon([w], scale="fro", K=1, direct_grads=True)
    (L.layer_norm(x, w, w, EPS) * c).sum().backward()
    opt.step()
    assert torch.equal(opt._groups[0].G[:24], want)


def test_norm_gradient_refuses_one_array_for_both_sums():
    x = torch.randn(6, 8, device="cuda")
    y, m, r = B.layer_norm(x, want_stats=True)
    both = torch.zeros(8, device="cuda")
    with pytest.raises(B.SignMuonError):
        B.layer_norm_backward(x, x, None, m, r, dweight=both, dbias=both)
    assert float(both.abs().max()) == 0.0


@pytest.mark.parametrize("n,vocab,kind", [((1 << 20) + 1, 40, "same"), ((1 << 21) + 5, 3000, "same"),
                                          ((1 << 20) - 7, 3, "same"), (1 << 20, 70000, "same"),
                                          ((1 << 22) + 77, 50, "zipf"),
                                          ((1 << 21) + 1, 5000, "half"),
                                          (1300000, 200000, "half")])
def test_embedding_backward_of_tokens_repeated_in_long_batches(n, vocab, kind):
    """A token that fills most of a batch past 2^20 tokens.  Entries 0, 1 and 2:
    every partial sum is an integer below 2^24 and so exact in float32."""
    print(f"long batch n={n} vocab={vocab} {kind}", flush=True)
    rng = np.random.default_rng(n + vocab)
    if kind == "half":
        t = np.where(rng.random(n) < 0.9, vocab - 2, rng.integers(0, vocab, n))
    else:
        t = _tokens(rng, kind, n, vocab)
    dy = rng.integers(0, 3, (n, 2)).astype(np.float32)
    want = np.stack([np.bincount(t, dy[:, k], minlength=vocab) for k in (0, 1)], 1)
    assert want.max() < 1 << 24
    T, DY = torch.from_numpy(t).cuda(), dev(dy)
    assert np.array_equal(host(B.embedding_backward(DY, T, vocab)), want)
    assert np.array_equal(host(B.embedding_backward(DY, T.int(), vocab)), want)
    keep = t != t[0]
    got = host(B.embedding_backward(DY, T, vocab, padding=int(t[0])))
    want[t[0]] = 0
    assert keep.any() == bool(want.any()) and np.array_equal(got, want)


def test_embedding_backward_of_the_longest_batch():
    """2^27 tokens, the most that a call takes, seven of eight of them the same:
    sums of ones are exact up to 2^24, and parts are joined in double."""
    n, vocab = 1 << 27, 2000
    T = torch.full((n,), 1234, device="cuda", dtype=torch.int32)
    T[::8] = torch.arange(n // 8, device="cuda", dtype=torch.int32) % vocab
    dy = torch.ones(n, 1, device="cuda", dtype=torch.bfloat16)
    got = host(B.embedding_backward(dy, T, vocab))[:, 0]
    want = np.bincount(np.arange(n // 8) % vocab, minlength=vocab).astype(np.float64)
    want[1234] += n - n // 8
    assert np.array_equal(got, want.astype(np.float32))


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1, 65536), (1, 65537), (3, 131071), (5, 40003), (100, 32769),
                                       (260, 33000), (31, 24577), (9, 16391), (2, 1 << 20)])
def test_norm_long_rows(rows, cols, x_dtype):
    """Rows past the registers: few, which blocks share, and many; strided,
    misaligned and in place; each gradient alone."""
    print(f"norm long rows {rows}x{cols} {x_dtype}", flush=True)
    rng = np.random.default_rng(rows + cols)
    x, dy = values(rng, (rows, cols), x_dtype, 1.5, 20.0), values(rng, (rows, cols), x_dtype)
    g, b = values(rng, cols, "f32", 0.3, 1.0), values(rng, cols, "f32", 0.3)
    wide = torch.full((rows, cols + 9), float("nan"), device="cuda", dtype=DT[x_dtype])
    wide[:, 1:cols + 1] = dev(x, x_dtype)
    X, DY, G, BB = dev(x, x_dtype), dev(dy, x_dtype), dev(g), dev(b)
    y, m, r = B.layer_norm(X, G, BB, EPS, want_stats=True)
    for a, w, e, name in zip((y, m, r), R.norm(x, g, b, EPS), R.norm_bounds(x, g, b, EPS, x_dtype),
                             ("y", "mean", "rstd")):
        within(host(a), w, e, name)
    assert torch.equal(bits(B.layer_norm(wide[:, 1:cols + 1], G, BB, EPS)), bits(y))
    same = X.clone()
    assert torch.equal(bits(B.layer_norm(same, G, BB, EPS, Y=same)), bits(y))
    got = B.layer_norm_backward(DY, X, G, m, r)
    for a, w, e, name in zip(got, R.norm_grad(dy, x, g, host(m), host(r)),
                             R.norm_grad_bounds(dy, x, g, host(m), host(r), x_dtype, "f32"),
                             ("dx", "dgamma", "dbeta")):
        within(host(a), w, e, name)
    for k in range(3):
        one = B.layer_norm_backward(DY, wide[:, 1:cols + 1], G, m, r, want_x=k == 0,
                                    want_weight=k == 1, want_bias=k == 2)
        assert torch.equal(bits(one[k]), bits(got[k]))
    inplace = B.layer_norm_backward(DY, X, G, m, r, dX=DY)
    for a, c in zip(got, inplace):
        assert torch.equal(bits(a), bits(c))


def test_norm_long_rows_of_unlike_parts():
    """Rows whose start says nothing of the rest: a step from 0 to 1000, a
    ramp, and one large entry among small ones."""
    cols = 50000
    x = np.zeros((3, cols), np.float32)
    x[0, 7:] = 1000.0
    x[0] += np.sin(np.arange(cols, dtype=np.float32))
    x[1] = np.arange(cols, dtype=np.float32)
    x[2] = np.cos(np.arange(cols, dtype=np.float32))
    x[2, 31] = 1e4
    y, m, r = B.layer_norm(dev(x), None, None, EPS, want_stats=True)
    for a, w, e, name in zip((y, m, r), R.norm(x, None, None, EPS),
                             R.norm_bounds(x, None, None, EPS, "f32"), ("y", "mean", "rstd")):
        within(host(a), w, e, name)


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(r, c) for r in (2048, 2049) for c in
                                       (1, 3, 4, 7, 8, 31, 33, 63, 65, 129, 257, 513, 767, 1001,
                                        1025)] + [(2048, 2047), (2048, 2049), (1025, 4071)])
def test_norm_backward_at_the_last_row_of_one_launch(rows, cols, x_dtype):
    test_norm_backward_large(rows, cols, x_dtype)


# every path of several launches: the sort and its sums, runs of a long batch,
# runs past 16-bit places, and rows past the registers
RUNS = [(5000, 90, 160), (70000, 300, 24), ((1 << 20) + 500, 40, 3), (60, 50, 20011)]


@pytest.mark.parametrize("n,vocab,dim", RUNS)
def test_several_launches_on_two_streams_at_once(n, vocab, dim):
    print(f"two streams {n} {vocab}x{dim}", flush=True)
    sets = [_batch(s, n, vocab, dim) for s in (21, 22)]
    want = [_all(*b) for b in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(4):
        for k in (0, 1):
            got[k].append(_all(*sets[k], stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for o in got[k]:
            for name in o:
                assert torch.equal(o[name], want[k][name]), (k, name)


@pytest.mark.parametrize("n,vocab,dim", RUNS)
def test_graphs_of_several_launches_match_eager(n, vocab, dim):
    """Replayed with changed inputs, eager work in between; the workspaces are
    the graph's own and allocated in it."""
    print(f"graph {n} {vocab}x{dim}", flush=True)
    b = _batch(31, n, vocab, dim)
    o = _all(*b)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        _all(*b, out=o)
    for rep in range(3):
        fresh = _batch(40 + rep, n, vocab, dim)
        for old, new in zip(b, fresh):
            old.copy_(new)
        for t in o.values():
            t.fill_(float("nan"))
        want = _all(*fresh)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(o[name], want[name]), (rep, name)


def test_captured_layers_return_their_gradients():
    """Forward and backward captured while an optimizer takes gradients
    directly: the replays' gradients are returned, the step's are left alone."""
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    rng = np.random.default_rng(5)
    w = torch.nn.Parameter(dev(values(rng, (64,), "f32", 0.3, 1.0)))
    table = torch.nn.Parameter(dev(values(rng, (30, 64), "f32")))
    opt = SO.SignMuon([w, table], scale="fro", K=1, direct_grads=True)
    t = torch.arange(50, device="cuda") % 30
    c = dev(values(rng, (50, 64), "f32"))

    def run():
        return torch.autograd.grad((L.layer_norm(L.embedding(t, table), w) * c).sum(), [w, table])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = run()
    for rep in range(3):
        c.copy_(dev(values(np.random.default_rng(60 + rep), (50, 64), "f32")))
        g.replay()
        torch.cuda.synchronize()
        want = run()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), rep
        assert not _filled(w) and not _filled(table)
    (L.layer_norm(L.embedding(t, table), w) * c).sum().backward()
    assert _filled(w) and torch.equal(w._signmuon_slot.grad, want[0])
    assert torch.equal(table._signmuon_slot.grad, want[1])


def test_direct_gradients_of_groups_added_and_of_saved_models():
    """Two parameter groups, one added later; a model saved and loaded again
    has ordinary gradients until an optimizer takes it."""
    import io
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    rng = np.random.default_rng(14)
    a, b = L.LayerNorm(40, device="cuda"), L.LayerNorm(40, bias=False, device="cuda")
    x = dev(values(rng, (9, 40), "f32"))
    c = dev(values(rng, (9, 40), "f32"))
    want = torch.autograd.grad((b(a(x)) * c).sum(), [a.weight, a.bias, b.weight])
    opt = SO.SignMuon(a.parameters(), scale="fro", K=1, direct_grads=True)
    opt.add_param_group({"params": list(b.parameters()), "lr": 0.5})
    (b(a(x)) * c).sum().backward()
    # the added group moves at its first step, and takes what is in p.grad then
    assert a.weight.grad is None and b.weight.grad is not None
    opt.step()
    assert torch.equal(opt._groups[0].G[:40], want[0])
    assert torch.equal(opt._groups[1].G[:40], want[2])
    opt.zero_grad(set_to_none=False)
    now = torch.autograd.grad((b(a(x)) * c).sum(), [a.weight, a.bias, b.weight])
    (b(a(x)) * c).sum().backward()
    opt.step()
    assert torch.equal(opt._groups[0].G[:40], now[0])
    assert torch.equal(opt._groups[1].G[:40], now[2])
    assert not opt.nonfinite()
    f = io.BytesIO()
    torch.save(a, f)
    f.seek(0)
    a2 = torch.load(f, weights_only=False)       # the file written above
    assert torch.equal(a2.weight, a.weight)
    (a2(x) * c).sum().backward()
    assert a2.weight.grad is not None and not _filled(a.weight)
    opt2 = SO.SignMuon(a2.parameters(), scale="fro", K=1, direct_grads=True)
    opt2.zero_grad()
    (a2(x) * c).sum().backward()
    assert a2.weight.grad is None and _filled(a2.weight)
