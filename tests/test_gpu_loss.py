"""Linear cross entropy on the GPU, forward and backward, against its definition
in 64 bits (tests/block_reference.py holds that and the error bounds)."""
import pytest

from distributed_bit_matrix_amd import binding as B
from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
IGNORE = -100


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


def within(got, want, bound, what):
    got = got.double()
    off = (got - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           off[bad][:4].tolist(), bound.expand(bad.shape)[bad][:4].tolist())


def inputs(rows, dim, vocab, dtype, seed, ignored=0.0, spread=2.0, bits_=64):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, dim, device="cuda", generator=gen).to(DT[dtype])
    w = (spread * dim ** -0.5 * torch.randn(vocab, dim, device="cuda", generator=gen)).to(DT[dtype])
    t = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    drop = torch.rand(rows, device="cuda", generator=gen) < ignored
    t = torch.where(drop, IGNORE, t)
    return x, w, t.to(torch.int64 if bits_ == 64 else torch.int32)


def check(x, w, t, reduction, dw_dtype=None, ignore=IGNORE):
    loss, lse = B.linear_cross_entropy(x, w, t, ignore, reduction, want_lse=True)
    t64 = t.long()
    each, want_lse = R.loss(x, w, t64, ignore)
    e_each, e_lse = R.loss_bounds(x, w, t64, ignore)
    within(lse, want_lse, e_lse, "lse")
    want, bound = (R.reduce_loss(v, t64, ignore, reduction) for v in (each, e_each))
    within(loss, want, bound + 2 * R.U32 * want.abs(), "loss")
    gen = torch.Generator(device="cuda").manual_seed(7)
    dloss = 1 + 0.3 * torch.randn(loss.shape, device="cuda", generator=gen)
    dw_dtype = dw_dtype or x.dtype
    dx, dw = B.linear_cross_entropy_backward(dloss, x, w, t, lse, ignore, reduction,
                                             dtype=dw_dtype)
    assert dw.dtype == dw_dtype and dx.dtype == x.dtype
    args = (dloss, x, w, t64, lse, ignore, reduction)
    wx, ww = R.loss_grad(*args)
    bx, bw = R.loss_grad_bounds(*args, dw_dtype)
    within(dx, wx, bx, "dx")
    within(dw, ww, bw, "dw")
    return loss, lse, dloss, dx, dw


# one row and column, sizes around tiles of 64, 128 and 256 and pieces of 8, odd ones
SHAPES = [(1, 1, 1), (1, 8, 2), (2, 1, 7), (3, 7, 5), (5, 16, 64), (63, 64, 65), (64, 72, 127),
          (65, 63, 128), (127, 65, 129), (128, 128, 255), (129, 96, 256), (255, 40, 257),
          (256, 33, 300), (257, 127, 511), (300, 129, 1000), (33, 1000, 33), (512, 256, 513),
          (777, 257, 1001), (1, 768, 5003), (8, 64, 4999)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,vocab", SHAPES)
def test_shapes(rows, dim, vocab, dtype):
    print(f"loss {rows}x{dim}x{vocab} {dtype}", flush=True)
    reduction = ("mean", "sum", "none")[(rows + vocab) % 3]
    x, w, t = inputs(rows, dim, vocab, dtype, rows * 7 + vocab, 0.25 if rows > 4 else 0.0,
                     bits_=32 if dim % 2 else 64)
    check(x, w, t, reduction, torch.float32 if vocab % 2 else None)


# long rows against small tables: the logits' sums over k are split
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,vocab", [(17, 2000, 2), (40, 1203, 91), (300, 2048, 513),
                                            (100, 1500, 1025), (1, 4096, 3), (2500, 1111, 17)])
def test_small_tables(rows, dim, vocab, dtype):
    for reduction in ("mean", "sum", "none"):
        print(f"loss {rows}x{dim}x{vocab} {dtype} {reduction}", flush=True)
        x, w, t = inputs(rows, dim, vocab, dtype, rows + vocab, 0.2 if rows > 1 else 0.0)
        check(x, w, t, reduction)


# float32 rows that are few for their weights: the weights are read as they lie
@pytest.mark.parametrize("rows,dim,vocab", [(3, 1030, 2500), (17, 520, 5001), (33, 2049, 1027),
                                            (100, 1031, 2049), (128, 64, 40000), (129, 1029, 16800),
                                            (300, 4099, 4100), (512, 260, 66000)])
def test_few_rows_for_a_large_table(rows, dim, vocab):
    print(f"loss {rows}x{dim}x{vocab}", flush=True)
    reduction = ("mean", "sum", "none")[rows % 3]
    x, w, t = inputs(rows, dim, vocab, "f32", rows, 0.3)
    check(x, w, t, reduction)


@pytest.mark.parametrize("rows,dim,vocab", [(40, 1033, 4500), (20, 1200, 61)])
def test_strides_and_alignment_beside_large_and_small_tables(rows, dim, vocab):
    x, w, t = inputs(rows, dim, vocab, "f32", 6, 0.2)
    gaps = torch.zeros(rows, dim + 7, device="cuda")[:, 3:3 + dim]
    gaps.copy_(x)
    w2 = torch.zeros(vocab * dim + 1, device="cuda")[1:].view(vocab, dim)
    w2.copy_(w)
    one = torch.ones((), device="cuda")
    out = []
    for xs, ws in ((x, w), (gaps, w2)):
        loss, lse = B.linear_cross_entropy(xs, ws, t, want_lse=True)
        out.append((loss, lse, *B.linear_cross_entropy_backward(one, xs, ws, t, lse)))
    assert all(torch.equal(bits(p), bits(q)) for p, q in zip(*out))


def test_a_small_table_with_rows_and_targets_that_do_not_count():
    """Where the sums are split: padding of NaN reaches nothing, a target outside the table
    has NaN for its row alone, and every row may be ignored."""
    x, w, t = inputs(60, 1500, 70, "bf16", 9, 0.3)
    drop = t == IGNORE
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    dx, dw = B.linear_cross_entropy_backward(loss, x, w, t, lse, IGNORE, "none")
    x2 = torch.where(drop[:, None], torch.full_like(x, float("nan")), x)
    loss2, lse2 = B.linear_cross_entropy(x2, w, t, IGNORE, "none", want_lse=True)
    dx2, dw2 = B.linear_cross_entropy_backward(loss, x2, w, t, lse2, IGNORE, "none")
    for a, b in ((loss, loss2), (lse, lse2), (dx, dx2), (dw, dw2)):
        assert torch.equal(bits(a), bits(b))
    live = int((~drop).nonzero()[0])
    t[live] = 70
    loss = B.linear_cross_entropy(x, w, t, IGNORE, "none")
    assert loss.isnan().nonzero().flatten().tolist() == [live]
    t.fill_(IGNORE)
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "mean", want_lse=True)
    dx, dw = B.linear_cross_entropy_backward(torch.full_like(loss, float("inf")), x, w, t, lse)
    assert loss == 0 and (lse == 0).all() and (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("rows,dim,vocab", [(5, 300, 4000), (20, 1200, 60), (128, 700, 900),
                                            (1500, 40, 300)])
def test_few_results_keep_two_values_of_g(rows, dim, vocab):
    """G as a sum of two bfloat16 is off by 2^-18 of an entry at most, its softmax by the
    logits' float32 errors, under 2^-17 here (lse included, |z| < 16, sums of dim terms of
    2^-24 each that average): as a whole under 2^-13, where one bfloat16 leaves about 2^-9."""
    x, w, t = inputs(rows, dim, vocab, "bf16", 21)
    _, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    gen = torch.Generator(device="cuda").manual_seed(22)
    dloss = 1 + 0.3 * torch.randn(rows, device="cuda", generator=gen)
    _, dw = B.linear_cross_entropy_backward(dloss, x, w, t, lse, IGNORE, "none", want_x=False,
                                            dtype=torch.float32)
    _, want = R.loss_grad(dloss, x, w, t, lse, IGNORE, "none")
    assert (dw.double() - want).norm() < 2.0 ** -13 * want.norm()


@pytest.mark.parametrize("rows,dim,vocab", [(2000, 96, 300), (20, 1200, 60)])
def test_a_factor_of_all_rows_is_not_rounded(rows, dim, vocab):
    """The gradients are the factor times those of the factor 1, though a bfloat16 holds it
    half a step off: two float32 roundings apart at most, one of each result."""
    x, w, t = inputs(rows, dim, vocab, "bf16", 3, 0.1)
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "sum", want_lse=True)
    one = torch.ones((), device="cuda")
    dw = B.linear_cross_entropy_backward(one, x, w, t, lse, IGNORE, "sum",
                                         dtype=torch.float32)[1]
    for c in (1 + 2.0 ** -8, 0.7 * 2.0 ** -12):
        c = torch.tensor(c, device="cuda")
        got = B.linear_cross_entropy_backward(c, x, w, t, lse, IGNORE, "sum",
                                              dtype=torch.float32)[1]
        within(got, dw.double() * c.double(), 2 * R.U32 * (dw.double() * c.double()).abs(), "dw")


@pytest.mark.parametrize("rows,dim,vocab", [(9, 64, 200), (300, 96, 300), (40, 1200, 60),
                                            (40, 260, 70000)])
@pytest.mark.parametrize("factor", [float("inf"), float("nan")])
def test_ignored_rows_have_zero_gradients_whatever_the_factor(rows, dim, vocab, factor):
    x, w, t = inputs(rows, dim, vocab, "f32", 3, 0.4)
    drop = t == IGNORE
    assert drop.any() and not drop.all()
    _, lse = B.linear_cross_entropy(x, w, t, IGNORE, "mean", want_lse=True)
    dx, _ = B.linear_cross_entropy_backward(torch.tensor(factor, device="cuda"), x, w, t, lse,
                                            IGNORE, "mean")
    assert (dx[drop] == 0).all() and not dx[~drop].isfinite().any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_around_the_form_for_few(dtype):
    """15, 16 and 17 rows, with padding among them, every reduction."""
    for rows in (1, 15, 16, 17):
        for reduction in ("none", "sum", "mean"):
            x, w, t = inputs(rows, 200, 1111, dtype, rows, 0.3)
            check(x, w, t, reduction)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [5, 100])
def test_ignored_rows_reach_nothing(rows, dtype):
    """Whatever they hold: NaN and infinities in the activations of padding change no
    bit of the others' results."""
    x, w, t = inputs(rows, 72, 333, dtype, 3, 0.4)
    t[1] = IGNORE
    loss, lse, dloss, dx, dw = check(x, w, t, "mean")
    x2 = x.clone()
    drop = t == IGNORE
    x2[drop] = torch.where(torch.arange(72, device="cuda") % 2 == 0, float("nan"), float("inf")).to(
        x.dtype)
    loss2, lse2 = B.linear_cross_entropy(x2, w, t, IGNORE, "mean", want_lse=True)
    dx2, dw2 = B.linear_cross_entropy_backward(dloss, x2, w, t, lse, IGNORE, "mean",
                                               dtype=x.dtype)
    for a, b in ((loss, loss2), (lse, lse2), (dx, dx2), (dw, dw2)):
        assert torch.equal(bits(a), bits(b))
    assert (dx2[drop] == 0).all() and (lse2[drop] == 0).all()


@pytest.mark.parametrize("rows", [7, 40])
def test_all_rows_ignored(rows):
    """A mean of nothing is 0 and has zero gradients."""
    x, w, _ = inputs(rows, 40, 50, "bf16", 1)
    t = torch.full((rows,), -1, device="cuda")
    for reduction in ("none", "sum", "mean"):
        loss, lse = B.linear_cross_entropy(x, w, t, -1, reduction, want_lse=True)
        assert (loss == 0).all() and (lse == 0).all()
        dx, dw = B.linear_cross_entropy_backward(torch.ones_like(loss), x, w, t, lse, -1, reduction)
        assert (dx == 0).all() and (dw == 0).all()
    # no rows at all
    loss, lse = B.linear_cross_entropy(x[:0], w, t[:0], want_lse=True)
    assert loss.item() == 0 and lse.shape == (0,)
    acc = torch.full((50, 40), 3.0, device="cuda")
    dx, dw = B.linear_cross_entropy_backward(loss, x[:0], w, t[:0], lse, dweight=acc,
                                             accumulate=True)
    assert dx.shape == (0, 40) and (dw == 3).all()
    assert (B.linear_cross_entropy_backward(loss, x[:0], w, t[:0], lse)[1] == 0).all()


@pytest.mark.parametrize("rows", [6, 50])
def test_targets_outside_the_table(rows):
    """Their rows' loss and gradients are NaN, no others' loss is."""
    x, w, t = inputs(rows, 40, 64, "f32", 2)
    t[2], t[4] = 64, -3
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[2] = bad[4] = True
    assert torch.equal(loss.isnan(), bad) and not lse.isnan().any()
    assert B.linear_cross_entropy(x, w, t, IGNORE, "mean").isnan()
    dx, dw = B.linear_cross_entropy_backward(torch.ones_like(loss), x, w, t, lse, IGNORE, "none")
    assert torch.equal(dx.isnan().all(1), bad) and torch.equal(dx.isnan().any(1), bad)
    assert dw.isnan().all()
    # an ignored index inside the table is ignored all the same
    t = torch.arange(rows, device="cuda") % 64
    loss = B.linear_cross_entropy(x, w, t, 3, "none")
    assert loss[3] == 0 and (loss != 0).sum() == rows - 1


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [9, 130])
def test_nonfinite_values(rows, dtype):
    """A NaN in a row that counts is its own row's; one in the table is everyone's."""
    x, w, t = inputs(rows, 64, 100, dtype, 4)
    x[3, 7] = float("nan")
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    assert loss.isnan().sum() == 1 and loss[3].isnan() and lse.isnan().sum() == 1
    dx, dw = B.linear_cross_entropy_backward(torch.ones_like(loss), x, w, t, lse, IGNORE, "none")
    assert dx.isnan().any(1).sum() == 1 and dx[3].isnan().all()
    assert dw.isnan().all()
    x, w, t = inputs(rows, 64, 100, dtype, 4)
    w[50, 3] = float("nan")
    assert B.linear_cross_entropy(x, w, t, IGNORE, "none").isnan().all()
    w[50, 3] = 0
    w[50] = 0
    x[:, 0], w[50, 0] = 1, float("-inf")      # a logit of -inf: probability zero
    t[t == 50] = 51
    loss, lse = B.linear_cross_entropy(x[:, :8], w[:, :8].contiguous(), t, IGNORE, "none",
                                       want_lse=True)
    if dtype == "bf16":                        # (planes of a float32 infinity are not finite)
        keep = torch.arange(100, device="cuda") != 50
        want = torch.logsumexp(x[:, :8].double() @ w[keep][:, :8].double().T, 1)
        assert (lse.double() - want).abs().max() < 1e-4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_large_logits(dtype):
    """Far apart and far from zero: the largest decides, nothing overflows."""
    x, w, t = inputs(200, 64, 300, dtype, 5, spread=100.0)
    loss, lse, *_ = check(x, w, t, "mean")
    assert lse.isfinite().all() and lse.abs().max() > 200


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [64, 65])
def test_strides_alignment_and_dimensions(dim, dtype):
    """Rows with gaps, starts off any 16 bytes, leading dimensions: the bits of
    contiguous calls."""
    x, w, t = inputs(60, dim, 200, dtype, 6, 0.2)
    want = check(x, w, t, "sum")
    pad = torch.zeros(60, dim + 7, device="cuda", dtype=x.dtype)
    flat = torch.zeros(200 * dim + 1, device="cuda", dtype=x.dtype)
    x2 = pad[:, 3:3 + dim]
    x2.copy_(x)
    w2 = flat[1:].view(200, dim)
    w2.copy_(w)
    for xs, ws in ((x2, w), (x, w2), (x2, w2)):
        loss, lse = B.linear_cross_entropy(xs, ws, t, IGNORE, "sum", want_lse=True)
        dx, dw = B.linear_cross_entropy_backward(want[2], xs, ws, t, lse, IGNORE, "sum",
                                                 dtype=x.dtype)
        for a, b in zip((loss, lse, dx, dw), (want[0], want[1], want[3], want[4])):
            assert torch.equal(bits(a), bits(b))
    x3, t3 = x.view(3, 4, 5, dim), t.view(3, 4, 5)
    loss, lse = B.linear_cross_entropy(x3, w, t3, IGNORE, "none", want_lse=True)
    assert loss.shape == lse.shape == (3, 4, 5)
    dx, _ = B.linear_cross_entropy_backward(loss, x3, w, t3, lse, IGNORE, "none")
    assert dx.shape == x3.shape


def test_outputs_one_by_one_in_place_and_added():
    x, w, t = inputs(90, 64, 300, "f32", 8, 0.1)
    loss, lse = B.linear_cross_entropy(x, w, t, want_lse=True)
    one = torch.ones((), device="cuda")
    dx, dw = B.linear_cross_entropy_backward(one, x, w, t, lse)
    a, b = B.linear_cross_entropy_backward(one, x, w, t, lse, want_x=False)
    assert a is None and torch.equal(b, dw)
    a, b = B.linear_cross_entropy_backward(one, x, w, t, lse, want_weight=False)
    assert b is None and torch.equal(a, dx)
    acc = torch.full_like(dw, 1.0)
    B.linear_cross_entropy_backward(one, x, w, t, lse, dweight=acc, accumulate=True)
    assert torch.equal(acc, 1.0 + dw)
    x2 = x.clone()
    B.linear_cross_entropy_backward(one, x2, w, t, lse, dX=x2, dweight=torch.empty_like(dw))
    assert torch.equal(x2, dx)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_pieces_of_the_vocabulary(dtype):
    """Sums that are exact in any order: logits all zero, so every probability is
    2^-16, and small integers elsewhere.  The gradient goes in several pieces of the
    vocabulary (2^30 bytes of it at a time); one row, token or piece lost or twice
    would show."""
    rows, dim, vocab = (20000, 16, 65536)
    x = torch.zeros(rows, dim, device="cuda", dtype=DT[dtype])
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randint(-3, 4, (vocab, dim), device="cuda", generator=gen).to(DT[dtype])
    t = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    t[::3] = IGNORE
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    keep = t != IGNORE
    ln = 16 * 0.6931471805599453
    assert (lse[keep] - ln).abs().max() < 1e-5 and (loss[keep] - ln).abs().max() < 1e-5
    dloss = torch.full((rows,), 65536.0, device="cuda")
    dx, _ = B.linear_cross_entropy_backward(dloss, x, w, t, torch.full_like(lse, ln), IGNORE,
                                            "none", want_weight=False, dX=torch.empty_like(x))
    # G is exp(-lse) 65536 = 1 to 2^-20, but for the target's 1 - 65536
    cols = w.double().sum(0)
    want = torch.where(keep[:, None], cols - 65536.0 * w.double()[t.clamp(min=0)], 0.0)
    tol = 2.0 ** -7 * 65536 * 4 if dtype == "bf16" else 2.0 ** -17 * 65536 * 20
    assert (dx.double() - want).abs().max() <= tol
    x.fill_(1.0)
    w.zero_()
    _, dw = B.linear_cross_entropy_backward(dloss, x, w, t, torch.full_like(lse, ln), IGNORE,
                                            "none", want_x=False)
    counts = torch.bincount(t[keep], minlength=vocab).double()
    want = (int(keep.sum()) - 65536.0 * counts)[:, None].expand(vocab, dim)
    tol = 65536 * counts.max() * 2.0 ** -8 + int(keep.sum()) * 2.0 ** -18
    assert (dw.double() - want).abs().max() <= tol
    empty = counts == 0
    assert (dw.double() - want)[empty].abs().max() <= int(keep.sum()) * 2.0 ** -18


@pytest.mark.parametrize("shapes", [((300, 64, 1000, "bf16"), (40, 128, 777, "f32"),
                                     (8, 128, 777, "bf16")),
                                    ((40, 1200, 60, "bf16"), (40, 1033, 4500, "f32"),
                                     (150, 515, 33000, "f32"))])
def test_streams_and_graphs(shapes):
    """Calls at once on streams of their own, and a graph replayed between eager
    calls with other inputs: the same bits each time."""
    cases = [inputs(*s, 11 + i, 0.2 if s[0] > 8 else 0.0) for i, s in enumerate(shapes)]

    def both(x, w, t):
        loss, lse = B.linear_cross_entropy(x, w, t, want_lse=True)
        dx, dw = B.linear_cross_entropy_backward(torch.ones_like(loss), x, w, t, lse)
        return loss, lse, dx, dw

    want = [both(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(3):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(both(*c))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(a, b))
    for c, b in zip(cases, want):
        static = [v.clone() for v in c]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            both(*static)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = both(*static)
        for turn in range(3):
            static[0].copy_(c[0] if turn != 1 else c[0] * 0.5)
            g.replay()
            ref = b if turn != 1 else both(c[0] * 0.5, *c[1:])
            torch.cuda.synchronize()
            assert all(torch.equal(bits(p), bits(q)) for p, q in zip(out, ref))


@pytest.mark.slow
def test_offsets_past_32_bits():
    """Rows 2^33 bytes apart in X, a table and a gradient of 2^32 bytes and more."""
    dim = 2048
    store = torch.zeros((1 << 32) + 8192, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((3, dim), (1 << 31, 1))
    x.normal_()
    gen = torch.Generator(device="cuda").manual_seed(3)
    vocab = (1 << 20) + 0
    w = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    w.normal_(std=0.05, generator=gen)
    t = torch.tensor([0, vocab - 1, vocab // 2 + 77], device="cuda")
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    z = x.float().contiguous() @ w.float().T
    want = torch.logsumexp(z.double(), 1)
    assert (lse.double() - want).abs().max() < 1e-4
    assert (loss.double() - (want - z.double()[torch.arange(3), t])).abs().max() < 1e-4
    dx, dw = B.linear_cross_entropy_backward(torch.ones_like(loss), x, w, t, lse, IGNORE, "none",
                                             dtype=torch.bfloat16)
    g = torch.exp(z - lse[:, None])
    g[torch.arange(3), t] -= 1
    ref = g @ w.float()
    assert ((dx.float() - ref).norm() / ref.norm()) < 2.0 ** -7
    for v in (0, 1, vocab // 2 + 77, vocab - 1):
        row = g[:, v] @ x.float().contiguous()
        assert (dw[v].float() - row).norm() <= 2.0 ** -7 * row.norm() + 1e-6


def confident(rows, dim, vocab, dtype, factor, tops, seed):
    """Rows whose target's logit is the largest: activations along the target's weights, times
    factor, and a first column that moves all of a row's logits, so that the target's is near
    tops[row] (None: as it comes).  (x, w, t, logits in 64 bits, the others' distances below
    the target's)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(vocab, dim, device="cuda", generator=gen)
    w[:, 0] = 1.0
    w = w.to(DT[dtype])
    t = torch.randint(vocab, (rows,), device="cuda", generator=gen)
    x = (factor * w[t].double()).to(DT[dtype])
    if tops is not None:
        x[:, 0] = 0.0
        x[:, 0] = (tops - (x.double() * w[t].double()).sum(1)).to(DT[dtype])
    z = x.double() @ w.double().T
    rest = torch.ones_like(z, dtype=torch.bool)
    rest[torch.arange(rows, device="cuda"), t] = False
    gap = (z.gather(1, t[:, None]) - z)[rest].view(rows, vocab - 1)
    return x, w, t, z, gap


# every form of the statistics: few rows; tiles of either size; split sums; float32 weights
# as they lie
FORMS = [(12, 64, 300, "f32"), (12, 64, 300, "bf16"), (300, 64, 1000, "f32"),
         (300, 64, 1000, "bf16"), (2500, 64, 5000, "f32"), (2500, 64, 5000, "bf16"),
         (40, 1203, 91, "f32"), (40, 1203, 91, "bf16"), (128, 64, 40000, "f32")]


@pytest.mark.parametrize("rows,dim,vocab,dtype", FORMS)
def test_a_certain_target_has_no_loss(rows, dim, vocab, dtype):
    """Its logit leads by 40 or more, so that all other terms together are below 2^-25: 1 and
    they are 1, whose logarithm is 0, and the loss is 0 to the last bit in every form,
    whatever the logits' size.  lse is the target's logit then."""
    steps = torch.linspace(0, 1, rows, device="cuda", dtype=torch.float64)
    sizes = 20.0 * 50.0 ** steps
    for factor, tops in ((12.0, sizes), (12.0, -sizes), (1e3, None), (2e9, None), (1e30, None)):
        x, w, t, z, gap = confident(rows, dim, vocab, dtype, factor, tops, rows + vocab)
        assert gap.min() > 40 + torch.log(torch.tensor(float(vocab)))
        loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
        assert (loss == 0).all(), (factor, loss.min().item(), loss.max().item())
        e = R.product_error(dim, x.dtype) * (x.double().abs() @ w.double().abs().T)
        within(lse, z.gather(1, t[:, None])[:, 0], e.gather(1, t[:, None])[:, 0] + R.TINY, "lse")
        assert B.linear_cross_entropy(x, w, t, IGNORE, "mean") == 0


@pytest.mark.parametrize("rows,dim,vocab,dtype", FORMS)
def test_a_likely_target_has_a_loss_of_its_own_size(rows, dim, vocab, dtype):
    """The target leads by little, at logits up to 1000: the loss is not negative, and off by
    errors of its own size, never by one of the logits' (R.likely_loss)."""
    steps = torch.linspace(0, 1, rows, device="cuda", dtype=torch.float64)
    sizes = 20.0 * 50.0 ** steps
    for tops in (sizes, -sizes):
        x, w, t, _, _ = confident(rows, dim, vocab, dtype, 0.3 if dim < 100 else 0.01, tops,
                                  rows + vocab)
        loss = B.linear_cross_entropy(x, w, t, IGNORE, "none")
        assert (loss >= 0).all(), loss.min().item()
        within(loss, *R.likely_loss(x, w, t), "loss")


@pytest.mark.parametrize("rows,dim,vocab,dtype", FORMS)
def test_logits_up_to_the_types_largest(rows, dim, vocab, dtype):
    """Logits of 1 to 1.75 times 2^127 and their negatives, past 2^128 / log2(e): all sums are
    exact, probabilities are 0 or 1, and losses, statistics and gradients are finite."""
    level = torch.tensor([1.0, 1.25, 1.5, -1.5, -1.25, -1.0], device="cuda", dtype=torch.float64)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    a = level[torch.randint(6, (vocab,), device="cuda", generator=gen)]
    a[7], a[11] = 1.75, -1.75
    w = torch.zeros(vocab, dim, device="cuda", dtype=DT[dtype])
    w[:, 0] = (a * 2.0 ** 63).to(DT[dtype])
    x = torch.zeros(rows, dim, device="cuda", dtype=DT[dtype])
    sign = torch.where(torch.arange(rows, device="cuda") % 3 == 1, -1.0, 1.0).double()
    x[:, 0] = (sign * 2.0 ** 64).to(DT[dtype])
    # targets on the row's own side: the distance from the largest stays in range
    same = [torch.nonzero(a * s > 0)[:, 0] for s in (1, -1)]
    pick = torch.randint(1 << 30, (rows,), device="cuda", generator=gen)
    t = torch.where(sign > 0, same[0][pick % len(same[0])], same[1][pick % len(same[1])])
    t[:4] = torch.where(sign[:4] > 0, 7, 11)
    top = torch.where(sign > 0, 7, 11)
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    assert (lse.double() == 1.75 * 2.0 ** 127).all()
    assert torch.equal(loss.double(), (a[top] - a[t]).abs() * 2.0 ** 127)
    one = torch.ones((rows,), device="cuda")
    dx, dw = B.linear_cross_entropy_backward(one, x, w, t, lse, IGNORE, "none",
                                             dtype=torch.float32)
    g = torch.zeros(rows, vocab, device="cuda", dtype=torch.float64)
    rows_ = torch.arange(rows, device="cuda")
    g[rows_, top] += 1
    g[rows_, t] -= 1
    assert torch.equal(dx.double(), g @ w.double())
    assert torch.equal(dw.double(), g.T.contiguous() @ x.double())


@pytest.mark.parametrize("rows,dim,vocab", [(12, 64, 300), (300, 64, 1000), (40, 1203, 91),
                                            (40, 1033, 4500)])
def test_finite_float32_activations_up_to_the_largest(rows, dim, vocab):
    """float32's largest values, a mask's for instance, past the largest bfloat16: beside small
    weights they are numbers like others."""
    x, w, t = inputs(rows, dim, vocab, "f32", 31, 0.1)
    big = torch.finfo(torch.float32).max
    x[:, 0] = torch.where(torch.arange(rows, device="cuda") % 2 == 0, big, -big)
    w[:, 0] = torch.where(torch.arange(vocab, device="cuda") % 3 == 0, 2.0 ** -126, -2.0 ** -126)
    loss, lse = B.linear_cross_entropy(x, w, t, IGNORE, "none", want_lse=True)
    want, want_lse = R.loss(x, w, t, IGNORE)
    e_each, e_lse = R.loss_bounds(x, w, t, IGNORE)
    within(lse, want_lse, e_lse, "lse")
    within(loss, want, e_each, "loss")
    args = (torch.ones(rows, device="cuda"), x, w, t, lse, IGNORE, "none")
    dx, _ = B.linear_cross_entropy_backward(*args, want_weight=False)
    # (but for the column of weights of 2^-126, whose products are below float32's range)
    within(dx[:, 1:], R.loss_grad(*args)[0][:, 1:],
           R.loss_grad_bounds(*args, torch.float32)[0][:, 1:], "dx")
