"""Gated feed-forward block on the GPU, forward and backward, against its definition
in 64 bits (tests/block_reference.py)."""
import pytest

from distributed_bit_matrix_amd import binding as B
from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t.view(torch.int32)


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           off[bad][:4].tolist(), bound.expand(bad.shape)[bad][:4].tolist())


def normal(seed, *shape, dtype="f32", std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(*shape, device="cuda", generator=gen)).to(DT[dtype])


def inputs(rows, dim, hidden, dtype, seed):
    x = normal(seed, rows, dim, dtype=dtype)
    wg = normal(seed + 1, hidden, dim, dtype=dtype, std=1.5 * dim ** -0.5)
    wu = normal(seed + 2, hidden, dim, dtype=dtype, std=dim ** -0.5)
    wd = normal(seed + 3, dim, hidden, dtype=dtype, std=hidden ** -0.5)
    return x, wg, wu, wd


def check_forward(x, wg, wu, wd, kind):
    y, pre = B.gated_mlp(x, wg, wu, wd, kind, want_pre=True)
    want, want_pre = R.mlp(x, wg, wu, wd, kind)
    b_y, b_pre = R.mlp_bounds(x, wg, wu, wd, kind)
    within(pre, want_pre, b_pre, "pre")
    within(y, want, b_y, "y")
    assert torch.equal(bits(B.gated_mlp(x, wg, wu, wd, kind)), bits(y))
    return y, pre


def check_backward(dy, x, wg, wu, wd, pre, kind, dw_dtype):
    got = B.gated_mlp_backward(dy, x, wg, wu, wd, pre, kind, dtype=dw_dtype)
    want = R.mlp_grad(dy, x, wg, wu, wd, pre, kind)
    bound = R.mlp_grad_bounds(dy, x, wg, wu, wd, pre, kind, dw_dtype)
    for g, w, b, name in zip(got, want, bound, ("dx", "dw_gate", "dw_up", "dw_down")):
        within(g, w, b, name)
    return got


# one row and column, sizes around 16 rows, tiles of 64, 128 and 256 and pieces of 8
SHAPES = [(1, 1, 1), (1, 8, 16), (2, 3, 5), (7, 40, 24), (15, 64, 65), (16, 129, 257),
          (17, 130, 256), (31, 256, 127), (64, 65, 128), (65, 127, 129), (128, 128, 64),
          (129, 256, 255), (256, 96, 512), (257, 33, 300), (300, 513, 130), (777, 257, 1001),
          (512, 256, 768), (1, 2048, 1000), (9, 1000, 2048)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim,hidden", SHAPES)
def test_shapes(rows, dim, hidden, dtype):
    print(f"mlp {rows}x{dim}x{hidden} {dtype}", flush=True)
    kind = "gelu" if (rows + dim) % 2 else "silu"
    x, wg, wu, wd = inputs(rows, dim, hidden, dtype, rows * 31 + dim)
    _, pre = check_forward(x, wg, wu, wd, kind)
    dy = normal(rows + 5, rows, dim, dtype=dtype)
    check_backward(dy, x, wg, wu, wd, pre, kind, DT["f32"] if hidden % 2 else DT[dtype])


# float32 rows that are few for their weights: the weights are read as they lie
@pytest.mark.parametrize("rows,dim,hidden", [(1, 700, 1100), (17, 515, 1400), (33, 1030, 700),
                                             (64, 64, 11000), (100, 1027, 1029), (128, 4100, 180),
                                             (129, 2050, 2800), (257, 1300, 4400),
                                             (512, 5700, 1000)])
def test_few_rows_for_large_weights(rows, dim, hidden):
    print(f"mlp {rows}x{dim}x{hidden}", flush=True)
    kind = "gelu" if rows % 2 else "silu"
    x, wg, wu, wd = inputs(rows, dim, hidden, "f32", rows * 31 + dim)
    _, pre = check_forward(x, wg, wu, wd, kind)
    dy = normal(rows + 5, rows, dim)
    check_backward(dy, x, wg, wu, wd, pre, kind, DT["f32"])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [6, 70])
@pytest.mark.parametrize("dim,hidden", [(64, 128), (65, 127)])
def test_strides_alignment_and_dimensions(dim, hidden, rows, dtype):
    """Rows with gaps, starts off any 16 bytes, leading dimensions: the bits of
    contiguous calls."""
    x, wg, wu, wd = inputs(rows, dim, hidden, dtype, 5)
    dy = normal(9, rows, dim, dtype=dtype)
    y, pre = check_forward(x, wg, wu, wd, "silu")
    want = check_backward(dy, x, wg, wu, wd, pre, "silu", x.dtype)

    def gaps(t):
        pad = torch.zeros(rows, dim + 5, device="cuda", dtype=t.dtype)
        pad[:, 3:3 + dim] = t
        return pad[:, 3:3 + dim]

    def off(t):
        flat = torch.zeros(t.numel() + 1, device="cuda", dtype=t.dtype)
        flat[1:] = t.flatten()
        return flat[1:].view(t.shape)

    for a in ((gaps(x), wg, wu, wd), (x, off(wg), wu, wd), (x, wg, off(wu), wd),
              (x, wg, wu, off(wd)), (gaps(x), off(wg), off(wu), off(wd))):
        y2, pre2 = B.gated_mlp(*a, want_pre=True)
        assert torch.equal(bits(y2), bits(y)) and torch.equal(pre2, pre)
        got = B.gated_mlp_backward(gaps(dy), *a, pre, dtype=x.dtype)
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(got, want))
    lead = (rows // 2, 2, dim)
    y3, pre3 = B.gated_mlp(x.view(lead), wg, wu, wd, want_pre=True)
    assert y3.shape == lead and pre3.shape == (rows // 2, 2, 2 * hidden)
    assert torch.equal(bits(y3.view(rows, dim)), bits(y))


def test_outputs_one_by_one_and_added():
    x, wg, wu, wd = inputs(50, 64, 96, "f32", 3)
    dy = normal(4, 50, 64)
    pre = B.gated_mlp(x, wg, wu, wd, want_pre=True)[1]
    want = B.gated_mlp_backward(dy, x, wg, wu, wd, pre)
    for i in range(4):
        got = B.gated_mlp_backward(dy, x, wg, wu, wd, pre,
                                   want=tuple(j == i for j in range(4)))
        # (another number of products in a launch may split their sums differently)
        assert [g is not None for g in got] == [j == i for j in range(4)]
        assert torch.equal(got[i], want[i])
    acc = [torch.full_like(g, 0.5) for g in want[1:]]
    B.gated_mlp_backward(dy, x, wg, wu, wd, pre, dw_gate=acc[0], dw_up=acc[1], dw_down=acc[2],
                         accumulate=True)
    assert all(torch.equal(a, 0.5 + g) for a, g in zip(acc, want[1:]))


def test_no_rows():
    x, wg, wu, wd = inputs(4, 16, 24, "bf16", 3)
    e = x[:0]
    y, pre = B.gated_mlp(e, wg, wu, wd, want_pre=True)
    assert y.shape == (0, 16) and pre.shape == (0, 48)
    dx, *dw = B.gated_mlp_backward(e, e, wg, wu, wd, pre, dtype=torch.bfloat16)
    assert dx.shape == (0, 16) and all((g == 0).all() for g in dw)
    acc = [torch.full(w.shape, 2.0, device="cuda") for w in (wg, wu, wd)]
    B.gated_mlp_backward(e, e, wg, wu, wd, pre, dw_gate=acc[0], dw_up=acc[1], dw_down=acc[2],
                         accumulate=True)
    assert all((a == 2).all() for a in acc)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("rows", [5, 60])
def test_gates_far_from_zero(rows, kind):
    """Gates where the exponentials overflow or vanish; NaN stays in its row."""
    dim, hidden = 32, 64
    x, wg, wu, wd = inputs(rows, dim, hidden, "f32", 3)
    wg = wg * 200
    y, pre = check_forward(x, wg, wu, wd, kind)
    assert pre.abs().max() > 500 and y.isfinite().all()
    dy = normal(4, rows, dim)
    got = check_backward(dy, x, wg, wu, wd, pre, kind, torch.float32)
    assert all(g.isfinite().all() for g in got)
    x[2, 3] = float("nan")
    y, pre = B.gated_mlp(x, wg, wu, wd, kind, want_pre=True)
    assert y.isnan().any(1).sum() == 1 and y[2].isnan().all()
    dx, *dw = B.gated_mlp_backward(dy, x, wg, wu, wd, pre, kind)
    assert dx.isnan().any(1).sum() == 1 and all(g.isnan().any() for g in dw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_that_are_exact(dtype):
    """Small integers through gates so large that silu is the identity: every product
    is exact in any order, so one row, feature or split lost or twice shows."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, device="cuda", generator=gen).to(DT[dtype])

    for rows, dim, hidden in ((2000, 96, 1500), (20, 5000, 64), (5000, 40, 72), (9, 4100, 520)):
        x = ints(0, 2, rows, dim) * 0
        x[:, 0] = 64
        x[:, 1] = ints(-1, 2, rows)
        wg = torch.zeros(hidden, dim, device="cuda", dtype=DT[dtype])
        wu, wd = wg.clone(), ints(-2, 3, dim, hidden)
        wg[:, 0] = 2                     # gate 128: silu(128) = 128
        wu[:, 1] = ints(-2, 3, hidden)
        y, pre = B.gated_mlp(x, wg, wu, wd, want_pre=True)
        g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
        assert torch.equal(pre.double(), torch.cat([g, u], 1))
        want = (g * u) @ wd.double().T
        assert torch.equal(y.double(), want.to(DT[dtype]).double())
        dy = ints(-1, 2, rows, dim)
        dx, dwg, dwu, dwd = B.gated_mlp_backward(dy, x, wg, wu, wd, pre)
        dh = dy.double() @ wd.double()
        # (dg and du are rounded to the operands' type; where the results are few, below
        # 4096 values, they have two bfloat16, which hold these integers as they are)
        dg, du = dh * u, dh * g
        if rows * min(dim, hidden) >= 4096:
            dg, du = (v.to(DT[dtype]).double() for v in (dg, du))
        assert torch.equal(dwd.double(), dy.double().T @ (g * u))
        assert torch.equal(dwg.double(), dg.T @ x.double())
        assert torch.equal(dwu.double(), du.T @ x.double())
        assert torch.equal(dx.double(), (dg @ wg.double() + du @ wu.double()).to(DT[dtype]).double())


@pytest.mark.parametrize("rows,dim,hidden", [(3, 200, 900), (16, 65, 700), (40, 90, 1000),
                                             (20, 2000, 90)])
def test_few_results_keep_two_values_between_the_products(rows, dim, hidden):
    """h as a sum of two bfloat16 is off by 2^-18 of a value at most, and its float32 sums
    by less: y is its own rounding, half a step, and 2^-15 of its terms' sizes."""
    x, wg, wu, wd = inputs(rows, dim, hidden, "bf16", 23)
    y, pre = B.gated_mlp(x, wg, wu, wd, want_pre=True)
    g, u = pre.double().chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    want, sizes = h @ wd.double().T, h.abs() @ wd.double().abs().T
    within(y, want, torch.finfo(torch.bfloat16).eps / 2 * want.abs() + 2.0 ** -15 * sizes, "y")


@pytest.mark.parametrize("shapes", [((300, 64, 256, "bf16"), (5, 128, 512, "bf16"),
                                     (70, 65, 90, "f32")),
                                    ((40, 1030, 1500, "f32"), (3, 64, 33, "bf16"),
                                     (20, 40, 90, "bf16"))])
def test_streams_and_graphs(shapes):
    """Calls at once on streams of their own, and a graph replayed between eager calls
    with other inputs."""
    cases = [(*inputs(r, d, h, dt, r), normal(7, r, d, dtype=dt)) for r, d, h, dt in shapes]

    def both(x, wg, wu, wd, dy):
        y, pre = B.gated_mlp(x, wg, wu, wd, "gelu", want_pre=True)
        return (y, pre, *B.gated_mlp_backward(dy, x, wg, wu, wd, pre, "gelu"))

    want = [both(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(both(*c))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(a, b))
    for c, b in zip(cases, want):
        static = [t.clone() for t in c]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = both(*static)
        for turn in range(3):
            static[0].copy_(c[0] if turn != 1 else c[0] * 2)
            g.replay()
            ref = b if turn != 1 else both(c[0] * 2, *c[1:])
            torch.cuda.synchronize()
            assert all(torch.equal(bits(p), bits(q)) for p, q in zip(out, ref))


def test_gradients_against_differences():
    """The library's own forward pass, in float32, moved along a direction: central
    differences of a loss of about 1 with a step of 2^-7 are off by the third
    derivative (2^-14 of it) and by the roundings over the step (2^-24 2^7)."""
    x, wg, wu, wd = inputs(40, 48, 80, "f32", 3)
    dy = normal(4, 40, 48) / (40 * 48)
    for kind in ("silu", "gelu"):
        pre = B.gated_mlp(x, wg, wu, wd, kind, want_pre=True)[1]
        grads = B.gated_mlp_backward(dy, x, wg, wu, wd, pre, kind)
        for i, g in enumerate(grads):
            args = [x, wg, wu, wd]
            way = normal(20 + i, *g.shape)
            way = way / way.abs().max()
            ends = []
            for sign in (1, -1):
                moved = list(args)
                moved[i] = args[i] + sign * 2.0 ** -7 * way
                ends.append((B.gated_mlp(*moved, kind).double() * dy.double()).sum().item())
            slope = (ends[0] - ends[1]) * 2.0 ** 6
            want = (g.double() * way.double()).sum().item()
            assert abs(slope - want) <= 2.0 ** -9 * max(1.0, abs(want)), (kind, i, slope, want)


def test_refusals():
    x, wg, wu, wd = inputs(4, 16, 24, "f32", 3)
    for call in (lambda: B.gated_mlp(x.half(), wg, wu, wd), lambda: B.gated_mlp(x, wg.bfloat16(), wu, wd),
                 lambda: B.gated_mlp(x, wg, wu, wd.t()), lambda: B.gated_mlp(x, wg, wu[:5], wd),
                 lambda: B.gated_mlp(x, wg[0], wu, wd), lambda: B.gated_mlp(x.t(), wg, wu, wd),
                 lambda: B.gated_mlp_backward(x, x, wg, wu, wd, torch.zeros(4, 24, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: B.gated_mlp(x, wg, wu, wd, "relu"), lambda: B.gated_mlp(x, wg.cpu(), wu, wd),
                 lambda: B.gated_mlp_backward(x, x, wg, wu, wd, torch.zeros(4, 48, device="cuda"),
                                              accumulate=True)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.SignMuonError):
        B.gated_mlp(x, wg, wu, wd, Y=x)


BIG = torch.finfo(torch.float32).max


# few rows; tiles with the gate in their epilogue; split sums; weights as they lie
@pytest.mark.parametrize("rows,dim,hidden", [(9, 96, 200), (300, 64, 1000), (40, 1203, 91),
                                             (40, 768, 1100)])
def test_finite_float32_values_up_to_the_largest(rows, dim, hidden):
    """float32's largest values, past the largest bfloat16, as activations, gradients and
    what lies between the products: beside small weights they are numbers like others."""
    sign = torch.where(torch.arange(rows, device="cuda") % 2 == 0, 1.0, -1.0)
    small = torch.where(torch.arange(hidden, device="cuda") % 3 == 0, 2.0 ** -126, -2.0 ** -126)
    x, wg, wu, wd = inputs(rows, dim, hidden, "f32", 41)
    x[:, 0] = sign * BIG
    wg[:, 0], wu[:, 0] = small, -small
    _, pre = check_forward(x, wg, wu, wd, "silu")
    dy = normal(42, rows, dim)
    dy[:, 0] = sign * BIG
    wd[0] = small
    got = B.gated_mlp_backward(dy, x, wg, wu, wd, pre, want=(True, False, False, False))[0]
    args = (dy, x, wg, wu, wd, pre, "silu")
    # (but for the column of weights of 2^-126, whose products are below float32's range)
    within(got[:, 1:], R.mlp_grad(*args)[0][:, 1:],
           R.mlp_grad_bounds(*args, torch.float32)[0][:, 1:], "dx")
    # act(gate) * up of a feature is the largest value itself
    x, wg, wu, wd = inputs(rows, dim, hidden, "f32", 43)
    x[:, 0] = 1.0
    wg[0], wu[0] = 0.0, 0.0
    wg[0, 0], wu[0, 0] = 2.0 ** 64, (1 - 2.0 ** -24) * 2.0 ** 64
    wd[:, 0] = torch.where(torch.arange(dim, device="cuda") % 3 == 0, 2.0 ** -126, -2.0 ** -126)
    _, pre = check_forward(x, wg, wu, wd, "silu")
    dy = 2.0 ** -20 * normal(44, rows, dim)
    got = B.gated_mlp_backward(dy, x, wg, wu, wd, pre, want=(False, False, False, True))[3]
    args = (dy, x, wg, wu, wd, pre, "silu")
    within(got, R.mlp_grad(*args)[3], R.mlp_grad_bounds(*args, torch.float32)[3], "dw_down")


@pytest.mark.parametrize("rows,dim,hidden", [(9, 96, 200), (300, 64, 1000), (40, 1203, 91),
                                             (40, 768, 1100)])
def test_small_float32_operands(rows, dim, hidden):
    """An operand is held to 2^-133 at least, below float32's normal range too: from 2^-109 on
    that is all of its 24 bits.  (Products with 1 and sums with 0 are exact.)"""
    gen = torch.Generator(device="cuda").manual_seed(6)
    part = 1 + torch.randint(1 << 23, (hidden,), device="cuda", generator=gen).double() * 2.0 ** -23
    wd = torch.zeros(dim, hidden, device="cuda")
    for power in (-100, -109, -110, -118, -126, -130, -140):
        small = (part * 2.0 ** power).float()
        x = torch.zeros(rows, dim, device="cuda")
        w = torch.zeros(hidden, dim, device="cuda")
        x[:, 0], w[:, 0] = 1, small
        want = small.double().repeat(2)
        off = (B.gated_mlp(x, w, w, wd, want_pre=True)[1].double() - want).abs().max()
        assert off == 0 if power >= -109 else off <= 2.0 ** -133
        x[:, 0], w[:, 0] = small[0], 1
        off = (B.gated_mlp(x, w, w, wd, want_pre=True)[1].double() - want[0]).abs().max()
        assert off == 0 if power >= -109 else off <= 2.0 ** -133
