"""Residual root-mean-square norm on the GPU, forward (also with 8-bit output) and
backward, against its definition in 64 bits (tests/block_reference.py)."""
import pytest

from distributed_bit_matrix_amd import binding as B
from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 2.0 ** -20


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist(),
                           off[bad][:4].tolist(), bound.expand(bad.shape)[bad][:4].tolist())


def normal(seed, *shape, dtype="f32", std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (std * torch.randn(*shape, device="cuda", generator=gen)).to(DT[dtype])


def check_codes(q, scales, y, e_y, block):
    """Scales within the error of their maxima; a code within half a step of its
    value over the scale."""
    want = R.e4m3_scales(y, block)
    within(scales, want, R.e4m3_scales(e_y, block) + 2 * R.U32 * want, "scales")
    cols = y.shape[-1]
    s = scales.double()
    s = s.expand(y.shape) if block is None else s.repeat_interleave(block, -1)[..., :cols]
    v = y / s
    bound = R.e4m3_half_step(v) + e_y / s + 2 * R.U32 * v.abs()
    within(q.float(), v, bound, "codes")


@pytest.mark.parametrize("block", [128, None])
@pytest.mark.parametrize("x_std,w_std", [(1e-18, 1e-14), (1e-18, 1e-25), (1e-3, 1e-36), (1e3, 1e28),
                                         (1e15, 1e18), (1e15, 1e-33), (1.0, 1e-38)])
def test_codes_over_float32s_range(x_std, w_std, block):
    """Products of a row and the weights past what the codes' shorter way takes, and scales
    at their least."""
    x = normal(5, 40, 300) * x_std
    w = normal(6, 300) * w_std
    q, scales = B.rms_norm_e4m3(x, w, None, EPS, block)
    want, _ = R.rms(x, w, EPS)
    e_y, _ = R.rms_bounds(x, w, EPS)
    # (values below float32's normal range may be flushed: to nothing beside the least scale)
    check_codes(q, scales, want, e_y + 2.0 ** -126, block)


# every boundary of the kernels' row widths, odd ones, one column and many
SHAPES = [(1, 1), (3, 1), (5, 2), (7, 3), (257, 4), (33, 7), (65, 8), (64, 9), (100, 31),
          (9, 32), (130, 33), (77, 63), (41, 64), (19, 65), (50, 127), (23, 128), (31, 255),
          (12, 256), (37, 257), (5, 511), (6, 512), (29, 513), (200, 768), (17, 1000),
          (18, 1001), (11, 1024), (10, 1025), (6, 2047), (7, 2048), (5, 2049), (3, 4095),
          (4, 4096), (3, 4097), (2, 8191), (3, 8192), (2, 8193), (3, 16384), (2, 16385),
          (2, 32768), (2, 32769), (1, 100003), (1500, 24), (1100, 96), (4100, 5), (2000, 1),
          (2100, 768)]


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, x_dtype):
    w_dtype = "bf16" if (rows + cols) % 2 else "f32"
    print(f"rms {rows}x{cols} {x_dtype} weight {w_dtype}", flush=True)
    x = normal(rows * 131 + cols, rows, cols, dtype=x_dtype, std=1.5)
    r = normal(rows * 131 + cols + 1, rows, cols, dtype=x_dtype, std=3.0)
    w = 1 + 0.3 * normal(cols, cols)
    w = w.to(DT[w_dtype])
    for residual, weight in ((r, w), (None, w), (r, None)):
        h = R.rms_sum(x, residual)
        want, want_r = R.rms(h, weight, EPS)
        e_y, e_r = R.rms_bounds(h, weight, EPS)
        y, hh, rstd = B.rms_norm(x, weight, residual, EPS, want_stats=True)
        assert torch.equal(bits(hh), bits(h))
        within(rstd, want_r, e_r, "rstd")
        within(y, want, R.stored(want, e_y, x.dtype), "y")
        if cols > 16384:
            continue
        for block in (128, None):
            q, scales, hh, rstd8 = B.rms_norm_e4m3(x, weight, residual, EPS, block,
                                                   want_stats=True)
            assert torch.equal(bits(hh), bits(h)) and torch.equal(bits(rstd8), bits(rstd))
            check_codes(q, scales, want, e_y, block)
    # in place and without statistics: the same bits
    want, want_h = B.rms_norm(x, w, r, EPS)
    for at in ("x", "r"):
        a, b = x.clone(), r.clone()
        y, h = B.rms_norm(a, w, b, EPS, H=a if at == "x" else b)
        assert torch.equal(bits(h), bits(want_h)) and torch.equal(bits(y), bits(want))
    a, b = x.clone(), r.clone()
    B.rms_norm(a, w, b, EPS, Y=a, H=b)
    assert torch.equal(bits(b), bits(want_h)) and torch.equal(bits(a), bits(want))
    a = x.clone()
    want = B.rms_norm(x, w, None, EPS)
    B.rms_norm(a, w, None, EPS, Y=a)
    assert torch.equal(bits(a), bits(want))


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, x_dtype):
    w_dtype = "f32" if (rows + cols) % 2 else "bf16"
    print(f"rms grad {rows}x{cols} {x_dtype} weight {w_dtype}", flush=True)
    seed = rows * 131 + cols
    h = normal(seed, rows, cols, dtype=x_dtype, std=2.0)
    dy = normal(seed + 1, rows, cols, dtype=x_dtype)
    dh = normal(seed + 2, rows, cols, dtype=x_dtype, std=0.5)
    w = (1 + 0.3 * normal(seed + 3, cols)).to(DT[w_dtype])
    rstd = R.rms(h, None, EPS)[1].float()
    dw_dtype = DT["bf16" if cols % 3 == 0 else "f32"]
    for weight, added in ((w, dh), (None, dh), (w, None)):
        dx, dw = B.rms_norm_backward(dy, h, weight, rstd, added, dtype=dw_dtype)
        wx, ww = R.rms_grad(dy, h, weight, rstd, added)
        bx, bw = R.rms_grad_bounds(dy, h, weight, rstd, added, dw_dtype)
        within(dx, wx, bx, "dx")
        within(dw, ww, bw, "dw")
    # one of the two alone, in place, added to: the same bits
    dx, dw = B.rms_norm_backward(dy, h, w, rstd, dh)
    assert B.rms_norm_backward(dy, h, w, rstd, dh, want_x=False)[0] is None
    assert torch.equal(B.rms_norm_backward(dy, h, w, rstd, dh, want_x=False)[1], dw)
    assert torch.equal(bits(B.rms_norm_backward(dy, h, w, rstd, dh, want_weight=False)[0]),
                       bits(dx))
    for at in ("dy", "dh"):
        a, b = dy.clone(), dh.clone()
        got, gw = B.rms_norm_backward(a, h, w, rstd, b, dX=a if at == "dy" else b)
        assert torch.equal(bits(got), bits(dx)) and torch.equal(gw, dw)
    acc = torch.full_like(dw, 2.0)
    B.rms_norm_backward(dy, h, w, rstd, dh, dweight=acc, accumulate=True)
    assert torch.equal(acc, 2.0 + dw)


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [768, 257, 20000])
def test_strides_and_alignment(cols, x_dtype):
    """Rows with gaps, starts off any 16 bytes, leading dimensions: the bits of
    contiguous calls, and nothing written between the rows."""
    rows = 12
    x, r, dh, dy = (normal(cols + i, rows, cols, dtype=x_dtype) for i in range(4))
    w = 1 + 0.2 * normal(9, cols)

    def gaps(t):
        pad = torch.full((rows, cols + 5), 7.0, device="cuda", dtype=t.dtype)
        pad[:, 3:3 + cols] = t
        return pad[:, 3:3 + cols]

    y, h, rstd = B.rms_norm(x, w, r, EPS, want_stats=True)
    y2, h2, rstd2 = B.rms_norm(gaps(x), w, gaps(r), EPS, want_stats=True)
    for a, b in ((y, y2), (h, h2), (rstd, rstd2)):
        assert torch.equal(bits(a), bits(b))
    dx, dw = B.rms_norm_backward(dy, h, w, rstd, dh)
    dx2, dw2 = B.rms_norm_backward(gaps(dy), gaps(h), w, rstd, gaps(dh))
    assert torch.equal(bits(dx), bits(dx2)) and torch.equal(dw, dw2)
    if cols <= 16384:
        q, s = B.rms_norm_e4m3(x, w, None, EPS)
        q2, s2 = B.rms_norm_e4m3(gaps(x), w, None, EPS)
        assert torch.equal(bits(q), bits(q2)) and torch.equal(s, s2)
        flat = torch.zeros(rows * cols + 3, dtype=torch.uint8, device="cuda")
        q3 = flat[1:1 + rows * cols].view(rows, cols).view(torch.float8_e4m3fn)
        B.rms_norm_e4m3(x, w, None, EPS, Q=q3)
        assert torch.equal(bits(q3), bits(q)) and flat[0] == 0 and (flat[-2:] == 0).all()
    lead = (3, 4, cols)
    y3, h3, rstd3 = B.rms_norm(x.view(lead), w, r.view(lead), EPS, want_stats=True)
    assert y3.shape == h3.shape == lead and rstd3.shape == (3, 4)
    assert torch.equal(bits(y3.view(rows, cols)), bits(y))
    dx3, _ = B.rms_norm_backward(dy.view(lead), h3, w, rstd3, dh.view(lead))
    assert torch.equal(bits(dx3.view(rows, cols)), bits(dx))
    if cols <= 16384:
        assert B.rms_norm_e4m3(x.view(lead), w, block=None)[1].shape == (3, 4, 1)


def test_no_rows():
    x = torch.zeros(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    y, h, rstd = B.rms_norm(x, w, x, want_stats=True)
    assert y.shape == h.shape == (0, 64) and rstd.shape == (0,)
    assert B.rms_norm_e4m3(x, w)[0].shape == (0, 64)
    dx, dw = B.rms_norm_backward(x, x, w, rstd)
    assert dx.shape == (0, 64) and (dw == 0).all()
    acc = torch.full((64,), 2.0, device="cuda")
    B.rms_norm_backward(x, x, w, rstd, dweight=acc, accumulate=True)
    assert (acc == 2).all()


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [5, 100, 768, 4096, 20000])
def test_values_out_of_range(cols, x_dtype):
    """A NaN is its own row's; zeros stay zeros, with the least scale; a sum of
    squares past float32 gives rstd 0."""
    x = normal(1, 6, cols, dtype=x_dtype)
    x[1, cols // 2] = float("nan")
    x[2] = 0
    x[3] = 3e19
    y, h, rstd = B.rms_norm(x, None, None, EPS, want_stats=True)
    assert y[1].isnan().all() and y.isnan().any(1).sum() == 1
    assert (y[2] == 0).all() and rstd[2] == 2.0 ** 10
    assert rstd[3] == 0 and (y[3] == 0).all()
    if cols > 16384:
        return
    for block in (128, None):
        q, s = B.rms_norm_e4m3(x, None, None, EPS, block)
        assert (q[2].float() == 0).all() and (s[2] == 2.0 ** -126).all()
        assert q[1].float().isnan().any() and not q[[0, 4, 5]].float().isnan().any()
        assert (q[[0, 4, 5]].float().abs().amax(1) == 448).all()


def test_streams_and_graphs():
    """Calls at once on streams of their own, and a graph replayed between eager calls
    with other inputs."""
    cases = [(3000, 768), (40, 1001), (3, 20000)]
    data = [[normal(i, r, c, dtype="bf16") for i in range(4)] for r, c in cases]

    def all_of(x, r, dy, dh):
        y, h, rstd = B.rms_norm(x, None, r, EPS, want_stats=True)
        return (y, h, rstd, *B.rms_norm_backward(dy, h, None, rstd, dh))

    want = [all_of(*d) for d in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(3):
        got = []
        for s, d in zip(streams, data):
            with torch.cuda.stream(s):
                got.append(all_of(*d))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(bits(p), bits(q)) for p, q in zip(a, b))
    # on a stream that is passed
    y, h = B.rms_norm(data[0][0], None, data[0][1], EPS, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(bits(y), bits(want[0][0]))
    for d, b in zip(data, want):
        static = [t.clone() for t in d]
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            out = all_of(*static)
        for turn in range(3):
            static[0].copy_(d[0] if turn != 1 else d[0] * 2)
            g.replay()
            ref = b if turn != 1 else all_of(d[0] * 2, *d[1:])
            torch.cuda.synchronize()
            assert all(torch.equal(bits(p), bits(q)) for p, q in zip(out, ref))


@pytest.mark.slow
def test_row_offsets_past_32_bits():
    cols = 1024
    store = torch.zeros((1 << 33) + cols, dtype=torch.bfloat16, device="cuda")
    x = store.as_strided((3, cols), (1 << 32, 1))
    v = normal(1, 3, cols, dtype="bf16")
    x.copy_(v)
    y, rstd = B.rms_norm(x, None, None, EPS, want_stats=True)[::2]
    assert torch.equal(bits(y), bits(B.rms_norm(v, None, None, EPS)))
    a, _ = B.rms_norm_backward(x, x, None, rstd, x)
    b, _ = B.rms_norm_backward(v, v, None, rstd, v)
    assert torch.equal(bits(a), bits(b))


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    for call in (lambda: B.rms_norm(x.half()), lambda: B.rms_norm(x, w.half()),
                 lambda: B.rms_norm(x, w[:4]), lambda: B.rms_norm(x, w, x.bfloat16()),
                 lambda: B.rms_norm(x, w, x[:2]), lambda: B.rms_norm(x.t(), w),
                 lambda: B.rms_norm_e4m3(x, Q=torch.zeros(4, 8, device="cuda")),
                 lambda: B.rms_norm_e4m3(x, scales=torch.zeros(4, 2, device="cuda")),
                 lambda: B.rms_norm_backward(x, x.bfloat16(), w, x[:, 0].contiguous())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: B.rms_norm_e4m3(x, block=64), lambda: B.rms_norm(x, H=x.clone()),
                 lambda: B.rms_norm(x, w.cpu()),
                 lambda: B.rms_norm_backward(x, x, w, x[:, 0].contiguous(), accumulate=True)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(B.SignMuonError):
        B.rms_norm(x, eps=-1.0)
    with pytest.raises(B.SignMuonError):
        B.rms_norm_e4m3(torch.zeros(1, 16385, device="cuda"))


@pytest.mark.parametrize("block", [128, None])
@pytest.mark.parametrize("x_std,w_std", [(1e-18, 1e-27), (1e-18, 1e-24), (1e17, 1e27), (1e17, 1e22)])
@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
def test_codes_where_row_times_weights_leaves_float32(x_std, w_std, x_dtype, block):
    """Y is an ordinary number though the products of the row as it is and the weights are
    past float32's largest, or below its least."""
    x = (normal(5, 40, 300).double() * x_std).to(DT[x_dtype])
    w = (normal(6, 300).double() * w_std).float()
    q, scales = B.rms_norm_e4m3(x, w, None, 0.0, block)
    want, _ = R.rms(x, w, 0.0)
    e_y, _ = R.rms_bounds(x, w, 0.0)
    check_codes(q, scales, want, e_y, block)


@pytest.mark.parametrize("block", [128, None])
def test_codes_where_the_squares_sum_past_float32(block):
    """rstd is 0 then, and so is Y, whatever the weights."""
    x = torch.full((3, 300), 3e19, device="cuda")
    w = torch.full((300,), 1e30, device="cuda")
    assert (B.rms_norm(x, w, None, EPS) == 0).all()
    q, scales = B.rms_norm_e4m3(x, w, None, EPS, block)
    assert (q.float() == 0).all() and (scales == 2.0 ** -126).all()


@pytest.mark.parametrize("block", [128, None])
@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
def test_codes_are_the_nearest_values_and_ties_stay_ties(x_dtype, block):
    """Of rows of 8-bit values without weights a code stands for 448 h / max |h|.  In units
    of half a code's step that is a multiple of 2^-3 / max, max an integer of 8 bits: 2^-11
    from a middle between two codes, an odd number, at least, unless it is one.  The
    quotient's rounding to float32 is 2^-19 of half a step at most.  So the code is the exact
    quotient's, and a tie stays one."""
    x, v = R.rows_with_ties(torch.device("cuda"))
    for power in (0, -7, 40):
        q, _ = B.rms_norm_e4m3((x * 2.0 ** power).to(DT[x_dtype]), None, None, EPS, block)
        want = R.e4m3_nearest(v)
        bad = q.float().double() != want
        assert not bad.any(), (int(bad.sum()), x[bad][:4].tolist(), want[bad][:4].tolist(),
                               q.float()[bad][:4].tolist())
