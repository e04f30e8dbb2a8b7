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
