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
