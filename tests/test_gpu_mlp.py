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
