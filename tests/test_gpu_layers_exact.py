"""Layer norm and embedding on inputs whose sums are exact in float32, so that
a lost row, column or token of any size of sum shows."""
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


def within(got, want, bound, what):
    off = np.abs(got - want)
    bad = ~(off <= bound)
    assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), off[bad][:4])


@pytest.mark.parametrize("x_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cols", [700, 16384, 16385, 24576, 24577, 40003, 1 << 20])
def test_norm_of_constant_rows_of_large_values(cols, x_dtype):
    """Constant rows of powers of two: every partial sum is exact (counts below
    2^24), so the mean is the constant, the deviations are zero and y is beta,
    also where the constant's square is past float32."""
    print(f"norm constant rows {cols} {x_dtype}", flush=True)
    value = np.array([2.0 ** 67, -2.0 ** 90, 2.0 ** 63, 1.0])
    x = np.broadcast_to(value[:, None], (4, cols)).astype(np.float32)
    b = np.linspace(-1, 1, cols).astype(np.float32)
    y, m, r = B.layer_norm(dev(x, x_dtype), None, dev(b), EPS, want_stats=True)
    assert np.array_equal(host(m), value)
    # one addition, a root and a reciprocal
    want = 1 / np.sqrt(EPS)
    assert (np.abs(host(r) - want) <= 4 * R.U32 * want).all()
    assert np.array_equal(host(y), np.broadcast_to(host(dev(b, x_dtype)), (4, cols)))


def test_traced_layers_run_the_kernels():
    from distributed_bit_matrix_amd import layers as L
    g = torch.Generator(device="cuda").manual_seed(4)
    x, x2 = (torch.randn(7, 40, device="cuda", generator=g) for _ in range(2))
    w, table = (torch.randn(s, device="cuda", generator=g) for s in ((40,), (30, 40)))
    t, t2 = (torch.randint(30, (7,), device="cuda", generator=g) for _ in range(2))
    norm = torch.jit.trace(lambda x: L.layer_norm(x, w), x)
    look = torch.jit.trace(lambda t: L.embedding(t, table), t)
    assert torch.equal(norm(x2), B.layer_norm(x2, w))
    assert torch.equal(look(t2), table[t2])


def test_direct_gradients_outlive_their_optimizer():
    """A backward pass on another stream, still under way when its optimizer
    and the gradients' array go: new tensors do not get its memory."""
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    t = torch.arange(3000, device="cuda")
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for rep in range(4):
        w = torch.nn.Parameter(torch.zeros(3000, 512, device="cuda"))
        opt = SO.SignMuon([w], scale="fro", K=1, direct_grads=True)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(20):
                busy @ busy
            L.embedding(t, w).sum().backward()
        assert w.grad is None
        del opt
        SO.SignMuon([w], scale="fro", K=1, direct_grads=True)      # drops the old array
        new = [torch.full((3000, 512), 7.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        for n in new:
            assert bool((n == 7.0).all()), rep


def test_step_outlives_its_optimizer():
    """A step on another stream, still under way when the optimizer goes: the
    weights move as they do without the deletion, and new tensors keep theirs."""
    from distributed_bit_matrix_amd import optim as SO
    g = torch.Generator(device="cuda").manual_seed(6)
    w0, grad = (torch.randn(512, 700, device="cuda", generator=g) for _ in range(2))

    def run(drop):
        w = torch.nn.Parameter(w0.clone())
        w.grad = grad.clone()
        opt = SO.SignMuon([w], scale="fro", K=2)
        opt._state(0, opt.param_groups[0])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(20):
                w0.t() @ w0
            opt.step()
        if drop:
            del opt
        new = [torch.full((512, 700), 7.0, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        return w.detach().clone(), all(bool((n == 7.0).all()) for n in new)

    want, _ = run(False)
    got, kept = run(True)
    assert kept and torch.equal(got, want) and not torch.equal(got, w0)


def test_a_kept_parameter_frees_the_optimizers_arrays():
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    w = torch.nn.Parameter(torch.zeros(4096, 512, device="cuda"))
    t = torch.arange(64, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    opt = SO.SignMuon([w], scale="fro", K=1, direct_grads=True)
    L.embedding(t, w).sum().backward()
    opt.step()
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before >= 2 * 4 * w.numel()
    del opt
    # the weights take the place of the parameter's own memory; nothing else stays
    assert torch.cuda.memory_allocated() - before < w.numel()
    L.embedding(t, w).sum().backward()
    assert w.grad is not None


def test_captured_backward_fills_the_parameters_grads():
    """A plain backward pass captured while an optimizer takes gradients
    directly: each replay's gradients are in p.grad, the step's array and the
    slots stay as they are, and the next eager pass writes to them again."""
    from distributed_bit_matrix_amd import layers as L
    from distributed_bit_matrix_amd import optim as SO
    g = torch.Generator(device="cuda").manual_seed(9)
    w, b, table = params = [torch.nn.Parameter(torch.randn(s, device="cuda", generator=g))
                            for s in ((64,), (64,), (30, 64))]
    opt = SO.SignMuon(params, scale="fro", K=1, direct_grads=True)
    t = torch.randint(30, (50,), device="cuda", generator=g)
    c = torch.randn(50, 64, device="cuda", generator=g)

    def run():      # no graph of the parameters lives on after it
        L.layer_norm(L.embedding(t, table), w, b).backward(c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    opt.zero_grad()
    flat = opt._groups[0].G
    flat.fill_(5.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    got = [p.grad for p in params]
    assert all(v is not None for v in got)
    for rep in range(4):
        c.copy_(torch.randn(50, 64, device="cuda", generator=g))
        t.copy_(torch.randint(30, (50,), device="cuda", generator=g))
        for v in got:
            v.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.autograd.grad(L.layer_norm(L.embedding(t, table), w, b), params, c)
        torch.cuda.synchronize()
        for p, v, e in zip(params, got, want):
            assert p.grad is v and torch.equal(v, e), rep
            assert not p._signmuon_slot.filled
        assert bool((flat == 5.0).all()), rep
    for p in params:
        p.grad = None
    run()
    for p, e in zip(params, want):
        assert p.grad is None and p._signmuon_slot.filled
        assert torch.equal(p._signmuon_slot.grad, e)


# one of every width of the kernels' rows, in registers and past them, and of
# every number of rows a block or a launch takes
EXACT = [(5, 1), (9, 2), (7, 7), (40, 64), (33, 129), (11, 511), (19, 768), (17, 1001),
         (2048, 257), (2049, 257), (3, 2049), (5, 4097), (3, 8192), (4, 8193), (3, 16384),
         (2, 16385), (3, 24577), (9, 32769), (40, 40003), (2, 100003), (1, 1 << 20)]


@pytest.mark.parametrize("rows,cols", EXACT)
def test_norm_loses_no_column(rows, cols):
    print(f"exact norm {rows}x{cols}", flush=True)
    for x_dtype in DT:
        x, want, bound = R.exact_norm(rows, cols, EPS, x_dtype)
        got = B.layer_norm(dev(x, x_dtype), None, None, EPS, want_stats=True)
        for a, w, e, name in zip(got, want, bound, ("y", "mean", "rstd")):
            within(host(a), w, e, (x_dtype, name))


def _exact_grad(rows, cols):
    for x_dtype in DT:
        dy, x, want, e = R.exact_norm_grad(rows, cols, x_dtype)
        DY, X = dev(dy, x_dtype), dev(x, x_dtype)
        m, r = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
        for dw_dtype in DT:
            dx, dg, db = B.layer_norm_backward(DY, X, None, m, r, dtype=DT[dw_dtype])
            within(host(dx), want[0], e, (x_dtype, "dx"))
            for a, w, name in ((dg, want[1], "dgamma"), (db, want[2], "dbeta")):
                w = R.bf16_values(w) if dw_dtype == "bf16" else w
                assert np.array_equal(host(a), w), (x_dtype, dw_dtype, name)
        old = np.arange(cols) % 7
        acc = [dev(old.astype(np.float32)) for _ in range(2)]
        B.layer_norm_backward(DY, X, None, m, r, want_x=False, dweight=acc[0], dbias=acc[1],
                              accumulate=True)
        for a, w in zip(acc, want[1:]):
            assert np.array_equal(host(a), w + old), x_dtype


@pytest.mark.parametrize("rows,cols", EXACT)
def test_norm_backward_loses_no_row_or_column(rows, cols):
    print(f"exact norm grad {rows}x{cols}", flush=True)
    _exact_grad(rows, cols)


@pytest.mark.parametrize("rows,cols", [(2049, 1), (140000, 3), (40000, 8), (70000, 24),
                                       (33000, 33), (4097, 65), (12289, 768), (4200, 1001),
                                       (2100, 2049), (3001, 4096), (513, 8193), (300, 16384),
                                       (1100, 16385), (600, 33000)])
def test_norm_backward_of_several_launches_loses_no_row(rows, cols):
    print(f"exact norm grad, several launches {rows}x{cols}", flush=True)
    assert B.layer_norm_backward_workspace(rows, cols) > 0
    _exact_grad(rows, cols)


def test_sums_over_rows_past_32_bits():
    """2^21 + 1 rows of 1024: dY and X are 1 or 2, in turns of their own, so that
    every sum is an integer below 2^23 and a bit."""
    n, dim = (1 << 21) + 1, 1024
    print(f"exact sums past 32 bits: {n} x {dim}", flush=True)
    i, c = torch.arange(n, device="cuda")[:, None], torch.arange(dim, device="cuda")[None]
    DY = torch.empty(n, dim, device="cuda", dtype=torch.bfloat16)
    X = torch.empty_like(DY)
    for a in range(0, n, 1 << 18):
        k = i[a:a + (1 << 18)]
        DY[a:a + (1 << 18)] = (1 + (k + c) % 2).bfloat16()
        X[a:a + (1 << 18)] = (1 + (k // 2 + c) % 2).bfloat16()
    m, r = torch.zeros(n, device="cuda"), torch.ones(n, device="cuda")
    _, dg, db = B.layer_norm_backward(DY, X, None, m, r, want_x=False)
    i, c = np.arange(4)[:, None], np.arange(dim)[None]      # the rows repeat after 4
    times = np.bincount(np.arange(n) % 4)[:, None]
    dy, x = 1 + (i + c) % 2, 1 + (i // 2 + c) % 2
    assert np.array_equal(host(db), (times * dy).sum(0))
    assert np.array_equal(host(dg), (times * dy * x).sum(0))
    T = torch.arange(n, device="cuda") % 4
    dW = B.embedding_backward(DY, T, 5, 0.5)
    assert np.array_equal(host(dW), 0.5 * np.concatenate([times * dy, 0 * dy[:1]]))


def _tokens(rng, kind, n, vocab):
    if kind == "same":
        return np.full(n, rng.integers(0, vocab))
    if kind == "positions":
        return np.arange(n) % vocab
    if kind == "skew":                  # many tokens of one residue
        return 5 + 256 * rng.integers(0, vocab // 256, n)
    if kind == "zipf":
        return np.minimum((vocab ** rng.random(n)).astype(np.int64) - 1, vocab - 1)
    return rng.integers(0, vocab, n)


@pytest.mark.parametrize("n,vocab,dim,kind", [
    (896, 513, 5, "same"), (2048, 300, 70, "same"), (2047, 5000, 260, "zipf"),
    (2048, 1000, 5, "skew"), (2049, 1000, 7, "skew"), (4000, 64, 1030, "zipf"),
    (12288, 50257, 96, "zipf"), (33000, 70000, 2, "zipf"), (50000, 4096, 3, "zipf"),
    (65536, 1024, 96, "positions"), (65536, 300, 20, "same"), (65537, 2000, 3, "zipf"),
    (70001, 1, 3, "same"), (70000, 100, 1, "uniform"), (131073, 3, 5, "same"),
    (150000, 30000, 2, "zipf"), (100001, 300000, 2, "skew"), (262145, 17, 2, "uniform"),
    (600001, 1048576, 1, "uniform")])
def test_embedding_backward_loses_no_token(n, vocab, dim, kind):
    print(f"exact embed grad n={n} {vocab}x{dim} {kind}", flush=True)
    rng = np.random.default_rng(n + vocab + dim)
    t = _tokens(rng, kind, n, vocab)
    dy = rng.integers(1, 4, (n, dim)).astype(np.float32)
    want = 0.5 * R.exact_embed_grad(dy, t, vocab)
    T, old = torch.from_numpy(t).cuda(), (np.arange(vocab) % 7)[:, None] + np.zeros(dim)
    for dy_dtype in DT:
        DY = dev(dy, dy_dtype)
        assert np.array_equal(host(B.embedding_backward(DY, T, vocab, 0.5)), want)
        got = B.embedding_backward(DY, T.int(), vocab, 0.5, dtype=torch.bfloat16)
        assert np.array_equal(host(got), R.bf16_values(want))
        acc = dev(old.astype(np.float32))
        B.embedding_backward(DY, T, vocab, 0.5, dW=acc, accumulate=True)
        assert np.array_equal(host(acc), want + old)


def test_rows_far_apart():
    """Rows 2^28 + 24 entries apart, as in a slice of a large matrix: the bits
    of the dense rows, and the memory between them stays."""
    gap, cols = (1 << 28) + 24, 768
    print("rows far apart", flush=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    big = torch.full((3, gap), 7.0, device="cuda", dtype=torch.bfloat16)
    X, DY = big[:, 5:5 + cols], big[:, 5 + 2 * cols:5 + 3 * cols]
    X.copy_(torch.randn(3, cols, device="cuda", generator=g))
    DY.copy_(torch.randn(3, cols, device="cuda", generator=g))
    x, dy = X.contiguous(), DY.contiguous()
    got, want = (B.layer_norm(a, None, None, EPS, want_stats=True) for a in (X, x))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(B.layer_norm_backward(DY, X, None, *got[1:]),
                    B.layer_norm_backward(dy, x, None, *got[1:])):
        assert torch.equal(a, b)
    T = torch.tensor([4, 1, 4], device="cuda")
    assert torch.equal(B.embedding_backward(DY, T, 6), B.embedding_backward(dy, T, 6))
    X.fill_(7.0)
    DY.fill_(7.0)
    assert bool((big == 7.0).all())
