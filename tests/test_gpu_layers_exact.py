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
