"""The residual norm, the gated block and the linear cross entropy together, as a
model trained with the optimizer uses them: a table shared by the lookup and the
loss, gradients of every parameter in both ways that the step takes them, a captured
pass, and single tokens against a whole batch."""
import pytest

from distributed_bit_matrix_amd import layers as L
from tests import block_reference as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
VOCAB, DIM, HIDDEN = 331, 64, 160


class Model(torch.nn.Module):
    def __init__(self, dtype, layers=2):
        super().__init__()
        kw = dict(device="cuda", dtype=dtype)
        self.table = L.Embedding(VOCAB, DIM, scale=DIM ** 0.5, **kw)
        self.norms = torch.nn.ModuleList(L.RMSNorm(DIM, **kw) for _ in range(layers + 1))
        self.blocks = torch.nn.ModuleList(
            L.GatedMLP(DIM, HIDDEN, "gelu" if i % 2 else "silu", **kw) for i in range(layers))
        self.loss = L.LinearCrossEntropy(VOCAB, DIM, weight=self.table.weight)

    def hidden(self, t):
        h, add = None, self.table(t)
        for norm, block in zip(self.norms, self.blocks):
            if h is None:
                h, y = add, norm(add)
            else:
                y, h = norm(add, h)
            add = block(y)
        return self.norms[-1](add, h)[0]

    def forward(self, t, targets):
        return self.loss(self.hidden(t), targets)


def model(dtype):
    torch.manual_seed(0)
    return Model(dtype)


def batch(seed, rows=6, length=21):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(VOCAB, (rows, length), device="cuda", generator=g)
    targets = t.roll(-1, 1)
    targets[:, -1] = -100
    targets[2, 9:] = -100
    return t, targets


def plain_loss(m, t, targets):
    """The same model in elementary operations, float64."""
    F = torch.nn.functional
    w = {n: p.detach().double().requires_grad_() for n, p in m.named_parameters()}

    def norm(h, i):
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * w[f"norms.{i}.weight"]

    h = DIM ** 0.5 * w["table.weight"][t]
    for i, block in enumerate(m.blocks):
        y = norm(h, i)
        act = F.silu if block.activation == "silu" else F.gelu
        gate, up = y @ w[f"blocks.{i}.w_gate"].T, y @ w[f"blocks.{i}.w_up"].T
        h = h + (act(gate) * up) @ w[f"blocks.{i}.w_down"].T
    z = norm(h, len(m.blocks)) @ w["table.weight"].T
    return F.cross_entropy(z.view(-1, VOCAB), targets.view(-1)), w


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_loss_and_gradients(dtype):
    """Against autograd in 64 bits.  Relative to a gradient's norm: some twenty roundings
    of the type lie between the loss and the first layer, each off by half a step and
    passed on by factors of about one; 64 half steps hold them."""
    m = model(DT[dtype])
    t, targets = batch(1)
    loss = m(t, targets)
    want, w = plain_loss(m, t, targets)
    half = R.HALF_STEP[DT[dtype]]
    assert abs(loss.item() - want.item()) <= 64 * half * want.item()
    loss.backward()
    names = [n for n, _ in m.named_parameters()]
    grads = torch.autograd.grad(want, [w[n] for n in names])
    for n, g in zip(names, grads):
        p = dict(m.named_parameters())[n]
        assert (p.grad.double() - g).norm() <= 64 * half * g.norm(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_direct_gradients_reach_the_step(dtype):
    """The flat array of the step holds the gradient that the ordinary path gives,
    summed over two passes; a step moves every weight by its rate."""
    from distributed_bit_matrix_amd import optim as SO
    plain, direct = model(DT[dtype]), model(DT[dtype])
    o1 = SO.SignMuon(plain.parameters(), scale="fro")
    o2 = SO.SignMuon(direct.parameters(), scale="fro", direct_grads=True)
    names = [n for n, _ in direct.named_parameters()]
    for step in range(2):
        for o, m in ((o1, plain), (o2, direct)):
            o.zero_grad()
            for k in range(2):
                m(*batch(10 * step + k)).backward()
        assert all(p.grad is None for p in direct.parameters())
        o1.step()
        o2.step()
        torch.cuda.synchronize()
        assert not o1.nonfinite() and not o2.nonfinite()
        a, b = o1._groups[0], o2._groups[0]
        for n, (r, c, off, _) in zip(names, b.layout):
            ga, gb = a.G[off:off + r * c], b.G[off:off + r * c]
            # ordinary gradients: a pass, its parts of the shared table and each sum
            # rounded to the type, of magnitudes up to twice the largest entry
            tol = 5 * (R.HALF_STEP[DT[dtype]] + 4 * R.U32) * 2 * gb.abs().max()
            assert (ga - gb).abs().max() <= tol and gb.abs().max() > 0, (step, n)
        with torch.no_grad():
            for p, q in zip(plain.parameters(), direct.parameters()):
                p.copy_(q)


def test_a_captured_pass():
    """Forward and backward in a graph, replayed between eager work on other inputs:
    the gradients of an eager pass, bit for bit."""
    m = model(torch.bfloat16)
    params = list(m.parameters())
    t, targets = batch(5)

    def run():
        m(t, targets).backward()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            for p in params:
                p.grad = None
            run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for p in params:
        p.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    got = [p.grad for p in params]
    for rep in range(4):
        t2, targets2 = batch(20 + rep)
        t.copy_(t2)
        targets.copy_(targets2)
        for g in got:
            g.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want = torch.autograd.grad(m(t, targets), params)
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g, w), rep


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_single_tokens_against_a_batch(dtype):
    """A row of few goes through other kernels than a row of many: the same values
    within the roundings that both have (a hidden state is off by some ten of them
    either way)."""
    m = model(DT[dtype])
    t, targets = batch(3)
    with torch.no_grad():
        whole = m.hidden(t)
        few = torch.cat([m.hidden(t[i:i + 1, j:j + 7]) for i in range(6) for j in range(0, 21, 7)])
        few = few.view(6, 21, DIM)
        half = R.HALF_STEP[DT[dtype]]
        assert (whole.double() - few.double()).norm() <= 32 * half * whole.double().norm()
        each = L.linear_cross_entropy(whole, m.table.weight, targets, reduction="none")
        rows = torch.stack([L.linear_cross_entropy(whole[i, j:j + 7], m.table.weight,
                                                   targets[i, j:j + 7], reduction="none")
                            for i in range(6) for j in range(0, 21, 7)]).view(6, 21)
        # (the same inputs: sums of products alone differ)
        assert (each - rows).abs().max() <= 2.0 ** -16


def test_with_gradients_and_without_are_the_same():
    m = model(torch.bfloat16)
    t, targets = batch(4)
    with torch.no_grad():
        want = m(t, targets)
    assert torch.equal(m(t, targets).detach(), want)


def test_two_devices_or_the_cpu_are_refused():
    m = model(torch.float32)
    t, targets = batch(4)
    with pytest.raises((ValueError, TypeError)):
        L.linear_cross_entropy(m.hidden(t), m.table.weight, targets.cpu())
    with pytest.raises((ValueError, TypeError)):
        L.rms_norm(m.hidden(t), m.norms[0].weight.cpu())
    with pytest.raises((ValueError, TypeError)):
        L.gated_mlp(m.hidden(t).cpu(), *(p.cpu() for p in m.blocks[0].parameters()))
