"""Autograd through the layers, on the CPU: the library's calls are replaced by
elementary torch operations, so that what layers.py and optim.py do around them
can be seen without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad as fw  # noqa: E402

from distributed_bit_matrix_amd import binding as B  # noqa: E402
from distributed_bit_matrix_amd import layers as L  # noqa: E402


def _norm(x, weight=None, bias=None, eps=1e-5, want_stats=False):
    x = x.detach()
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[..., None]
    y = y if weight is None else y * weight.detach()
    y = y if bias is None else y + bias.detach()
    return (y, mean, rstd) if want_stats else y


def _sums(out, value, dtype, accumulate):
    if out is None:
        return value.to(dtype or torch.float32)
    return out.add_(value) if accumulate else out.copy_(value)


def _norm_backward(dy, x, weight, mean, rstd, want_x=True, want_weight=True, want_bias=True,
                   dweight=None, dbias=None, dtype=None, accumulate=False):
    xh = (x - mean[..., None]) * rstd[..., None]
    g = dy if weight is None else dy * weight
    dx = rstd[..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    cols = x.shape[-1]
    return (dx if want_x else None,
            _sums(dweight, (dy * xh).reshape(-1, cols).sum(0), dtype, accumulate)
            if want_weight else None,
            _sums(dbias, dy.reshape(-1, cols).sum(0), dtype, accumulate) if want_bias else None)


def _embedding(tokens, weight, scale=1.0):
    return scale * weight.detach()[tokens]


def _embedding_backward(dy, tokens, vocab, scale=1.0, padding=None, dW=None, dtype=None,
                        accumulate=False):
    keep = torch.ones_like(tokens, dtype=torch.bool) if padding is None else tokens != padding
    dw = torch.zeros(vocab, dy.shape[-1]).index_add_(0, tokens[keep], scale * dy[keep])
    return _sums(dW, dw, dtype, accumulate)


@pytest.fixture
def calls(monkeypatch):
    monkeypatch.setattr(B, "layer_norm", _norm)
    monkeypatch.setattr(B, "layer_norm_backward", _norm_backward)
    monkeypatch.setattr(B, "embedding", _embedding)
    monkeypatch.setattr(B, "embedding_backward", _embedding_backward)


def _tensors(seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, generator=g) for s in ((5, 6), (6,), (6,), (9, 6))]


@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_are_refused(calls, grad):
    """A tangent of any input, with or without requires_grad, is not dropped."""
    x, w, b, table = _tensors()
    t = torch.tensor([1, 4])
    with fw.dual_level(), torch.set_grad_enabled(grad):
        dual = [fw.make_dual(v, torch.ones_like(v)) for v in (x, w, b, table)]
        for call in (lambda: L.layer_norm(dual[0]), lambda: L.layer_norm(x, dual[1]),
                     lambda: L.layer_norm(x, w, dual[2]), lambda: L.layer_norm(x, None, dual[2]),
                     lambda: L.embedding(t, dual[3])):
            with pytest.raises(NotImplementedError):
                call()
        # without a tangent nothing changes
        assert torch.equal(L.layer_norm(x, w, b), _norm(x, w, b))
        assert torch.equal(L.embedding(t, table), table[t])


def test_traced_layers_run_again(calls):
    """A trace holds the layers themselves, not the memory that they return
    (the kernels are hidden from it)."""
    x, w, b, table = _tensors()
    t = torch.tensor([1, 4, 0])
    norm = torch.jit.trace(lambda x: L.layer_norm(x, w, b), x)
    look = torch.jit.trace(lambda t: L.embedding(t, table, 2.0), t)
    assert "_LayerNorm" in str(norm.graph) and "_Embedding" in str(look.graph)
    x2, t2 = _tensors(1)[0], torch.tensor([8, 8, 2])
    assert torch.equal(norm(x2), _norm(x2, w, b))
    assert torch.equal(look(t2), 2.0 * table[t2])


class _State:
    """Stands for the optimizer's flat arrays of one group."""

    def __init__(self):
        self.log = []

    def wait(self):
        self.log.append("wait")

    def mark(self):
        self.log.append("mark")


def _with_slot(p, state):
    from distributed_bit_matrix_amd import optim as SO
    p = torch.nn.Parameter(p)
    p._signmuon_slot = SO.GradSlot(state, torch.full_like(p, float("nan")))
    return p


@pytest.fixture
def not_capturing(monkeypatch):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


@pytest.mark.parametrize("with_x", [True, False])
@pytest.mark.parametrize("form", ["weight", "bias", "both"])
def test_direct_gradients_of_every_form(calls, not_capturing, form, with_x):
    """A weight alone, a bias alone and both, with and without the input's
    gradient, over two passes that add up."""
    state = _State()
    x, w, b, _ = _tensors()
    x.requires_grad_(with_x)
    w = _with_slot(w, state) if form != "bias" else None
    b = _with_slot(b, state) if form != "weight" else None
    params = [p for p in (w, b) if p is not None]
    c = torch.arange(30.).view(5, 6)
    want = torch.autograd.grad((L.layer_norm(x, w, b) * c).sum(), params)
    assert not any(p._signmuon_slot.filled for p in params)
    for turn in (1, 2):
        (L.layer_norm(x, w, b) * c).sum().backward()
        for p, g in zip(params, want):
            assert p.grad is None and p._signmuon_slot.filled
            assert torch.equal(p._signmuon_slot.grad, turn * g)
    assert (x.grad is not None) == with_x


class _Stream:
    pass


class _Array:
    """Stands for a tensor on a GPU: its streams are remembered."""
    device = None

    def __init__(self):
        self.streams = []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_a_write_on_another_stream_keeps_the_array(monkeypatch):
    """The flat gradient may go with its optimizer while a backward pass still
    writes it on a stream that the allocator does not know of."""
    from distributed_bit_matrix_amd import optim as SO
    state = SO._GroupState.__new__(SO._GroupState)
    log = []

    class Event:
        def record(self, stream):
            log.append(stream)

    state.G, state.event = _Array(), Event()
    stream = _Stream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    slot = SO.GradSlot(state, torch.zeros(4))
    slot.close()
    assert slot.filled and log == [stream] and state.G.streams == [stream]


def test_a_step_on_another_stream_keeps_its_arrays(monkeypatch):
    from distributed_bit_matrix_amd import optim as SO
    opt = SO.SignMuon([torch.nn.Parameter(torch.zeros(4))])
    state = SO._GroupState.__new__(SO._GroupState)
    arrays = [_Array() for _ in range(5)]
    state.G, state.W, state.Mom, state.bits = arrays[:4]
    state.slots, state.params, state.stride = [], [], 1
    ran = []

    class Plan:
        ws = arrays[4]

        def set_eta(self, eta):
            pass

        def __call__(self, *args):
            ran.append(args[:4])

    state.plan = Plan()
    opt._groups[0] = state
    stream = _Stream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    opt.step()
    assert len(ran) == 1 and all(a.streams == [stream] for a in arrays)


def test_a_slot_does_not_keep_the_array():
    """A parameter that outlives its optimizer holds nothing of its arrays."""
    import weakref
    from distributed_bit_matrix_amd import optim as SO
    state, flat = _State(), torch.zeros(100)
    p = torch.nn.Parameter(torch.zeros(4))
    p._signmuon_slot = SO.GradSlot(state, flat[8:12])
    assert p._signmuon_slot.grad.data_ptr() == flat.data_ptr() + 32
    gone = []
    weakref.finalize(p._signmuon_slot.grad, gone.append, True)
    del state
    assert gone == [True] and not p._signmuon_slot.alive()


def test_an_optimizer_may_go_during_a_pass(calls, not_capturing):
    """The state that took a gradient lives until the gradient is written."""
    x, w, _, _ = _tensors()
    state = _State()
    w = _with_slot(w, state)
    log = state.log
    y = L.layer_norm(x, w).sum()

    real = B.layer_norm_backward

    def drop(*args, **kw):
        nonlocal state
        state = None                # the last reference outside of the pass
        return real(*args, **kw)

    B.layer_norm_backward = drop
    try:
        y.backward()
    finally:
        B.layer_norm_backward = real
    assert log == ["wait", "mark"] and w.grad is None and not w._signmuon_slot.alive()


def test_parameters_with_a_slot_load_as_weights_only():
    """torch.load's default: parameters saved by themselves (a state_dict holds
    plain tensors), as they were before an optimizer took their gradients."""
    import io
    state = _State()
    p = _with_slot(torch.arange(4.), state)
    f = io.BytesIO()
    torch.save({"p": p}, f)
    f.seek(0)
    q = torch.load(f, weights_only=True)["p"]
    assert torch.equal(q.detach(), p.detach())
    assert q.__dict__.get("_signmuon_slot") is None and p._signmuon_slot.alive()


@pytest.mark.parametrize("capturing", [False, True])
def test_a_captured_pass_returns_its_gradients(calls, monkeypatch, capturing):
    """backward() in a capture puts the gradients into p.grad and leaves the
    slots alone; the same pass outside of one fills the slots."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    x, w, b, table = _tensors()
    state = _State()
    params = [w, b, table] = [_with_slot(p, state) for p in (w, b, table)]
    t = torch.tensor([1, 4, 1, 0, 8])
    c = torch.arange(30.).view(5, 6)
    want = torch.autograd.grad((L.layer_norm(L.embedding(t, table), w, b) * c).sum(), params)
    (L.layer_norm(L.embedding(t, table), w, b) * c).sum().backward()
    for p, g in zip(params, want):
        slot = p._signmuon_slot
        assert slot.filled != capturing and (p.grad is None) != capturing
        assert torch.equal(p.grad if capturing else slot.grad, g)
        assert not capturing or bool(slot.grad.isnan().all())
    assert (state.log == []) == capturing
