"""Autograd through the residual norm, the gated block and the linear cross entropy,
on the CPU: the library's calls are replaced by elementary torch operations, so that
what layers.py does around them can be seen without a GPU."""
import pytest

torch = pytest.importorskip("torch")

from torch.autograd import forward_ad as fw  # noqa: E402

from distributed_bit_matrix_amd import binding as B  # noqa: E402
from distributed_bit_matrix_amd import layers as L  # noqa: E402
from tests import block_reference as R  # noqa: E402


def _sums(out, value, dtype, accumulate):
    if out is None:
        assert not accumulate
        return value.to(dtype or torch.float32)
    return out.add_(value) if accumulate else out.copy_(value)


def _rms(x, weight=None, residual=None, eps=1e-6, want_stats=False):
    x = x.detach()
    h = x if residual is None else x + residual.detach()
    y, rstd = R.rms(h, None if weight is None else weight.detach(), eps)
    y, rstd = y.to(x.dtype), rstd.float()
    if want_stats:
        return y, h, rstd
    return y if residual is None else (y, h)


def _rms_backward(dy, h, weight, rstd, dH=None, want_x=True, want_weight=True, dweight=None,
                  dtype=None, accumulate=False):
    flat = [t if t is None else t.reshape(-1, h.shape[-1]) for t in (dy, h, dH)]
    dx, dw = R.rms_grad(flat[0], flat[1], weight, rstd.reshape(-1), flat[2])
    return (dx.view(h.shape).to(h.dtype) if want_x else None,
            _sums(dweight, dw, dtype, accumulate) if want_weight else None)


def _mlp(x, wg, wu, wd, activation="silu", want_pre=False):
    y, pre = R.mlp(x.detach().reshape(-1, x.shape[-1]), wg.detach(), wu.detach(), wd.detach(),
                   activation)
    y = y.view(x.shape).to(x.dtype)
    return (y, pre.float()) if want_pre else y


def _mlp_backward(dy, x, wg, wu, wd, pre, activation="silu", want=(True,) * 4, dw_gate=None,
                  dw_up=None, dw_down=None, dtype=None, accumulate=False):
    flat = [t.reshape(-1, x.shape[-1]) for t in (dy, x)]
    dx, *dw = R.mlp_grad(*flat, wg, wu, wd, pre, activation)
    return (dx.view(x.shape).to(x.dtype) if want[0] else None,
            *(_sums(o, g, dtype, accumulate) if w else None
              for o, g, w in zip((dw_gate, dw_up, dw_down), dw, want[1:])))


def _loss(x, weight, targets, ignore=-100, reduction="mean", want_lse=False):
    each, lse = R.loss(x.detach().reshape(-1, x.shape[-1]), weight.detach(), targets.reshape(-1),
                       ignore)
    out = R.reduce_loss(each, targets.reshape(-1), ignore, reduction).float()
    if reduction == "none":
        out = out.view(targets.shape)
    return (out, lse.float().view(targets.shape)) if want_lse else out


def _loss_backward(dloss, x, weight, targets, lse, ignore=-100, reduction="mean", want_x=True,
                   want_weight=True, dweight=None, dtype=None, accumulate=False):
    dx, dw = R.loss_grad(dloss.reshape(-1) if reduction == "none" else dloss,
                         x.reshape(-1, x.shape[-1]), weight, targets.reshape(-1), lse.reshape(-1),
                         ignore, reduction)
    return (dx.view(x.shape).to(x.dtype) if want_x else None,
            _sums(dweight, dw, dtype, accumulate) if want_weight else None)


@pytest.fixture
def calls(monkeypatch):
    for name, f in (("rms_norm", _rms), ("rms_norm_backward", _rms_backward),
                    ("gated_mlp", _mlp), ("gated_mlp_backward", _mlp_backward),
                    ("linear_cross_entropy", _loss),
                    ("linear_cross_entropy_backward", _loss_backward)):
        monkeypatch.setattr(B, name, f)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)


def tensors(seed=0):
    g = torch.Generator().manual_seed(seed)
    shapes = dict(x=(2, 5, 6), r=(2, 5, 6), w=(6,), wg=(7, 6), wu=(7, 6), wd=(6, 7), table=(9, 6))
    t = {k: torch.randn(s, generator=g) for k, s in shapes.items()}
    t["t"] = torch.tensor([[1, 4, -100, 0, 8], [2, 2, 8, -100, 7]])
    return t


def model(t):
    """What a gated transformer's layer and its end are, but for the attention."""
    y, h = L.rms_norm(t["x"], t["w"], t["r"])
    y, h = L.rms_norm(L.gated_mlp(y, t["wg"], t["wu"], t["wd"]), t["w"], h)
    return L.linear_cross_entropy(y + 0.1 * h, t["table"], t["t"])


def plain(t):
    F = torch.nn.functional
    norm = lambda h: h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * t["w"]  # noqa: E731
    h = t["x"] + t["r"]
    y = norm(h)
    h = h + (F.silu(y @ t["wg"].T) * (y @ t["wu"].T)) @ t["wd"].T
    return F.cross_entropy(((norm(h) + 0.1 * h) @ t["table"].T).view(-1, 9), t["t"].view(-1))


PARAMS = ("w", "wg", "wu", "wd", "table")


def test_gradients_reach_every_input(calls):
    """Through both outputs of the norm, the residual among them, against autograd
    through elementary operations (float32 either way: 2^-14 of the largest entry is
    a thousand roundings, more than any entry here goes through)."""
    t = {k: v.requires_grad_() if v.is_floating_point() else v for k, v in tensors().items()}
    names = [k for k in t if k != "t"]
    loss, want = model(t), plain(t)
    assert abs(loss.item() - want.item()) < 2 ** -14
    got = torch.autograd.grad(loss, [t[k] for k in names])
    ref = torch.autograd.grad(want, [t[k] for k in names])
    for k, a, b in zip(names, got, ref):
        assert (a - b).abs().max() <= 2 ** -14 * b.abs().max(), k


def test_only_what_needs_a_gradient_gets_one(calls):
    t = tensors()
    for k in PARAMS:
        t[k].requires_grad_()
    for k in ("x", "r"):
        assert torch.autograd.grad(model(t), t["w"])[0].shape == (6,)
    t = tensors()
    t["r"].requires_grad_()
    model(t).backward()
    assert t["r"].grad is not None and all(t[k].grad is None for k in PARAMS)


def test_the_sum_alone(calls):
    """A use of the norm's second output only: its gradient goes to both inputs,
    none to the weight."""
    t = tensors()
    for k in ("x", "r", "w"):
        t[k].requires_grad_()
    _, h = L.rms_norm(t["x"], t["w"], t["r"])
    (h * 3).sum().backward()
    assert torch.equal(t["x"].grad, torch.full_like(t["x"], 3.0))
    assert torch.equal(t["r"].grad, t["x"].grad) and t["w"].grad is None


@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_derivatives_are_refused(calls, grad):
    t = tensors()
    with fw.dual_level(), torch.set_grad_enabled(grad):
        d = {k: fw.make_dual(v, torch.ones_like(v)) for k, v in t.items() if k != "t"}
        for call in (lambda: L.rms_norm(d["x"]), lambda: L.rms_norm(t["x"], d["w"]),
                     lambda: L.rms_norm(t["x"], t["w"], d["r"]),
                     lambda: L.gated_mlp(d["x"], t["wg"], t["wu"], t["wd"]),
                     lambda: L.gated_mlp(t["x"], t["wg"], t["wu"], d["wd"]),
                     lambda: L.linear_cross_entropy(d["x"], t["table"], t["t"]),
                     lambda: L.linear_cross_entropy(t["x"], d["table"], t["t"])):
            with pytest.raises(NotImplementedError):
                call()
        assert torch.equal(L.rms_norm(t["x"], t["w"]), _rms(t["x"], t["w"]))


def test_gradients_are_not_differentiated_again(calls):
    t = {k: v.requires_grad_() if v.is_floating_point() else v for k, v in tensors().items()}
    g, = torch.autograd.grad(model(t), t["table"], create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


class _State:
    """Stands for the optimizer's flat arrays of one group."""

    def wait(self):
        pass

    def mark(self):
        pass


def with_slot(p, state):
    from distributed_bit_matrix_amd import optim as SO
    p = torch.nn.Parameter(p)
    p._signmuon_slot = SO.GradSlot(state, torch.full_like(p, float("nan")))
    return p


def test_direct_gradients(calls):
    """Gradients of every parameter go to their places and add up over two passes; a
    weight that two norms share gets both."""
    state, t = _State(), tensors()
    for k in PARAMS:
        t[k] = with_slot(t[k], state)
    params = [t[k] for k in PARAMS]
    want = torch.autograd.grad(model(t), params)
    assert not any(p._signmuon_slot.filled for p in params)
    for turn in (1, 2):
        model(t).backward()
        for p, g in zip(params, want):
            assert p.grad is None and p._signmuon_slot.filled
            # (the shared weight's two parts meet in another order)
            assert (p._signmuon_slot.grad - turn * g).abs().max() <= 2 ** -20 * g.abs().max()


def test_direct_gradients_of_some(calls):
    """One weight of the block is frozen, one not the optimizer's, one holds a
    gradient already."""
    state, t = _State(), tensors()
    t["wg"] = with_slot(t["wg"], state)
    t["wd"] = torch.nn.Parameter(t["wd"])
    y = lambda: L.gated_mlp(t["x"], t["wg"], t["wu"], t["wd"], "gelu").sum()  # noqa: E731
    wg, wd = torch.autograd.grad(y(), [t["wg"], t["wd"]])
    for turn in (1, 2):
        t["wd"].grad = None
        y().backward()
        assert torch.equal(t["wg"]._signmuon_slot.grad, turn * wg)
        assert torch.equal(t["wd"].grad, wd)


def test_one_parameter_in_two_places(calls):
    """As gate and up: the sum is returned, not written to its place twice."""
    state, t = _State(), tensors()
    t["wg"] = with_slot(t["wg"], state)
    L.gated_mlp(t["x"], t["wg"], t["wg"], t["wd"]).sum().backward()
    assert not t["wg"]._signmuon_slot.filled
    a, b = t["wg"].detach().clone().requires_grad_(), t["wg"].detach().clone().requires_grad_()
    ga, gb = torch.autograd.grad(L.gated_mlp(t["x"], a, b, t["wd"]).sum(), [a, b])
    assert torch.equal(t["wg"].grad, ga + gb)


def test_reductions_and_shapes(calls):
    t = tensors()
    none = L.linear_cross_entropy(t["x"], t["table"], t["t"], reduction="none")
    assert none.shape == (2, 5) and none[0, 2] == 0
    total = L.linear_cross_entropy(t["x"], t["table"], t["t"], reduction="sum")
    mean = L.linear_cross_entropy(t["x"], t["table"], t["t"])
    assert total.shape == mean.shape == ()
    assert abs(total - none.sum()) < 1e-4 and abs(mean - total / 8) < 1e-5
    t["x"].requires_grad_()
    each = L.linear_cross_entropy(t["x"], t["table"], t["t"], reduction="none")
    g, = torch.autograd.grad((each * torch.arange(10.).view(2, 5)).sum(), t["x"])
    assert g.shape == t["x"].shape and (g[0, 2] == 0).all() and (g[0, 0] == 0).all()


def test_modules(calls):
    norm, mlp = L.RMSNorm(6), L.GatedMLP(6, 7, "gelu")
    head = L.LinearCrossEntropy(9, 6, reduction="sum")
    assert [tuple(p.shape) for m in (norm, mlp, head) for p in m.parameters()] == [
        (6,), (7, 6), (7, 6), (6, 7), (9, 6)]
    t = tensors()
    y, h = norm(t["x"], t["r"])
    head(mlp(y) + h, t["t"]).backward()
    assert all(p.grad is not None for m in (norm, mlp, head) for p in m.parameters())
    table = L.Embedding(9, 6)
    assert L.LinearCrossEntropy(9, 6, weight=table.weight).weight is table.weight
    with pytest.raises(ValueError):
        L.LinearCrossEntropy(8, 6, weight=table.weight)
