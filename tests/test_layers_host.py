"""Host-only checks of the layer operators: exported symbols, refusals before
any GPU work, and the 64-bit reference with its error bounds."""
import ctypes
import os
import re

import numpy as np
import pytest

from distributed_bit_matrix_amd import binding as B
from tests import layer_reference as R

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
built = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libsignmuon.so not built")

# never dereferenced: validation fails first
P, Q, S = (ctypes.c_void_p(k << 20) for k in (1, 2, 3))
ODD = ctypes.c_void_p((1 << 20) + 1)
NAN, INF = float("nan"), float("inf")


@built
def test_declared_symbols_are_exported():
    text = open(os.path.join(ROOT, "include", "signmuon_layers.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(signmuon_\w+)\s*\(", text))
    assert names == set(B.LAYER_EXPORTS)
    for n in names:
        assert hasattr(B.lib(), n), n


def _norm(X=P, xd=0, xs=8, g=None, b=None, wd=0, rows=4, cols=8, eps=1e-5, Y=Q, m=None, r=None):
    return B.lib().signmuon_layer_norm(X, xd, xs, g, b, wd, rows, cols, eps, Y, m, r, None)


@built
def test_norm_refusals():
    assert _norm(rows=0, X=None, Y=None) == B.SM_OK
    for bad in (dict(xd=2), dict(wd=-1), dict(rows=-1), dict(rows=1 << 31), dict(cols=0),
                dict(cols=(1 << 20) + 1, xs=1 << 21), dict(eps=-1e-9), dict(eps=NAN),
                dict(eps=INF), dict(X=None), dict(Y=None), dict(xs=7), dict(xs=1 << 40),
                dict(Y=P, xs=9), dict(X=ODD), dict(Y=ODD), dict(g=ODD), dict(b=ODD),
                dict(m=ODD), dict(r=ODD), dict(xd=1, X=ODD)):
        assert _norm(**bad) == B.SM_EINVAL, bad


def _norm_grad(dY=P, dys=8, X=Q, xd=0, xs=8, g=None, wd=0, m=S, r=S, rows=4, cols=8, dX=S, dg=S,
               db=S, dwd=0, acc=0, ws=P, nbytes=None):
    if nbytes is None:
        nbytes = B.lib().signmuon_layer_norm_backward_workspace(4, 8)
    return B.lib().signmuon_layer_norm_backward(dY, dys, X, xd, xs, g, wd, m, r, rows, cols, dX,
                                                dg, db, dwd, acc, ws, nbytes, None)


@built
def test_norm_grad_refusals():
    assert _norm_grad(dX=None, dg=None, db=None) == B.SM_OK     # nothing is wanted
    for bad in (dict(xd=3), dict(wd=9), dict(dwd=2), dict(rows=-1), dict(cols=0), dict(acc=2),
                dict(acc=1, dwd=1), dict(dY=None), dict(X=None), dict(m=None), dict(r=None),
                dict(dys=7), dict(xs=7), dict(dX=Q), dict(dX=P, dys=9), dict(dX=ODD),
                dict(dg=ODD), dict(db=ODD), dict(dY=ODD), dict(X=ODD), dict(g=ODD),
                dict(m=ODD), dict(r=ODD)):
        assert _norm_grad(**bad) == B.SM_EINVAL, bad
    need = B.layer_norm_backward_workspace(5000, 8)
    assert need > 0 and need % 256 == 0
    assert _norm_grad(rows=5000, nbytes=need - 1) == B.SM_EWORKSPACE
    assert _norm_grad(rows=5000, ws=None, nbytes=need) == B.SM_EWORKSPACE
    assert _norm_grad(rows=5000, ws=ctypes.c_void_p((1 << 20) + 16),
                      nbytes=need) == B.SM_EWORKSPACE
    assert B.layer_norm_backward_workspace(4, 8) == 0           # one launch
    for rows, cols in ((-1, 8), (4, 0), (1 << 31, 8), (4, (1 << 20) + 1)):
        with pytest.raises(B.SignMuonError) as e:
            B.layer_norm_backward_workspace(rows, cols)
        assert e.value.status == B.SM_EINVAL


def _embed(W=P, wd=0, vocab=9, dim=8, t=Q, bits=64, n=5, scale=1.0, Y=S, yd=0):
    return B.lib().signmuon_embedding(W, wd, vocab, dim, t, bits, n, scale, Y, yd, None)


@built
def test_a_norm_gradient_that_is_an_input_is_refused():
    """But dX, which may be dY."""
    gamma, dx, dg, db = (ctypes.c_void_p(k << 20) for k in (5, 6, 7, 8))
    for rows in (4, 5000):
        full = dict(g=gamma, rows=rows, nbytes=1 << 34)
        for bad in (P, Q, S, gamma, dx):
            assert _norm_grad(dX=dx, dg=bad, db=db, **full) == B.SM_EINVAL, bad
            assert _norm_grad(dX=dx, dg=dg, db=bad, **full) == B.SM_EINVAL, bad
        for bad in (Q, S, gamma):
            assert _norm_grad(dX=bad, dg=dg, db=db, **full) == B.SM_EINVAL, bad


@built
def test_embedding_refusals():
    assert _embed(n=0, W=None, t=None, Y=None) == B.SM_OK
    for bad in (dict(wd=2), dict(yd=2), dict(bits=16), dict(n=-1), dict(n=(1 << 30) + 1), dict(vocab=0),
                dict(vocab=(1 << 20) + 1), dict(dim=0), dict(dim=(1 << 20) + 1), dict(scale=NAN),
                dict(scale=INF), dict(W=None), dict(t=None), dict(Y=None), dict(W=ODD),
                dict(t=ctypes.c_void_p((1 << 20) + 4)), dict(Y=ODD), dict(yd=1, Y=ODD)):
        assert _embed(**bad) == B.SM_EINVAL, bad


def _embed_grad(dY=P, dyd=0, dys=8, t=Q, bits=64, n=5, pad=-1, scale=1.0, dW=S, dwd=0, vocab=9,
                dim=8, acc=0, ws=P, nbytes=1 << 30):
    return B.lib().signmuon_embedding_backward(dY, dyd, dys, t, bits, n, pad, scale, dW, dwd,
                                               vocab, dim, acc, ws, nbytes, None)


@built
def test_embedding_grad_refusals():
    assert _embed_grad(n=0, acc=1, dW=None, ws=None) == B.SM_OK
    for bad in (dict(dyd=2), dict(dwd=2), dict(bits=8), dict(n=-1), dict(n=(1 << 27) + 1),
                dict(vocab=0), dict(dim=0), dict(pad=-2), dict(pad=9), dict(scale=NAN),
                dict(acc=2), dict(acc=1, dwd=1), dict(dW=None), dict(dW=ODD), dict(dY=None),
                dict(t=None), dict(dys=7), dict(dY=ODD), dict(t=ctypes.c_void_p((1 << 20) + 4))):
        assert _embed_grad(**bad) == B.SM_EINVAL, bad
    big = dict(n=5000, vocab=900, dim=8)
    need = B.embedding_backward_workspace(5000, 900, 8)
    assert need > 2 * 5000 * 4 and need % 256 == 0
    assert _embed_grad(**big, nbytes=need - 1) == B.SM_EWORKSPACE
    assert _embed_grad(**big, ws=None) == B.SM_EWORKSPACE
    assert _embed_grad(**big, ws=ctypes.c_void_p((1 << 20) + 64)) == B.SM_EWORKSPACE
    assert B.embedding_backward_workspace(5, 9, 8) == 0         # one launch
    for args in ((-1, 9, 8), (5, 0, 8), (5, 9, 0), ((1 << 27) + 1, 9, 8), (5, (1 << 20) + 1, 8)):
        with pytest.raises(B.SignMuonError) as e:
            B.embedding_backward_workspace(*args)
        assert e.value.status == B.SM_EINVAL


def test_cpu_tensors_are_refused():
    x, t = torch.zeros(3, 4), torch.zeros(3, dtype=torch.int64)
    for call in (lambda: B.layer_norm(x), lambda: B.layer_norm_backward(x, x, None, x, x),
                 lambda: B.embedding(t, x), lambda: B.embedding_backward(x, t, 4)):
        with pytest.raises(TypeError):
            call()


def test_rows_of_a_tensor():
    x = torch.zeros(4, 6, 8)
    assert B._rows(x, "x") == (24, 8, 8)
    assert B._rows(x[:, 0, :5], "x") == (4, 5, 48)
    assert B._rows(x[0], "x") == (6, 8, 8)
    assert B._rows(torch.zeros(8), "x") == (1, 8, 8)
    assert B._rows(torch.zeros(5, 9)[:, :1], "x") == (5, 1, 9)
    assert B._rows(torch.zeros(0, 8), "x") == (0, 8, 8)
    for bad in (x.transpose(0, 1), x[..., ::2], x[0].t(), torch.zeros(1, 8).expand(4, 8),
                torch.zeros(8, 1).expand(8, 4), torch.zeros(40).as_strided((4, 8), (4, 1))):
        with pytest.raises(TypeError):
            B._rows(bad, "x")
    with pytest.raises(ValueError):
        B._rows(torch.zeros(()), "x")


def test_layers_arguments():
    from distributed_bit_matrix_amd import layers as L
    e = L.Embedding(7, 3, scale=2.0, padding_idx=1)
    assert e.weight.shape == (7, 3) and float(e.weight.detach().abs().max()) < 0.2
    n = L.LayerNorm(5, bias=False)
    assert n.bias is None and n.weight.detach().tolist() == [1.0] * 5
    for pad in (-1, 7):
        with pytest.raises(ValueError):
            L.embedding(torch.zeros(2, dtype=torch.int64), e.weight, padding_idx=pad)
    with pytest.raises(TypeError):           # no CPU path
        n(torch.zeros(2, 5))
    x = torch.zeros(6, 4).expand(3, 6, 4)
    assert L._dense_rows(x).is_contiguous() and L._dense_rows(x[0]) is not None


# The bounds have to hold for an evaluation in float32 and to reject mistakes.
def _norm32(x, g, b, eps):
    x = x.astype(np.float32)
    mean = x.mean(1, dtype=np.float32)
    d = x - mean[:, None]
    rstd = np.float32(1) / np.sqrt((d * d).mean(1, dtype=np.float32) + np.float32(eps))
    return d * rstd[:, None] * g + b, mean, rstd


def test_norm_bounds_accept_float32_and_reject_mistakes():
    rng = np.random.default_rng(0)
    for cols in (1, 7, 300):
        x = (3 * rng.standard_normal((20, cols)) + 1).astype(np.float32)
        g = (1 + 0.3 * rng.standard_normal(cols)).astype(np.float32)
        b = rng.standard_normal(cols).astype(np.float32)
        y, m, r = R.norm(x, g, b, 1e-5)
        by, bm, br = R.norm_bounds(x, g, b, 1e-5, "f32")
        y32, m32, r32 = _norm32(x, g, b, 1e-5)
        assert (np.abs(y32 - y) <= by).all() and (np.abs(m32 - m) <= bm).all()
        assert (np.abs(r32 - r) <= br).all()
        if cols > 1:
            wrong = x.std(1, ddof=1)[:, None]            # divided by cols - 1
            y_wrong = (x - m[:, None]) / wrong * g + b
            assert not (np.abs(y_wrong - y) <= by).all()
            assert not (np.abs(np.roll(y, 1, axis=1) - y) <= by).all()
            assert not (np.abs(y - b - y) <= by).all()   # a bias left out


def test_norm_grad_bounds_reject_mistakes():
    rng = np.random.default_rng(1)
    x, dy = (rng.standard_normal((40, 33)).astype(np.float32) for _ in range(2))
    g = (1 + 0.3 * rng.standard_normal(33)).astype(np.float32)
    _, m, r = R.norm(x, None, None, 1e-5)
    dx, dg, db = R.norm_grad(dy, x, g, m, r)
    ex, eg, eb = R.norm_grad_bounds(dy, x, g, m, r, "f32", "f32")
    # differences of the definition
    h, i, j = 1e-5, 3, 7
    hi, lo = x.astype(np.float64), x.astype(np.float64)
    hi[i, j] += h
    lo[i, j] -= h
    diff = (dy * (R.norm(hi, g, None, 1e-5)[0] - R.norm(lo, g, None, 1e-5)[0])).sum() / (2 * h)
    assert abs(diff - dx[i, j]) < 1e-7
    few = R.norm_grad(dy[:-1], x[:-1], g, m[:-1], r[:-1])       # the last row left out
    assert not (np.abs(few[1] - dg) <= eg).all() and not (np.abs(few[2] - db) <= eb).all()
    no_gamma = R.norm_grad(dy, x, None, m, r)[0]
    assert not (np.abs(no_gamma - dx) <= ex).all()
    y32 = (dy * ((x - m[:, None].astype(np.float32)) * r[:, None].astype(np.float32))).sum(
        0, dtype=np.float32)
    want = R.norm_grad(dy, x, g, m.astype(np.float32), r.astype(np.float32))[1]
    assert (np.abs(y32 - want) <= eg).all()


def test_embed_grad_bounds_reject_mistakes():
    rng = np.random.default_rng(2)
    dy = rng.standard_normal((500, 6)).astype(np.float32)
    t = rng.integers(0, 20, 500)
    dw, mag, counts = R.embed_grad(dy, t, 22, 0.5)
    e = R.embed_grad_bounds(dw, mag, counts, "f32")
    assert counts.sum() == 500 and (dw[20:] == 0).all() and (e[20:] <= 1e-30).all()
    moved = t.copy()
    moved[17] = (moved[17] + 1) % 20                             # one row to another token
    assert not (np.abs(R.embed_grad(dy, moved, 22, 0.5)[0] - dw) <= e).all()
    assert not (np.abs(2 * dw - dw) <= e).all()                  # the scale left out
    s32 = np.zeros((22, 6), np.float32)
    for i in range(500):
        s32[t[i]] += dy[i]
    assert (np.abs(np.float32(0.5) * s32 - dw) <= e).all()


@built
def test_norm_grad_refuses_one_array_for_both_sums():
    both = ctypes.c_void_p(9 << 20)
    assert _norm_grad(dg=both, db=both) == B.SM_EINVAL
    assert _norm_grad(dX=None, dg=both, db=both) == B.SM_EINVAL


class _Probe(torch.autograd.Function):
    """x * w that records whether the pass adds to the grads of x and w."""
    seen = []

    @staticmethod
    def forward(ctx, x, w):
        ctx.save_for_backward(x, w)
        return x * w

    @staticmethod
    def backward(ctx, g):
        from distributed_bit_matrix_amd import layers as L
        x, w = ctx.saved_tensors
        _Probe.seen.append(tuple(L._accumulates(ctx, i) for i in (0, 1)))
        return g * w, g * x


def test_a_pass_knows_whether_it_adds_to_a_leaf():
    x, w = torch.ones(3, requires_grad=True), torch.nn.Parameter(torch.ones(3))

    def run(call):
        _Probe.seen.clear()
        call(_Probe.apply(x, w).sum())
        return _Probe.seen[0]

    assert run(lambda y: y.backward()) == (True, True)
    assert run(lambda y: y.backward(inputs=[x])) == (True, False)
    assert run(lambda y: y.backward(inputs=[w])) == (False, True)
    assert run(lambda y: torch.autograd.grad(y, [w])) == (False, False)
    assert run(lambda y: torch.autograd.grad(y, [x])) == (False, False)
    assert run(lambda y: torch.autograd.grad(y, [x, w])) == (False, False)


def test_parameters_with_a_slot_can_be_saved_and_copied():
    import copy
    import io
    from distributed_bit_matrix_amd import optim as SO

    class State:
        pass

    state, p = State(), torch.nn.Parameter(torch.arange(4.))
    p._signmuon_slot = SO.GradSlot(state, torch.zeros(4))
    f = io.BytesIO()
    torch.save(p, f)
    f.seek(0)
    q = torch.load(f, weights_only=False)          # the file written above
    for r in (q, copy.deepcopy(p)):
        assert torch.equal(r.detach(), p.detach())
        assert r.__dict__.get("_signmuon_slot") is None
    assert p._signmuon_slot.alive()
    del state
    assert not p._signmuon_slot.alive()


def test_direct_gradients_need_parameters_on_a_gpu():
    from distributed_bit_matrix_amd import optim as SO
    p = torch.nn.Parameter(torch.zeros(4))
    with pytest.raises(ValueError):
        SO.SignMuon([p], direct_grads=True)
    assert "_signmuon_slot" not in p.__dict__
    opt = SO.SignMuon([p])              # without them, they may move later
    opt.zero_grad()
    with pytest.raises(ValueError):
        opt.step()


@built
def test_row_strides_are_limited():
    """More than memory holds is refused, whatever the number of rows."""
    far = 1 << 39
    for bad in (dict(xs=far + 1), dict(xs=far, rows=(1 << 21) + 1), dict(xs=-8)):
        assert _norm(**bad) == B.SM_EINVAL, bad
        assert _norm_grad(**bad) == B.SM_EINVAL, bad
    for bad in (dict(dys=far + 1), dict(dys=far, n=(1 << 21) + 1, nbytes=1 << 62)):
        assert _embed_grad(**bad) == B.SM_EINVAL, bad
