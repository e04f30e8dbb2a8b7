"""Host-only checks of the residual norm, the gated block and the linear cross
entropy: refusals before any GPU work, workspaces, and the 64-bit reference with its
error bounds."""
import ctypes
import os

import pytest

from distributed_bit_matrix_amd import binding as B
from tests import block_reference as R

torch = pytest.importorskip("torch")

built = pytest.mark.skipif(not os.path.exists(B.LIB_PATH), reason="libsignmuon.so not built")

# never dereferenced: validation fails first
P, Q, S, T, U, V = (ctypes.c_void_p(k << 20) for k in (1, 2, 3, 4, 5, 6))
ODD = ctypes.c_void_p((1 << 20) + 1)
NAN, INF = float("nan"), float("inf")


def _rms(X=P, xs=8, R_=None, rs=8, xd=0, g=None, wd=0, rows=4, cols=8, eps=1e-6, H=None, Y=Q,
         r=None):
    return B.lib().signmuon_rms_norm(X, xs, R_, rs, xd, g, wd, rows, cols, eps, H, Y, r, None)


def _rms8(X=P, xs=8, R_=None, rs=8, xd=0, g=None, wd=0, rows=4, cols=8, eps=1e-6, block=128, H=None,
          Y=Q, sc=S, r=None):
    return B.lib().signmuon_rms_norm_e4m3(X, xs, R_, rs, xd, g, wd, rows, cols, eps, block, H, Y,
                                          sc, r, None)


@built
def test_rms_refusals():
    for call in (_rms, _rms8):
        assert call(rows=0, X=None, Y=None) == B.SM_OK
        for bad in (dict(xd=2), dict(wd=-1), dict(rows=-1), dict(rows=1 << 31), dict(cols=0),
                    dict(cols=(1 << 20) + 1, xs=1 << 21), dict(eps=-1e-9), dict(eps=NAN),
                    dict(eps=INF), dict(X=None), dict(Y=None), dict(xs=7), dict(xs=1 << 40),
                    dict(Y=P, xs=9), dict(X=ODD), dict(g=ODD), dict(r=ODD), dict(xd=1, X=ODD),
                    dict(R_=S), dict(R_=S, H=T, rs=7), dict(R_=ODD, H=T), dict(R_=S, H=ODD),
                    dict(R_=S, H=P, xs=9), dict(R_=S, H=S, rs=9), dict(R_=S, H=Q),
                    dict(R_=Q, H=T)):
            assert call(**bad) == B.SM_EINVAL, (call, bad)
    for bad in (dict(Y=P), dict(sc=None), dict(sc=ODD), dict(block=64), dict(block=-1),
                dict(cols=16385, xs=16385)):
        assert _rms8(**bad) == B.SM_EINVAL, bad
    assert _rms(Y=ODD) == B.SM_EINVAL


def _rms_grad(dY=P, dys=8, H=Q, hs=8, dH=None, dhs=8, xd=0, g=None, wd=0, r=S, rows=4, cols=8,
              dX=T, dg=U, dwd=0, acc=0, ws=None, nbytes=0):
    return B.lib().signmuon_rms_norm_backward(dY, dys, H, hs, dH, dhs, xd, g, wd, r, rows, cols, dX,
                                              dg, dwd, acc, ws, nbytes, None)


@built
def test_one_array_for_two_outputs_is_refused():
    for bad in (dict(r=P), dict(r=Q), dict(r=T, R_=T, H=S), dict(r=S, R_=T, H=S)):
        assert _rms(**bad) == _rms8(**{"sc": U, **bad}) == B.SM_EINVAL, bad
    for bad in (dict(sc=Q), dict(sc=P), dict(sc=T, r=T)):
        assert _rms8(**bad) == B.SM_EINVAL, bad
    for same in (P, Q, S, T, U):
        assert _mlp(pre=same) == B.SM_EINVAL
    for bad in (dict(loss=U), dict(loss=P), dict(loss=Q), dict(loss=S), dict(lse=P), dict(lse=Q),
                dict(lse=S)):
        assert _loss(**bad) == B.SM_EINVAL, bad


@built
def test_rms_grad_refusals():
    assert _rms_grad(dX=None, dg=None) == B.SM_OK            # nothing is wanted
    for bad in (dict(xd=3), dict(wd=9), dict(dwd=2), dict(rows=-1), dict(cols=0), dict(acc=2),
                dict(acc=1, dwd=1), dict(dY=None), dict(H=None), dict(r=None), dict(dys=7),
                dict(hs=7), dict(dH=V, dhs=7), dict(dX=Q), dict(dX=P, dys=9),
                dict(dH=V, dX=V, dhs=9), dict(dY=ODD), dict(H=ODD), dict(dH=ODD), dict(g=ODD),
                dict(r=ODD), dict(dX=ODD), dict(dg=ODD)):
        assert _rms_grad(**bad) == B.SM_EINVAL, bad
    need = B.rms_norm_backward_workspace(5000, 8)
    assert need > 0 and need % 256 == 0
    big = dict(rows=5000, ws=P)
    assert _rms_grad(**big, nbytes=need - 1) == B.SM_EWORKSPACE
    assert _rms_grad(rows=5000, nbytes=need) == B.SM_EWORKSPACE
    assert _rms_grad(rows=5000, ws=ctypes.c_void_p((1 << 20) + 64), nbytes=need) == B.SM_EWORKSPACE
    assert B.rms_norm_backward_workspace(5, 8) == 0           # one launch
    for args in ((-1, 8), (5, 0), (1 << 31, 8), (5, (1 << 20) + 1)):
        with pytest.raises(B.SignMuonError):
            B.rms_norm_backward_workspace(*args)


@built
def test_an_output_that_is_an_input_is_refused():
    """But where a call says that it may be."""
    gamma = ctypes.c_void_p(9 << 20)
    for bad in (dict(g=Q), dict(g=S, r=S), dict(g=S, R_=T, H=S)):
        assert _rms(**bad) == _rms8(**{"sc": U, **bad}) == B.SM_EINVAL, bad
    for bad in (dict(g=S), dict(R_=S, H=T), dict(sc=T, R_=V, H=T)):
        assert _rms8(**bad) == B.SM_EINVAL, bad
    # every size: few rows go in one launch that reads all inputs and writes all outputs
    big = dict(rows=5000, cols=8, ws=ctypes.c_void_p(11 << 20), nbytes=BIG)
    for bad in (dict(dg=P), dict(dg=Q), dict(dg=S), dict(dg=T), dict(dg=gamma), dict(dX=S),
                dict(dX=gamma), dict(dH=V, dg=V)):
        assert _rms_grad(g=gamma, **bad) == B.SM_EINVAL, bad
        assert _rms_grad(g=gamma, **big, **bad) == B.SM_EINVAL, bad
    for bad in (P, Q, S, U, V):
        assert _loss_grad(dW=bad) == B.SM_EINVAL, bad
        assert bad is P or _loss_grad(dX=bad) == B.SM_EINVAL, bad


BIG = 1 << 34


def _mlp(X=P, xs=8, g=Q, u=S, d=T, dt=0, act=0, rows=4, dim=8, hid=16, Y=U, pre=None, ws=P,
         nbytes=BIG):
    return B.lib().signmuon_gated_mlp(X, xs, g, u, d, dt, act, rows, dim, hid, Y, pre, ws, nbytes,
                                      None)


def _mlp_grad(dY=V, dys=8, X=P, xs=8, g=Q, u=S, d=T, pre=U, dt=0, act=0, rows=4, dim=8, hid=16,
              out=(7, 8, 9, 10), dwd=0, acc=0, ws=P, nbytes=BIG):
    out = [o if o is None or isinstance(o, ctypes.c_void_p) else ctypes.c_void_p(o << 20)
           for o in out]
    return B.lib().signmuon_gated_mlp_backward(dY, dys, X, xs, g, u, d, pre, dt, act, rows, dim, hid,
                                               *out, dwd, acc, ws, nbytes, None)


@built
def test_mlp_refusals():
    assert _mlp(rows=0, X=None, Y=None, ws=None) == B.SM_OK
    assert _mlp_grad(out=(None,) * 4) == B.SM_OK
    shared = (dict(dt=2), dict(act=2), dict(act=-1), dict(rows=-1), dict(rows=(1 << 22) + 1),
              dict(dim=0), dict(dim=(1 << 16) + 1, xs=1 << 17), dict(hid=0),
              dict(hid=(1 << 16) + 1), dict(X=None), dict(g=None), dict(u=None), dict(d=None),
              dict(xs=7), dict(xs=1 << 40), dict(X=ODD), dict(g=ODD), dict(u=ODD), dict(d=ODD),
              dict(pre=ODD))
    for bad in shared + (dict(Y=None), dict(Y=P), dict(Y=Q), dict(Y=S), dict(Y=T), dict(Y=ODD)):
        assert _mlp(**bad) == B.SM_EINVAL, bad
    for bad in shared + (dict(dY=None), dict(pre=None), dict(dys=7), dict(dY=ODD), dict(dwd=2),
                         dict(acc=2), dict(acc=1, dwd=1), dict(out=(7, 8, 8, 9)),
                         dict(out=(7, 7, 8, 9)), dict(out=(7, 8, 9, 7)), dict(out=(P, 8, 9, 10)),
                         dict(out=(7, Q, 9, 10)), dict(out=(7, 8, U, 10)), dict(out=(V, 8, 9, 10)),
                         dict(out=(ODD, 8, 9, 10)), dict(out=(7, 8, ODD, 10))):
        assert _mlp_grad(**bad) == B.SM_EINVAL, bad
    for call, back in ((_mlp, False), (_mlp_grad, True)):
        need = B.gated_mlp_workspace(40, 8, 16, torch.float32, back)
        assert need > 0 and need % 256 == 0
        assert call(rows=40, nbytes=need - 1) == B.SM_EWORKSPACE
        assert call(rows=40, ws=None) == B.SM_EWORKSPACE
        assert call(rows=40, ws=ctypes.c_void_p((1 << 20) + 64)) == B.SM_EWORKSPACE
    assert B.gated_mlp_workspace(0, 8, 16, torch.bfloat16, True) == 0
    for args in ((-1, 8, 8), (5, 0, 8), (5, 8, 0), ((1 << 22) + 1, 8, 8), (5, (1 << 16) + 1, 8)):
        with pytest.raises(B.SignMuonError):
            B.gated_mlp_workspace(*args, torch.float32, False)


def _loss(X=P, xs=8, W=Q, dt=0, t=S, bits=64, rows=20, dim=8, vocab=9, ignore=-100, red=2, loss=T,
          lse=U, ws=P, nbytes=BIG):
    return B.lib().signmuon_linear_cross_entropy(X, xs, W, dt, t, bits, rows, dim, vocab, ignore,
                                                 red, loss, lse, ws, nbytes, None)


def _loss_grad(dl=V, X=P, xs=8, W=Q, dt=0, t=S, bits=64, lse=U, rows=20, dim=8, vocab=9,
               ignore=-100, red=2, dX=ctypes.c_void_p(7 << 20), dW=ctypes.c_void_p(8 << 20), dwd=0,
               acc=0, ws=P, nbytes=BIG):
    return B.lib().signmuon_linear_cross_entropy_backward(
        dl, X, xs, W, dt, t, bits, lse, rows, dim, vocab, ignore, red, dX, dW, dwd, acc, ws, nbytes,
        None)


@built
def test_loss_refusals():
    assert _loss(rows=0, red=0, X=None, loss=None, ws=None) == B.SM_OK
    assert _loss_grad(dX=None, dW=None) == B.SM_OK
    assert _loss_grad(rows=0, dX=None, acc=1, ws=None) == B.SM_OK
    shared = (dict(dt=2), dict(bits=16), dict(rows=-1), dict(rows=(1 << 22) + 1), dict(dim=0),
              dict(dim=(1 << 16) + 1, xs=1 << 17), dict(vocab=0), dict(vocab=(1 << 20) + 1),
              dict(red=3), dict(red=-1), dict(X=None), dict(W=None), dict(t=None), dict(lse=None),
              dict(xs=7), dict(xs=1 << 40), dict(X=ODD), dict(W=ODD), dict(lse=ODD),
              dict(t=ctypes.c_void_p((1 << 20) + 4)))
    for bad in shared + (dict(loss=None), dict(loss=ODD)):
        assert _loss(**bad) == B.SM_EINVAL, bad
    for bad in shared + (dict(dl=None), dict(dl=ODD), dict(dwd=2), dict(acc=2), dict(acc=1, dwd=1),
                         dict(dX=Q), dict(dX=P, xs=9), dict(dW=P), dict(dW=Q), dict(dX=ODD),
                         dict(dW=ODD), dict(dX=ctypes.c_void_p(8 << 20))):
        assert _loss_grad(**bad) == B.SM_EINVAL, bad
    for call, back in ((_loss, False), (_loss_grad, True)):
        need = B.linear_cross_entropy_workspace(20, 8, 9, torch.float32, back)
        assert need > 0 and need % 256 == 0
        assert call(nbytes=need - 1) == B.SM_EWORKSPACE
        assert call(ws=None) == B.SM_EWORKSPACE
        assert call(ws=ctypes.c_void_p((1 << 20) + 64)) == B.SM_EWORKSPACE
    for args in ((-1, 8, 9), (5, 0, 9), (5, 8, 0), ((1 << 22) + 1, 8, 9), (5, 8, (1 << 20) + 1)):
        with pytest.raises(B.SignMuonError):
            B.linear_cross_entropy_workspace(*args, torch.float32, False)


@built
def test_the_logits_are_not_kept():
    """A workspace holds a piece of the logits' gradient at most: 12288 rows over
    50257 tokens in bfloat16 would be 1.2 GB of them."""
    need = B.linear_cross_entropy_workspace(12288, 768, 50257, torch.bfloat16, False)
    assert need < 200 << 20
    wide = B.linear_cross_entropy_workspace(16384, 64, 1 << 20, torch.bfloat16, True)
    assert wide < 2.5 * (1 << 30) < 16384 * (1 << 20) * 2


def test_cpu_tensors_are_refused():
    x, t, w = torch.zeros(3, 4), torch.zeros(3, dtype=torch.int64), torch.zeros(5, 4)
    s = torch.zeros(())
    for call in (lambda: B.rms_norm(x), lambda: B.rms_norm_e4m3(x),
                 lambda: B.rms_norm_backward(x, x, None, t.float()),
                 lambda: B.gated_mlp(x, w, w, w.T.contiguous()),
                 lambda: B.gated_mlp_backward(x, x, w, w, w.T.contiguous(), torch.zeros(3, 10)),
                 lambda: B.linear_cross_entropy(x, w, t),
                 lambda: B.linear_cross_entropy_backward(s, x, w, t, t.float())):
        with pytest.raises(TypeError):
            call()


def test_an_index_to_be_ignored_past_64_bits_is_refused():
    """Its low 64 bits are another index, the ordinary one for instance."""
    x, t, w = torch.zeros(3, 4), torch.zeros(3, dtype=torch.int64), torch.zeros(5, 4)
    for ignore in (-(1 << 63), -100, 4, (1 << 63) - 1):
        assert B._loss_args(x, w, t, ignore, "mean", -1)[:4] == (3, 4, 4, 5)
    for ignore in ((1 << 64) - 100, 1 << 63, -(1 << 63) - 1):
        with pytest.raises(ValueError, match="ignore_index"):
            B._loss_args(x, w, t, ignore, "mean", -1)


# --- the reference and its bounds ------------------------------------------

DTYPES = [torch.float32, torch.bfloat16]


def gen(seed=0):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, dtype=torch.float32, std=1.0):
    return (std * torch.randn(shape, generator=g)).to(dtype)


def inside(got, want, bound):
    return bool(((got.double() - want).abs() <= bound).all())


def loss_inputs(dtype, rows=40, dim=24, vocab=50):
    g = gen()
    x, w = normal(g, rows, dim, dtype=dtype), normal(g, vocab, dim, dtype=dtype, std=0.4)
    t = torch.randint(vocab, (rows,), generator=g)
    t[::7] = -100
    return x, w, t


@pytest.mark.parametrize("dtype", DTYPES)
def test_loss_bounds_take_float32_and_no_mistake(dtype):
    x, w, t = loss_inputs(dtype)
    each, lse = R.loss(x, w, t, -100)
    e_each, e_lse = R.loss_bounds(x, w, t, -100)
    keep = t != -100
    z = x.float() @ w.float().T
    got_lse = torch.where(keep, torch.logsumexp(z, 1), 0.0)
    picked = z.gather(1, t.clamp(min=0)[:, None])[:, 0]
    got = torch.where(keep, got_lse - picked, 0.0)
    assert inside(got_lse, lse, e_lse) and inside(got, each, e_each)
    # one logit left out, one twice, a target off by one, the padding counted
    assert not inside(torch.where(keep, torch.logsumexp(z[:, 1:], 1), 0.0), lse, e_lse)
    assert not inside(torch.where(keep, torch.logsumexp(torch.cat([z, z[:, :1]], 1), 1), 0.0), lse,
                      e_lse)
    off = z.gather(1, (t.clamp(min=0)[:, None] + 1) % 50)[:, 0]
    assert not inside(torch.where(keep, got_lse - off, 0.0), each, e_each)
    assert not inside(torch.logsumexp(z, 1) - picked, each, e_each)


@pytest.mark.parametrize("dtype", DTYPES)
def test_likely_loss_takes_float32_and_no_errors_of_the_logits_size(dtype):
    g = gen(3)
    w = normal(g, 300, 64)
    w[:, 0] = 1.0
    w = w.to(dtype)
    t = torch.randint(300, (200,), generator=g)
    x = (0.3 * w[t].float()).to(dtype)
    x[:, 0] = torch.linspace(-1000, 1000, 200)
    want, bound = R.likely_loss(x, w, t)
    z = x.float() @ w.float().T
    top, at = z.amax(1, keepdim=True), z.gather(1, t[:, None])
    log2e = torch.tensor(1.4426950408889634)

    def evaluate(power):
        return ((top - at)[:, 0] + torch.log(torch.exp2(power).sum(1)))

    got = evaluate((z - top) * log2e)
    assert inside(got, want, bound) and (got >= 0).all()
    # the largest logit's product with log2(e) rounded, and the difference from it exact
    got = evaluate((z.double() * log2e.double() - (top * log2e).double()).float())
    assert not inside(got, want, bound) and (got < 0).any()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_loss_grad_bounds_take_float32_and_no_mistake(dtype, reduction):
    x, w, t = loss_inputs(dtype)
    lse = R.loss(x, w, t, -100)[1].float()
    dloss = 1 + 0.3 * normal(gen(1), *((40,) if reduction == "none" else ()))
    args = (dloss, x, w, t, lse, -100, reduction)
    dx, dw = R.loss_grad(*args)
    bx, bw = R.loss_grad_bounds(*args, dtype)

    def evaluate(shift=0, drop=False, count=None):
        keep = t != -100
        z = x.float() @ w.float().T
        g = torch.exp(z - lse[:, None])
        g[torch.arange(40), (t.clamp(min=0) + shift) % 50] -= 1
        scale = torch.where(keep | drop, dloss, 0.0)
        if reduction == "mean":
            scale = scale / (count or int(keep.sum()))
        g = (g * scale[:, None]).to(dtype).float()
        return (g @ w.float()).to(dtype), (g.T @ x.float()).to(dtype)

    got = evaluate()
    assert inside(got[0], dx, bx) and inside(got[1], dw, bw)
    wrong = [evaluate(shift=1), evaluate(drop=True)]
    if reduction == "mean":
        wrong.append(evaluate(count=40))
    for a, b in wrong:
        assert not inside(a, dx, bx) and not inside(b, dw, bw)
    # against autograd
    x64, w64 = x.double().requires_grad_(), w.double().requires_grad_()
    f = torch.nn.functional.cross_entropy(x64 @ w64.T, t, reduction=reduction)
    a, b = torch.autograd.grad(f, (x64, w64), dloss.double())
    assert (a - dx).abs().max() < 1e-6 and (b - dw).abs().max() < 1e-6   # (lse is float32)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_bounds_take_float32_and_no_mistake(dtype):
    g = gen()
    x, r = normal(g, 20, 33, dtype=dtype), normal(g, 20, 33, dtype=dtype)
    w = 1 + 0.3 * normal(g, 33)
    h = R.rms_sum(x, r)
    y, rstd = R.rms(h, w, 1e-6)
    e_y, e_r = R.rms_bounds(h, w, 1e-6)
    b_y = R.stored(y, e_y, dtype)

    def evaluate(h, cols=33):
        f = h.float()
        rs = torch.rsqrt(f.square().sum(1) / cols + 1e-6)
        return (f * rs[:, None] * w).to(dtype), rs

    got = evaluate(h)
    assert inside(got[0], y, b_y) and inside(got[1], rstd, e_r)
    # the width off by one, the sum not rounded (bfloat16), the residual left out
    assert not inside(evaluate(h, 34)[1], rstd, e_r)
    assert not inside(evaluate(x)[0], y, b_y)
    if dtype == torch.bfloat16:
        assert not inside(evaluate(x.float() + r.float())[1], rstd, e_r)
    s = R.e4m3_scales(y, 16)
    assert s.shape == (20, 3)
    q = (y / s.repeat_interleave(16, 1)[:, :33])
    code = q.float().to(torch.float8_e4m3fn).double()
    half = R.e4m3_half_step(q) * (1 + 2 ** -20)
    assert inside(code, q, half) and code.abs().max() == 448
    assert not inside(code.roll(1, 1), q, half)
    v = torch.tensor([1.0, 1.125, 448.0, 2.0 ** -6, 2.0 ** -9, 0.0], dtype=torch.float64)
    assert R.e4m3_half_step(v).tolist() == [2.0 ** -4, 2.0 ** -4, 16.0, 2.0 ** -10, 2.0 ** -10,
                                            2.0 ** -10]


def test_nearest_codes_take_a_rounded_quotient_and_no_other():
    x, v = R.rows_with_ties()
    k = v / R.e4m3_half_step(v)
    tie = (k % 2 == 1) & (v != 0)
    assert tie.sum() > 1000 and tie.any(1).all()
    off = ((k - 1) % 2 - 1).abs()                # 1 on a middle
    assert (1 - off[~tie]).min() >= 2.0 ** -11
    code = lambda q: q.to(torch.float8_e4m3fn).double()  # noqa: E731
    want = R.e4m3_nearest(v)
    assert torch.equal(code(v.float()), want)
    # the maximum's reciprocal rounded first; halves away from zero
    most = x.float().amax(1, keepdim=True)
    assert not torch.equal(code(x.float() * (448 / most)), want)
    step = 2 * R.e4m3_half_step(v)
    assert not torch.equal(torch.sign(v) * torch.floor(v.abs() / step + 0.5) * step, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rms_grad_bounds_take_float32_and_no_mistake(dtype):
    g = gen()
    dy, h, dh = (normal(g, 20, 33, dtype=dtype) for _ in range(3))
    w = 1 + 0.3 * normal(g, 33)
    rstd = R.rms(h, None, 1e-6)[1].float()
    dx, dw = R.rms_grad(dy, h, w, rstd, dh)
    bx, bw = R.rms_grad_bounds(dy, h, w, rstd, dh, torch.float32)
    xh = h.float() * rstd[:, None]
    gg = dy.float() * w
    got = (rstd[:, None] * (gg - xh * (gg * xh).mean(1, keepdim=True)) + dh.float()).to(dtype)
    sums = (dy.float() * xh).sum(0)
    assert inside(got, dx, bx) and inside(sums, dw, bw)
    assert not inside((got.float() - dh.float()).to(dtype), dx, bx)
    assert not inside((dy.float() * xh)[1:].sum(0), dw, bw)
    mean = rstd[:, None] * (gg - gg.mean(1, keepdim=True)) + dh.float()      # a layer norm's
    assert not inside(mean.to(dtype), dx, bx)
    h64, w64 = h.double().requires_grad_(), w.double().requires_grad_()
    y = h64 * torch.rsqrt(h64.square().mean(1, keepdim=True) + 1e-6) * w64
    a, b = torch.autograd.grad(y, (h64, w64), dy.double())
    assert (a + dh.double() - dx).abs().max() < 1e-5 and (b - dw).abs().max() < 1e-5


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_mlp_bounds_take_float32_and_no_mistake(dtype, kind):
    g = gen()
    x = normal(g, 30, 24, dtype=dtype)
    wg, wu = (normal(g, 40, 24, dtype=dtype, std=0.3) for _ in range(2))
    wd = normal(g, 24, 40, dtype=dtype, std=0.2)
    dy = normal(g, 30, 24, dtype=dtype)
    F = torch.nn.functional
    f = F.silu if kind == "silu" else F.gelu
    other = F.gelu if kind == "silu" else F.silu
    y, pre = R.mlp(x, wg, wu, wd, kind)
    b_y, b_pre = R.mlp_bounds(x, wg, wu, wd, kind)
    xf, gf, uf, df = (t.float() for t in (x, wg, wu, wd))

    def evaluate(act, flip=False):
        a, b = xf @ gf.T, xf @ uf.T
        if flip:
            a, b = b, a
        return ((act(a) * b).to(dtype).float() @ df.T).to(dtype), torch.cat([a, b], 1)

    got = evaluate(f)
    assert inside(got[0], y, b_y) and inside(got[1], pre, b_pre)
    assert not inside(evaluate(other)[0], y, b_y)
    assert not inside(evaluate(f, True)[0], y, b_y) and not inside(evaluate(f, True)[1], pre, b_pre)
    kept = pre.float()
    want = R.mlp_grad(dy, x, wg, wu, wd, kept, kind)
    bound = R.mlp_grad_bounds(dy, x, wg, wu, wd, kept, kind, dtype)

    def grads(act):
        p = kept.clone().requires_grad_()
        a, b = p.chunk(2, 1)
        h = act(a) * b
        dh = dy.float() @ df
        dp, = torch.autograd.grad(h, p, dh)
        dp = dp.to(dtype).float()
        dg, du = dp.chunk(2, 1)
        hh = h.detach().to(dtype).float()
        return [t.to(dtype) for t in (dg @ gf + du @ uf, dg.T @ xf, du.T @ xf, dy.float().T @ hh)]

    for a, b, c in zip(grads(f), want, bound):
        assert inside(a, b, c)
    for a, b, c in zip(grads(other), want, bound):
        assert not inside(a, b, c)
    # against autograd in 64 bits, which has no rounded pre-activations
    args = [t.double().requires_grad_() for t in (x, wg, wu, wd)]
    out = (f(args[0] @ args[1].T) * (args[0] @ args[2].T)) @ args[3].T
    for a, b in zip(torch.autograd.grad(out, args, dy.double()), want):
        assert (a - b).abs().max() < 1e-5
