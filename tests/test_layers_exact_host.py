"""The inputs with exact sums (tests/layer_reference.py) accept a float32
evaluation and reject what is lost from it, at sizes like those on the GPU."""
import numpy as np
import pytest

from tests import layer_reference as R

EPS = float(np.float32(1e-5))


def _ok(got, want, bound):
    return bool((np.abs(np.asarray(got, np.float64) - want) <= bound).all())


def _norm32(x, eps, lost=0, lost_squares=0):
    """In float32, the last columns left out of the sums."""
    f = np.float32
    n = x.shape[1]
    mean = x[:, :n - lost].sum(1, dtype=f) / f(n)
    d = x - mean[:, None]
    q = (d * d)[:, :n - lost_squares].sum(1, dtype=f) * (f(1) / f(n))
    rstd = f(1) / np.sqrt(q + f(eps))
    return d * rstd[:, None], mean, rstd


@pytest.mark.parametrize("rows,cols", [(9, 2), (7, 7), (5, 768), (3, 8193), (3, 16384), (2, 32769),
                                       (2, 100003), (1, 1 << 20)])
def test_a_lost_column_of_the_forward_pass_shows(rows, cols):
    x, want, bound = R.exact_norm(rows, cols, EPS, "f32")
    got = _norm32(x, EPS)
    assert all(_ok(g, w, e) for g, w, e in zip(got, want, bound))
    ref = R.norm(x, None, None, EPS)
    assert all(np.allclose(r, w, rtol=1e-12, atol=1e-12) for r, w in zip(ref, want))
    lost = _norm32(x, EPS, lost=1)
    assert not _ok(lost[1], want[1], bound[1])
    lost = _norm32(x, EPS, lost_squares=1 + cols % 2)        # the last of odd ones is 0
    assert not _ok(lost[2], want[2], bound[2])


def _grad32(dy, x, lost=0):
    f = np.float32
    n = dy.shape[1]
    inv = f(1) / f(n)
    c1 = dy[:, :n - lost].sum(1, dtype=f, keepdims=True) * inv
    c2 = (dy * x)[:, :n - lost].sum(1, dtype=f, keepdims=True) * inv
    return dy - c1 - x * c2


@pytest.mark.parametrize("rows,cols", [(5, 2), (9, 768), (4, 8193), (3, 16385), (3, 100003),
                                       (140000, 3), (70000, 24), (12289, 100)])
def test_a_lost_row_or_column_of_the_backward_pass_shows(rows, cols):
    dy, x, want, e = R.exact_norm_grad(rows, cols, "f32")
    ref = R.norm_grad(dy, x, None, np.zeros(rows), np.ones(rows))
    assert np.allclose(ref[0], want[0], rtol=0, atol=1e-10)
    assert np.array_equal(ref[1], want[1]) and np.array_equal(ref[2], want[2])
    assert _ok(_grad32(dy, x), want[0], e)
    assert not _ok(_grad32(dy, x, lost=2), want[0], e)
    live = slice(0, cols - cols % 2)
    for keep in (np.arange(rows) > 0, np.arange(rows) < rows - 1,
                 np.arange(rows) // max(1, rows // 512) != 1, np.zeros(rows, bool)):
        if keep.all():
            continue
        assert (dy[keep].sum(0) != want[2])[live].any()
        assert ((dy * x)[keep].sum(0) != want[1])[live].all()


def test_a_lost_token_shows():
    rng = np.random.default_rng(0)
    for n, vocab in ((131073, 3), (262145, 17)):
        t, dy = rng.integers(0, vocab, n), rng.integers(1, 4, (n, 2))
        want = R.exact_embed_grad(dy, t, vocab)
        s32 = np.zeros((vocab, 2), np.float32)
        np.add.at(s32, t, dy.astype(np.float32))
        assert np.array_equal(s32, want)
        for keep in (slice(1, None), slice(0, n - 1), slice(0, n - 512), slice(0, 0)):
            assert not np.array_equal(R.exact_embed_grad(dy[keep], t[keep], vocab)
                                      if dy[keep].size else 0 * want, want)
