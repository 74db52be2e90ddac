"""The oracle of the norm, the 8-bit product and the log probabilities against
differences of its own forward and hand-worked values (CPU)."""
import numpy as np
import pytest

from oracle import readout as ro


def diff(f, x, d=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += d
        b[i] -= d
        g[i] = (f(a) - f(b)) / (2 * d)
    return g


@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (2, 16)])
def test_norm_gradient(rows, dim):
    rng = np.random.default_rng(rows * 100 + dim)
    h, w = rng.normal(size=(rows, dim)), rng.normal(size=dim)
    dout, dh = rng.normal(size=(rows, dim)), rng.normal(size=(rows, dim))
    loss = lambda h, w: (dout * ro.add_rmsnorm_fwd(h, w, 1e-3)[0]).sum() + (dh * h).sum()  # noqa: E731
    d, dw = ro.add_rmsnorm_bwd(h, w, 1e-3, dout, dh)
    assert np.allclose(d, diff(lambda x: loss(x, w), h), atol=1e-7)
    assert np.allclose(dw, diff(lambda x: loss(h, x), w), atol=1e-7)


@pytest.mark.parametrize("V,scale", [(1, 1.0), (5, 0.7), (30, 2.0)])
def test_logprob_gradient(V, scale):
    rng = np.random.default_rng(V)
    x = rng.normal(size=(4, V))
    if V > 3:
        x[1, [0, 2]] = -np.inf
    tok = np.array([0, V // 2 if V != 5 else 3, -1, V - 1])
    dl, dH = rng.normal(size=4), rng.normal(size=4)

    def loss(x):
        o = ro.token_logprobs(x, tok, scale)
        return (dl * o["logprobs"] * (tok >= 0)).sum() + (dH * o["entropy"]).sum()
    got = ro.token_logprobs_bwd(x, tok, scale, dl, dH)
    with np.errstate(all="ignore"):
        want = np.where(np.isinf(x), 0.0, diff(loss, x))
    assert np.allclose(got, want, atol=1e-7)


def test_logprob_values():
    x = np.log([[1.0, 2.0, 1.0, 4.0]])
    o = ro.token_logprobs(x, [1], 1.0, 3)
    assert np.allclose(o["logprobs"], np.log(0.25)) and np.allclose(o["lse"], np.log(8))
    p = np.array([1, 2, 1, 4]) / 8
    assert np.allclose(o["entropy"], -(p * np.log(p)).sum())
    assert list(o["top_tokens"][0]) == [3, 1, 0]        # the tie of 0 and 2 goes to 0
    o = ro.token_logprobs(np.full((1, 3), -np.inf), [1], 1.0, 2)
    assert o["lse"][0] == o["logprobs"][0] == -np.inf and o["entropy"][0] == 0
    assert list(o["top_tokens"][0]) == [-1, -1]


def test_half_steps():
    vals = np.unique(ro.code_values(np.arange(127, dtype=np.uint8), "e4m3"))
    gaps = np.diff(vals)
    # the step above each value, and so twice half_steps there
    assert np.array_equal(gaps, 2 * ro.half_steps(vals[:-1], "e4m3"))


def test_matmul_values():
    a, w = np.array([[1.0, -2, 3]]), np.array([[4.0, 5, 6], [0, 0, 1]])
    out = ro.scaled_matmul(a, np.array([2.0]), w, np.array([0.5, 10.0]), np.array([1.0, -1.0]))
    assert np.allclose(out, [[2 * 0.5 * 12 + 1, 2 * 10 * 3 - 1]])
