"""Pins of the delta-rule oracle (CPU): the gradient against central
differences, packing, resuming, closed forms, and the chunked algebra."""
import numpy as np
import pytest

from oracle import delta as od


def draw(rng, b=1, L=7, H=4, P=3, N=5, G=2):
    n = rng.standard_normal
    k = n((b, L, G, N))
    return dict(q=n((b, L, G, N)), k=k / np.linalg.norm(k, axis=-1, keepdims=True),
                v=n((b, L, H, P)), g=-np.abs(n((b, L, H))), beta=rng.uniform(0, 1, (b, L, H)),
                init=n((b, H, P, N)))


def test_gradient_matches_central_differences():
    rng = np.random.default_rng(0)
    for seq in (None, np.array([[0, 0, 0, 1, 1, 4, 4]], np.int32)):
        d = draw(rng)
        dy, df = rng.standard_normal(d["v"].shape), rng.standard_normal(d["init"].shape)

        def loss(d):
            y, S = od.delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.7, d["init"], seq)
            return (y * dy).sum() + (S * df).sum()
        got = od.delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.7, dy, d["init"], seq, df)
        got = {n[1:]: x for n, x in got.items()}
        got["init"] = got.pop("initial_states")
        h = 1e-6    # truncation ~ h^2, cancellation ~ 1e-16 / h: both below 1e-8
        for name in d:
            num = np.empty_like(d[name])
            for i in np.ndindex(d[name].shape):
                e = {n: x.copy() for n, x in d.items()}
                e[name][i] += h
                up = loss(e)
                e[name][i] -= 2 * h
                num[i] = (up - loss(e)) / (2 * h)
            assert np.abs(num - got[name]).max() < 1e-6 * max(1, np.abs(num).max()), name


def test_packed_row_is_its_sequences_one_by_one():
    rng = np.random.default_rng(1)
    d = draw(rng, L=9)
    seq = np.array([[3] * 4 + [5] * 5], np.int32)
    y, S = od.delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], 1.0, d["init"], seq)
    for lo, hi, init in ((0, 4, d["init"]), (4, 9, None)):
        part = [d[n][:, lo:hi] for n in ("q", "k", "v", "g", "beta")]
        yy, SS = od.delta_fwd(*part, 1.0, init)
        assert np.allclose(yy, y[:, lo:hi], atol=1e-13)
    assert np.allclose(SS, S, atol=1e-13)


def test_closed_forms():
    rng = np.random.default_rng(2)
    d = draw(rng, L=3, G=4)
    zero, one = np.zeros_like(d["g"]), np.ones_like(d["beta"])
    # strength 1 and a unit key: the state then answers the key with the value
    k = d["k"]
    y, S = od.delta_fwd(k, k, d["v"], d["g"], one, 1.0, d["init"])
    assert np.allclose(y, d["v"], atol=1e-12)
    # strength 0: the state only decays
    y, S = od.delta_fwd(d["q"], k, d["v"], d["g"], zero, 1.0, d["init"])
    assert np.allclose(S, np.exp(d["g"].sum(1))[..., None, None] * d["init"], atol=1e-13)


@pytest.mark.parametrize("C", [1, 4, 16])
def test_chunk_algebra_is_the_recurrence(C):
    """The triangular system of a chunk (the kernels' formulas) against the
    token-by-token recurrence, forward and reverse."""
    rng = np.random.default_rng(3)
    L, P, N, scale = C, 3, 5, 0.6
    d = draw(rng, L=L, H=1, G=1, P=P, N=N)
    q, k, v = (d[n][0, :, 0] for n in ("q", "k", "v"))
    g, beta, S0 = d["g"][0, :, 0], d["beta"][0, :, 0], d["init"][0, 0].T
    gam = np.cumsum(g)
    E = np.tril(np.exp(gam[:, None] - gam[None]))
    e, o = np.exp(gam), np.exp(gam[-1] - gam)
    M = np.tril(E * (k @ k.T), -1) * beta
    w = np.linalg.solve(np.eye(L) + M, v - e[:, None] * (k @ S0))
    A = scale * E * (q @ k.T) * beta
    y = scale * e[:, None] * (q @ S0) + A @ w
    S1 = e[-1] * S0 + ((o * beta)[:, None] * k).T @ w
    ry, rS = od.delta_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale, d["init"])
    assert np.allclose(y, ry[0, :, 0], atol=1e-12) and np.allclose(S1, rS[0, 0].T, atol=1e-12)
    dy, D1 = rng.standard_normal((L, P)), rng.standard_normal((N, P))
    r = np.linalg.solve((np.eye(L) + M).T, A.T @ dy + (beta * o)[:, None] * (k @ D1))
    D0 = e[-1] * D1 + (e[:, None] * scale * q).T @ dy - (e[:, None] * k).T @ r
    ref = od.delta_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], scale, dy[None, :, None],
                       d["init"], None, D1.T[None, None])
    assert np.allclose(r, ref["dv"][0, :, 0], atol=1e-11)
    assert np.allclose(D0, ref["dinitial_states"][0, 0].T, atol=1e-11)


def test_verification_keeps_the_targets_distribution():
    """Over many random numbers the first token is distributed as the target,
    whatever the draft."""
    rng = np.random.default_rng(4)
    V, n = 5, 40000
    p, q = rng.dirichlet(np.ones(V)), rng.dirichlet(np.ones(V))
    target = np.broadcast_to(p, (n, 2, V))
    draft = np.broadcast_to(q, (n, 1, V))
    tokens = rng.choice(V, size=(n, 1), p=q)
    out, _ = od.verify_draft(target, draft, tokens, rng.uniform(size=(n, 1)),
                             rng.exponential(size=(n, V)))
    freq = np.bincount(out[:, 0], minlength=V) / n
    # five standard deviations of a frequency of n draws
    assert np.all(np.abs(freq - p) < 5 * np.sqrt(p * (1 - p) / n))


@pytest.mark.parametrize("form,err", [("int8", 0.5 / 127), ("e4m3", 2.0 ** -4)])
def test_cache_error_is_half_a_step(form, err):
    """int8: half a step of amax/127; e4m3: half an ulp of 2^-3 relative (down
    to its subnormals, 2^-10 of a 448th)."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 3, 4, 33)).astype(np.float32)
    y, scale = od.cache_roundtrip(x, form)
    big = np.abs(x).max(-1, keepdims=True)
    bound = err * big if form == "int8" else np.maximum(err * np.abs(x), big / 448 * 2.0 ** -10)
    assert np.all(np.abs(y - x) <= bound * (1 + 1e-5))
    assert np.allclose(scale, big[..., 0] / (127 if form == "int8" else 448))
