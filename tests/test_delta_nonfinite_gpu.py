"""Infinities and NaN in the gated delta rule's inputs (GPU): a packed row's
sequences do not meet, whatever they hold and wherever in a chunk they begin.

One token of one sequence is spoilt.  By definition it reaches the outputs of
its own sequence from that token on (q: of that token alone), and the gradients
of v up to it.  Everything else is compared with the oracle's results for the
row with that token as it was; the tolerances are test_delta_gpu's."""
import numpy as np
import pytest
import torch

from tests.test_delta_gpu import TOL, close, device, draw, reference

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16
INF, NAN = float("inf"), float("nan")


def packed(L, H, P, N, G, dtype, starts, seed=0):
    d = draw(1, L, H, P, N, G, dtype, seed=seed, init=True, dfinal=True)
    cuts = np.zeros((1, L), np.int32)
    cuts[0, starts] = 1
    d["seq_idx"] = torch.from_numpy(np.cumsum(cuts, 1).astype(np.int32))
    return d


def spoil(d, name, t, value):
    e = {n: None if x is None else x.clone() for n, x in d.items()}
    e[name][0, t] = value
    return e


def run(d, grad=True):
    dev = device(d, grad=grad)
    dev.fwd()
    if grad:
        dev.bwd()
    assert dev.device_status() == 0
    return {n: x.numpy() for n, x in dev.results().items()}


def check(d, ref, name, t, value, chunk, exact):
    """`exact`: the definition's reach; else every token of the sequence that
    is in the spoilt one's chunk may be reached too."""
    dtype, L = d["v"].dtype, d["v"].shape[1]
    seq = d["seq_idx"][0].numpy()
    got = run(spoil(d, name, t, value))
    at = np.arange(L)
    mine, near = seq == seq[t], at // chunk == t // chunk
    after, before = mine & (at >= t), mine & (at <= t)
    if not exact:
        after, before = mine & ((at >= t) | near), mine & ((at <= t) | near)
    reach = dict(y=after, dv=before)
    if name == "q":
        reach["y"] = mine & near if not exact else at == t
    if name == "v":
        reach["dv"] = at < 0        # dv does not depend on v
    if name == "dy":
        reach["y"] = at < 0
    # the other gradients: within the chunks that hold tokens of the sequence
    around = np.isin(at // chunk, at[mine] // chunk)
    for n in ("dq", "dk", "dg", "dbeta"):
        reach[n] = around
    what = (name, t, value)
    for n, r in reach.items():
        keep = ~r
        if keep.any():
            close(got[n][:, keep], ref[n][:, keep], TOL[dtype], what + (n,))
    if mine.sum() and seq[t] != seq[-1] or name in ("q", "dy"):
        close(got["final_states"], ref["final_states"], TOL[dtype], what + ("final",))
    if seq[t] != seq[0] or name == "v":
        close(got["dinitial_states"], ref["dinitial_states"], TOL[dtype], what + ("dinit",))


STARTS = [1, 31, 33, 63, 65, 100]
VALUES = [("v", INF), ("k", NAN), ("q", INF), ("g", NAN), ("beta", INF), ("dy", INF)]


def both_sides(L, H, P, N, G, dtype, starts, chunk, exact):
    d = packed(L, H, P, N, G, dtype, starts)
    ref = reference(d, N ** -0.5)
    edges = [0] + starts + [L]
    # a token early in each sequence, its last one, and one in the middle of the last sequence
    tokens = {min(lo + 3, hi - 1) for lo, hi in zip(edges, edges[1:])}
    tokens |= {hi - 1 for hi in edges[1:]} | {(starts[-1] + L) // 2}
    for i, t in enumerate(sorted(tokens)):
        for name, value in VALUES:
            check(d, ref, name, t, value if i % 2 else (NAN if value == INF else INF), chunk, exact)


@pytest.mark.parametrize("start", STARTS)
@pytest.mark.parametrize("P,N,dtype", [(16, 16, F), (20, 200, F), (24, 40, B)])
def test_one_start_fp32_kernels(start, P, N, dtype):
    both_sides(190, 2, P, N, 1, dtype, [start], 32, True)


@pytest.mark.parametrize("dtype", [F, B])
def test_many_starts_fp32_kernels(dtype):
    both_sides(150, 4, 40, 56, 2, dtype, [1, 10, 12, 31, 32, 70, 95, 96, 97, 127], 32, True)


@pytest.mark.parametrize("start", STARTS)
@pytest.mark.parametrize("H,P,N", [(2, 64, 64), (1, 128, 128)])
def test_one_start_tensor_cores(start, H, P, N):
    both_sides(250, H, P, N, 1, B, [start], 64, False)


# 16, 32 and 64 columns a CTA, whole chains and pieces of them
@pytest.mark.parametrize("L,H,N,starts", [
    (200, 2, 128, [1, 10, 12, 63, 64, 70, 127, 128, 129]), (200, 44, 64, [5, 70, 71, 192]),
    (150, 80, 64, [33, 100]), (150, 77, 128, [60, 130]), (600, 2, 64, [100, 130, 320, 321, 590]),
    (520, 44, 128, [250, 300]),
])
def test_many_starts_tensor_cores(L, H, N, starts):
    both_sides(L, H, 64, N, 1, B, starts, 64, False)


@pytest.mark.parametrize("P,N,dtype,chunk", [(16, 16, F, 32), (64, 64, B, 64)])
def test_forgotten_states(P, N, dtype, chunk):
    """A decay of -inf, or below -100, forgets an infinite state as a sequence's
    start does, inside a chunk and at its first token."""
    for t in (0, 5, 64, 77):
        for g in (-INF, -101.0):
            d = draw(1, 130, 2, P, N, 1, dtype, init=True)
            d["g"][0, t] = g
            if t == 0:
                e = {**d, "init": torch.full_like(d["init"], NAN)}
            else:
                e = spoil(d, "v", t - 1, INF)
            ref = reference(d, N ** -0.5, grad=False)
            got = run(e, grad=False)
            close(got["y"][:, t:], ref["y"][:, t:], TOL[dtype], (t, g))
            close(got["final_states"], ref["final_states"], TOL[dtype], (t, g))


@pytest.mark.parametrize("P,N,dtype,chunk", [(16, 16, F, 32), (64, 128, B, 64)])
def test_a_state_that_is_not_finite_ends_with_its_sequence(P, N, dtype, chunk):
    for start in STARTS:
        d = packed(200, 2, P, N, 1, dtype, [start])
        ref = reference(d, N ** -0.5)
        e = {**d, "init": d["init"].clone()}
        e["init"][0, :, 0, 0] = NAN
        got = run(e)
        rest = slice(start, None)
        close(got["y"][:, rest], ref["y"][:, rest], TOL[dtype], start)
        close(got["final_states"], ref["final_states"], TOL[dtype], start)
        close(got["dv"], ref["dv"], TOL[dtype], start)
        behind = slice(-(-start // chunk) * chunk, None)
        for n in ("dq", "dk", "dg", "dbeta"):
            close(got[n][:, behind], ref[n][:, behind], TOL[dtype], (start, n))
        # and a gradient of the last state that is not
        e = {**d, "dfinal": d["dfinal"].clone()}
        e["dfinal"][0, :, 1] = INF
        got = run(e)
        first = slice(0, start)
        close(got["dv"][:, first], ref["dv"][:, first], TOL[dtype], start)
        close(got["dinitial_states"], ref["dinitial_states"], TOL[dtype], start)
