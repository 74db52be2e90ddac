"""The gated delta rule's kernels against the float64 oracle (GPU): forward,
gradient, recurrent step; head layouts, odd sizes, packed rows, strides,
states of both types, decays that forget.

Tolerances, on the 2-norm of the difference over the 2-norm of the result.
fp32: a value passes through sums of up to 256 terms and a chain of states
whose error decays with them: about sqrt(256) roundings of 2^-24, 1e-6; a
token's gradient sums three such chains; 2e-5 leaves a factor of six.  bf16:
the result's own rounding is 2^-9 / sqrt(3) = 1.1e-3 and at most five rounded
operands of that size stand between it and the inputs, 2.8e-3 in quadrature;
1e-2 leaves a factor of three.  Single elements: 20 times as much of the
largest value."""
import numpy as np
import pytest
import torch

from oracle import delta as od

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2e-5, torch.bfloat16: 1e-2}


def draw(b, L, H, P, N, G, dtype, seed=0, nseq=1, init=False, state_dtype=None, dfinal=False):
    rng = np.random.default_rng(seed)
    n = rng.standard_normal

    def unit(x):
        x = x / (1 + np.exp(-x))
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    t = lambda x, dt=dtype: torch.from_numpy(np.ascontiguousarray(x)).to(dt)  # noqa: E731
    d = dict(q=t(unit(n((b, L, G, N)))), k=t(unit(n((b, L, G, N)))), v=t(n((b, L, H, P))),
             g=t(-np.exp(rng.uniform(np.log(1e-3), np.log(2.0), (b, L, H)))),
             beta=t(1 / (1 + np.exp(-n((b, L, H))))), dy=t(n((b, L, H, P))),
             seq_idx=None, init=None, dfinal=None)
    st = state_dtype or dtype
    if init:
        d["init"] = t(0.3 * n((b, H, P, N)), st)
    if dfinal:
        d["dfinal"] = t(n((b, H, P, N)), st)
    if nseq > 1:
        cuts = np.zeros((b, L), np.int32)
        for i in range(b):
            cuts[i, 1 + rng.choice(L - 1, nseq - 1, replace=False)] = 1
        d["seq_idx"] = torch.from_numpy(np.cumsum(cuts, 1).astype(np.int32))
    return d


def f64(t):
    return None if t is None else t.double().numpy()


def reference(d, scale, grad=True):
    a = [f64(d[x]) for x in ("q", "k", "v", "g", "beta")]
    seq = None if d["seq_idx"] is None else d["seq_idx"].numpy()
    y, fin = od.delta_fwd(*a, scale, f64(d["init"]), seq)
    out = dict(y=y, final_states=fin)
    if grad:
        out.update(od.delta_bwd(*a, scale, f64(d["dy"]), f64(d["init"]), seq, f64(d["dfinal"])))
        if d["init"] is None:
            del out["dinitial_states"]
    return out


def close(got, ref, tol, what=""):
    got, norm = np.asarray(got, np.float64), np.linalg.norm(ref)
    assert np.isfinite(got).all(), what
    if norm == 0:
        assert not got.any(), what
        return
    off = np.linalg.norm(got - ref) / norm
    assert off <= tol, (what, off)
    assert np.abs(got - ref).max() <= 20 * tol * np.abs(ref).max(), what


def device(d, scale=None, state_dtype=None, grad=True, **over):
    from mamba_selective_state_gb300 import runner
    c = {n: None if t is None else t.cuda() for n, t in d.items()}
    c.update(over)
    return runner.DeltaDevice(c["q"], c["k"], c["v"], c["g"], c["beta"], scale,
                              initial_states=c["init"], seq_idx=c["seq_idx"],
                              dy=c["dy"] if grad else None,
                              dfinal_states=c["dfinal"] if grad else None,
                              state_dtype=state_dtype or d["v"].dtype)


def check(d, scale=None, state_dtype=None, grad=True, **over):
    dev = device(d, scale, state_dtype, grad, **over)
    dev.fwd()
    if grad:
        dev.bwd()
    assert dev.device_status() == 0
    got = dev.results()
    ref = reference(d, scale or d["q"].shape[-1] ** -0.5, grad)
    tol = TOL[d["v"].dtype]
    assert set(got) == set(ref)
    for n in ref:
        close(got[n].numpy(), ref[n], tol, n)
    return dev


F, B = torch.float32, torch.bfloat16


@pytest.mark.parametrize("b,L,H,P,N,G,dtype,nseq,init,dfinal", [
    (1, 1, 1, 1, 1, 1, F, 1, False, False),         # the least problem
    (1, 1, 2, 8, 16, 1, F, 1, True, True),
    (2, 33, 4, 16, 16, 2, F, 1, True, True),        # one token past a chunk
    (1, 64, 3, 5, 7, 3, F, 1, False, True),         # odd heads, whole chunks
    (2, 77, 6, 40, 56, 3, F, 3, True, True),
    (1, 95, 2, 17, 129, 1, F, 4, True, False),      # just past a register class
    (1, 50, 2, 256, 256, 2, F, 1, True, True),      # the largest heads
    (1, 130, 8, 64, 128, 1, F, 5, True, True),      # eight heads share q and k
    (2, 70, 4, 24, 40, 2, B, 3, True, True),        # bf16 outside the tensor-core set
    (1, 1, 4, 64, 128, 2, B, 1, False, False),      # bf16 inside it
    (1, 1, 4, 64, 64, 2, B, 1, True, True),
    (2, 63, 4, 64, 128, 1, B, 1, True, True),
    (1, 64, 4, 64, 128, 4, B, 1, True, True),
    (2, 65, 8, 64, 64, 1, B, 1, False, True),
    (1, 200, 16, 64, 128, 2, B, 7, True, True),     # packed, heads share
    (1, 333, 3, 32, 64, 3, B, 5, False, False),
    (2, 190, 6, 128, 128, 3, B, 3, True, True),     # wide values
    (1, 150, 2, 96, 64, 1, B, 2, True, True),
    (1, 321, 24, 64, 128, 2, B, 1, True, True),     # twelve heads share
    (1, 129, 40, 64, 64, 1, B, 1, False, True),     # forty
    (1, 100, 2, 256, 128, 1, B, 2, True, False),    # the widest values
    (3, 70, 30, 128, 64, 30, B, 1, True, True),     # enough chains for 64 columns a CTA
    (20, 66, 8, 64, 128, 4, B, 1, True, True),
])
def test_forward_and_gradient(b, L, H, P, N, G, dtype, nseq, init, dfinal):
    check(draw(b, L, H, P, N, G, dtype, seed=L, nseq=nseq, init=init, dfinal=dfinal))


@pytest.mark.parametrize("L,H,P,N,starts", [
    (700, 2, 64, 64, []),                             # packed in name only
    (700, 2, 64, 128, [1]),
    (700, 2, 64, 64, [64, 128, 320, 448, 576]),       # sequences of whole chunks
    (1301, 2, 64, 128, [63, 65, 640, 641, 1299]),     # starts at both ends of a chunk
    (1301, 1, 128, 64, [650, 655, 660, 700, 1024]),   # several in a chunk
    (1301, 2, 64, 64, [1281]),                        # in the last chunk alone
    (1301, 2, 64, 64, list(range(1, 1301))),          # sequences of one token
    (513, 40, 64, 64, [255, 256, 257, 512]),          # 64 columns a CTA
])
def test_packed_chains_in_pieces(L, H, P, N, starts):
    d = draw(1, L, H, P, N, 1, B, seed=L + len(starts), init=True, dfinal=True)
    cuts = np.zeros((1, L), np.int32)
    cuts[0, starts] = 1
    d["seq_idx"] = torch.from_numpy(np.cumsum(cuts, 1).astype(np.int32))
    check(d)


@pytest.mark.parametrize("dtype,N", [(F, 48), (B, 128)])
def test_forward_alone_matches(dtype, N):
    d = draw(2, 140, 4, 64, N, 2, dtype, init=True)
    a, b = check(d, grad=False), check(d)
    assert torch.equal(a.y, b.y) and torch.equal(a.final, b.final)


@pytest.mark.parametrize("dtype,P,N", [(F, 20, 24), (B, 64, 64)])
def test_column_blocks_of_one_projection(dtype, P, N):
    """q, k and v as strided views of one tensor."""
    b, L, H, G = 2, 90, 4, 2
    d = draw(b, L, H, P, N, G, dtype, init=True, dfinal=True)
    wide = torch.zeros(b, L, 2 * G * N + H * P + 64, dtype=dtype, device="cuda")
    at, views = 0, {}
    for name, heads, width in (("q", G, N), ("k", G, N), ("v", H, P)):
        w = wide[..., at:at + heads * width]
        w.copy_(d[name].reshape(b, L, -1))
        views[name] = w.view(b, L, heads, width)
        at += heads * width
    assert not views["v"].is_contiguous()
    check(d, **views)


@pytest.mark.parametrize("dtype,P,N", [(F, 20, 24), (B, 64, 128)])
@pytest.mark.parametrize("state_dtype", [F, B])
def test_state_types(dtype, P, N, state_dtype):
    d = draw(1, 100, 4, P, N, 2, dtype, init=True, dfinal=True, state_dtype=state_dtype)
    dev = device(d, state_dtype=state_dtype)
    dev.fwd()
    dev.bwd()
    got, ref = dev.results(), reference(d, N ** -0.5)
    for n in ref:
        # a state that leaves in bf16 is rounded to it
        close(got[n].numpy(), ref[n], TOL[B if state_dtype == B and "states" in n else dtype], n)


@pytest.mark.parametrize("dtype,P,N", [(F, 16, 16), (B, 64, 64)])
def test_decays_at_their_limits(dtype, P, N):
    """-inf and huge negative decays forget the state and have no gradient;
    0 keeps it; strengths of 0, 1 and 2 write nothing, all and twice."""
    d = draw(1, 150, 4, P, N, 2, dtype, init=True, dfinal=True)
    d["g"][0, 10], d["g"][0, 64], d["g"][0, 100] = -float("inf"), -3e38, -1000.0
    d["g"][0, 70:80] = 0.0
    d["beta"][0, 20:25], d["beta"][0, 30:33], d["beta"][0, 40] = 0.0, 1.0, 2.0
    dev = check(d)
    for t in (10, 64, 100):
        assert not dev.dg[0, t].any()


def test_sequence_start_hides_what_came_before():
    """Infinite values in one sequence of a packed row stay in it."""
    for dtype, P, N in ((F, 16, 16), (B, 64, 64)):
        d = draw(1, 130, 2, P, N, 1, dtype)
        d["seq_idx"] = torch.zeros(1, 130, dtype=torch.int32)
        d["seq_idx"][0, 64:] = 1
        ref = reference(d, N ** -0.5, grad=False)
        d["v"][0, 3] = float("inf")
        dev = device(d, grad=False)
        dev.fwd()
        close(dev.y[0, 64:].double().cpu().numpy(), ref["y"][0, 64:], TOL[dtype], "y")
        close(dev.final.double().cpu().numpy(), ref["final_states"], TOL[dtype], "final")


def test_results_are_reproducible():
    d = draw(2, 200, 8, 64, 128, 2, B, init=True, dfinal=True, nseq=3)
    runs = []
    for _ in range(2):
        dev = device(d)
        dev.fwd()
        dev.bwd()
        runs.append(dev.results())
    for n in runs[0]:
        assert torch.equal(runs[0][n], runs[1][n]), n


def test_other_stream():
    d = draw(1, 130, 4, 64, 64, 2, B, init=True)
    s = torch.cuda.Stream()
    dev = device(d)
    s.wait_stream(torch.cuda.current_stream())
    dev.fwd(stream=s)
    dev.bwd(stream=s)
    s.synchronize()
    got, ref = dev.results(), reference(d, 64 ** -0.5)
    for n in ref:
        close(got[n].numpy(), ref[n], TOL[B], n)


def test_gradient_matches_differences():
    """fp32, along a random direction of every input: central differences of
    the kernel's own loss, in 64 bits from its fp32 outputs.  Steps of 1e-2 of
    unit directions: truncation ~1e-4, rounding ~1e-6 / 1e-2."""
    d = draw(1, 70, 4, 24, 40, 2, F, init=True, dfinal=True, nseq=2)
    dev = device(d)
    dev.fwd()
    dev.bwd()
    rng = np.random.default_rng(7)
    grads = dict(q=dev.dq, k=dev.dk, v=dev.dv, g=dev.dg, beta=dev.dbeta, init=dev.dinit)

    def loss(e):
        x = device(e)
        x.fwd()
        return float((x.y.double() * x.dy.double()).sum()
                     + (x.final.double() * x.dfinal.double()).sum())
    for name, grad in grads.items():
        u = rng.standard_normal(d[name].shape)
        u = torch.from_numpy((u / np.linalg.norm(u)).astype(np.float32))
        want = float((grad.double().cpu() * u.double()).sum())
        sides = []
        for h in (1e-2, -1e-2):
            e = {n: None if t is None else t.clone() for n, t in d.items()}
            e[name] += h * u
            sides.append(loss(e))
        num = (sides[0] - sides[1]) / 2e-2
        assert abs(num - want) <= 2e-3 * max(1.0, float(grad.double().norm())), name


# ---- the recurrent step ---------------------------------------------------
@pytest.mark.parametrize("b,T,H,P,N,G,dtype", [
    (1, 1, 1, 1, 1, 1, F), (3, 1, 4, 64, 128, 2, B), (2, 5, 6, 40, 57, 3, F),
    (4, 8, 4, 64, 16, 1, B), (1, 20, 2, 128, 256, 2, F), (5, 17, 2, 33, 64, 1, B),
])
@pytest.mark.parametrize("ragged", [False, True])
def test_step(b, T, H, P, N, G, dtype, ragged):
    from mamba_selective_state_gb300 import runner
    d = draw(b, T, H, P, N, G, dtype, seed=b + T, init=True, state_dtype=F)
    rng = np.random.default_rng(3)
    nslots = b + 2
    slots = rng.permutation(nslots)[:b].astype(np.int32)
    pool = torch.from_numpy(rng.standard_normal((nslots, H, P, N)).astype(np.float32))
    pool[torch.from_numpy(slots).long()] = d["init"]
    lengths = rng.integers(0, T + 1, b).astype(np.int32) if ragged else None
    x = {n: d[n].cuda() for n in ("q", "k", "v", "g", "beta")}
    sl = torch.from_numpy(slots).cuda()
    le = None if lengths is None else torch.from_numpy(lengths).cuda()
    want, y = pool.double().numpy().copy(), None
    args = [f64(d[n]) for n in ("q", "k", "v", "g", "beta")]
    y, fin, path = od.delta_fwd(*args, N ** -0.5, f64(d["init"]), states=True)
    path.append(fin)
    for i in range(b):
        want[slots[i]] = path[T if lengths is None else lengths[i]][i]
    out = torch.full_like(pool, 7.0).cuda()
    dev = runner.DeltaStepDevice(pool.cuda(), out)
    got = dev.step(*x.values(), slots=sl, lengths=le)
    close(got.double().cpu().numpy(), y, TOL[dtype], "y")
    close(out[sl.long()].double().cpu().numpy(), want[slots], TOL[F], "states")
    rest = np.setdiff1d(np.arange(nslots), slots)
    assert bool((out[torch.from_numpy(rest).cuda()] == 7.0).all())      # nothing else is written
    place = runner.DeltaStepDevice(pool.cuda())                          # in place
    assert place.step(*x.values(), slots=sl, lengths=le, outputs=False) is None
    assert torch.equal(place.states[sl.long()], out[sl.long()])
    same = runner.DeltaStepDevice(pool.cuda())                           # no update
    assert torch.equal(same.step(*x.values(), slots=sl, lengths=le, update=False), got)
    assert torch.equal(same.states.cpu(), pool)


def test_step_padding_and_shared_slots():
    from mamba_selective_state_gb300 import runner
    d = draw(4, 3, 2, 16, 32, 1, B, init=True, state_dtype=F)
    x = [d[n].cuda() for n in ("q", "k", "v", "g", "beta")]
    pool = d["init"].cuda()
    dev = runner.DeltaStepDevice(pool.clone())
    # -1 and 9 are padding; two sequences read slot 2 (nothing is written)
    slots = torch.tensor([2, -1, 9, 2], dtype=torch.int32, device="cuda")
    y = dev.step(*x, slots=slots, update=False)
    assert not y[1].any() and not y[2].any()
    ref, _ = od.delta_fwd(*[f64(t.cpu())[[0, 3]] for t in x], 32 ** -0.5,
                          f64(d["init"])[[2, 2]])
    close(y[[0, 3]].double().cpu().numpy(), ref, TOL[B], "y")
    dev.step(*x, slots=torch.tensor([-1, 4, -1, 2 ** 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(dev.states, pool)


def test_step_continues_the_chunked_forward():
    d = draw(2, 101, 4, 64, 64, 2, B, init=True, state_dtype=F)
    from mamba_selective_state_gb300 import runner
    x = {n: d[n].cuda() for n in ("q", "k", "v", "g", "beta")}
    head = [t[:, :96].contiguous() for t in x.values()]
    tail = [t[:, 96:].contiguous() for t in x.values()]
    pre = runner.DeltaDevice(*head, initial_states=d["init"].cuda())
    pre.fwd()
    y = runner.DeltaStepDevice(pre.final).step(*tail)
    ref = reference(d, 64 ** -0.5, grad=False)
    close(y.double().cpu().numpy(), ref["y"][:, 96:], TOL[B], "y")
    close(pre.final.double().cpu().numpy(), ref["final_states"], TOL[B], "states")
