"""Draft verification and the 8-bit state cache against their definitions
(GPU).  Tokens and counts are whole numbers and are equal; the cache's values
come from the same fp32 products and are equal too."""
import numpy as np
import pytest
import torch

from oracle import delta as od

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16


def draft_case(b, K, V, dtype, seed=0, ragged=False):
    rng = np.random.default_rng(seed)
    logits = 2 * rng.standard_normal((b, K + 1, V))
    soft = lambda x: np.exp(x - x.max(-1, keepdims=True))  # noqa: E731
    p = soft(logits)
    q = soft(logits[:, :K] + 0.7 * rng.standard_normal((b, K, V)))
    p, q = p / p.sum(-1, keepdims=True), q / q.sum(-1, keepdims=True)
    tokens = (np.argmax(q / rng.exponential(size=q.shape), -1) if K else
              np.zeros((b, 0))).astype(np.int32)
    t = lambda x, dt: torch.from_numpy(np.ascontiguousarray(x)).to(dt)  # noqa: E731
    return dict(target=t(p, dtype), draft=t(q, dtype), tokens=t(tokens, torch.int32),
                uniform=t(rng.uniform(size=(b, K)), F), noise=t(rng.exponential(size=(b, V)), F),
                lengths=t(rng.integers(0, K + 1, b), torch.int32) if ragged else None)


def verify(c):
    from mamba_selective_state_gb300 import runner
    d = {n: None if t is None else t.cuda() for n, t in c.items()}
    tokens, kept = runner.verify_draft(d["target"], d["draft"], d["tokens"], d["uniform"],
                                       d["noise"], lengths=d["lengths"])
    n = lambda t: None if t is None else t.float().numpy()  # noqa: E731
    want = od.verify_draft(n(c["target"]), n(c["draft"]), c["tokens"].numpy(),
                           n(c["uniform"]), n(c["noise"]),
                           None if c["lengths"] is None else c["lengths"].numpy())
    assert np.array_equal(tokens.cpu().numpy(), want[0])
    assert np.array_equal(kept.cpu().numpy(), want[1])
    return tokens.cpu().numpy(), kept.cpu().numpy()


@pytest.mark.parametrize("b,K,V,dtype", [
    (1, 0, 1, F), (1, 1, 2, F), (3, 4, 300, B), (5, 7, 2049, F), (2, 40, 1000, F),
    (4, 5, 32000, B), (17, 3, 5003, B), (2, 2, 100003, F), (1, 33, 8192, B),
])
@pytest.mark.parametrize("ragged", [False, True])
def test_verification(b, K, V, dtype, ragged):
    verify(draft_case(b, K, V, dtype, seed=V + K, ragged=ragged))


def test_verification_without_draft_probabilities():
    c = draft_case(64, 3, 50, F)
    c["draft"] = None
    c["target"] = torch.softmax(40 * c["target"], -1)
    kept = verify(c)[1]
    assert 0 < kept.sum() < 64 * 3


def test_verification_at_its_limits():
    c = draft_case(12, 2, 4000, F)
    V = 4000
    c["tokens"][0, 0], c["tokens"][1, 1] = -5, V           # no such token: refused
    c["uniform"][2:6] = 0.0                                # all kept
    c["draft"][6, 0], c["target"][6, 0] = 0.0, 0.0         # nothing left: token 0
    c["uniform"][7, 0] = 1.0                               # equal rows refused: falls back to p
    c["draft"][7, 0] = c["target"][7, 0]
    c["target"][8, 0, :] = float("nan")
    c["uniform"][9, 0] = 2.0
    c["noise"][9, ::2] = 0.0                               # infinite ratios tie: the lowest index
    c["noise"][10, 5] = float("nan")
    c["uniform"][11, 0] = 2.0
    c["target"][11, 0, 17] = float("inf")
    c["lengths"] = torch.tensor([2] * 10 + [-3, 99], dtype=torch.int32)
    tokens, kept = verify(c)
    assert kept[0] == 0 and kept[6] == 0 and tokens[6, 0] == 0 and tokens[11, 0] == 17


@pytest.mark.parametrize("noise,weight", [(1e38, 1.0), (3e38, 1.0), (1e-30, 1.0), (1.0, 1e-38),
                                          (1e-3, 1e-44)])
def test_verification_at_extreme_ratios(noise, weight):
    """Divisors and ratios at the ends of the fp32 range: still the largest
    quotient, in the words' order."""
    rng = np.random.default_rng(9)
    b, V = 2, 3000
    t = lambda x: torch.from_numpy(x.astype(np.float32))  # noqa: E731
    verify(dict(target=t(weight * rng.uniform(0.1, 1, (b, 1, V))), draft=torch.zeros(b, 0, V),
                tokens=torch.zeros(b, 0, dtype=torch.int32), uniform=torch.zeros(b, 0),
                noise=t(noise * rng.uniform(0.5, 1, (b, V))), lengths=None))


def test_verification_ties_take_the_lowest_index():
    b, V = 3, 20000
    c = dict(target=torch.full((b, 1, V), 1.0 / V), draft=torch.zeros(b, 0, V),
             tokens=torch.zeros(b, 0, dtype=torch.int32), uniform=torch.zeros(b, 0),
             noise=torch.ones(b, V), lengths=None)
    c["noise"][1, :777] = 2.0
    c["noise"][2, [5000, 19999]] = 0.25
    tokens, _ = verify(c)
    assert tokens[:, 0].tolist() == [0, 777, 5000]


@pytest.mark.parametrize("b,H,P,N,form", [
    (1, 1, 1, 1, "int8"), (2, 3, 5, 7, "e4m3"), (3, 4, 64, 128, "int8"), (2, 2, 16, 130, "int8"),
    (3, 2, 40, 72, "e4m3"), (1, 4, 8, 256, "e4m3"), (2, 5, 33, 57, "int8"), (1, 2, 64, 16, "e4m3"),
    (2, 3, 24, 20, "int8"),
])
def test_cache_roundtrip(b, H, P, N, form):
    from mamba_selective_state_gb300 import runner
    rng = np.random.default_rng(N)
    x = (rng.standard_normal((b, H, P, N)) * np.exp(3 * rng.standard_normal((b, H, P, 1))))
    x = x.astype(np.float32)
    nslots = b + 3
    slots = torch.from_numpy(rng.permutation(nslots)[:b].astype(np.int32)).cuda()
    cache = runner.StateCache(nslots, H, P, N, form)
    cache.values.fill_(3)
    cache.store(torch.from_numpy(x).cuda(), slots)
    out = torch.empty(b, H, P, N, device="cuda")
    cache.load(slots, out)
    want, scale = od.cache_roundtrip(x, form)
    assert np.array_equal(out.cpu().numpy(), want)
    assert np.array_equal(cache.scales[slots.long()].cpu().numpy(), scale)
    rest = np.setdiff1d(np.arange(nslots), slots.cpu().numpy())
    assert bool((cache.values[torch.from_numpy(rest).cuda()] == 3).all())
    assert not cache.scales[torch.from_numpy(rest).cuda()].any()


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("N", [12, 33])
def test_cache_odd_rows(form, N):
    """Zero rows, rows of the least and largest magnitudes, rows with infinite
    values and NaN; ties; padding slots; one slot read twice."""
    from mamba_selective_state_gb300 import runner
    x = np.random.default_rng(1).standard_normal((2, 1, 8, N)).astype(np.float32)
    x[0, 0, 0] = 0.0
    x[0, 0, 1] = 1e-45
    x[0, 0, 2] *= 1e-37
    x[0, 0, 3] *= 1e37
    x[0, 0, 4, 2] = np.inf
    x[0, 0, 5, 3] = np.nan
    x[0, 0, 6] = np.arange(N) + 0.5
    x[0, 0, 6, -1] = 127.0
    x[0, 0, 7] *= 2.0 ** -118
    cache = runner.StateCache(2, 1, 8, N, form)
    cache.store(torch.from_numpy(x).cuda())
    slots = torch.tensor([1, 0, -1, 2, 0], dtype=torch.int32, device="cuda")
    out = torch.full((5, 1, 8, N), 5.0, device="cuda")
    cache.load(slots, out)
    want, _ = od.cache_roundtrip(x, form)
    got = out.cpu().numpy()
    assert np.array_equal(got[[0, 1, 4]], want[[1, 0, 0]], equal_nan=True)
    assert not got[2:4].any()
    cache.store(torch.zeros(2, 1, 8, N, device="cuda"),
                torch.tensor([-1, 2], dtype=torch.int32, device="cuda"))
    cache.load(slots, out)
    assert np.array_equal(out.cpu().numpy(), got, equal_nan=True)
