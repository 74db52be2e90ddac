"""What the delta-rule, verification and state-cache entry points refuse, and
their buffer sizes (CPU: the calls return before any CUDA call)."""
import ctypes

import pytest
import torch

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from mamba_selective_state_gb300 import build_ext
    build_ext.build()
    from mamba_selective_state_gb300 import _lib
    return _lib


def prob(lib, **kw):
    d = dict(batch=2, seqlen=300, nheads=8, headdim=64, dstate=128, ngroups=2, scale=0.1,
             dtype=lib.SSD_BF16, state_dtype=lib.SSD_F32, flags=0)
    d.update(kw)
    return lib.make_delta_problem(**d)


@pytest.mark.parametrize("bad", [
    dict(batch=0), dict(seqlen=0), dict(nheads=0), dict(headdim=0), dict(dstate=0),
    dict(ngroups=0), dict(ngroups=3), dict(headdim=257), dict(dstate=257), dict(dtype=2),
    dict(state_dtype=9), dict(flags=16), dict(flags=1 << 30), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(q_stride=255), dict(k_stride=-1), dict(v_stride=511),
    dict(batch=1 << 40), dict(seqlen=1 << 40), dict(batch=1 << 20, seqlen=1 << 30),
])
def test_invalid_delta_problems_have_no_buffers(lib, bad):
    p = prob(lib, **bad)
    assert lib.ssd_delta_fwd_workspace_bytes(p) == 0
    assert lib.ssd_delta_bwd_workspace_bytes(p) == 0
    assert lib.ssd_delta_saved_bytes(p) == 0


def test_delta_buffer_sizes(lib):
    for kw in (dict(), dict(dtype=0, headdim=17, dstate=33), dict(seqlen=1), dict(headdim=256, dstate=256),
               dict(q_stride=4096, k_stride=256, v_stride=1 << 20)):
        p = prob(lib, **kw)
        sizes = [lib.ssd_delta_fwd_workspace_bytes(p), lib.ssd_delta_bwd_workspace_bytes(p),
                 lib.ssd_delta_saved_bytes(p)]
        assert all(n > 0 and n % 256 == 0 for n in sizes), kw
        flags = prob(lib, flags=lib.SSD_HAS_INIT | lib.SSD_WANT_DINIT, **kw)
        assert lib.ssd_delta_bwd_workspace_bytes(flags) == sizes[1]
        longer = prob(lib, **dict(kw, seqlen=1000))
        assert lib.ssd_delta_saved_bytes(longer) > sizes[2]


FWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, initial_states=None, seq_idx=None, y=FAKE,
           final_states=FAKE, saved=FAKE, workspace=FAKE)
BWD = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, seq_idx=None, dy=FAKE, dfinal_states=None,
           dq=FAKE, dk=FAKE, dv=FAKE, dg=FAKE, dbeta=FAKE, dinitial_states=None, saved=FAKE,
           workspace=FAKE)


def call(lib, fn, p, base, saved_bytes=1 << 50, workspace_bytes=1 << 50, **over):
    return fn(p, **dict(base, **over), saved_bytes=saved_bytes, workspace_bytes=workspace_bytes,
              stream=0, check=False)


def test_delta_argument_errors(lib):
    bad, small = lib.SSD_ERR_INVALID_ARGUMENT, lib.SSD_ERR_WORKSPACE_TOO_SMALL
    fwd = lambda p=prob(lib), **o: call(lib, lib.ssd_delta_fwd, p, FWD, **o)  # noqa: E731
    bwd = lambda p=prob(lib), **o: call(lib, lib.ssd_delta_bwd, p, BWD, **o)  # noqa: E731
    for n in ("q", "k", "v", "g", "beta", "y", "workspace"):
        assert fwd(**{n: None}) == bad, n
    for n in ("q", "k", "v", "g", "beta", "dy", "dq", "dk", "dv", "dg", "dbeta", "saved", "workspace"):
        assert bwd(**{n: None}) == bad, n
    for n in FWD:
        assert fwd(prob(lib, flags=3), **{"initial_states": FAKE, "seq_idx": FAKE, n: FAKE + 8}) == bad, n
    for n in BWD:
        full = dict(seq_idx=FAKE, dfinal_states=FAKE, dinitial_states=FAKE)
        assert bwd(prob(lib, flags=14), **{**full, n: FAKE + 4}) == bad, n
    assert fwd(initial_states=FAKE) == bad and fwd(seq_idx=FAKE) == bad       # flag missing
    assert fwd(prob(lib, flags=1)) == bad and fwd(prob(lib, flags=2)) == bad  # pointer missing
    assert fwd(prob(lib, flags=4)) == bad and fwd(prob(lib, flags=8)) == bad  # the backward's
    assert bwd(prob(lib, flags=4)) == bad and bwd(dfinal_states=FAKE) == bad
    assert bwd(prob(lib, flags=8)) == bad and bwd(dinitial_states=FAKE) == bad
    assert fwd(workspace_bytes=8) == small and fwd(saved_bytes=8) == small
    assert bwd(workspace_bytes=8) == small and bwd(saved_bytes=8) == small
    assert fwd(prob(lib, headdim=300)) == lib.SSD_ERR_UNSUPPORTED
    assert lib.LIB.ssd_delta_fwd(None, *([None] * 10), 0, None, 0, None) == bad
    assert lib.LIB.ssd_delta_bwd(None, *([None] * 15), 0, None, 0, None) == bad


def test_step_argument_errors(lib):
    bad = lib.SSD_ERR_INVALID_ARGUMENT
    base = dict(q=FAKE, k=FAKE, v=FAKE, g=FAKE, beta=FAKE, nslots=2, states_in=FAKE,
                states_out=FAKE, slots=None, lengths=None, y=FAKE)

    def step(p=prob(lib), **o):
        return lib.ssd_delta_step(p, **dict(base, **o), stream=0, check=False)
    for n in ("q", "k", "v", "g", "beta", "states_in"):
        assert step(**{n: None}) == bad, n
    for n in ("q", "states_in", "states_out", "slots", "lengths", "y"):
        assert step(**{n: FAKE + 4}) == bad, n
    assert step(y=None, states_out=None) == bad             # nothing to do
    assert step(nslots=1) == bad and step(nslots=0, slots=FAKE) == bad
    assert step(prob(lib, state_dtype=1)) == bad and step(prob(lib, flags=1)) == bad
    assert step(nslots=1 << 40, slots=FAKE) == lib.SSD_ERR_UNSUPPORTED
    assert lib.LIB.ssd_delta_step(None, *([None] * 5), 1, *([None] * 5), None) == bad


def test_verify_argument_errors(lib):
    bad = lib.SSD_ERR_INVALID_ARGUMENT
    base = dict(target_probs=FAKE, draft_probs=FAKE, draft_tokens=FAKE, lengths=None,
                uniform=FAKE, noise=FAKE, out_tokens=FAKE, accepted=FAKE)

    def verify(b=2, K=3, V=100, dtype=0, **o):
        return lib.ssd_verify_draft(lib.make_verify_problem(b, K, V, dtype), **dict(base, **o),
                                    stream=0, check=False)
    for n in ("target_probs", "draft_tokens", "uniform", "noise", "out_tokens", "accepted"):
        assert verify(**{n: None}) == bad, n
    for n in base:
        assert verify(**{n: FAKE + 8}) == bad, n
    assert verify(b=0) == bad and verify(K=-1) == bad and verify(V=0) == bad and verify(dtype=3) == bad
    assert verify(V=1 << 31) == lib.SSD_ERR_UNSUPPORTED
    assert verify(b=1 << 20, K=100, V=1 << 20) == lib.SSD_ERR_UNSUPPORTED
    assert lib.LIB.ssd_verify_draft(None, *([None] * 8), None) == bad


def test_cache_argument_errors(lib):
    bad = lib.SSD_ERR_INVALID_ARGUMENT

    def both(b=2, H=4, P=8, N=16, nslots=2, fmt=0, states=FAKE, slots=None, cache=FAKE, scales=FAKE):
        p = lib.make_cache_problem(b, H, P, N, nslots, fmt)
        rcs = {lib.ssd_state_cache_store(p, states, slots, cache, scales, stream=0, check=False),
               lib.ssd_state_cache_load(p, cache, scales, slots, states, stream=0, check=False)}
        assert len(rcs) == 1
        return rcs.pop()
    for n in ("states", "cache", "scales"):
        assert both(**{n: None}) == bad and both(**{n: FAKE + 4}) == bad, n
    assert both(slots=FAKE + 2) == bad
    for n in ("b", "H", "P", "N", "nslots"):
        assert both(**{n: 0}) == bad, n
    assert both(fmt=2) == bad and both(nslots=1) == bad
    assert both(N=257) == lib.SSD_ERR_UNSUPPORTED
    assert both(nslots=1 << 40) == lib.SSD_ERR_UNSUPPORTED
    assert lib.LIB.ssd_state_cache_store(None, *([None] * 4), None) == bad


def test_struct_sizes(lib):
    assert ctypes.sizeof(lib.ssd_delta_problem) == 9 * 8 + 4 * 4
    assert ctypes.sizeof(lib.ssd_verify_problem) == 32
    assert ctypes.sizeof(lib.ssd_cache_problem) == 48


def test_runner_refuses_wrong_tensors(lib):
    from mamba_selective_state_gb300 import runner
    q = torch.zeros(1, 4, 2, 8)
    v, g = torch.zeros(1, 4, 4, 16), torch.zeros(1, 4, 4)
    for bad in (dict(k=torch.zeros(1, 4, 2, 9)), dict(k=q.bfloat16()), dict(g=g[:, :3]),
                dict(v=torch.zeros(1, 4, 4, 16).double()), dict(v=torch.zeros(1, 4, 16, 4).transpose(2, 3)),
                dict(init=torch.zeros(1, 4, 16, 9)), dict(seq=torch.zeros(1, 4)),
                dict(state_dtype=torch.float16), dict(dfinal=torch.zeros(1, 4, 16, 8))):
        a = dict(q=q, k=q, v=v, g=g, beta=g, init=None, seq=None, state_dtype=torch.float32, dfinal=None)
        a.update(bad)
        with pytest.raises(ValueError):
            runner.DeltaDevice(a["q"], a["k"], a["v"], a["g"], a["beta"], initial_states=a["init"],
                               seq_idx=a["seq"], dfinal_states=a["dfinal"],
                               state_dtype=a["state_dtype"])
    with pytest.raises(ValueError):
        runner.DeltaStepDevice(torch.zeros(2, 4, 16))
    with pytest.raises(ValueError):
        runner.DeltaStepDevice(torch.zeros(2, 4, 16, 9)).step(q, q, v, g, g)
    with pytest.raises(ValueError):
        runner.StateCache(2, 4, 16, 8, "int4", device="cpu")
    with pytest.raises(ValueError):
        runner.StateCache(2, 4, 16, 8, device="cpu").store(torch.zeros(1, 4, 16, 9))
    with pytest.raises(ValueError):
        runner.verify_draft(torch.zeros(1, 3, 9), torch.zeros(1, 3, 9), torch.zeros(1, 2, dtype=torch.int32),
                            torch.zeros(1, 2), torch.zeros(1, 9))
