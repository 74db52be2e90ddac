"""The whole chain on a stream of the caller's, forward and backward, and what
lies behind the norm's outputs (GPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import readout as ro

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("named", [True, False])        # the stream as an argument, or current
@pytest.mark.parametrize("rows", [1, 70, 300])
def test_forward_and_backward_on_another_stream(rows, named):
    from mamba_selective_state_gb300 import runner
    g = torch.Generator(device="cuda").manual_seed(rows)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, r, w = rn(rows, 520).to(BF16), rn(rows, 520), 1 + 0.1 * rn(520)
    tok = torch.randint(0, 3001, (rows,), generator=g, device="cuda", dtype=torch.int32)
    norm8 = runner.AddNormDevice(x, w, residual=r, form="int8")
    norm = runner.AddNormDevice(x, w, residual=r, dout=rn(rows, 520).to(BF16), dh=rn(rows, 520))
    lin = runner.Linear8.from_weight(rn(3001, 520) * 0.1, out_dtype=F32)
    logits = torch.empty(rows, 3001, device="cuda")
    lp = runner.LogProbsDevice(logits, tok, ntop=5, dlogprobs=rn(rows), dentropy=rn(rows))
    outs = (norm8.h, norm8.codes.view(torch.uint8), norm8.scales, norm.out, norm.dx, norm.dresidual, norm.dweight,
            logits, lp.logprobs, lp.entropy, lp.lse, lp.stats, lp.top_tokens, lp.top_logprobs, lp.dlogits)

    def go(stream):
        norm8.fwd(stream=stream)
        lin(norm8.codes, norm8.scales, out=logits, stream=stream)
        lp.fwd(stream=stream)
        lp.bwd(stream=stream)
        norm.fwd(stream=stream)
        norm.bwd(stream=stream)
    go(None)
    want = [t.clone() for t in outs]
    for t in outs:
        t.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        wait = rn(4000, 4000)
        for _ in range(5):                              # work that the chain has to stay behind
            wait = wait @ wait
            wait = wait / wait.abs().max()
        x.copy_(x.clone())
        if not named:
            go(None)
    if named:
        go(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("form", [None, "int8", "e4m3"])
@pytest.mark.parametrize("rt", [BF16, F32])
@pytest.mark.parametrize("rows,dim", [(2003, 1), (1500, 7), (1501, 9), (1300, 1237), (1250, 4095), (5, 7), (40, 520)])
def test_norm_writes_its_rows_and_no_more(rows, dim, rt, form):
    """Nothing behind h, the output and the scales is touched; rows with an infinity
    or NaN have the scale NaN, or the formula's values."""
    from mamba_selective_state_gb300 import _lib
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, r, w = rn(rows, dim).to(BF16), rn(rows, dim).to(rt), 1 + 0.3 * rn(dim)
    bad = sorted({rows // 3, rows - 2, rows - 1})
    x[bad[0], dim // 2], r[bad[1], 0], x[bad[2], dim - 1] = math.nan, math.inf, -math.inf

    def room(n, dt):
        """n values and 64 behind them, in bytes of 0x5a."""
        buf = torch.full(((n + 64) * dt.itemsize,), 0x5a, dtype=torch.uint8, device="cuda")
        return buf, buf[n * dt.itemsize:], buf[:n * dt.itemsize].view(dt)
    ot = BF16 if form is None else torch.int8 if form == "int8" else torch.float8_e4m3fn
    h, out, scales = room(rows * dim, rt), room(rows * dim, ot), room(rows, F32)
    kind = {None: _lib.SSD_OUT_PLAIN, "int8": _lib.SSD_OUT_INT8, "e4m3": _lib.SSD_OUT_E4M3}[form]
    prob = _lib.make_add_norm_problem(rows, dim, 1e-5, BF16, rt, kind)
    _lib.ssd_add_rmsnorm_fwd(prob, x, r, w, h[0], out[0], None if form is None else scales[0])
    torch.cuda.synchronize()
    for what in (h, out) + (() if form is None else (scales,)):
        assert bool((what[1] == 0x5a).all())
    hs = h[2].view(rows, dim).double().cpu().numpy()
    want, _ = ro.add_rmsnorm_fwd(hs, w.double().cpu().numpy(), 1e-5)
    if form is None:
        got = out[2].view(rows, dim).double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isnan(got[bad]).any(1).all()
        fine = np.isfinite(want)
        # 48 roundings in fp32 and the output's own
        assert (np.abs(got - want)[fine] <= (48 * 2.0 ** -24 + 2.0 ** -8) * np.abs(want[fine])).all()
    else:
        s = scales[2].cpu().numpy()
        assert np.isnan(s[bad]).all() and np.isnan(s).sum() == len(bad)
        assert not out[2].view(torch.uint8).view(rows, dim)[bad].any()


def test_training_step_captured_and_replayed():
    """Forward and backward of the norm and of the log probabilities in one graph:
    replays with new inputs give the bits of eager calls."""
    from mamba_selective_state_gb300 import runner
    rows, dim, V = 400, 264, 1003
    g = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, r, w, E = rn(rows, dim).to(BF16), rn(rows, dim), 1 + 0.1 * rn(dim), rn(V, dim) * dim ** -0.5
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    dout, logits = torch.empty(rows, dim, dtype=BF16, device="cuda"), torch.empty(rows, V, device="cuda")
    norm = runner.AddNormDevice(x, w, residual=r, dout=dout, dh=rn(rows, dim))
    lp = runner.LogProbsDevice(logits, tok, dlogprobs=rn(rows), dentropy=rn(rows), dlogits=logits)

    def step():
        norm.fwd()
        torch.matmul(norm.out.float(), E.T, out=logits)
        lp.fwd()
        lp.bwd()
        dout.copy_(logits @ E)
        norm.bwd()

    def results():
        return [t.clone() for t in (norm.out, norm.dx, norm.dresidual, norm.dweight, lp.logprobs, lp.entropy, logits)]
    first, second = (rn(rows, dim).to(BF16), rn(rows, dim)), (rn(rows, dim).to(BF16), rn(rows, dim))
    want = []
    for xs, rs in (first, second):
        x.copy_(xs)
        r.copy_(rs)
        step()
        want.append(results())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (0, 1, 0):
        x.copy_((first, second)[i][0])
        r.copy_((first, second)[i][1])
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(want[i], results()))
