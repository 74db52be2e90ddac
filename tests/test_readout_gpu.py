"""The norm with residual, the 8-bit product and the log probabilities against
the float64 oracle (GPU).  The tolerances count roundings: U is half a step of
fp32 relative to the value, HALF of the outputs' type."""
import math

import numpy as np
import pytest
import torch

from oracle import readout as ro

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def close(got, want, tol, what=""):
    """|got - want| <= tol where want is finite, the same elsewhere."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    want = np.asarray(want, np.float64)
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    with np.errstate(invalid="ignore"):
        over = np.abs(got - want)[fine] - np.broadcast_to(tol, want.shape)[fine]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()))


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rn(g, *s):
    return torch.randn(s, generator=g, device="cuda")


# ------------------------------------------------------------------- the norm
# A row's sum of squares: a thread's products one after the other (at most 32 of
# them), then 5 + 16 additions; mean, eps, the root (2 units) and two products.
# The root halves the relative error: under 48 roundings in all.
NORM = 48 * U


def norm_case(rows, dim, dt, rt, seed, resid=True, spread=1.0, stride=None):
    g = gen(seed)
    x = (rn(g, rows, stride or dim) * spread).to(dt)[:, :dim]
    r = (2 * rn(g, rows, dim) * spread).to(rt) if resid else None
    return x, r, 1 + 0.3 * rn(g, dim)


def stored(x, r):
    return x if r is None else (x.float() + r.float()).to(r.dtype)


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (2, 33), (7, 256), (2, 1237), (700, 520), (400, 2048), (3, 4104),
          (1, 8192), (2, 16384), (310, 16383), (320, 12000)]
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm_forward(rows, dim, dt, rt):
    from mamba_selective_state_gb300 import runner
    x, r, w = norm_case(rows, dim, dt, rt, rows + dim)
    dev = runner.AddNormDevice(x, w, residual=r, eps=1e-5)
    dev.fwd()
    want_h = stored(x.cpu(), r.cpu())
    assert torch.equal(dev.h.cpu(), want_h)
    want, _ = ro.add_rmsnorm_fwd(f64(want_h), f64(w), 1e-5)
    close(dev.out, want, (NORM + HALF[dt]) * np.abs(want))


@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm_codes(rows, dim, dt, rt, form):
    from mamba_selective_state_gb300 import runner
    x, r, w = norm_case(rows, dim, dt, rt, rows * 3 + dim)
    dev = runner.AddNormDevice(x, w, residual=r, eps=1e-6, form=form)
    dev.fwd()
    out, _ = ro.add_rmsnorm_fwd(f64(stored(x, r)), f64(w), 1e-6)
    scales = np.abs(out).max(-1) / ro.TOP[form]
    close(dev.scales, scales, (NORM + 2 * U) * scales)
    # off by half a step, and by the errors of the value and of the factor
    y = out / scales[:, None]
    close(ro.code_values(raw(dev.codes), form), y, ro.half_steps(y, form) + (2 * NORM + 4 * U) * np.abs(y))


def test_norm_without_residual_and_strided():
    from mamba_selective_state_gb300 import runner
    for stride, dim in ((200, 96), (97, 96), (4096, 1000)):     # whole vectors, odd rows, columns
        x, _, w = norm_case(9, dim, BF16, BF16, stride, resid=False, stride=stride)
        dev = runner.AddNormDevice(x, w)
        dev.fwd()
        assert dev.h is x
        want, _ = ro.add_rmsnorm_fwd(f64(x), f64(w), 1e-5)
        close(dev.out, want, (NORM + HALF[BF16]) * np.abs(want))


# Many rows whose ends are not those of 16-byte vectors: each row but the first
# begins inside a vector that holds other rows' values too.
@pytest.mark.parametrize("form", [None, "int8", "e4m3"])
@pytest.mark.parametrize("rt", [BF16, F32])
@pytest.mark.parametrize("rows,dim", [(2003, 1), (2001, 3), (1500, 7), (1501, 9), (1237, 100), (1300, 1237), (1250, 4095),
                                      (1221, 16367), (1221, 16371)])
def test_norm_many_odd_rows(rows, dim, rt, form):
    from mamba_selective_state_gb300 import runner
    x, r, w = norm_case(rows, dim, BF16, rt, rows * 5 + dim)
    x[11, dim // 2], r[rows - 3, 0], x[rows - 1, dim - 1] = float("nan"), float("inf"), float("-inf")
    room = rows * dim                                # the stream in place, with room behind it that stays as it was
    buf = torch.full((room + 64,), 3.0, dtype=rt, device="cuda")
    buf[:room] = r.flatten()
    inplace = buf[:room].view(rows, dim)
    dev = runner.AddNormDevice(x, w, residual=inplace, h_out=inplace, form=form)
    want_h = stored(x.cpu(), r.cpu())
    fine = torch.ones(rows, dtype=torch.bool)
    fine[[11, rows - 3, rows - 1]] = False
    dev.fwd()
    torch.testing.assert_close(dev.h.cpu(), want_h, rtol=0, atol=0, equal_nan=True)
    assert bool((buf[room:] == 3).all())
    want, _ = ro.add_rmsnorm_fwd(f64(want_h[fine]), f64(w), 1e-5)
    if form is None:
        close(dev.out.cpu()[fine], want, (NORM + HALF[BF16]) * np.abs(want))
        return
    scales = np.abs(want).max(-1) / ro.TOP[form]
    got = dev.scales.cpu()
    close(got[fine], scales, (NORM + 2 * U) * scales)
    assert bool(got[11].isnan()) and bool(got[rows - 1].isnan())
    y = want / np.where(scales > 0, scales, 1)[:, None]
    codes = ro.code_values(raw(dev.codes), form)[fine.numpy()]
    close(codes, y, ro.half_steps(y, form) + (2 * NORM + 4 * U) * np.abs(y))


def test_norm_updates_the_residual_in_place():
    from mamba_selective_state_gb300 import runner
    x, r, w = norm_case(500, 1024, BF16, F32, 5)
    want = stored(x, r)
    dev = runner.AddNormDevice(x, w, residual=r, h_out=r, form="int8")
    dev.fwd()
    assert torch.equal(r, want) and dev.h is r


@pytest.mark.parametrize("form", ["int8", "e4m3"])
def test_norm_rows_of_nothing_and_not_finite(form):
    from mamba_selective_state_gb300 import runner
    x, r, w = norm_case(6, 300, F32, F32, 8)
    x[0] = r[0] = 0
    x[1, 5] = math.inf
    x[2, 299] = math.nan
    x[3] = r[3] = 1e-40
    x[4, 7], r[4, 7] = math.inf, -math.inf
    dev = runner.AddNormDevice(x, w, residual=r, form=form, eps=1e-5)
    dev.fwd()
    s, c = f64(dev.scales), ro.code_values(raw(dev.codes), form)
    assert s[0] == 0 and not c[0].any()
    assert s[3] == 0 and not c[3].any()         # 1e-40 / sqrt(eps) is below 2^-118
    assert np.isnan(s[[1, 2, 4]]).all() and np.isfinite(s[5]) and np.isfinite(c).all()
    want, _ = ro.add_rmsnorm_fwd(f64(x[5:] + r[5:]), f64(w), 1e-5)
    assert np.abs(c[5] * s[5] - want[0]).max() <= np.abs(want).max() * (0.5 / 127 if form == "int8" else 2.0 ** -4)


@pytest.mark.parametrize("dt,rt", TYPES)
@pytest.mark.parametrize("rows,dim", SHAPES + [(2500, 64)])
@pytest.mark.parametrize("with_dh", [True, False])
def test_norm_backward(rows, dim, dt, rt, with_dh):
    from mamba_selective_state_gb300 import runner
    g = gen(rows + 7 * dim)
    x, r, w = norm_case(rows, dim, dt, rt, rows + 7 * dim)
    dout, dh = rn(g, rows, dim).to(dt), rn(g, rows, dim).to(rt) if with_dh else None
    dev = runner.AddNormDevice(x, w, residual=r, eps=1e-3, dout=dout, dh=dh)
    dev.fwd()
    dev.bwd()
    h = f64(stored(x, r))
    d, dw = ro.add_rmsnorm_bwd(h, f64(w), 1e-3, f64(dout), None if dh is None else f64(dh))
    _, rstd = ro.add_rmsnorm_fwd(h, f64(w), 1e-3)
    n, gg = h * rstd, f64(dout) * f64(w)
    # each term's size times the roundings of the root, of the mean of g n and of its own products
    size = rstd * (np.abs(gg) + np.abs(n) * np.abs(gg * n).mean(-1, keepdims=True))
    size = size + (0 if dh is None else np.abs(f64(dh)))
    close(dev.dx, d, 2 * NORM * size + HALF[dt] * np.abs(d), "dx")
    close(dev.dresidual, d, 2 * NORM * size + HALF[rt] * np.abs(d), "dresidual")
    assert (dev.dresidual is dev.dx) == (dt is rt)
    # a column's sum: at most 2500 / 152 rows to a CTA, 1216 / 16 slices to a warp, 16 warps
    close(dev.dweight, dw, (NORM + 112 * U) * np.abs(f64(dout) * n).sum(0), "dweight")


def test_norm_backward_without_residual():
    from mamba_selective_state_gb300 import runner
    x, _, w = norm_case(40, 513, F32, F32, 3, resid=False)
    dout = rn(gen(4), 40, 513)
    dev = runner.AddNormDevice(x, w, dout=dout)
    dev.fwd()
    dev.bwd()
    d, dw = ro.add_rmsnorm_bwd(f64(x), f64(w), 1e-5, f64(dout))
    assert dev.dresidual is None
    assert np.abs(f64(dev.dx) - d).max() < 1e-5 * np.abs(d).max()
    assert np.abs(f64(dev.dweight) - dw).max() < 1e-5 * np.abs(dw).max()


def test_norm_gradient_by_differences():
    """The kernels' own gradient against differences of the kernels' own output
    (fp32, a step of 2^-6: the outputs' rounding weighs 2^-24 / 2^-6)."""
    from mamba_selective_state_gb300 import runner
    rows, dim, eps = 3, 24, 0.1
    x, r, w = norm_case(rows, dim, F32, F32, 9)
    dout, dh = rn(gen(1), rows, dim), rn(gen(2), rows, dim)
    dev = runner.AddNormDevice(x, w, residual=r, eps=eps, dout=dout, dh=dh)
    dev.fwd()
    dev.bwd()
    dx = f64(dev.dx)

    def loss():
        dev.fwd()
        return (f64(dev.out) * f64(dout)).sum() + (f64(dev.h) * f64(dh)).sum()
    for i, j in ((0, 0), (1, 11), (2, 23)):
        x0, est = float(x[i, j]), []
        for s in (2.0 ** -6, 2.0 ** -5):
            x[i, j] = x0 + s
            up = loss()
            x[i, j] = x0 - s
            est.append((up - loss()) / (2 * s))
            x[i, j] = x0
        # Richardson: the error of the steps goes with the fourth power
        assert abs((4 * est[0] - est[1]) / 3 - dx[i, j]) < 2e-3 * np.abs(dx).max()


def test_norm_reproducible():
    from mamba_selective_state_gb300 import runner
    x, r, w = norm_case(3000, 1000, BF16, F32, 3)
    dout = rn(gen(3), 3000, 1000).to(BF16)
    dev = runner.AddNormDevice(x, w, residual=r, dout=dout)
    got = []
    for _ in range(2):
        dev.fwd()
        dev.bwd()
        got.append([t.clone() for t in (dev.out, dev.dx, dev.dresidual, dev.dweight)])
    assert all(torch.equal(a, b) for a, b in zip(*got))


# ---------------------------------------------------------------- the product
def some_codes(g, rows, k, form):
    if form == "int8":      # |code| <= 60: 4096 products stay below 2^24 in sum
        return torch.randint(-60, 61, (rows, k), generator=g, device="cuda").to(torch.int8)
    return (rn(g, rows, k) * 40).clamp(-448, 448).to(torch.float8_e4m3fn)


def values(t):
    return ro.code_values(raw(t), "int8" if t.dtype is torch.int8 else "e4m3")


MATS = [(1, 1, 1), (1, 10304, 4096), (1, 17, 100), (2, 5, 3), (3, 300, 64), (4, 1000, 1000), (7, 130, 4096),
        (8, 64, 16), (9, 64, 48), (16, 777, 80), (17, 129, 272), (31, 100, 1040), (33, 2048, 512), (61, 515, 4096),
        (64, 256, 128), (65, 256, 128), (100, 1, 64), (128, 100, 192), (129, 257, 63), (200, 640, 2048),
        (255, 33, 4096), (257, 513, 129), (300, 1000, 1000), (520, 776, 384), (1000, 4100, 256), (2049, 300, 64), (40, 50, 1),
        (3000, 40, 1), (9000, 1030, 3)]


def check_product(a, sa, w, sw, bias, out, out_dtype):
    av, wv = values(a), values(w)
    want = ro.scaled_matmul(av, f64(sa), wv, f64(sw), None if bias is None else f64(bias))
    prod = (np.abs(av) @ np.abs(wv).T) * np.abs(f64(sa))[:, None] * np.abs(f64(sw))
    k = a.shape[1]
    # int8: the sums are exact, three roundings follow; e4m3: sums of 16 products
    # with a rounding each (to zero at worst: 2 U), and their joins
    err = 0.0 if a.dtype is torch.int8 else (k / 16 + 16) * 2 * U
    size = np.abs(want) + (0 if bias is None else 2 * np.abs(f64(bias)))
    close(out, want, err * prod + 3 * U * size + HALF[out_dtype] * np.abs(want))


@pytest.mark.parametrize("out_dtype", [BF16, F32])
@pytest.mark.parametrize("form", ["int8", "e4m3"])
@pytest.mark.parametrize("m,n,k", MATS)
def test_product(m, n, k, form, out_dtype):
    from mamba_selective_state_gb300 import runner
    g = gen(m * 7 + n + k)
    a, w = some_codes(g, m, k, form), some_codes(g, n, k, form)
    sa, sw = torch.rand(m, generator=g, device="cuda") + 0.1, torch.rand(n, generator=g, device="cuda") + 0.1
    bias = rn(g, n) * 100 if (m + n) % 2 else None
    lin = runner.Linear8(w, sw, bias=bias, out_dtype=out_dtype)
    out = torch.full((m + 1, n), 7.0, dtype=out_dtype, device="cuda")
    lin(a, sa, out=out[:m])
    assert (out[m] == 7).all()                  # the row behind the last token
    assert lin.device_status() == 0
    check_product(a, sa, w, sw, bias, out[:m], out_dtype)


@pytest.mark.parametrize("m", [1, 5, 40, 300])
def test_product_of_every_code(m):
    """All 256 codes of int8, -128 among them, and every finite one of e4m3."""
    from mamba_selective_state_gb300 import runner
    for dt, codes in ((torch.int8, range(256)), (torch.float8_e4m3fn, [c for c in range(256) if c & 127 != 127])):
        every = torch.tensor(list(codes), dtype=torch.uint8, device="cuda")
        a = torch.stack([every.roll(i) for i in range(m)]).view(dt)
        w = torch.stack([every.roll(-3 * i) for i in range(70)]).view(dt)
        one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
        out = runner.Linear8(w, one(70), out_dtype=F32)(a, one(m))
        check_product(a, one(m), w, one(70), None, out, F32)


@pytest.mark.parametrize("m,n,k", [(3, 70, 96), (50, 300, 256), (200, 300, 256)])
def test_product_keeps_what_is_not_finite_in_its_place(m, n, k):
    from mamba_selective_state_gb300 import runner
    g = gen(m)
    for form in ("int8", "e4m3"):
        a, w = some_codes(g, m, k, form), some_codes(g, n, k, form)
        sa, sw = torch.ones(m, device="cuda"), torch.ones(n, device="cuda")
        sa[1], sw[2] = math.nan, math.inf
        if form == "e4m3":
            a.view(torch.uint8)[0, k - 1] = 0x7f        # NaN
            w.view(torch.uint8)[n - 1, 0] = 0xff
        out = f64(runner.Linear8(w, sw, out_dtype=F32)(a, sa))
        bad = np.zeros((m, n), bool)
        bad[1], bad[:, 2] = True, True
        if form == "e4m3":
            bad[0], bad[:, n - 1] = True, True
        assert np.isfinite(out[~bad]).all() and not np.isfinite(out[bad]).any()


def test_linear8_from_weight():
    from mamba_selective_state_gb300 import runner
    w = rn(gen(1), 40, 100) * torch.exp(3 * rn(gen(2), 40, 1))
    w[3], w[4, 7], w[5] = 0, math.inf, 1e-37
    for form in ("int8", "e4m3"):
        lin = runner.Linear8.from_weight(w, form)
        s, c = f64(lin.scales), values(lin.codes)
        assert s[3] == s[5] == 0 and np.isnan(s[4]) and not c[[3, 4, 5]].any()
        fine = [i for i in range(40) if i not in (3, 4, 5)]
        y = f64(w)[fine] / s[fine][:, None]
        assert (np.abs(c[fine] - y) <= ro.half_steps(y, form) + 8 * U * np.abs(y)).all()


# ------------------------------------------------------- the log probabilities
def logp_case(rows, V, dt, seed, masked=0.0, stride=None):
    g = gen(seed)
    z = 3 * rn(g, rows, stride or V)
    if masked:
        z[torch.rand(z.shape, generator=g, device="cuda") < masked] = -math.inf
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    return z.to(dt)[:, :V], tok


def check_logp(dev, logits, tok, scale, ntop):
    x, V = f64(logits), logits.shape[1]
    want = ro.token_logprobs(x, tok.cpu().numpy(), scale, ntop)
    with np.errstate(all="ignore"):
        z = np.where(np.isfinite(x), scale * x, np.nan)
        m = np.nanmax(np.where(np.isnan(z), -np.inf, z), 1)
        spread = np.nansum(np.exp(z - m[:, None]) * np.abs(z - m[:, None]), 1) / np.nansum(np.exp(z - m[:, None]), 1)
        spread = np.nan_to_num(spread)          # rows without a word have no sums
    # a sum's relative error: a thread's words one after the other and the joins;
    # an exponential's: two units and the rounding of its exponent (up to 16 of
    # those words that weigh)
    rel = (V / 256 + 64) * U + 32 * U
    with np.errstate(all="ignore"):
        close(dev.lse, want["lse"], rel + 2 * U * (np.abs(m) + np.abs(want["lse"])), "lse")
        close(dev.logprobs, want["logprobs"], rel + 4 * U * np.abs(want["logprobs"]), "logprobs")
        close(dev.entropy, want["entropy"], rel * (2 + 2 * spread) + 4 * U * np.abs(want["entropy"]), "entropy")
        if ntop:
            assert np.array_equal(dev.top_tokens.cpu().numpy(), want["top_tokens"])
            close(dev.top_logprobs, want["top_logprobs"], rel + 4 * U * np.abs(want["top_logprobs"]), "top")
    return want, rel


VOCABS = [(1, 1), (5, 2), (3, 7), (9, 31), (2, 300), (700, 130), (3, 1025), (4, 5003), (320, 4096), (2, 32000),
          (1, 100003), (30, 20000)]


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows,V", VOCABS)
@pytest.mark.parametrize("ntop", [0, 1, 20, 32])
def test_logprobs(rows, V, dt, ntop):
    from mamba_selective_state_gb300 import runner
    logits, tok = logp_case(rows, V, dt, rows + V)
    dev = runner.LogProbsDevice(logits, tok, scale=0.8, ntop=ntop)
    dev.fwd()
    check_logp(dev, logits, tok, float(np.float32(0.8)), ntop)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_logprobs_masks_ties_and_padding(dt):
    from mamba_selective_state_gb300 import runner
    V = 2100
    logits, tok = logp_case(16, V, dt, 6, masked=0.5)
    low = torch.finfo(dt).min
    logits[0] = -math.inf                       # nothing is left
    logits[1] = -math.inf
    logits[1, [2, 77, 2000]] = 1.0              # fewer words than alternatives, equal
    logits[2] = 0.25                            # every word equal
    logits[3] = low
    logits[3, 4:7] = 1.5                        # masked by the type's lowest value
    logits[4] = low                             # all of them
    logits[5, 9] = math.nan
    logits[6, 9] = math.inf
    logits[7] = math.nan
    logits[8, :600] = 9.0                       # more equal words than a list holds
    logits[9] = 0.0
    logits[9, ::2] = -0.0                       # zeros are equal
    logits[10] = -1e30
    logits[10, 5] = 1e30
    tok[:16] = torch.tensor([3, 77, 5, 5, 9, 1, 1, 1, 2099, 0, 5, -1, V, 10 ** 9, 0, -2 ** 31], dtype=torch.int32)
    dev = runner.LogProbsDevice(logits, tok, scale=1.0, ntop=20)
    dev.fwd()
    check_logp(dev, logits, tok, 1.0, 20)
    got = f64(dev.logprobs)
    assert (got[[11, 12, 13, 15]] == 0).all()


@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("stride", [0, 5008, 5011])
@pytest.mark.parametrize("which", ["both", "logprobs", "entropy"])
def test_logprobs_backward(dt, stride, which):
    from mamba_selective_state_gb300 import runner
    rows, V, scale = 11, 5003, 1.5
    logits, tok = logp_case(rows, V, dt, 8, masked=0.3, stride=stride or None)
    logits[2] = -math.inf
    logits[3, 8] = math.nan
    tok[4] = -1
    dl, dH = rn(gen(1), rows), rn(gen(2), rows)
    kw = dict(dlogprobs=dl if which != "entropy" else None, dentropy=dH if which != "logprobs" else None)
    dev = runner.LogProbsDevice(logits, tok, scale=scale, **kw)
    dev.fwd()
    dev.bwd()
    assert dev.dlogits.shape == (rows, V)
    want, rel = check_logp(dev, logits, tok, scale, 0)
    check_grad(dev.dlogits, logits, tok, scale, rel, want, dt, **kw)


@pytest.mark.parametrize("dt", [BF16, F32])
def test_logprobs_of_large_logits(dt):
    """Rows whose logits are large, or all of them the type's lowest value: the
    sums are relative to the row's largest, in the gradient too."""
    from mamba_selective_state_gb300 import runner
    rows, V = 4, 700
    logits, tok = logp_case(rows, V, dt, 3)
    logits[0] = torch.finfo(dt).min
    logits[1] = (logits[1].float() + 30000).to(dt)
    logits[2] = -1e30
    dl, dH = rn(gen(1), rows), rn(gen(2), rows)
    dev = runner.LogProbsDevice(logits, tok, dlogprobs=dl, dentropy=dH)
    dev.fwd()
    dev.bwd()
    x, got = f64(logits), f64(dev.dlogits)
    for i in range(rows):
        z = x[i] - x[i].max()
        lp = z - np.log(np.exp(z).sum())
        p, t = np.exp(lp), int(tok[i])
        H = -(p * lp).sum()
        d = -p * (float(dl[i]) + float(dH[i]) * (lp + H))
        d[t] += float(dl[i])
        # (V / 256 + 96 roundings of the sum, 4 of an exponent of at most 32)
        tol = (V / 256 + 96 + 128) * U * p * (abs(float(dl[i])) + abs(float(dH[i])) * (np.abs(lp) + H + 1))
        tol = tol + 2 * U * abs(float(dl[i])) + HALF[dt] * np.abs(d) + 1e-40
        assert (np.abs(got[i] - d) <= tol).all(), i


# Rows that are nearly all one word: their log probabilities and entropies keep
# their digits, however small.  In roundings relative to each: a word's exponent d,
# below 64 here, and the exponent of each rebasing (64 at most in all) put 0.7 d on
# its exponential, 45 each, as does the factor log2(e) scale for the entropy; an
# exponential is within 4 and there are fewer than 10 rebasings; the chains of sums
# are 16 + 13 + 5 + 4 + 8 long: under 256.  Rows whose sum is 1.5 or more have
# logarithms from 0.4 on and lose a factor of 2.5 to it: 640.
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("rows,V,ntop", [(3, 1, 0), (50, 2, 1), (200, 7, 0), (400, 300, 5), (300, 5003, 0), (1000, 5003, 3),
                                         (300, 40001, 0), (4, 40001, 2), (1, 100003, 0)])
def test_logprobs_of_likely_words(rows, V, ntop, dt):
    from mamba_selective_state_gb300 import runner
    for turn in range(4 if rows < 10 else 1):
        g = gen(rows + V + turn)
        logits = 2 * rn(g, rows, V)
        # the word anywhere in the row: in its first and last vectors, in the middle
        tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
        tok[::5] = torch.randint(0, min(V, 4), (len(tok[::5]),), generator=g, device="cuda", dtype=torch.int32)
        tok[1::5] = V - 1
        lift = 8 + 17 * torch.rand(rows, generator=g, device="cuda")
        logits[torch.arange(rows, device="cuda"), tok.long()] = lift
        if V > 7:
            logits[2::7, 3] = logits[2::7].max(-1).values       # one more as likely, or the same word
            logits[4::7, :2] = -math.inf
            logits[4::7, 2] = 24.0
            tok[4::7] = 2
        logits = logits.to(dt)
        dl, dH = rn(g, rows), rn(g, rows)
        dev = runner.LogProbsDevice(logits, tok, scale=1.25, ntop=ntop, dlogprobs=dl, dentropy=dH)
        dev.fwd()
        dev.bwd()
        t = tok.cpu().numpy()
        want = ro.token_logprobs(f64(logits), t, 1.25, ntop)
        near = lambda x: 640 * U * np.abs(x) + 1e-14    # (64 bits lose what they add to 1)  # noqa: E731
        close(dev.logprobs, want["logprobs"], near(want["logprobs"]), "logprobs")
        # the likely word's own exponent is the rounding of its product with log2(e) scale (below 64: 64 U at most), and it is
        # taken back times a sum within 8 U
        close(dev.entropy, want["entropy"], near(want["entropy"]) + 512 * U * U, "entropy")
        if ntop:
            close(dev.top_logprobs[:, 0], want["top_logprobs"][:, 0], near(want["top_logprobs"][:, 0]), "top")
        # the gradient: a word's p with its exponent's roundings (64 of them and the exponential's), the token's 1 - p with
        # those of its log probability
        lp = 1.25 * f64(logits) - want["lse"][:, None]
        with np.errstate(invalid="ignore"):
            p, off = np.exp(lp), np.where(lp > -np.inf, np.abs(lp), 0) + want["entropy"][:, None]
        size = p * (np.abs(f64(dl))[:, None] + np.abs(f64(dH))[:, None] * off)
        at = np.arange(rows), t
        size[at] = np.abs(f64(dl) * np.expm1(want["logprobs"])) + np.abs(f64(dH)) * p[at] * off[at]
        d = ro.token_logprobs_bwd(f64(logits), t, 1.25, f64(dl), f64(dH))
        close(dev.dlogits, d, 1.25 * (1300 * U * size + 1e-11) + HALF[dt] * np.abs(d), "dlogits")


def test_logprobs_without_tokens():
    """Only what is asked for is written."""
    from mamba_selective_state_gb300 import _lib
    logits, _ = logp_case(7, 900, F32, 4)
    prob = _lib.make_logprob_problem(7, 900, 1.0, 0, F32)
    lse = torch.zeros(7, device="cuda")
    _lib.ssd_token_logprobs(prob, logits, None, None, None, lse)
    assert torch.allclose(lse, torch.logsumexp(logits, -1))
    top, val = torch.zeros(7, 2, dtype=torch.int32, device="cuda"), torch.zeros(7, 2, device="cuda")
    _lib.ssd_token_logprobs(_lib.make_logprob_problem(7, 900, 1.0, 2, F32), logits, None, None, None, None, None, top, val)
    assert torch.equal(top[:, 0].long(), logits.argmax(-1))


def check_grad(got, logits, tok, scale, rel, want, dt, dlogprobs, dentropy):
    x, t = f64(logits), tok.cpu().numpy()
    dl = np.zeros(len(x)) if dlogprobs is None else f64(dlogprobs)
    dH = 0 * dl if dentropy is None else f64(dentropy)
    d = ro.token_logprobs_bwd(x, t, scale, None if dlogprobs is None else dl, None if dentropy is None else dH)
    with np.errstate(all="ignore"):
        lp = np.maximum(scale * x - want["lse"][:, None], -1e4)
        p = np.exp(lp)
        # p's relative error: that of lse (its sum's, and the rounding of its value) and of the exponent;
        # the token's own term is added last
        e = rel + 2 * U * (np.abs(want["lse"])[:, None] + 2 * np.abs(np.maximum(lp, -100))) + 8 * U
        size = p * (np.abs(dl)[:, None] + np.abs(dH)[:, None] * (np.abs(lp) + want["entropy"][:, None] + 1))
        tol = scale * (e * size + 2 * U * np.abs(dl)[:, None]) + HALF[dt] * np.abs(d) + 2.0 ** -149
        tol = np.where(np.isfinite(tol), tol, 0.0)
    close(got, d, tol, "dlogits")


@pytest.mark.parametrize("rows,V", [(1, 1), (1, 100003), (700, 33), (620, 4001)])
def test_logprobs_backward_in_place(rows, V):
    from mamba_selective_state_gb300 import runner
    for dt in (BF16, F32):
        logits, tok = logp_case(rows, V, dt, rows)
        dl, dH = rn(gen(1), rows), rn(gen(2), rows)
        apart = runner.LogProbsDevice(logits, tok, dlogprobs=dl, dentropy=dH)
        apart.fwd()
        apart.bwd()
        kept = logits.clone()
        dev = runner.LogProbsDevice(logits, tok, dlogprobs=dl, dentropy=dH, dlogits=logits)
        dev.fwd()
        dev.bwd()
        assert torch.equal(apart.dlogits, logits)
        want, rel = check_logp(dev, kept, tok, 1.0, 0)
        check_grad(logits, kept, tok, 1.0, rel, want, dt, dl, dH)


def test_logprobs_leave_the_columns_between_rows():
    from mamba_selective_state_gb300 import runner
    logits, tok = logp_case(6, 1000, F32, 2)
    grad = torch.full((6, 1003), 5.0, device="cuda")
    dev = runner.LogProbsDevice(logits, tok, dlogprobs=rn(gen(1), 6), dlogits=grad[:, :1000])
    dev.fwd()
    dev.bwd()
    assert (grad[:, 1000:] == 5).all()
    dense = runner.LogProbsDevice(logits, tok, dlogprobs=dev.dlogprobs)
    dense.fwd()
    dense.bwd()
    assert torch.equal(dense.dlogits, grad[:, :1000])


# -------------------------------------------------------------- all together
def pipeline(x, r, w, lin, tok):
    from mamba_selective_state_gb300 import runner
    norm = runner.AddNormDevice(x, w, residual=r, form="int8")
    logits = torch.empty(len(x), len(lin.scales), dtype=lin.out_dtype, device="cuda")
    lp = runner.LogProbsDevice(logits, tok, ntop=5)

    def go():
        norm.fwd()
        lin(norm.codes, norm.scales, out=logits)
        lp.fwd()
    return norm, logits, lp, go


@pytest.mark.parametrize("rows", [1, 70, 200])
def test_from_the_residual_to_the_answer(rows):
    """Norm, readout product and log probabilities in one go, also captured and
    replayed with new inputs, and on another stream: the same bits each time,
    and each step right for what it was given."""
    from mamba_selective_state_gb300 import runner
    g = gen(rows)
    x, r, w = norm_case(rows, 512, BF16, F32, rows)
    lin = runner.Linear8.from_weight(rn(g, 3001, 512) * 0.1, out_dtype=F32)
    tok = torch.randint(0, 3001, (rows,), generator=g, device="cuda", dtype=torch.int32)
    norm, logits, lp, go = pipeline(x, r, w, lin, tok)

    def results():
        return [t.clone() for t in (norm.h, norm.codes.view(torch.uint8), norm.scales, logits, lp.logprobs,
                                    lp.entropy, lp.top_tokens, lp.top_logprobs)]
    go()
    first = results()
    check_product(norm.codes, norm.scales, lin.codes, lin.scales, None, logits, F32)
    check_logp(lp, logits, tok, 1.0, 5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    keep = x.clone()
    x.copy_(rn(g, rows, 512))
    graph.replay()
    second = results()
    assert not torch.equal(first[3], second[3])
    check_product(norm.codes, norm.scales, lin.codes, lin.scales, None, logits, F32)
    check_logp(lp, logits, tok, 1.0, 5)
    x.copy_(keep)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, results()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    norm.out = None
    logits.zero_()
    side.wait_stream(torch.cuda.current_stream())
    norm.fwd(stream=side)
    out = lin(norm.codes, norm.scales, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first[3])


# each way that a product can go: few tokens, some, pairs of CTAs with and without rows written out before
WAYS = [(5, 300, 256, "int8"), (5, 300, 250, "int8"), (20, 300, 256, "e4m3"), (100, 500, 512, "int8"),
        (100, 500, 500, "e4m3"), (9000, 1100, 256, "int8"), (9000, 1100, 250, "e4m3"), (9000, 1100, 256, "e4m3")]


@pytest.mark.parametrize("m,n,k,form", WAYS)
def test_product_captured_and_on_two_streams(m, n, k, form):
    """Replays with new inputs, and two calls of one map at once on two streams,
    give the bits of calls one by one."""
    from mamba_selective_state_gb300 import runner
    g = gen(m + k)
    w, sw = some_codes(g, n, k, form), torch.rand(n, generator=g, device="cuda")
    ins = [(some_codes(g, m, k, form), torch.rand(m, generator=g, device="cuda")) for _ in range(2)]
    lin = runner.Linear8(w, sw)
    want = [lin(a, s).clone() for a, s in ins]
    check_product(*ins[0], w, sw, None, want[0], BF16)
    assert not torch.equal(*want)
    a, s = ins[0][0].clone(), ins[0][1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lin(a, s)
    for i in (1, 0):
        a.copy_(ins[i][0])
        s.copy_(ins[i][1])
        graph.replay()
        assert torch.equal(out, want[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[], []]
    for _ in range(5):
        for i in (0, 1):
            outs[i].append(lin(*ins[i], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in (0, 1) for o in outs[i])
    assert lin.device_status() == 0


def test_product_reproducible_and_rowwise():
    """A token's result does not depend on the tokens around it where the same
    kernel takes them, and the same call gives the same bits."""
    from mamba_selective_state_gb300 import runner
    g = gen(5)
    for form, m in (("int8", 20), ("e4m3", 100), ("int8", 100), ("int8", 3000), ("e4m3", 3000)):
        w, a = some_codes(g, 700, 640, form), some_codes(g, m, 640, form)
        lin = runner.Linear8(w, torch.ones(700, device="cuda"), out_dtype=F32)
        one = lin(a, torch.ones(m, device="cuda"))
        assert torch.equal(one, lin(a, torch.ones(m, device="cuda")))
        b = a.clone()
        tail = b[m // 2:].view(torch.uint8)
        tail.copy_(tail.roll(1, 0))
        assert torch.equal(one[:m // 2], lin(b, torch.ones(m, device="cuda"))[:m // 2])


def test_offsets_beyond_32_bits():
    """The last rows of tensors of more than 2^31 elements."""
    from mamba_selective_state_gb300 import runner
    g = gen(11)
    rows, V = 21500, 100003
    logits = torch.zeros(rows, V, dtype=BF16, device="cuda")
    logits[-2:] = (3 * rn(g, 2, V)).to(BF16)
    tok = torch.full((rows,), 77, dtype=torch.int32, device="cuda")
    dl, dH = rn(g, rows), rn(g, rows)
    dev = runner.LogProbsDevice(logits, tok, ntop=3, dlogprobs=dl, dentropy=dH)
    dev.fwd()
    dev.bwd()
    small = runner.LogProbsDevice(logits[-2:].clone(), tok[-2:].clone(), ntop=3, dlogprobs=dl[-2:].clone(),
                                  dentropy=dH[-2:].clone())
    small.fwd()
    small.bwd()
    check_logp(small, small.logits, small.tokens, 1.0, 3)
    assert torch.equal(dev.top_tokens[-2:], small.top_tokens)
    assert torch.allclose(dev.logprobs[-2:], small.logprobs, rtol=1e-5)
    assert torch.allclose(dev.dlogits[-2:].float(), small.dlogits.float(), rtol=2.0 ** -7, atol=1e-12)
    assert torch.equal(dev.top_tokens[:-2], torch.tensor([0, 1, 2], device="cuda", dtype=torch.int32).expand(rows - 2, 3))
    del logits, dev
    rows, dim = 135000, 16384
    x = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    x[-3:] = rn(g, 3, dim).to(BF16)
    w = 1 + 0.1 * rn(g, dim)
    dev = runner.AddNormDevice(x, w, form="int8")
    dev.fwd()
    out, _ = ro.add_rmsnorm_fwd(f64(x[-3:]), f64(w), 1e-5)
    got = ro.code_values(raw(dev.codes[-3:]), "int8") * f64(dev.scales[-3:])[:, None]
    assert np.abs(got - out).max() <= 0.51 / 127 * np.abs(out).max()
    assert not dev.scales[:-3].any() and not dev.codes[0].any()
    del x, dev
    torch.cuda.empty_cache()
    m, n, k = 210000, 10304, 64
    a, wc = some_codes(g, m, k, "int8"), some_codes(g, n, k, "int8")
    lin = runner.Linear8(wc, torch.ones(n, device="cuda"))
    out = lin(a, torch.ones(m, device="cuda"))
    check_product(a[-300:], torch.ones(300, device="cuda"), wc, lin.scales, None, out[-300:], BF16)


def test_gradients_through_the_chain():
    """A training step's chain -- norm on the residual stream, readout, log
    probabilities and entropy of sampled tokens, and back -- against float64
    differentiation, in fp32."""
    from mamba_selective_state_gb300 import runner
    g = gen(21)
    rows, dim, V, eps = 33, 96, 500, 1e-5
    x, r, w = norm_case(rows, dim, F32, F32, 21)
    E = rn(g, V, dim) * dim ** -0.5
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tok[3] = -1
    adv, dH, dh = rn(g, rows), 0.1 * rn(g, rows), rn(g, rows, dim)
    dout = torch.empty(rows, dim, device="cuda")
    norm = runner.AddNormDevice(x, w, residual=r, eps=eps, dout=dout, dh=dh)
    norm.fwd()
    logits = norm.out @ E.T
    lp = runner.LogProbsDevice(logits, tok, dlogprobs=adv, dentropy=dH)
    lp.fwd()
    lp.bwd()
    dout.copy_(lp.dlogits @ E)
    norm.bwd()
    xd, rd, wd, Ed = (t.detach().double().cpu().requires_grad_() for t in (x, r, w, E))
    h = xd + rd
    z = (h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * wd) @ Ed.T
    logp = torch.log_softmax(z, -1)
    t = tok.cpu().long()
    loss = ((logp.gather(1, t.clamp(min=0)[:, None])[:, 0] * (t >= 0)) * adv.cpu().double()).sum()
    loss = loss - ((logp.exp() * logp).sum(-1) * dH.cpu().double()).sum() + (h * dh.cpu().double()).sum()
    loss.backward()
    # five steps in fp32, sums of at most 500 terms: 1e-4 of the largest is 1600 roundings
    for got, want in ((norm.dx, xd.grad), (norm.dweight, wd.grad), (norm.dresidual, rd.grad)):
        assert np.abs(f64(got) - want.numpy()).max() < 1e-4 * np.abs(want.numpy()).max()


def test_refusals_of_misaligned_tensors():
    from mamba_selective_state_gb300 import _lib, runner
    x = torch.zeros(5, 7, device="cuda")
    with pytest.raises(_lib.SSDError):
        runner.AddNormDevice(x[1:], torch.ones(7, device="cuda")).fwd()
    with pytest.raises(_lib.SSDError):
        runner.LogProbsDevice(x[1:], torch.zeros(4, dtype=torch.int32, device="cuda")).fwd()
    c = torch.zeros(5, 7, dtype=torch.int8, device="cuda")
    lin = runner.Linear8(c, torch.ones(5, device="cuda"))
    with pytest.raises(_lib.SSDError):
        lin(c[1:], torch.ones(4, device="cuda"))
    for bad in (dict(codes=c.float()), dict(codes=c.cpu()), dict(codes=c[:, :5]), dict(codes=c[0]),
                dict(scales=torch.ones(4, device="cuda")), dict(scales=torch.ones(5)),
                dict(out=torch.zeros(5, 5, device="cuda"))):
        with pytest.raises(ValueError):
            lin(**dict(dict(codes=c, scales=torch.ones(5, device="cuda")), **bad))


def test_serving_example_scores_what_it_generated():
    """The example's 8-bit scores against the same readout in float64: 8 bits of
    the outputs (a row's largest over 254) and of the embeddings weigh in the
    logits as independent errors of half a step each."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "delta_serving.py")
    spec = importlib.util.spec_from_file_location("delta_serving", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    layer = ex.Layer(vocab=64, width=64, nheads=4, headdim=64, dstate=64)
    tokens = torch.randint(0, 64, (90,), generator=gen(1), device="cuda", dtype=torch.int32)
    got = ex.score(layer, tokens, top=4)
    pre = ex.runner.DeltaDevice(*layer.inputs(tokens[None, :-1]))
    pre.fwd()
    h = f64((pre.y[0].float().flatten(1) @ layer.wo).bfloat16())
    out, E = h, f64(layer.embed)
    z = out @ E.T
    want = ro.token_logprobs(z, tokens[1:].cpu().numpy(), 1.0)
    # (1 % more for what fp32 rounds)
    # |z - z8| <= half a step of one operand on the sum of the other's sizes, and the product of both
    so, se = np.abs(out).max(-1) / 254, np.abs(E).max(-1) / 254
    tol = so[:, None] * np.abs(E).sum(-1) + se * np.abs(out).sum(-1)[:, None] + 64 * so[:, None] * se
    worst = tol.max(-1) * 1.01
    assert (np.abs(f64(got.logits) - z) <= tol * 1.01).all()
    # a log probability moves by at most the largest error of its row, twice
    assert (np.abs(f64(got.logprobs) - want["logprobs"]) <= 2 * worst).all()
    assert (got.top_logprobs[:, :-1] >= got.top_logprobs[:, 1:]).all() and (got.logprobs <= 0).all()
