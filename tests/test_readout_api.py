"""What the entry points of the norm with residual, the 8-bit product and the
log probabilities refuse (CPU: the calls return before any CUDA call)."""
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


def test_struct_sizes(lib):
    assert ctypes.sizeof(lib.ssd_add_norm_problem) == 48
    assert ctypes.sizeof(lib.ssd_matmul_problem) == 40
    assert ctypes.sizeof(lib.ssd_logprob_problem) == 48


def norm(lib, flags=None, **kw):
    d = dict(rows=4, dim=64, eps=1e-5, dtype=lib.SSD_BF16)
    d.update(kw)
    p = lib.make_add_norm_problem(**d)
    if flags is not None:
        p.flags = flags
    return p


def test_norm_problems(lib):
    size = lib.ssd_add_rmsnorm_bwd_workspace_bytes
    for bad in (dict(rows=0), dict(dim=0), dict(x_stride=63), dict(x_stride=-64), dict(eps=0.0), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(dtype=2), dict(residual_dtype=3),
                dict(out_format=3), dict(out_format=-1), dict(flags=1), dict(residual=False, residual_dtype=0),
                dict(dtype=0, residual_dtype=1), dict(dim=16385), dict(rows=1 << 40, dim=1024),
                dict(x_stride=1 << 31)):
        assert size(norm(lib, **bad)) == 0, bad
    assert size(norm(lib)) >= 4 * 64 * 4 and size(norm(lib, rows=10 ** 6)) % 256 == 0
    assert size(norm(lib, rows=10 ** 6)) == size(norm(lib, rows=10 ** 9))


def test_norm_arguments(lib):
    bad = lib.SSD_ERR_INVALID_ARGUMENT
    base = dict(x=FAKE, residual=FAKE, weight=FAKE, h=FAKE, out=FAKE, scales=None)
    fwd = lambda p=norm(lib), **o: lib.ssd_add_rmsnorm_fwd(p, **dict(base, **o), stream=0, check=False)  # noqa: E731
    for n in ("x", "residual", "weight", "out"):
        assert fwd(**{n: None}) == bad, n
    for n in base:
        assert fwd(norm(lib, out_format=1 if n == "scales" else 0), **{n: FAKE + 8}) == bad, n
    assert fwd(scales=FAKE) == bad and fwd(norm(lib, out_format=1)) == bad
    assert fwd(norm(lib, residual=False)) == bad            # a residual without its flag
    assert fwd(norm(lib, dim=20000)) == lib.SSD_ERR_UNSUPPORTED
    base2 = dict(h=FAKE, weight=FAKE, dout=FAKE, dh=FAKE, dx=FAKE, dresidual=FAKE, dweight=FAKE, workspace=FAKE)
    bwd = lambda p=norm(lib), nb=1 << 40, **o: lib.ssd_add_rmsnorm_bwd(  # noqa: E731
        p, **dict(base2, **o), workspace_bytes=nb, stream=0, check=False)
    for n in ("h", "weight", "dout", "dx", "dweight", "workspace"):
        assert bwd(**{n: None}) == bad, n
    for n in base2:
        assert bwd(**{n: FAKE + 4}) == bad, n
    assert bwd(norm(lib, residual=False)) == bad            # dresidual without a residual
    assert bwd(nb=8) == lib.SSD_ERR_WORKSPACE_TOO_SMALL
    assert lib.LIB.ssd_add_rmsnorm_fwd(None, *([None] * 6), None) == bad
    assert lib.LIB.ssd_add_rmsnorm_bwd(None, *([None] * 8), 0, None) == bad


def test_matmul_refusals(lib):
    bad, uns = lib.SSD_ERR_INVALID_ARGUMENT, lib.SSD_ERR_UNSUPPORTED
    base = dict(a=FAKE, a_scales=FAKE, w=FAKE, w_scales=FAKE, bias=None, out=FAKE, workspace=FAKE)

    def call(m=4, n=8, k=16, fmt=0, out_dtype=1, nb=1 << 50, **o):
        p = lib.make_matmul_problem(m, n, k, fmt, out_dtype)
        if "flags" in o:
            p.flags = o.pop("flags")
        rc = lib.ssd_scaled_matmul(p, **dict(base, **o), workspace_bytes=nb, stream=0, check=False)
        assert (lib.ssd_scaled_matmul_workspace_bytes(p) == 0) == (rc in (bad, uns) and not o)
        return rc
    for n in ("m", "n", "k"):
        assert call(**{n: 0}) == bad and call(**{n: -1}) == bad and call(**{n: (1 << 22) + 1}) == uns, n
    assert call(fmt=2) == bad and call(out_dtype=2) == bad
    p = lib.make_matmul_problem(4, 8, 16, 0, 1)
    p.flags = 1
    assert lib.ssd_scaled_matmul_workspace_bytes(p) == 0
    assert call(m=1 << 22, k=1 << 22) == uns and call(m=1 << 22, n=1 << 22) == uns and call(n=1 << 22, k=1 << 22) == uns
    for n in base:
        if n != "bias":
            assert call(**{n: None}) == bad, n
        assert call(**{n: FAKE + 8}) == bad, n
    assert call(nb=8) == lib.SSD_ERR_WORKSPACE_TOO_SMALL
    assert call(k=(1 << 20) + 1) == uns
    for dims in ((1, 1, 1), (1, 10304, 4096), (64, 8, 17), (65, 8, 17), (4001, 2048, 4096), (1000, 1, 1)):
        for fmt in (0, 1):
            assert lib.ssd_scaled_matmul_workspace_bytes(lib.make_matmul_problem(*dims, fmt, 0)) >= 256
    assert lib.LIB.ssd_scaled_matmul(None, *([None] * 7), 0, None) == bad


def test_logprob_refusals(lib):
    bad, uns = lib.SSD_ERR_INVALID_ARGUMENT, lib.SSD_ERR_UNSUPPORTED
    base = dict(logits=FAKE, tokens=FAKE, logprobs=FAKE, entropy=FAKE, lse=FAKE, stats=FAKE, top_tokens=FAKE,
                top_logprobs=FAKE)
    base2 = dict(logits=FAKE, tokens=FAKE, stats=FAKE, entropy=FAKE, dlogprobs=FAKE, dentropy=FAKE, dlogits=2 * FAKE)

    def prob(rows=4, vocab=100, scale=1.0, ntop=3, dtype=1, **kw):
        return lib.make_logprob_problem(rows, vocab, scale, ntop, dtype, **kw)
    fwd = lambda p=prob(), **o: lib.ssd_token_logprobs(p, **dict(base, **o), stream=0, check=False)  # noqa: E731
    bwd = lambda p=prob(), **o: lib.ssd_token_logprobs_bwd(p, **dict(base2, **o), stream=0, check=False)  # noqa: E731
    for kw in (dict(rows=0), dict(vocab=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(ntop=-1), dict(dtype=2), dict(logit_stride=99), dict(grad_stride=99),
               dict(logit_stride=-100)):
        assert fwd(prob(**kw)) == bad and bwd(prob(**kw)) == bad, kw
    for kw in (dict(ntop=33), dict(vocab=1 << 31), dict(rows=1 << 28), dict(rows=1 << 20, logit_stride=1 << 20)):
        assert fwd(prob(**kw)) == uns and bwd(prob(**kw)) == uns, kw
    for n in ("logits", "tokens", "top_tokens", "top_logprobs"):
        assert fwd(**{n: None}) == bad, n
    for n in base:
        assert fwd(**{n: FAKE + 4}) == bad, n
    assert fwd(prob(ntop=0)) == bad                          # alternatives without a number
    assert fwd(prob(ntop=0), logprobs=None) == bad           # tokens without logprobs
    assert fwd(prob(ntop=0), logprobs=None, tokens=None, entropy=None, lse=None, stats=None, top_tokens=None,
               top_logprobs=None) == bad                     # nothing to do
    for n in ("logits", "stats", "dlogits", "tokens", "entropy"):
        assert bwd(**{n: None}) == bad, n
    for n in base2:
        assert bwd(**{n: FAKE + 4}) == bad, n
    assert bwd(dlogprobs=None) == bad and bwd(dentropy=None) == bad
    assert bwd(dlogprobs=None, tokens=None, dentropy=None, entropy=None) == bad
    assert bwd(prob(logit_stride=128), dlogits=FAKE) == bad  # in place with other strides
    assert lib.LIB.ssd_token_logprobs(None, *([None] * 8), None) == bad
    assert lib.LIB.ssd_token_logprobs_bwd(None, *([None] * 7), None) == bad


def test_runner_refuses_wrong_tensors(lib):
    from mamba_selective_state_gb300 import runner
    x, w, z = torch.zeros(4, 8), torch.ones(8), torch.zeros(4)
    for bad in (dict(x=torch.zeros(2, 4, 8)), dict(x=x.double()), dict(x=torch.zeros(8, 4).t()), dict(form="int4"),
                dict(residual=x.bfloat16()), dict(residual=x[:3]), dict(weight=w[:7]), dict(dh=x), dict(dout=x[:, :7]),
                dict(x=torch.zeros(4, 9)[:, :8], dout=x), dict()):     # (the last: tensors off the GPU)
        a = dict(dict(x=x, weight=w), **bad)
        with pytest.raises(ValueError):
            runner.AddNormDevice(a.pop("x"), a.pop("weight"), **a)
    c = torch.zeros(4, 8, dtype=torch.int8)
    for bad in (dict(codes=x), dict(codes=c[0]), dict(out_dtype=torch.float16), dict(scales=torch.zeros(5)), dict()):
        a = dict(dict(codes=c, scales=z), **bad)
        with pytest.raises(ValueError):
            runner.Linear8(a.pop("codes"), a.pop("scales"), **a)
    with pytest.raises(ValueError):
        runner.Linear8.from_weight(x, "int4")
    t = torch.zeros(4, dtype=torch.int32)
    for bad in (dict(logits=x.half()), dict(logits=x[0]), dict(logits=torch.zeros(8, 4).t()), dict(tokens=t[:3]),
                dict(tokens=t.long()), dict(dlogprobs=z[:3]), dict(dlogits=x), dict(dentropy=z, dlogits=x[:, :7]), dict()):
        a = dict(dict(logits=x, tokens=t), **bad)
        with pytest.raises(ValueError):
            runner.LogProbsDevice(a.pop("logits"), a.pop("tokens"), **a)
