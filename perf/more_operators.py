"""Cases and plain forms of the operators between a layer's residual stream and
a model's answer: the norm that takes in the residual (forward with its output
in 8 bits, and forward with gradient), the product of 8-bit codes that reads
it, and the log probabilities of given tokens with their entropy, their top
alternatives and their gradient.

Every case is one pass through one operator (``proj``: through the norm and the
product behind it).  ``run`` computes it with elementary torch operations in 32
bits (``own`` false) or through this repository's entry points (``own`` true);
``exact`` computes it in 64 bits from the definition.

    norm      h = x + residual, rounded to the residual's type
              out = h / sqrt(mean(h^2) + eps) * weight
    8 bits    a = max |out| of the row, scale = a / top, code = out / scale to the
              nearest (int8: top 127; e4m3: top 448)
    product   out[m, n] = a_scale[m] w_scale[n] sum_k a[m, k] w[n, k] + bias[n]
    logprobs  z = scale * logits, lse = log sum exp z, logprob = z[token] - lse,
              entropy = -sum p log p; alternatives by the logit, ties to the
              lowest index
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
TOP = {"int8": 127.0, "e4m3": 448.0}


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def _norm(name, op, rows, dim, dtype, resid, form=None):
    return dict(name=name, op=op, rows=rows, dim=dim, dtype=dtype, resid=resid, form=form)


def _matmul(name, m, n, k, form, out, bias=False):
    return dict(name=name, op="matmul", m=m, n=n, k=k, form=form, out=out, bias=bias)


def _logp(name, op, rows, vocab, dtype, top=0, masked=False):
    return dict(name=name, op=op, rows=rows, vocab=vocab, dtype=dtype, top=top, masked=masked)


def listed():
    return [
        # a decode step of four sequences: the norm before a projection, latency counts
        _norm("norm8_b4_D4096_e4m3", "norm8", 4, 4096, "bf16", "bf16", "e4m3"),
        # the same before a prefill's projections (batch 2 of 8192 tokens)
        _norm("norm8_L16384_D4096_e4m3", "norm8", 16384, 4096, "bf16", "bf16", "e4m3"),
        # a training step's norm on an fp32 residual stream, with every gradient
        _norm("norm_train_L16384_D4096", "norm_train", 16384, 4096, "bf16", "f32"),
        # a numerical check of a small model in fp32, at an odd width
        _norm("norm_train_L1001_D1237_f32", "norm_train", 1001, 1237, "f32", "f32"),
        # one token: norm to 8 bits and the layer's input projection (z, x, B, C, dt
        # of 64 heads of 64, 8 groups of 128)
        dict(name="proj_b1_int8", op="proj", m=1, n=10304, k=4096, form="int8", out="bf16",
             bias=False),
        # the projection for a serving batch of an odd number of tokens
        _matmul("matmul_b61_int8", 61, 10304, 4096, "int8", "bf16"),
        # the projection for a prefill
        _matmul("matmul_L16384_int8", 16384, 10304, 4096, "int8", "bf16"),
        # an output projection for a prompt of an odd length, in e4m3, with a bias
        _matmul("matmul_L4001_e4m3", 4001, 2048, 4096, "e4m3", "bf16", bias=True),
        # what a server returns beside four sequences' tokens: latency counts
        _logp("logp_b4_V32000_f32", "logp", 4, 32000, "f32", top=5),
        # a prompt scored over a large odd vocabulary
        _logp("logp_L4096_V100003_bf16", "logp", 4096, 100003, "bf16", top=20),
        # a training step on sampled tokens: log probability and entropy, with the
        # logits' gradient
        _logp("logp_train_L4096_V32000_bf16", "logp_train", 4096, 32000, "bf16"),
        # the same in fp32 with words that a grammar excludes, padded rows among them
        _logp("logp_train_L300_V5003_f32", "logp_train", 300, 5003, "f32", masked=True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm8", "norm_train", "proj", "matmul", "matmul", "logp", "logp_train"])
    if op in ("norm8", "norm_train"):
        dim = rng.choice([rng.randint(1, 8192), 8 * rng.randint(8, 1024), 64 * rng.randint(4, 128)])
        rows = _logint(rng, 1, min(16384, 16384 * 4096 // dim))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        case = _norm("", op, rows, dim, dtype, "f32" if dtype == "f32" else rng.choice(["bf16", "f32"]),
                     "e4m3" if op == "norm8" else None)
    elif op in ("proj", "matmul"):
        m = _logint(rng, 1, 64 if op == "proj" else 16384)
        n = rng.choice([rng.randint(1, 10304), 64 * rng.randint(1, 161)])
        k = rng.choice([rng.randint(1, 4096), 16 * rng.randint(1, 256), 64 * rng.randint(1, 64)])
        case = _matmul("", m, n, k, rng.choice(["int8", "int8", "e4m3"]), rng.choice(["bf16", "f32"]),
                       rng.random() < 0.3)
        case["op"] = op
        if op == "proj":
            case["bias"] = False
    else:
        vocab = _logint(rng, 300, 100003)
        rows = _logint(rng, 1, min(4096, (4096 * 32000 if op == "logp_train" else 4096 * 100003) // vocab))
        dtype = rng.choice(["bf16", "f32"])
        if dtype == "f32":
            rows = max(1, rows // 2)
        case = _logp("", op, rows, vocab, dtype, rng.choice([0, 1, 5, 20]) if op == "logp" else 0,
                     rng.random() < 0.3)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# What a program has in hand before the call
# ---------------------------------------------------------------------------
def _type(name):
    return BF16 if name == "bf16" else F32


def _codes(x, form):
    """8-bit codes of x's rows and the rows' scales."""
    a = x.abs().amax(-1, keepdim=True)
    y = x * (TOP[form] / a)
    y = torch.round(y).to(torch.int8) if form == "int8" else y.to(torch.float8_e4m3fn)
    return y, (a / TOP[form])[:, 0]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm8", "norm_train", "proj"):
        rows, dim = (case["m"], case["k"]) if op == "proj" else (case["rows"], case["dim"])
        dt, rt = (BF16, BF16) if op == "proj" else (_type(case["dtype"]), _type(case["resid"]))
        # a residual stream that has grown over the layers, some of its columns large
        s["residual"] = (n(rows, dim) * 2.0 * torch.exp(0.5 * n(dim))).to(rt)
        s["x"] = n(rows, dim).to(dt)
        s["weight"] = 1.0 + 0.2 * n(dim)
        s["eps"] = 1e-5
        if op == "norm_train":
            s["dout"], s["dh"] = n(rows, dim).to(dt), n(rows, dim).to(rt)
        if op != "proj":
            return s
    if op in ("matmul", "proj"):
        if op == "matmul":
            s["a"], s["a_scales"] = _codes(n(case["m"], case["k"]), case["form"])
        s["w"], s["w_scales"] = _codes(n(case["n"], case["k"]) * case["k"] ** -0.5, case["form"])
        s["bias"] = n(case["n"]) if case["bias"] else None
        return s
    rows, V = case["rows"], case["vocab"]
    z = n(rows, V)
    z *= 2.0
    # most of a distribution lies on few words: the sampled one is among the likely
    s["tokens"] = (z[:, : min(V, 4096)] + n(rows, min(V, 4096))).argmax(-1).to(torch.int32)
    z.scatter_add_(1, s["tokens"].long()[:, None], 6.0 * torch.rand(rows, 1, generator=gen, device="cuda"))
    if case["masked"]:
        out = torch.rand(rows, V, generator=gen, device="cuda") < 0.4
        out.scatter_(1, s["tokens"].long()[:, None], False)
        z.masked_fill_(out, -math.inf)
        s["tokens"][torch.rand(rows, generator=gen, device="cuda") < 0.1] = -1   # padding
    s["logits"] = z.to(_type(case["dtype"]))
    s["scale"] = 1.25
    if op == "logp_train":
        s["dlogprobs"], s["dentropy"] = n(rows), 0.01 * n(rows)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _plain_norm(s):
    """h in the residual's type, the fp32 values that it stands for, their
    reciprocal root mean square, and the fp32 output."""
    h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    v = h.float()
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + s["eps"])
    return h, v, r, v * r * s["weight"]


def _plain_matmul(a, a_scales, s):
    acc = a.float() @ s["w"].float().t()
    out = acc * a_scales[:, None] * s["w_scales"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(_type(s["case"]["out"]))


def _plain_top(logits, lse, scale, k):
    """The k largest of each row by one selection over keys of the value above
    the word's index counted from the end; what is excluded is none of them."""
    rows, V = logits.shape
    bits = (logits.float() + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() << 32
    key |= torch.arange(V - 1, -1, -1, device=logits.device)
    best = torch.topk(key, min(k, V), dim=1, sorted=True).values
    at = (V - 1) - (best & 0xFFFFFFFF)
    val = logits.gather(1, at).float() * scale - lse[:, None]
    at = torch.where(torch.isinf(val), -1, at).to(torch.int32)
    pad = (0, k - at.shape[1])
    return (torch.nn.functional.pad(at, pad, value=-1),
            torch.nn.functional.pad(val, pad, value=-math.inf))


def _plain_logp(s):
    c = s["case"]
    z = s["logits"].float() * s["scale"]
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = torch.exp(d)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total[:, 0] - torch.where(e > 0, e * d, 0.0).sum(-1) / total[:, 0]
    lse = (m + log_total)[:, 0]
    tok = s["tokens"].long()
    on = tok >= 0
    lp = torch.where(on, z.gather(1, tok.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
    out = {"logprobs": lp, "entropy": entropy, "lse": lse}
    if c["top"]:
        out["top_tokens"], out["top_logprobs"] = _plain_top(s["logits"], lse, s["scale"], c["top"])
    if c["op"] == "logp_train":
        dlp = torch.where(on, s["dlogprobs"], 0.0)
        p = e / total
        logp = torch.where(e > 0, d - log_total, 0.0)
        dz = -p * (dlp[:, None] + s["dentropy"][:, None] * (logp + entropy[:, None]))
        dz.scatter_add_(1, tok.clamp(min=0)[:, None], dlp[:, None])
        out["dlogits"] = (dz * s["scale"]).to(s["logits"].dtype)
    return out


def _plain(s):
    op = s["case"]["op"]
    if op in ("logp", "logp_train"):
        return _plain_logp(s)
    if op == "matmul":
        return {"out": _plain_matmul(s["a"], s["a_scales"], s)}
    h, v, r, out = _plain_norm(s)
    if op == "norm8":
        codes, scales = _codes(out, s["case"]["form"])
        return {"h": h, "codes": codes, "scales": scales}
    if op == "proj":
        return {"h": h, "out": _plain_matmul(*_codes(out, s["case"]["form"]), s)}
    g = s["dout"].float() * s["weight"]
    n = v * r
    dh = s["dh"].float() + r * (g - n * (g * n).mean(-1, keepdim=True))
    return {"h": h, "out": out.to(s["x"].dtype), "dx": dh.to(s["x"].dtype),
            "dresidual": dh.to(s["residual"].dtype), "dweight": (s["dout"].float() * n).sum(0)}


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------
def _own(s):
    from mamba_selective_state_gb300 import runner
    c, op, dev = s["case"], s["case"]["op"], s.get("dev")
    if op in ("norm8", "norm_train", "proj"):
        if dev is None:
            dev = s["dev"] = runner.AddNormDevice(s["x"], s["weight"], residual=s["residual"],
                                                  eps=s["eps"], form=c.get("form"),
                                                  dout=s.get("dout"), dh=s.get("dh"))
        dev.fwd()
        if op == "norm8":
            return {"h": dev.h, "codes": dev.codes, "scales": dev.scales}
        if op == "norm_train":
            dev.bwd()
            return {"h": dev.h, "out": dev.out, "dx": dev.dx, "dresidual": dev.dresidual,
                    "dweight": dev.dweight}
        s["a"], s["a_scales"] = dev.codes, dev.scales
    if op in ("proj", "matmul"):
        lin = s.get("lin")
        if lin is None:
            lin = s["lin"] = runner.Linear8(s["w"], s["w_scales"], bias=s["bias"],
                                            out_dtype=_type(c["out"]))
        out = lin(s["a"], s["a_scales"])
        return {"h": dev.h, "out": out} if op == "proj" else {"out": out}
    if dev is None:
        dev = s["dev"] = runner.LogProbsDevice(s["logits"], s["tokens"], scale=s["scale"],
                                               ntop=c["top"], dlogprobs=s.get("dlogprobs"),
                                               dentropy=s.get("dentropy"))
    dev.fwd()
    out = {"logprobs": dev.logprobs, "entropy": dev.entropy, "lse": dev.lse}
    if c["top"]:
        out["top_tokens"], out["top_logprobs"] = dev.top_tokens, dev.top_logprobs
    if op == "logp_train":
        dev.bwd()
        out["dlogits"] = dev.dlogits
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# Bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("norm8", "norm_train"):
        n, e, r = case["rows"] * case["dim"], size[case["dtype"]], size[case["resid"]]
        if op == "norm8":   # x, residual, weight in; h, codes, scales out
            return {"bytes": n * (e + 2 * r + 1) + 4 * (case["dim"] + case["rows"]), "flops": 8 * n}
        # and dout, dh in; out, dx, dresidual, dweight out
        return {"bytes": n * (4 * e + 4 * r) + 8 * case["dim"], "flops": 16 * n}
    if op in ("matmul", "proj"):
        m, n, k = case["m"], case["n"], case["k"]
        b = n * k + m * n * size[case["out"]] + 4 * (m + n) + (4 * n if case["bias"] else 0)
        # the projection reads x, residual and the norm's weight, and writes h
        b += m * k * 6 + 4 * k if op == "proj" else m * k
        return {"bytes": b, "flops": 2 * m * n * k}
    n, rows = case["rows"] * case["vocab"], case["rows"]
    b = n * size[case["dtype"]] + rows * (16 + 8 * case["top"])
    if op == "logp":
        return {"bytes": b, "flops": 6 * n}
    return {"bytes": b + n * size[case["dtype"]] + 8 * rows, "flops": 14 * n}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_logp(case, s):
    f = torch.float64
    parts = []
    for lo in range(0, case["rows"], 512):      # rows do not see each other
        raw = s["logits"][lo:lo + 512].to(f)
        z = s["scale"] * raw
        tok = s["tokens"][lo:lo + 512].long()
        lse = torch.logsumexp(z, -1)
        logp = z - lse[:, None]
        p = torch.exp(logp)
        plogp = torch.where(p > 0, p * logp, torch.zeros((), dtype=f, device=z.device))
        H = -plogp.sum(-1)
        on = (tok >= 0).to(f)
        rows = torch.arange(len(tok), device=z.device)
        one = {"logprobs": torch.where(tok >= 0, logp[rows, tok.clamp(min=0)], 0.0), "entropy": H,
               "lse": lse}
        if case["op"] == "logp_train":
            dl = s["dlogprobs"][lo:lo + 512].to(f) * on
            dH = s["dentropy"][lo:lo + 512].to(f)
            # d logp(tok) / d z = 1[tok] - p,  dH / d z = -p (logp + H)
            g = -dl[:, None] * p - dH[:, None] * (plogp + p * H[:, None])
            g[rows, tok.clamp(min=0)] += dl
            one["dlogits"] = s["scale"] * g
        if case["top"]:
            k = min(case["top"], case["vocab"])
            one["top_logprobs"] = torch.nn.functional.pad(
                logp.topk(k, -1).values, (0, case["top"] - k), value=-math.inf)
            one["top_tokens"] = None
        parts.append(one)
    return {n: None if parts[0][n] is None else torch.cat([p[n] for p in parts]) for n in parts[0]}


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    op = case["op"]
    if op in ("logp", "logp_train"):
        return _exact_logp(case, s)
    if op == "matmul":
        out = (s["a"].to(f) @ s["w"].to(f).t()) * s["a_scales"].to(f)[:, None] * s["w_scales"].to(f)
        return {"out": out if s["bias"] is None else out + s["bias"].to(f)}
    # the norm reads the value that the residual stream holds
    h = (s["x"].to(f) + s["residual"].to(f)).to(s["residual"].dtype).to(f)
    w = s["weight"].to(f)
    r = 1.0 / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / h.shape[-1] + s["eps"])
    out = h * r * w
    if op == "norm8":
        scales = out.abs().amax(-1) / TOP[case["form"]]
        return {"h": h, "codes": out / scales[:, None], "scales": scales}
    if op == "proj":
        scales = out.abs().amax(-1, keepdim=True) / TOP[case["form"]]
        codes = out / scales
        codes = torch.round(codes) if case["form"] == "int8" else codes.to(torch.float8_e4m3fn).to(f)
        return {"h": h, "out": scales * (codes @ s["w"].to(f).t()) * s["w_scales"].to(f)}
    do, dh = s["dout"].to(f), s["dh"].to(f)
    n = h * r
    proj = (do * w * n).sum(-1, keepdim=True) / h.shape[-1]
    dh = dh + r * (do * w - proj * n)
    return {"h": h, "out": out, "dx": dh, "dresidual": dh, "dweight": (do * n).sum(0)}
