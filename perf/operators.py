"""Cases and plain forms of the delta-rule operators: the gated delta rule over
whole sequences (forward, and forward with its gradient), its recurrent form
for single and drafted tokens, the verification of drafted tokens, and the
8-bit cache of recurrent states.

Every case is one pass through one operator.  ``run`` computes it with
elementary torch operations in 32 bits (``own`` false) or through this
repository's entry points (``own`` true); ``exact`` computes it in 64 bits from
the operator's definition, token by token.

The gated delta rule, per batch row and head, with a state S of headdim x
dstate values, decay a_t = exp(g_t) and a writing strength beta_t:

    S'  = a_t S_{t-1}
    u_t = beta_t (v_t - S' k_t)
    S_t = S' + u_t (outer) k_t
    y_t = scale * S_t q_t

A token whose seq_idx differs from its predecessor's starts from S' = 0.
Head h reads group floor(h * ngroups / nheads) of q and k.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def _delta(name, op, b, L, H, P, N, G, dtype, nseq=1, carry=False):
    return dict(name=name, op=op, batch=b, seqlen=L, nheads=H, headdim=P, dstate=N, ngroups=G,
                dtype=dtype, nseq=nseq, carry=carry)


def listed():
    return [
        # a training batch's forward, or a batched prefill: the layer workload this
        # repository's benchmark is quoted on
        _delta("fwd_b2_L8192_bf16", "fwd", 2, 8192, 64, 64, 128, 8, "bf16"),
        # one prompt of an odd length that continues a cached state: few chains
        _delta("fwd_prompt_L4001_bf16", "fwd", 1, 4001, 32, 64, 128, 1, "bf16", carry=True),
        # the smallest layer, in fp32: one short row, latency counts
        _delta("fwd_tiny_L256_fp32", "fwd", 1, 256, 4, 16, 16, 1, "f32", carry=True),
        # a training step on the same workload (forward and all gradients)
        _delta("train_b2_L8192_bf16", "train", 2, 8192, 64, 64, 128, 8, "bf16"),
        # sixteen sequences of odd lengths packed into one row
        _delta("train_packed_L20011_bf16", "train", 1, 20011, 64, 64, 64, 4, "bf16", nseq=16),
        # an fp32 step at odd head sizes, as a numerical check of a model runs it
        _delta("train_odd_L1000_fp32", "train", 2, 1000, 6, 40, 56, 3, "f32", carry=True),
        # token generation: one token for each sequence of a serving batch
        dict(name="step_b64_T1_bf16", op="step", batch=64, tokens=1, nheads=64, headdim=64,
             dstate=128, ngroups=8, dtype="bf16", ragged=False),
        # a small batch advanced by the accepted ones of its drafted tokens
        dict(name="step_b4_T5_bf16", op="step", batch=4, tokens=5, nheads=48, headdim=64,
             dstate=16, ngroups=1, dtype="bf16", ragged=True),
        # drafted tokens of a few sequences: latency counts
        dict(name="verify_b4_K4_fp32", op="verify", batch=4, draft=4, vocab=32000, dtype="f32"),
        # a large serving batch with a large odd vocabulary and unequal drafts
        dict(name="verify_b128_K6_bf16", op="verify", batch=128, draft=6, vocab=100003,
             dtype="bf16"),
        # the states of a batch's prefixes put away in 8 bits and taken out again
        dict(name="cache_b64_int8", op="cache", batch=64, nheads=64, headdim=64, dstate=128,
             form="int8"),
        # one small layer's states, odd sizes
        dict(name="cache_b3_e4m3", op="cache", batch=3, nheads=48, headdim=40, dstate=72,
             form="e4m3"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["fwd", "fwd", "train", "train", "step", "verify", "cache"])
    if op in ("fwd", "train"):
        G = rng.choice([1, 2, 3, 4, 8])
        if rng.random() < 0.7:      # bf16 at the head sizes that layers use
            P, N = rng.choice([64, 64, 128]), rng.choice([64, 128])
            H = G * rng.choice([1, 2, 4, 8])
            dtype, most, longest = "bf16", 2 * 8192 * 64, 16384
        else:                       # fp32, any head size
            P, N, H = rng.randint(1, 128), rng.randint(1, 128), G * rng.choice([1, 2, 3])
            dtype, most, longest = "f32", 2 * 1000 * 16, 2048
        L = _logint(rng, 1, longest)
        b = _logint(rng, 1, 8)
        while b * L * H * P * N > most * 64 * 128:
            b, L = max(1, b // 2), max(1, L // 2 + 1)
        nseq = rng.randint(2, 8) if L >= 64 and rng.random() < 0.3 else 1
        case = _delta("", op, b, L, H, P, N, G, dtype, nseq=nseq, carry=rng.random() < 0.5)
        del case["name"]
        return case
    if op == "step":
        G = rng.choice([1, 2, 4, 8])
        return dict(op=op, batch=_logint(rng, 1, 64), tokens=rng.choice([1, 1, 2, 3, 5, 8]),
                    nheads=G * rng.choice([1, 2, 4, 8]), headdim=rng.choice([16, 40, 64, 128]),
                    dstate=rng.choice([16, 57, 64, 128]), ngroups=G,
                    dtype=rng.choice(["bf16", "f32"]), ragged=rng.random() < 0.5)
    if op == "verify":
        return dict(op=op, batch=_logint(rng, 1, 128), draft=rng.randint(1, 6),
                    vocab=_logint(rng, 300, 100003), dtype=rng.choice(["bf16", "f32"]))
    return dict(op=op, batch=_logint(rng, 1, 64), nheads=_logint(rng, 1, 64),
                headdim=rng.choice([16, 40, 64]), dstate=rng.choice([16, 57, 64, 128]),
                form=rng.choice(["int8", "e4m3"]))


# ---------------------------------------------------------------------------
# What a program has in hand before the call
# ---------------------------------------------------------------------------
def _dtype(case):
    return BF16 if case["dtype"] == "bf16" else F32


def _gates(gen, b, L, H, dt):
    """Log decays -A * softplus(raw + bias) and strengths sigmoid(raw), drawn
    as a selective layer's: A in [1, 16], time steps around 1e-3 .. 1e-1."""
    r = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    A = torch.exp(r(H) * math.log(16.0))
    target = torch.exp(math.log(1e-3) + r(H) * math.log(100.0))
    bias = torch.log(torch.expm1(target))
    g = -A * torch.nn.functional.softplus(n(b, L, H) + bias)
    return g.to(dt), torch.sigmoid(n(b, L, H)).to(dt)


def _unit(gen, *shape):
    """Rows of unit length through a SiLU, as keys and queries come from a
    layer's convolution: they are correlated."""
    x = torch.nn.functional.silu(torch.randn(shape, generator=gen, device="cuda"))
    return x / (x.norm(dim=-1, keepdim=True) + 1e-6)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    u = lambda *s: torch.rand(s, generator=gen, device="cuda")  # noqa: E731
    op = case["op"]
    s = {"case": dict(case)}
    if op in ("fwd", "train", "step"):
        dt = _dtype(case)
        b, H, P, N, G = (case[k] for k in ("batch", "nheads", "headdim", "dstate", "ngroups"))
        L = case["tokens"] if op == "step" else case["seqlen"]
        s["q"], s["k"] = _unit(gen, b, L, G, N).to(dt), _unit(gen, b, L, G, N).to(dt)
        s["v"] = n(b, L, H, P).to(dt)
        s["g"], s["beta"] = _gates(gen, b, L, H, dt)
        s["scale"] = 1.0 / math.sqrt(N)
        if op == "step":
            s["states"] = 0.1 * n(b, H, P, N)
            s["slots"] = torch.randperm(b, generator=gen, device="cuda").to(torch.int32)
            s["lengths"] = None
            if case["ragged"]:
                s["lengths"] = torch.randint(0, L + 1, (b,), generator=gen, device="cuda",
                                             dtype=torch.int32)
            return s
        # a bf16 layer hands its states over in bf16: its products round to it
        s["init"] = (0.1 * n(b, H, P, N)).to(dt) if case["carry"] else None
        s["seq_idx"] = None
        if case["nseq"] > 1:
            cuts = torch.rand(b, L, generator=gen, device="cuda")
            cuts[:, 0] = -1.0
            starts = torch.zeros(b, L, dtype=torch.int32, device="cuda")
            starts.scatter_(1, cuts.topk(case["nseq"] - 1, dim=1).indices, 1)
            s["seq_idx"] = torch.cumsum(starts, 1).to(torch.int32)
        if op == "train":
            s["dy"] = n(b, L, H, P).to(dt)
        return s
    if op == "verify":
        b, K, V, dt = case["batch"], case["draft"], case["vocab"], _dtype(case)
        logits = 2.0 * n(b, K + 1, V)
        s["target"] = torch.softmax(logits, -1).to(dt)
        draft = torch.softmax(logits[:, :K] + 0.7 * n(b, K, V), -1)
        race = torch.empty(b, K, V, device="cuda").exponential_(generator=gen)
        s["tokens"] = (draft / race).argmax(-1).to(torch.int32)
        s["draft"] = draft.to(dt)
        s["lengths"] = torch.randint(0, K + 1, (b,), generator=gen, device="cuda",
                                     dtype=torch.int32)
        s["uniform"] = u(b, K)
        s["noise"] = torch.empty(b, V, device="cuda").exponential_(generator=gen)
        return s
    b, H, P, N = (case[k] for k in ("batch", "nheads", "headdim", "dstate"))
    # rows of very different sizes: a state's rows decay at their heads' rates
    s["states"] = n(b, H, P, N) * torch.exp(2.0 * n(b, H, P, 1))
    s["slots"] = torch.randperm(b, generator=gen, device="cuda").to(torch.int32)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
CHUNK = 64


def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular A by halves:
    [[X, 0], [C, Y]]^-1 = [[X', 0], [-Y' C X', Y']]."""
    n = A.shape[-1]
    if n == 1:
        return torch.ones_like(A)
    h = n // 2
    both = _unit_lower_inverse(torch.stack((A[..., :h, :h], A[..., h:, h:])))
    low = -(both[1] @ A[..., h:, :h] @ both[0])
    return torch.cat((torch.cat((both[0], torch.zeros_like(low)), -1),
                      torch.cat((low, both[1]), -1)), -2)


def _plain_delta(q, k, v, g, beta, scale, init, seq_idx):
    """y (b, L, H, P) and the last state (b, H, P, N) in fp32, chunk by chunk:
    inside a chunk the written vectors solve a triangular system, and the state
    goes from chunk to chunk."""
    b, L, H, P = v.shape
    G, N = k.shape[2:]
    C, nc = CHUNK, -(-L // CHUNK)
    pad = nc * C - L

    def lay(x, heads):      # (b, L, heads, d) -> (b, H, nc, C, d)
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad))
        x = x.reshape(b, nc, C, heads, -1).permute(0, 3, 1, 2, 4)
        return x.repeat_interleave(H // heads, 1)

    q, k, v = lay(q, G), lay(k, G), lay(v, H)
    g, beta = lay(g[..., None], H)[..., 0], lay(beta[..., None], H)[..., 0]
    seg = torch.zeros(b, 1, nc, C, dtype=torch.int32, device=v.device)
    if seq_idx is not None:
        new = torch.zeros(b, nc * C, dtype=torch.int32, device=v.device)
        new[:, 1:L] = (seq_idx[:, 1:] != seq_idx[:, :-1]).to(torch.int32)
        seg = torch.cumsum(new.reshape(b, 1, nc, C), -1)
    gam = torch.cumsum(g, -1)
    low = torch.ones(C, C, dtype=torch.bool, device=v.device).tril()
    pair = low & (seg[..., :, None] == seg[..., None, :])
    E = torch.exp(torch.where(pair, gam[..., :, None] - gam[..., None, :], -math.inf))
    into = torch.exp(torch.where(seg == 0, gam, -math.inf))
    out = torch.exp(torch.where(seg == seg[..., -1:], gam[..., -1:] - gam, -math.inf))
    M = (k @ k.transpose(-1, -2) * E).tril(-1)
    T = _unit_lower_inverse(M * beta[..., None, :])
    W, U = T @ (into[..., None] * k), T @ v
    A = (q @ k.transpose(-1, -2)) * E * beta[..., None, :]
    kd, qi = k * (out * beta)[..., None], q * into[..., None]
    S = v.new_zeros(b, H, N, P) if init is None else init.transpose(-1, -2)
    ys = []
    for c in range(nc):     # each chunk's state is the next one's start
        u = U[:, :, c] - W[:, :, c] @ S
        ys.append(qi[:, :, c] @ S + A[:, :, c] @ u)
        S = into[:, :, c, -1, None, None] * S + kd[:, :, c].transpose(-1, -2) @ u
    y = scale * torch.stack(ys, 2).permute(0, 2, 3, 1, 4).reshape(b, nc * C, H, P)[:, :L]
    return y, S.transpose(-1, -2)


def _plain_step(s):
    c = s["case"]
    hpg = c["nheads"] // c["ngroups"]
    q, k = (s[x].float().repeat_interleave(hpg, 2) for x in ("q", "k"))
    v, g, beta = s["v"].float(), s["g"].float(), s["beta"].float()
    S = s["states"][s["slots"].long()]
    kept = S
    ys = []
    for t in range(c["tokens"]):    # the recurrence itself
        S = torch.exp(g[:, t, :, None, None]) * S
        u = beta[:, t, :, None] * (v[:, t] - (S * k[:, t, :, None]).sum(-1))
        S = S + u[..., None] * k[:, t, :, None]
        ys.append(s["scale"] * (S * q[:, t, :, None]).sum(-1))
        on = True if s["lengths"] is None else (s["lengths"] > t)[:, None, None, None]
        kept = S if on is True else torch.where(on, S, kept)
    states = torch.empty_like(s["states"])
    states[s["slots"].long()] = kept
    return {"y": torch.stack(ys, 1).to(s["v"].dtype), "states": states}


def _plain_verify(s):
    p, d, tok = s["target"].float(), s["draft"].float(), s["tokens"].long()
    b, K, V = d.shape
    at = torch.arange(K, device=p.device)
    pt = p[:, :K].gather(2, tok[..., None])[..., 0]
    dt = d.gather(2, tok[..., None])[..., 0]
    ok = (s["uniform"] * dt < pt) & (at < s["lengths"][:, None])
    acc = torch.cumprod(ok.to(torch.int32), 1).sum(1)
    rows = torch.arange(b, device=p.device)
    target = p[rows, acc]
    drafted = torch.where((acc < s["lengths"])[:, None], d[rows, acc.clamp(max=K - 1)], 0.0)
    w = (target - drafted).clamp(min=0.0)
    w = torch.where((w > 0).any(1, keepdim=True), w, target)
    score = w / s["noise"]
    best = torch.where(score == score.amax(1, keepdim=True), torch.arange(V, device=p.device), V)
    out = torch.where(at[None] < acc[:, None], tok, -1)
    out = torch.cat((out, torch.full_like(out[:, :1], -1)), 1)
    out[rows, acc] = best.amin(1)
    return {"accepted": acc.to(torch.int32), "tokens": out.to(torch.int32)}


TOP = {"int8": 127.0, "e4m3": 448.0}


def _plain_cache(s):
    x, top = s["states"], TOP[s["case"]["form"]]
    big = x.abs().amax(-1, keepdim=True)
    y = x * (top / big)
    y = torch.round(y) if s["case"]["form"] == "int8" else y.to(torch.float8_e4m3fn).float()
    scales = big / top
    put = torch.empty_like(scales[..., 0])
    put[s["slots"].long()] = scales[..., 0]
    return {"scales": put, "states": y * scales}


def _plain(s):
    op = s["case"]["op"]
    if op == "step":
        return _plain_step(s)
    if op == "verify":
        return _plain_verify(s)
    if op == "cache":
        return _plain_cache(s)
    dt = s["v"].dtype
    wide = [s[x].float() for x in ("q", "k", "v", "g", "beta")]
    init = None if s["init"] is None else s["init"].float()
    if op == "fwd":
        y, S = _plain_delta(*wide, s["scale"], init, s["seq_idx"])
        return {"y": y.to(dt), "final": S.to(dt)}
    leaves = [x.requires_grad_() if x is not o else x.clone().requires_grad_()
              for x, o in zip(wide, (s[x] for x in ("q", "k", "v", "g", "beta")))]
    names = ["dq", "dk", "dv", "dg", "dbeta"]
    if init is not None:
        init = init.clone().requires_grad_()
        leaves.append(init)
        names.append("dinit")
    y, _ = _plain_delta(*leaves[:5], s["scale"], init, s["seq_idx"])
    grads = torch.autograd.grad(y, leaves, s["dy"].float())
    return {"y": y.detach().to(dt), **{n: x.to(dt) for n, x in zip(names, grads)}}


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------
def _own(s):
    from mamba_selective_state_gb300 import runner
    op, dev = s["case"]["op"], s.get("dev")
    if op in ("fwd", "train"):
        if dev is None:
            dev = s["dev"] = runner.DeltaDevice(
                s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], initial_states=s["init"],
                seq_idx=s["seq_idx"], dy=s.get("dy"), state_dtype=s["v"].dtype)
        dev.fwd()
        if op == "fwd":
            return {"y": dev.y, "final": dev.final}
        dev.bwd()
        out = {"y": dev.y, "dq": dev.dq, "dk": dev.dk, "dv": dev.dv, "dg": dev.dg,
               "dbeta": dev.dbeta}
        if s["init"] is not None:
            out["dinit"] = dev.dinit
        return out
    if op == "step":
        if dev is None:
            dev = s["dev"] = runner.DeltaStepDevice(s["states"], torch.empty_like(s["states"]))
        y = dev.step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["scale"], slots=s["slots"],
                     lengths=s["lengths"])
        return {"y": y, "states": dev.states_out}
    if op == "verify":
        tokens, accepted = runner.verify_draft(s["target"], s["draft"], s["tokens"], s["uniform"],
                                               s["noise"], lengths=s["lengths"])
        return {"accepted": accepted, "tokens": tokens}
    if dev is None:
        c = s["case"]
        dev = s["dev"] = runner.StateCache(c["batch"], c["nheads"], c["headdim"], c["dstate"],
                                           c["form"])
        s["out"] = torch.empty_like(s["states"])
    dev.store(s["states"], s["slots"])
    dev.load(s["slots"], s["out"])
    return {"scales": dev.scales, "states": s["out"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# Bytes and operations that a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op in ("fwd", "train", "step"):
        e = 2 if case["dtype"] == "bf16" else 4
        b, H, P, N, G = (case[k] for k in ("batch", "nheads", "headdim", "dstate", "ngroups"))
        L = case["tokens"] if op == "step" else case["seqlen"]
        qk, v, gates, st = b * L * G * N * e, b * L * H * P * e, b * L * H * e, b * H * P * N
        fwd = 2 * qk + 2 * v + 2 * gates        # q, k, v, g, beta in, y out
        # per token and head: S' k, u k, S q
        flops = 3 * 2 * b * L * H * P * N
        if op == "step":
            return {"bytes": fwd + 2 * st * 4, "flops": flops}
        carry = st * e if case["carry"] else 0
        if op == "fwd":
            return {"bytes": fwd + carry + st * e, "flops": flops}
        # the backward reads q, k, v, g, beta, dy and writes dq, dk, dv, dg, dbeta
        bwd = 4 * qk + 3 * v + 4 * gates + 2 * carry
        return {"bytes": fwd + carry + bwd, "flops": 3 * flops}
    if op == "verify":
        e = 2 if case["dtype"] == "bf16" else 4
        b, K, V = case["batch"], case["draft"], case["vocab"]
        # one row of each distribution and of the noise for each sequence
        return {"bytes": b * V * (2 * e + 4) + b * K * (2 * e + 8), "flops": 2 * b * V}
    n = case["batch"] * case["nheads"] * case["headdim"]
    # the states in, 8 bits and scales out; those in again, the states out
    return {"bytes": 2 * n * (case["dstate"] * 5 + 4), "flops": 4 * n * case["dstate"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_token(S, q, k, v, a, beta):
    """One token of the recurrence: the decayed state, the error it corrects,
    and the state after it."""
    S1 = a[..., None, None] * S
    err = v - torch.einsum("bhpn,bhn->bhp", S1, k)
    return S1, err, S1 + (beta[..., None] * err)[..., None] * k[..., None, :]


def _exact_delta(case, s):
    f = torch.float64
    hpg = case["nheads"] // case["ngroups"]
    q, k = (s[x].to(f).repeat_interleave(hpg, 2) for x in ("q", "k"))
    v, g, beta = (s[x].to(f) for x in ("v", "g", "beta"))
    b, L, H, P = v.shape
    N, scale = q.shape[-1], s["scale"]
    a = torch.exp(g)
    if s["seq_idx"] is not None:
        a[:, 1:] *= (s["seq_idx"][:, 1:] == s["seq_idx"][:, :-1])[..., None]
    start = torch.zeros(b, H, P, N, dtype=f, device=v.device)
    if s["init"] is not None:
        start += s["init"].to(f)
    S, y, marks, every = start, torch.empty_like(v), [], 64
    for t in range(L):
        if t % every == 0:
            marks.append(S)
        _, _, S = _exact_token(S, q[:, t], k[:, t], v[:, t], a[:, t], beta[:, t])
        y[:, t] = scale * torch.einsum("bhpn,bhn->bhp", S, q[:, t])
    if case["op"] == "fwd":
        return {"y": y, "final": S}
    dy = s["dy"].to(f)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg, dbeta = torch.empty_like(g), torch.empty_like(beta)
    D = torch.zeros_like(start)     # the gradient of S_t
    for c in range(len(marks) - 1, -1, -1):
        lo, hi = c * every, min(L, (c + 1) * every)
        S, path = marks[c], []
        for t in range(lo, hi):
            S1, err, S2 = _exact_token(S, q[:, t], k[:, t], v[:, t], a[:, t], beta[:, t])
            path.append((S, S1, err, S2))
            S = S2
        for t in range(hi - 1, lo - 1, -1):
            S0, S1, err, S2 = path.pop()
            D = D + scale * dy[:, t, ..., None] * q[:, t, :, None]
            dq[:, t] = scale * torch.einsum("bhpn,bhp->bhn", S2, dy[:, t])
            du = torch.einsum("bhpn,bhn->bhp", D, k[:, t])
            derr = beta[:, t, :, None] * du
            dbeta[:, t] = (err * du).sum(-1)
            dv[:, t] = derr
            dk[:, t] = (torch.einsum("bhpn,bhp->bhn", D, beta[:, t, :, None] * err)
                        - torch.einsum("bhpn,bhp->bhn", S1, derr))
            D = D - derr[..., None] * k[:, t, :, None]
            dg[:, t] = a[:, t] * (D * S0).sum((-1, -2))
            D = a[:, t, :, None, None] * D
    G = case["ngroups"]
    out = {"y": y, "dq": dq.reshape(b, L, G, hpg, N).sum(3), "dk": dk.reshape(b, L, G, hpg, N).sum(3),
           "dv": dv, "dg": dg, "dbeta": dbeta}
    if s["init"] is not None:
        out["dinit"] = D
    return out


def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None         # whole numbers: they are compared as they are
    s = prepare(case, seed)
    f = torch.float64
    if op in ("fwd", "train"):
        return _exact_delta(case, s)
    if op == "step":
        hpg = case["nheads"] // case["ngroups"]
        q, k = (s[x].to(f).repeat_interleave(hpg, 2) for x in ("q", "k"))
        v, a, beta = s["v"].to(f), torch.exp(s["g"].to(f)), s["beta"].to(f)
        states, y = s["states"].to(f), torch.empty_like(v)
        for i in range(case["batch"]):      # sequence by sequence
            slot = int(s["slots"][i])
            S = states[slot][None]
            last = case["tokens"] if s["lengths"] is None else int(s["lengths"][i])
            for t in range(case["tokens"]):
                _, _, S = _exact_token(S, q[i:i + 1, t], k[i:i + 1, t], v[i:i + 1, t],
                                       a[i:i + 1, t], beta[i:i + 1, t])
                y[i, t] = s["scale"] * torch.einsum("bhpn,bhn->bhp", S, q[i:i + 1, t])[0]
                if t + 1 == last:
                    states[slot] = S[0]
        return {"y": y, "states": states}
    # the stored values follow from the scales; the scales have an exact value
    x = s["states"].to(f)
    scales = torch.empty(x.shape[:3], dtype=f, device=x.device)
    scales[s["slots"].long()] = x.abs().amax(-1) / TOP[case["form"]]
    return {"scales": scales, "states": None}
