"""Float64 oracle of the gated delta rule, token by token, with its reverse
mode derived by hand, and the definitions of the draft verification and of the
8-bit state cache.  Test infrastructure only; shares no code with csrc/.

Shapes as in include/ssd.h: q, k (b, L, G, N), v (b, L, H, P), g, beta
(b, L, H), states (b, H, P, N), seq_idx (b, L).
"""
from __future__ import annotations

import numpy as np


def _heads(x, H):
    """(b, L, G, N) -> (b, L, H, N): head h reads group floor(h * G / H)."""
    G = x.shape[2]
    return x[:, :, (np.arange(H) * G) // H]


def _decay(g, seq_idx):
    a = np.exp(g)
    if seq_idx is not None:
        a[:, 1:][seq_idx[:, 1:] != seq_idx[:, :-1]] = 0.0
    return a


def delta_fwd(q, k, v, g, beta, scale, initial_states=None, seq_idx=None, states=False):
    """y (b, L, H, P) and the final state; with ``states`` also the list of
    the states before every token."""
    b, L, H, P = v.shape
    q, k, a = _heads(q, H), _heads(k, H), _decay(g, seq_idx)
    S = np.zeros((b, H, P, q.shape[-1])) if initial_states is None else initial_states.copy()
    y, path = np.empty_like(v), []
    for t in range(L):
        path.append(S)
        S1 = a[:, t, :, None, None] * S
        w = v[:, t] - np.einsum("bhpn,bhn->bhp", S1, k[:, t])
        S = S1 + np.einsum("bhp,bhn->bhpn", beta[:, t, :, None] * w, k[:, t])
        y[:, t] = scale * np.einsum("bhpn,bhn->bhp", S, q[:, t])
    return (y, S, path) if states else (y, S)


def delta_bwd(q, k, v, g, beta, scale, dy, initial_states=None, seq_idx=None, dfinal_states=None):
    """Gradients of sum(y * dy) + sum(final * dfinal)."""
    b, L, H, P = v.shape
    G, N = q.shape[2:]
    _, _, path = delta_fwd(q, k, v, g, beta, scale, initial_states, seq_idx, states=True)
    qh, kh, a = _heads(q, H), _heads(k, H), _decay(g, seq_idx)
    dq, dk = np.zeros((b, L, H, N)), np.zeros((b, L, H, N))
    dv, dg, dbeta = np.zeros_like(v), np.zeros_like(g), np.zeros_like(beta)
    D = np.zeros((b, H, P, N)) if dfinal_states is None else dfinal_states.copy()
    for t in range(L - 1, -1, -1):
        at, bt = a[:, t, :, None, None], beta[:, t, :, None]
        S1 = at * path[t]
        w = v[:, t] - np.einsum("bhpn,bhn->bhp", S1, kh[:, t])
        S2 = S1 + np.einsum("bhp,bhn->bhpn", bt * w, kh[:, t])
        D = D + scale * np.einsum("bhp,bhn->bhpn", dy[:, t], qh[:, t])
        dq[:, t] = scale * np.einsum("bhpn,bhp->bhn", S2, dy[:, t])
        du = np.einsum("bhpn,bhn->bhp", D, kh[:, t])
        dbeta[:, t] = (du * w).sum(-1)
        dw = bt * du
        dv[:, t] = dw
        dk[:, t] = (np.einsum("bhpn,bhp->bhn", D, bt * w) - np.einsum("bhpn,bhp->bhn", S1, dw))
        D1 = D - np.einsum("bhp,bhn->bhpn", dw, kh[:, t])
        dg[:, t] = (D1 * S1).sum((-1, -2))
        D = at * D1
    fold = lambda x: x.reshape(b, L, G, H // G, N).sum(3)  # noqa: E731
    return dict(dq=fold(dq), dk=fold(dk), dv=dv, dg=dg, dbeta=dbeta, dinitial_states=D)


def verify_draft(target, draft, tokens, uniform, noise, lengths=None):
    """The kept tokens and the next one, by the definition's fp32 comparisons
    and ratios.  draft may be None."""
    f = np.float32
    b, K1, V = target.shape
    K = K1 - 1
    out, accepted = np.full((b, K1), -1, np.int32), np.zeros(b, np.int32)
    for i in range(b):
        n = K if lengths is None else min(max(int(lengths[i]), 0), K)
        kept = 0
        while kept < n:
            x = int(tokens[i, kept])
            if not 0 <= x < V:
                break
            qv = f(1) if draft is None else f(draft[i, kept, x])
            if not f(uniform[i, kept]) * qv < f(target[i, kept, x]):
                break
            kept += 1
        p = target[i, kept].astype(f)
        w = p.copy()
        if kept < n:
            if draft is not None:
                w = p - draft[i, kept].astype(f)
            elif 0 <= int(tokens[i, kept]) < V:
                w[int(tokens[i, kept])] -= f(1)
        out[i, :kept] = tokens[i, :kept]
        out[i, kept] = 0
        for weights in (w, p):
            with np.errstate(all="ignore"):
                r = np.where(weights > 0, weights / noise[i].astype(f), f(0))
            r = np.where(r > 0, r, f(0))        # NaN ratios are passed over
            if r.max() > 0:
                out[i, kept] = int(np.argmax(r))
                break
        accepted[i] = kept
    return out, accepted


def e4m3_values():
    """The finite values of the 8-bit format (sign, 4-bit exponent of bias 7,
    3-bit mantissa; all ones is NaN), by code."""
    v = np.full(256, np.nan)
    for code in range(256):
        s, e, m = code >> 7, (code >> 3) & 15, code & 7
        if e == 15 and m == 7:
            continue
        v[code] = (-1.0) ** s * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return v


def cache_roundtrip(states, form):
    """What a state reads back as, and the rows' scales, both fp32."""
    f = np.float32
    top = f(127) if form == "int8" else f(448)
    x = states.astype(f)
    with np.errstate(all="ignore"):
        big = np.abs(x).max(-1, keepdims=True)
        bad = ~np.isfinite(x).all(-1, keepdims=True)
        empty = ~(big >= f(2.0 ** -118))
        y = (x * np.where(empty, f(0), (f(1) / big) * top)).astype(f)
        scale = np.where(bad, f(np.nan), np.where(empty, f(0), big * (f(1) / top))).astype(f)
    y = np.where(bad, f(0), y)
    if form == "int8":
        y = np.clip(np.rint(y), -127, 127)
    else:   # nearest finite value, ties to the even code
        vals = e4m3_values()
        pos = vals[:127]
        mag = np.abs(y).astype(np.float64)
        hi = np.clip(np.searchsorted(pos, mag), 1, 126)
        lo = hi - 1
        dl, dh = mag - pos[lo], pos[hi] - mag
        code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
        y = np.sign(y) * pos[code]
    return (y.astype(f) * scale).astype(f), scale[..., 0]
