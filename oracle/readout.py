"""Float64 oracle of the operators between the residual stream and a model's
answer: the norm that takes in the residual (with its 8-bit output and its
gradient), the product of 8-bit codes, and the tokens' log probabilities.

TEST INFRASTRUCTURE ONLY (see the package docstring).  Plain numpy, from the
definitions:

    v = x + residual (as the stream stores it),  r = 1 / sqrt(mean v^2 + eps)
    out = v r w
    L = <dout, out> + <dh, v>:  dv = dh + r (g - n mean(g n)),  g = dout w, n = v r
    out[m, n] = as[m] ws[n] sum_k a[m, k] w[n, k] + bias[n]
    z = scale logits,  lse = log sum exp z,  H = -sum p log p
    L = <dlp, z[tok] - lse> + <dH, H>:  dz = dlp (1[tok] - p) - dH p (log p + H)
"""
from __future__ import annotations

import numpy as np

from .delta import e4m3_values

TOP = {"int8": 127.0, "e4m3": 448.0}


def add_rmsnorm_fwd(h, weight, eps):
    """(out, rstd) of the stored h (rows, dim)."""
    h = np.asarray(h, np.float64)
    with np.errstate(all="ignore"):
        r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
        return h * r * weight, r


def add_rmsnorm_bwd(h, weight, eps, dout, dh=None):
    """(dh in all, dweight)."""
    h = np.asarray(h, np.float64)
    _, r = add_rmsnorm_fwd(h, weight, eps)
    n, g = h * r, dout * weight
    d = r * (g - n * (g * n).mean(-1, keepdims=True))
    return (d if dh is None else d + dh), (dout * n).sum(0)


def code_values(codes, form):
    """What codes (uint8 bytes, or int8) stand for, without their scale."""
    if form == "int8":
        return codes.view(np.int8).astype(np.float64)
    return e4m3_values()[codes.view(np.uint8)]


def half_steps(values, form):
    """Half the distance between neighbouring codes at a value in units of the
    scale: the most that rounding may be off."""
    if form == "int8":
        return np.full_like(values, 0.5)
    e = np.floor(np.log2(np.maximum(np.abs(values), 2.0 ** -6)))
    return 2.0 ** (e - 4)


def scaled_matmul(a, a_scales, w, w_scales, bias=None):
    """a, w: the codes' values."""
    with np.errstate(all="ignore"):
        out = (a @ w.T) * a_scales[:, None] * w_scales
    return out if bias is None else out + bias


def token_logprobs(logits, tokens, scale=1.0, ntop=0):
    """dict of logprobs, entropy, lse and, with ntop, top_tokens and
    top_logprobs, by the header's rules for what is excluded or not finite."""
    x = np.asarray(logits, np.float64)
    rows, V = x.shape
    out = dict(logprobs=np.zeros(rows), entropy=np.zeros(rows), lse=np.zeros(rows))
    if ntop:
        out["top_tokens"] = np.full((rows, ntop), -1, np.int64)
        out["top_logprobs"] = np.full((rows, ntop), -np.inf)
    for i in range(rows):
        t = int(tokens[i]) if tokens is not None else -1
        known = 0 <= t < V
        words = [v for v in np.argsort(-x[i], kind="stable") if x[i, v] > -np.inf][:ntop] if ntop else []
        if np.isnan(x[i]).any() or (x[i] == np.inf).any():
            m = ln = lse = H = lp = np.nan
        elif (x[i] == -np.inf).all():
            m = ln = lse = lp = -np.inf
            H = 0.0
        else:
            z = scale * x[i]
            m = z.max()
            ln = np.log(np.exp(z - m).sum())
            lse = m + ln        # (where z is huge, this does not hold ln)
            on = z > -np.inf
            H = -(np.exp(z[on] - m - ln) * (z[on] - m - ln)).sum()
            lp = z[t] - m - ln if known else 0.0
        out["lse"][i], out["entropy"][i], out["logprobs"][i] = lse, H, lp if known else 0.0
        for j, v in enumerate(words):
            out["top_tokens"][i, j] = v
            out["top_logprobs"][i, j] = scale * x[i, v] - m - ln
    return out


def token_logprobs_bwd(logits, tokens, scale, dlogprobs=None, dentropy=None):
    x = np.asarray(logits, np.float64)
    rows, V = x.shape
    f = token_logprobs(x, tokens, scale)
    d = np.zeros_like(x)
    for i in range(rows):
        t = int(tokens[i]) if tokens is not None and dlogprobs is not None else -1
        dl = float(dlogprobs[i]) if 0 <= t < V else 0.0
        dH = float(dentropy[i]) if dentropy is not None else 0.0
        if f["lse"][i] == -np.inf or (not 0 <= t < V and dH == 0):
            continue                # nothing is left, or nothing comes in
        if np.isnan(f["lse"][i]):
            d[i] = np.nan
            continue
        lp = np.maximum(scale * x[i] - f["lse"][i], -1e4)
        p = np.exp(lp)
        d[i] = -p * (dl + dH * (lp + f["entropy"][i]))
        if 0 <= t < V:
            d[i, t] += dl
    return scale * d
