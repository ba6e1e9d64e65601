"""Float64 reference of a calibration pass's operators: rotary positions, attention
over packed prompts with its gradients, log probabilities of tokens with theirs.
Plain loops and the definitions; used by tests only."""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------- rotary positions

def frequencies(dim, base, scaling="plain", factor=1.0, original=0.0, low=1.0, high=4.0):
    out = []
    for i in range(dim // 2):
        w = base ** (-2.0 * i / dim)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "parts":
            keep = (original * w / (2 * math.pi) - low) / (high - low)
        elif scaling == "index":
            at = [dim * math.log(original / (2 * math.pi * r)) / (2 * math.log(base)) for r in (high, low)]
            a, b = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
            keep = 1 - (i - a) / max(b - a, 0.001)
        keep = min(max(keep, 0.0), 1.0)
        out.append(keep * w + (1 - keep) * w / factor)
    return np.array(out)


def tables(first, positions, f, magnitude=1.0):
    angle = np.arange(first, first + positions, dtype=np.longdouble)[:, None] * f.astype(np.longdouble)
    return np.cos(angle) * magnitude, np.sin(angle) * magnitude


def pairs(rot, neighbours):
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if neighbours else (i, i + rot // 2)


def rotate(x, pos, cos, sin, neighbours, back):
    """x [rows, heads, dim]; rows of pos < 0 come back None."""
    one, two = pairs(2 * cos.shape[1], neighbours)
    out = []
    for r, p in enumerate(pos):
        if p < 0:
            out.append(None)
        elif p >= cos.shape[0]:
            out.append(np.full(x.shape[1:], np.nan))
        else:
            c, s = cos[p].astype(np.float64), sin[p].astype(np.float64) * (-1 if back else 1)
            y = x[r].copy()
            y[:, one] = x[r][:, one] * c - x[r][:, two] * s
            y[:, two] = x[r][:, two] * c + x[r][:, one] * s
            out.append(y)
    return out


# ---------------------------------------------------------------- attention over packed prompts

def seen(n, window):
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    return (j <= i) & (j > i - window) if window else j <= i


def prompt_attention(q, k, v, cu, scale, window=0):
    """(out, lse); rows of no sequence are NaN.  What a row does not see has no part
    in it, whatever it holds."""
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    share = q.shape[1] // k.shape[1]
    for b in range(len(cu) - 1):
        at, n = cu[b], cu[b + 1] - cu[b]
        for h in range(q.shape[1]):
            for i in range(n):
                lo = max(0, i - window + 1) if window else 0
                keys = slice(at + lo, at + i + 1)
                s = scale * (k[keys, h // share] @ q[at + i, h])
                m = s.max()
                w = np.exp(s - m)
                lse[at + i, h] = m + np.log(w.sum())
                out[at + i, h] = (w / w.sum()) @ v[keys, h // share]
    return out, lse


def prompt_attention_grad(dout, q, k, v, cu, scale, window=0):
    """(dq, dk, dv) and, of the same shapes, the sums of their terms' sizes that
    error bounds are made of."""
    dq, dk, dv = np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(v.shape, np.nan)
    size = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)]
    share = q.shape[1] // k.shape[1]
    for b in range(len(cu) - 1):
        at, n = cu[b], cu[b + 1] - cu[b]
        here = slice(at, at + n)
        dk[here] = dv[here] = 0
        mask = seen(n, window)
        for h in range(q.shape[1]):
            g = h // share
            s = np.where(mask, scale * (q[here, h] @ k[here, g].T), -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True, initial=-np.inf)) if n else s
            p = p / p.sum(-1, keepdims=True) if n else p
            dp = dout[here, h] @ v[here, g].T
            delta = (p * dp).sum(-1, keepdims=True)
            ds = p * (dp - delta)
            dq[here, h] = scale * ds @ k[here, g]
            dk[here, g] += scale * ds.T @ q[here, h]
            dv[here, g] += p.T @ dout[here, h]
            # sizes: |dP| <= sum |dO| |v|, |delta| <= sum |p| |dP|
            adp = np.abs(dout[here, h]) @ np.abs(v[here, g]).T
            ads = p * (adp + (p * adp).sum(-1, keepdims=True))
            size[0][here, h] = scale * ads @ np.abs(k[here, g])
            size[1][here, g] += scale * ads.T @ np.abs(q[here, h])
            size[2][here, g] += p.T @ np.abs(dout[here, h])
    return (dq, dk, dv), size


# ---------------------------------------------------------------- log probabilities

def token_logprobs(x, targets, top):
    """dict of lse, logp, entropy, top_logp, top_ids, and `far` = sum p |l - max|."""
    rows, vocab = x.shape
    got = dict(lse=np.zeros(rows), logp=np.zeros(rows), entropy=np.zeros(rows), far=np.zeros(rows),
               top_logp=np.zeros((rows, top)), top_ids=np.zeros((rows, top), dtype=np.int64))
    for r in range(rows):
        l = x[r]
        t = targets[r]
        if np.isnan(l).any() or (l == np.inf).any():
            for n in ("lse", "entropy", "top_logp"):
                got[n][r] = np.nan
            got["logp"][r] = np.nan if t >= 0 else 0.0
            got["top_ids"][r] = -1
            continue
        order = np.argsort(-l, kind="stable")[:top]      # equal ones by index
        got["top_ids"][r] = order
        m = l.max()
        if m == -np.inf:
            got["lse"][r] = got["top_logp"][r] = -np.inf
            got["logp"][r] = 0.0 if t < 0 else -np.inf if t < vocab else np.nan
            continue
        e = np.exp(l - m)
        total = e.sum()
        logp = (l - m) - np.log(total)
        p = e / total
        some = p > 0
        got["lse"][r] = m + np.log(total)
        got["entropy"][r] = -(p[some] * logp[some]).sum()
        got["far"][r] = (p[some] * (m - l[some])).sum()
        got["logp"][r] = 0.0 if t < 0 else logp[t] if t < vocab else np.nan
        got["top_logp"][r] = logp[order]
    return got


def token_logprobs_grad(x, targets, lse, d_logp=None, entropy=None, d_entropy=None, top_ids=None, d_top=None):
    """The gradient and the size of its terms."""
    rows, vocab = x.shape
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    for r in range(rows):
        if lse[r] == -np.inf:
            continue
        with np.errstate(over="ignore"):
            logp = x[r] - lse[r]
            p = np.exp(logp)
        t = targets[r] if targets is not None else -1
        g = d_logp[r] if d_logp is not None and t >= 0 else 0.0
        pairs_ = [(t, g)] if t >= 0 else []
        if d_top is not None:
            pairs_ += [(i, e) for i, e in zip(top_ids[r], d_top[r]) if 0 <= i < vocab]
        whole = sum(e for _, e in pairs_)
        d = -p * whole
        size[r] = p * sum(abs(e) for _, e in pairs_)
        if d_entropy is not None:
            some = p > 0
            term = np.zeros(vocab)
            term[some] = p[some] * (logp[some] + entropy[r])
            d = d - d_entropy[r] * term
            size[r, some] += abs(d_entropy[r]) * p[some] * (np.abs(logp[some]) + abs(entropy[r]))
        if t >= vocab:
            d[:] = np.nan
        for i, e in pairs_:
            if i < vocab:
                d[i] += e
                size[r, i] += abs(e)
        out[r] = d
    return out, size
