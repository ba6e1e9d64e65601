"""Bounds of the calibration pass's operators, by arithmetic."""
from __future__ import annotations

import numpy as np
import torch

from oracle import calib_oracle as C

DEV = "cuda:0"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}  # of the least ones
U = 2.0 ** -24


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def typed(x, dtype) -> torch.Tensor:
    """A host tensor of the type, whose values are then the exact inputs."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(dtype)


def near(got, want, tol, what=""):
    """NaN and infinities at the same places, the rest within tol."""
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), "%s: NaN at %s" % (what, np.argwhere(np.isnan(got) != nan)[:4].tolist())
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), "%s: infinities" % what
    fine = ~(nan | inf)
    far = np.where(fine, np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)) - tol, -1)
    assert far.size == 0 or far.max() <= 0, "%s: off by %.3g over the bound, at %s" % (
        what, far.max(), np.unravel_index(far.argmax(), far.shape))


def rotate_bound(x, pos, cos, sin, neighbours, back, dtype):
    """Two products and a sum in fp32, each rounded, and the result's rounding."""
    size = C.rotate(np.abs(x), pos, np.abs(cos), -np.abs(sin), neighbours, False)
    size2 = C.rotate(np.abs(x), pos, np.abs(cos), np.abs(sin), neighbours, False)
    want = C.rotate(x, pos, cos, sin, neighbours, back)
    tol = []
    for a, b, w in zip(size, size2, want):
        if a is None:
            tol.append(None)
            continue
        terms = np.maximum(np.abs(a), np.abs(b))         # |u c| + |v s| on each side
        tol.append(1.01 * (np.nan_to_num(terms) * 2 * U + np.abs(np.nan_to_num(w)) * HALF[dtype]) + TINY[dtype])
    return want, tol


def sum_error(want, vocab):
    """Relative error of S: a term e^d is off by d's rounding and its product's with
    log2 e (2 |d| U), exp2 (2 U) and at most 16 turns to a new maximum and their
    exponents; sums are of vocab / 256 terms a thread, 8 + 8 joins (segments: fewer
    terms, 16 joins more).  Weighted by the terms: |d| becomes `far`."""
    return U * (vocab / 256 + 96 + 4 * want["far"])


def check_logprobs(got, x, targets, top, entropy=True):
    """x: the exact logits; targets: numpy."""
    vocab = x.shape[1]
    want = C.token_logprobs(x, targets, top)
    es = sum_error(want, vocab)
    with np.errstate(invalid="ignore", over="ignore"):
        log_s = np.log2(vocab) * 0.7 + 0.1               # at least log S
        near(f64(got["lse"]), want["lse"], 1.05 * (es + 4 * U * log_s + 2 * U * np.abs(want["lse"])) + 1e-30, "lse")
        if "logp" in got:
            t = np.abs(np.nan_to_num(want["logp"], posinf=0, neginf=0))
            near(f64(got["logp"]), want["logp"], 1.05 * (es + 4 * U * (log_s + t)) + 1e-30, "logp")
        if entropy:
            # T / S: each term of T as S's, and its product with d
            tol = 1.05 * (es * (2 + 3 * want["far"]) + 4 * U * (log_s + want["far"])) + 1e-30
            near(f64(got["entropy"]), want["entropy"], tol, "entropy")
        if top:
            assert np.array_equal(got["top_ids"].cpu().numpy(), want["top_ids"]), "top_ids"
            t = np.abs(np.nan_to_num(want["top_logp"], posinf=0, neginf=0))
            near(f64(got["top_logp"]), want["top_logp"], 1.05 * (es[:, None] + 4 * U * (log_s + t)) + 1e-30, "top_logp")
    return want


def check_logprobs_grad(got, x, dtype, targets, lse, **kw):
    """lse, entropy: the fp32 values that the call was given."""
    want, size = C.token_logprobs_grad(x, targets, lse, **kw)
    with np.errstate(invalid="ignore", over="ignore"):
        logp = np.abs(np.nan_to_num(x - lse[:, None], nan=0, posinf=0, neginf=0))
    # p: l - lse rounded, its product with log2 e, exp2; p below fp32's least is 0; sums
    # of up to 64 gradients, and three products and sums
    e = np.minimum(3 * logp, 400) * U + 4 * U + 72 * U
    tol = 1.05 * (size * e + np.abs(np.nan_to_num(want)) * HALF[dtype]) + 2 * TINY[dtype] + 1e-37
    near(got, want, tol, "grad")


# ---------------------------------------------------------------- prompts

def prompt_case(lengths, qh, kh, dim, dtype, seed, before=0, behind=0, loud=1.0):
    """q, k, v, dout (host, typed) of rows of sequences, with rows of none around."""
    rng = np.random.default_rng(seed)
    rows = before + sum(lengths) + behind
    cu = (before + np.concatenate([[0], np.cumsum(lengths)])).astype(np.int32)
    q = typed(rng.normal(size=(rows, qh, dim)) * loud, dtype)
    k, v = (typed(rng.normal(size=(rows, kh, dim)), dtype) for _ in "kv")
    return q, k, v, typed(rng.normal(size=(rows, qh, dim)), dtype), cu


def _weight_error(b, s, dim, lse):
    """Relative error of a weight exp(S - m): products are summed in fp32 (dim additions),
    scaled (2 roundings), taken from the maximum or started from -lse / scale, lse itself
    rounded (4 |lse| U in all); exp2 4 U."""
    return U * (b * (dim + 2) + np.abs(s) * 4 + 4 * np.abs(lse) + 4 + 2 * np.abs(s - lse))


def prompt_reference(q, k, v, cu, scale, window, dtype):
    """64-bit (out, lse) and their bounds; rows of no sequence are NaN.  Dense, for finite
    inputs.

    A weight is off by a factor 1 + e: 2 e in out.  Weights are rounded to the type of v
    (half a step; fp16: no finer than 2^-25 beside a largest of at least 1); sums of up to
    `keys` terms and their turns to new maxima are fp32."""
    out, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    tol, ltol = np.zeros(q.shape), np.zeros(q.shape[:2])
    share, dim = q.shape[1] // k.shape[1], q.shape[2]
    for b in range(len(cu) - 1):
        here, n = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
        if n == 0:
            continue
        mask = C.seen(n, window)
        for h in range(q.shape[1]):
            g = h // share
            s = scale * q[here, h] @ k[here, g].T
            big = scale * np.abs(q[here, h]) @ np.abs(k[here, g]).T
            m = np.where(mask, s, -np.inf).max(-1, keepdims=True)
            w = np.where(mask, np.exp(np.minimum(s - m, 0)), 0)
            total = w.sum(-1, keepdims=True)
            p = w / total
            l = m + np.log(total)
            e = np.where(mask, _weight_error(big, s, dim, l), 0)
            out[here, h], lse[here, h] = p @ v[here, g], l[:, 0]
            av = np.abs(v[here, g])
            up = HALF[dtype] if dtype != torch.float32 else 0
            t = p @ av * (up + (1.5 * n + 64) * U) + (p * e) @ av + (p * e).sum(-1, keepdims=True) * (p @ av)
            if dtype == torch.float16:
                t = t + mask.sum(-1, keepdims=True) * 2.0 ** -25 * av.max() / total
            tol[here, h] = 1.05 * (t + np.abs(out[here, h]) * HALF[dtype]) + TINY[dtype]
            ltol[here, h] = 1.05 * ((p * e).sum(-1) + (n + 8) * U + 4 * U * np.abs(l[:, 0]))
    return out, lse, tol, ltol


def prompt_grad_reference(dout, q, k, v, out, lse, cu, scale, window, dtype):
    """64-bit (dq, dk, dv) and their bounds.  out and lse are what the call is given:
    delta is off by what they are off by.

    ds = p (dP - delta) is off by p's error e times its size, and by p times the errors of
    dP (dim additions) and delta; it and p are rounded to the type (fp16: no finer than
    2^-36 of a column's largest); sums are fp32."""
    want = [np.full(x.shape, np.nan) for x in (q, k, v)]
    tol = [np.zeros(x.shape) for x in (q, k, v)]
    share, dim = q.shape[1] // k.shape[1], q.shape[2]
    up = HALF[dtype] if dtype != torch.float32 else 0
    for b in range(len(cu) - 1):
        here, n = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
        if n == 0:
            continue
        for x in (1, 2):
            want[x][here] = 0
        mask = C.seen(n, window)
        for h in range(q.shape[1]):
            g = h // share
            qh, kg, vg, do = q[here, h], k[here, g], v[here, g], dout[here, h]
            s = scale * qh @ kg.T
            big = scale * np.abs(qh) @ np.abs(kg).T
            ms = np.where(mask, s, -np.inf)
            m = ms.max(-1, keepdims=True)
            p = np.exp(ms - m)
            p /= p.sum(-1, keepdims=True)
            l = lse[here, h][:, None]
            e = np.where(mask, _weight_error(big, s, dim, l), 0)
            dp, adp = do @ vg.T, np.abs(do) @ np.abs(vg).T
            delta = (p * dp).sum(-1, keepdims=True)
            given = (do * out[here, h]).sum(-1, keepdims=True)
            agiven = (np.abs(do) * np.abs(out[here, h])).sum(-1, keepdims=True)
            ds = p * (dp - delta)
            ed = p * (np.abs(dp - delta) * e + adp * (dim + 2) * U + np.abs(given - delta) + agiven * (dim + 4) * U)
            es, ep = ed + np.abs(ds) * (up + 2 * U), p * (e + up)
            if dtype == torch.float16:
                es = es + mask * (2.0 ** -36 * np.maximum(np.abs(ds).max(0, keepdims=True), np.abs(ds).max(-1, keepdims=True)))
                ep = ep + mask * (2.0 ** -36 * p.max(0, keepdims=True))
            acc = (n * share + 64) * U
            want[0][here, h] = scale * ds @ kg
            want[1][here, g] += scale * ds.T @ qh
            want[2][here, g] += p.T @ do
            tol[0][here, h] = scale * (es + np.abs(ds) * acc) @ np.abs(kg)
            tol[1][here, g] += scale * (es + np.abs(ds) * acc).T @ np.abs(qh)
            tol[2][here, g] += (ep + p * acc).T @ np.abs(do)
    tol = [1.05 * (t + np.abs(np.nan_to_num(w)) * HALF[dtype]) + TINY[dtype] for t, w in zip(tol, want)]
    return want, tol


def sequences_equal(got, want, tol, cu, before, what):
    """Rows of sequences are near, the others are as they were."""
    inside = np.zeros(got.shape[0], dtype=bool)
    for b in range(len(cu) - 1):
        inside[cu[b]:cu[b + 1]] = True
    assert (got[~inside] == before).all(), "%s: a row of no sequence was written" % what
    near(got[inside], want[inside], tol[inside], what)
