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
