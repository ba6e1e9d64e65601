"""Inputs of the key/value cache tests, and bounds of their results."""
from __future__ import annotations

import numpy as np
import torch

from oracle import kv_oracle as K

DEV = "cuda:0"
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}   # half a step


class Case:
    """A cache with content, a batch and queries: numpy on one side, torch on the
    device on the other."""

    def __init__(self, lengths, heads=2, share=2, dim=64, page=16, dtype=torch.float32, seed=0, rot=0,
                 neighbours=False, padding=0, columns=None, device=DEV, qscale=1.0, spread=0.5):
        rng = np.random.default_rng(seed)
        self.lengths, self.heads, self.share, self.dim, self.page = lengths, heads, share, dim, page
        self.dtype, self.device = dtype, device
        need = [-(-max(c, 0) // page) for c, _ in lengths]
        self.pages = sum(need) + 2
        ids = rng.permutation(self.pages)
        columns = max(need + [1]) if columns is None else columns
        self.table = np.full((len(lengths), columns), -7, dtype=np.int32)     # entries that are not needed
        at = 0
        for i, n in enumerate(need):
            n = min(n, columns)
            self.table[i, :n] = ids[at:at + n]
            at += need[i]
        self.ctx = np.array([c for c, _ in lengths], dtype=np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for _, n in lengths])]).astype(np.int32)
        self.rows = int(self.cu[-1]) + padding
        shape = (self.pages, heads, page)
        self.cache = {}
        for nm in "kv":
            self.cache[nm + "_codes"] = rng.integers(0, 256, shape + (dim // 2,), dtype=np.uint8)
            s = np.exp(rng.normal(size=shape) * spread) * 0.1
            w = s.astype(np.float32).view(np.uint32) & np.uint32(0xFFFFFFF0)
            self.cache[nm + "_grid"] = w | rng.integers(0, 16, shape).astype(np.uint32)
        self.rope = None
        if rot:
            n = max(int(self.ctx.max(initial=1)), 1)
            ang = np.arange(n)[:, None] * 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)
            self.rope = (np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32), neighbours)
        self.q = self.typed(rng.normal(size=(self.rows, heads * share, dim)) * qscale)
        self.k = self.typed(rng.normal(size=(self.rows, heads, dim)))
        self.v = self.typed(rng.normal(size=(self.rows, heads, dim)))

    def typed(self, x):
        """A tensor of the case's type (host), and so the exact values."""
        return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(self.dtype)

    @property
    def batch(self):
        return self.table, self.ctx, self.cu

    def dev(self, kq):
        """(cache, batch, rope) on the device."""
        d = self.device
        t = {n: torch.from_numpy(a.view(np.int32) if a.dtype == np.uint32 else a.copy()).clone().to(d)
             for n, a in self.cache.items()}
        cache = kq.KVCache(t["k_codes"], t["v_codes"], t["k_grid"], t["v_grid"])
        batch = kq.KVBatch(*(torch.from_numpy(x.copy()).to(d) for x in self.batch))
        rope = None
        if self.rope is not None:
            rope = kq.Rope(torch.from_numpy(self.rope[0]).to(d), torch.from_numpy(self.rope[1]).to(d), self.rope[2])
        return cache, batch, rope


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def cache_equal(cache, ref) -> None:
    for nm in ("k_codes", "v_codes"):
        assert np.array_equal(getattr(cache, nm).cpu().numpy(), ref[nm]), nm
    for nm in ("k_grid", "v_grid"):
        assert np.array_equal(getattr(cache, nm).cpu().numpy().view(np.uint32), ref[nm]), nm


def attention_bound(size, out, dtype, dim, keys, rotated):
    """How far an output may be from the 64-bit one, by arithmetic.

    Scores: with B = scale sum |q| |k| a product of q rounded by u_q and summed
    in fp32 (dim additions) is off by B (u_q + dim 2^-24) and by 8 roundings of
    fp32 to and from it; u_q is 2^-22 where q is held in two parts (fp32, fp16),
    half a step of fp16 (2^-11) for a rotated bf16 query and 0 for one as it
    came.  Keys of bf16's many rows carry their scale: 2 2^-11 more.  A score off
    by e changes a weight by the factor 1 + e (e small), numerator and
    denominator alike: 2 e sum w |v| in out.
    Weights times scales: u_p = 2^-11 of each (2^-22 in two parts), 3 2^-11 where
    values carry their scale; or where they are no normal fp16 numbers 2^-25
    against a row's largest of at least 2^5, so 2^-30 of that, times a code of at
    most 15, for each key (values with their scale: weights' 2^-25 against 2^6 and
    scales' 2^10 against 2^1, so 2^-22).
    exp2 itself 2^-22, and sums of `keys` terms in fp32, 32 at a time in the
    matrix cores.  The result is rounded to its type.  Second orders: 5 %."""
    wv, b, top = size[..., :dim], size[..., dim:dim + 1], size[..., dim + 1:]
    fold = dtype == torch.bfloat16
    uq = (2.0 ** -11 * (int(rotated) + 2)) if fold else 2.0 ** -22
    e = b * (uq + (dim + 8) * 2.0 ** -24)
    up = {torch.float32: 2.0 ** -22, torch.float16: 2.0 ** -11, torch.bfloat16: 3 * 2.0 ** -11}[dtype]
    low = 2.0 ** -22 if fold else 2.0 ** -30
    w = up + 2.0 ** -22 + (keys / 32 + 64) * 2.0 ** -24
    return 1.05 * (wv * (2 * e + w) + keys * 15 * low * top + np.abs(out) * HALF[dtype] + 1e-30)


def check_attention(case, out, lse, scale=None, window=0, sinks=0, before=None):
    """Every row against the 64-bit reference."""
    scale = case.dim ** -0.5 if scale is None else scale
    want, wlse, size = K.attention(case.cache, case.batch, f64(case.q), scale, window, sinks, case.rope)
    got, glse = f64(out), None if lse is None else f64(lse)
    for r in range(case.rows):
        if want[r] is None:
            if before is not None:
                assert np.array_equal(got[r], before[r]), "row %d of no sequence was written" % r
            continue
        nan = np.isnan(want[r])
        assert np.array_equal(np.isnan(got[r]), nan), "row %d: NaN" % r
        keys = int(case.ctx.max())
        tol = attention_bound(size[r], np.where(nan, 0, want[r]), case.dtype, case.dim, keys, case.rope is not None)
        with np.errstate(invalid="ignore"):
            far = np.where(nan, 0, np.abs(got[r] - want[r]) - tol)
        # beyond the type's largest number a result is infinite, as any rounding to the type makes it
        over = np.isinf(got[r]) & (np.sign(got[r]) == np.sign(want[r])) & \
            (np.abs(want[r]) + tol >= float(torch.finfo(case.dtype).max))
        far = np.where(over, 0, far)
        assert far.max() <= 0, "row %d: off by %.3g over the bound" % (r, far.max())
        if glse is not None:
            for h in range(got.shape[1]):
                x, y = glse[r, h], wlse[r, h]
                if np.isnan(want[r][h]).any():
                    continue                  # not defined
                if np.isinf(y):
                    assert x == y
                else:
                    b = size[r][h, case.dim]
                    uq = 3 * 2.0 ** -11 if case.dtype == torch.bfloat16 else 2.0 ** -22
                    assert abs(x - y) <= 1.05 * (b * (uq + (case.dim + 8) * 2.0 ** -24) + 2.0 ** -20 + abs(y) * 2.0 ** -22)
