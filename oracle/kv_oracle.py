"""float64 CPU oracle of the 4-bit paged key/value cache: rounding to the grid,
append, read back and attention.  Test infrastructure, written from the
definitions in include/kronq.h with plain loops over tokens; it shares no code
with the HIP path.

A cache is a dict of numpy arrays: k_codes, v_codes uint8 (pages, heads, page,
dim / 2) and k_grid, v_grid uint32 (pages, heads, page).  A batch is (table,
ctx, cu) of integers.  A rope is (cos, sin, neighbours) or None.
"""
from __future__ import annotations

import math

import numpy as np

NAN_WORD = 0x7FC00000


def scale_word(want: float) -> int:
    """fp32 bits of `want` with 20 significant bits (rounded twice: to fp32, then
    to 20 bits, ties to even each time), at least 2^-126."""
    w = int(np.float32(max(want, 2.0 ** -126)).view(np.uint32))
    low = w & 15
    w -= low
    if low > 8 or (low == 8 and (w >> 4) & 1):
        w += 16
    return w


def word_scale(word) -> float:
    return float(np.uint32(int(word) & ~15).view(np.float32))


def to_grid(x: np.ndarray):
    """(codes, word) of one group of float64 values."""
    if not np.all(np.isfinite(x)):
        return np.zeros(len(x), dtype=np.uint8), NAN_WORD
    lo, hi = min(0.0, float(x.min())), max(0.0, float(x.max()))
    if lo == hi:
        lo, hi = -1.0, 1.0
    word = scale_word((hi - lo) / 15.0)
    s = word_scale(word)
    z = min(max(float(np.rint(-lo / s)), 0.0), 15.0)
    codes = np.clip(np.rint(x / s + z), 0, 15).astype(np.uint8)
    return codes, word | int(z)


def from_grid(codes: np.ndarray, word) -> np.ndarray:
    return word_scale(word) * (codes.astype(np.float64) - (int(word) & 15))


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[0::2] | (codes[1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty(2 * len(packed), dtype=np.uint8)
    out[0::2], out[1::2] = packed & 15, packed >> 4
    return out


def rotate(x: np.ndarray, pos: int, rope) -> np.ndarray:
    """One head's values (float64) at a position."""
    if rope is None:
        return x.copy()
    cos, sin, neighbours = rope
    c, s = cos[pos].astype(np.float64), sin[pos].astype(np.float64)
    half = len(c)
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if neighbours else (np.arange(half), np.arange(half) + half)
    y = x.copy()
    y[a] = x[a] * c - x[b] * s
    y[b] = x[b] * c + x[a] * s
    return y


def rows_of(batch, rows: int):
    """(sequence, position) of each row; None for a row of no sequence."""
    _, ctx, cu = batch
    out = [None] * rows
    for i in range(len(ctx)):
        for r in range(int(cu[i]), int(cu[i + 1])):
            out[r] = (i, int(ctx[i]) - int(cu[i + 1]) + r)
    return out


def place(cache, batch, seq: int, pos: int):
    """(page, slot), or None where there is none in range."""
    table = batch[0]
    pages, _, page, _ = cache["k_codes"].shape
    if pos < 0 or pos // page >= table.shape[1]:
        return None
    p = int(table[seq, pos // page])
    return (p, pos % page) if 0 <= p < pages else None


def append(cache, batch, k: np.ndarray, v: np.ndarray, rope=None) -> None:
    for r, at in enumerate(rows_of(batch, len(k))):
        if at is None or at[1] < 0 or (rope is not None and at[1] >= len(rope[0])):
            continue
        where = place(cache, batch, *at)
        if where is None:
            continue
        p, slot = where
        for h in range(k.shape[1]):
            with np.errstate(invalid="ignore"):
                kx = rotate(k[r, h].astype(np.float64), at[1], rope)
            for nm, x in (("k", kx), ("v", v[r, h].astype(np.float64))):
                codes, word = to_grid(x)
                cache[nm + "_codes"][p, h, slot] = pack(codes)
                cache[nm + "_grid"][p, h, slot] = word


def held(cache, batch, seq: int, pos: int, nm: str) -> np.ndarray:
    """The values held for a position (heads, dim); NaN where there is no page."""
    _, heads, _, half = cache["k_codes"].shape
    where = place(cache, batch, seq, pos)
    if where is None:
        return np.full((heads, 2 * half), np.nan)
    p, slot = where
    return np.stack([from_grid(unpack(cache[nm + "_codes"][p, h, slot]), cache[nm + "_grid"][p, h, slot])
                     for h in range(heads)])


def read(cache, batch, rows: int, nm: str):
    """Rows' held values; None for a row of no sequence."""
    return [None if at is None else held(cache, batch, at[0], at[1], nm) for at in rows_of(batch, rows)]


def visible(pos: int, window: int, sinks: int) -> np.ndarray:
    j = np.arange(max(pos + 1, 0))
    return j if not window else j[(j > pos - window) | (j < sinks)]


def attention(cache, batch, q: np.ndarray, scale: float, window=0, sinks=0, rope=None):
    """(out, lse, size), lists of rows (None for a row of no sequence) but for
    lse: out (q_heads, dim), NaN where it is not defined, and what error bounds
    are made of, size (q_heads, dim + 2): sum_j w_j |v_j| for each value, then
    max_j scale sum |q| |k_j| and max_j w_j |s_j|, weights w of sum 1."""
    rows, qheads, dim = q.shape
    heads = cache["k_codes"].shape[1]
    share = qheads // heads
    out, lse, size = [None] * rows, np.full((rows, qheads), np.nan), [None] * rows
    seen = {}
    for r, at in enumerate(rows_of(batch, rows)):
        if at is None:
            continue
        b, pos = at
        out[r], size[r] = np.zeros((qheads, dim)), np.zeros((qheads, dim + 2))
        js = visible(pos, window, sinks)
        lse[r] = -np.inf
        if not len(js):
            continue
        if rope is not None and pos >= len(rope[0]):
            out[r][:], lse[r] = np.nan, np.nan
            continue
        for j in js:
            if (b, j) not in seen:
                where = place(cache, batch, b, int(j))
                words = np.full(heads, NAN_WORD) if where is None else cache["v_grid"][where[0], :, where[1]]
                seen[b, j] = (held(cache, batch, b, int(j), "k"), held(cache, batch, b, int(j), "v"),
                              np.array([word_scale(w) for w in words]))
        K = np.stack([seen[b, j][0] for j in js])
        V = np.stack([seen[b, j][1] for j in js])
        S = np.stack([seen[b, j][2] for j in js])
        for h in range(qheads):
            x = q[r, h].astype(np.float64)
            with np.errstate(invalid="ignore"):
                x = rotate(x, pos, rope)
                kh, vh = K[:, h // share], V[:, h // share]
                score = scale * (kh @ x)
                if not np.all(np.isfinite(score)):
                    out[r][h], lse[r, h] = np.nan, np.nan
                    continue
                top = score.max()
                w = np.exp(score - top)
                out[r][h] = (w @ vh) / w.sum()
                lse[r, h] = top + math.log(w.sum())
                size[r][h, :dim] = (w @ np.abs(vh)) / w.sum()
                size[r][h, dim] = (scale * (np.abs(kh) @ np.abs(x))).max()
                size[r][h, dim + 1] = (w * np.abs(S[:, h // share])).max() / w.sum()
    return out, lse, size
