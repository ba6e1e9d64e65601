"""Attention over the 4-bit cache, held to what its kernels promise: a second part
of queries or weights that were lost, or scales rounded into the operands (as those
of many rows in bf16 are), would be outside these bounds."""
import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import kv_oracle as K
from kv_helpers import DEV, HALF, Case, f64

TYPES = [torch.float32, torch.bfloat16, torch.float16]
ids = [str(t).replace("torch.", "") for t in TYPES]


def case(dtype, dim, new=1, keys=24, qscale=0.05, device=DEV, seed=0):
    # small queries and some keys, so that scores' own errors do not hide the weights',
    # and values are small beside what they are sums of; or large queries and one or two
    # keys, whose logarithm is a score
    return Case([(keys, new), (max(keys - 5, new), new), (1 + new, new)], share=4, dim=dim, dtype=dtype, qscale=qscale,
                seed=seed, device=device)


def bounds(size, out, lse, dtype, dim, keys):
    """Of out and lse.  Queries are not rotated, so exact in bf16 and in two parts
    (2^-22) else; a score is summed in fp32 and rounded eight times: e = B (u_q + (dim
    + 8) 2^-24).  Weights: 2^-22 in two parts, 2^-11 in bf16; a product below the
    normal fp16 numbers is off by 2^-25 against a row's largest of 2^5, times a code
    of at most 15.  exp2 2^-22; sums of `keys` terms, 32 at a time.  A result is
    rounded to its type, below its normal numbers by half their step."""
    wv, b, top = size[..., :dim], size[..., dim:dim + 1], size[..., dim + 1:]
    e = b * ((0 if dtype == torch.bfloat16 else 2.0 ** -22) + (dim + 8) * 2.0 ** -24)
    w = (2.0 ** -11 if dtype == torch.bfloat16 else 2.0 ** -22) + 2.0 ** -22 + (keys / 32 + 64) * 2.0 ** -24
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    far = 1.05 * (wv * (2 * e + w) + keys * 15 * 2.0 ** -30 * top + np.abs(out) * HALF[dtype] + tiny)
    return far, 1.05 * (e[..., 0] + 2.0 ** -20 + np.abs(lse) * 2.0 ** -22)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new", [1, 3, 6])
@pytest.mark.parametrize("keys,qscale", [(24, 0.05), (1, 2.0)])
def test_few_rows_keep_their_precision(dtype, dim, new, keys, qscale):
    c = case(dtype, dim, new, max(keys, new), qscale, seed=dim + new)
    cache, batch, _ = c.dev(kq)
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, want_lse=True)
    want, wlse, size = K.attention(c.cache, c.batch, f64(c.q), dim ** -0.5)
    for r in range(c.rows):
        far, lfar = bounds(size[r], want[r], wlse[r], dtype, dim, 24)
        assert (np.abs(f64(out)[r] - want[r]) <= far).all(), r
        assert (np.abs(f64(lse)[r] - wlse[r]) <= lfar).all(), r


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=["float32", "float16"])
@pytest.mark.parametrize("dim,new", [(64, 30), (64, 90), (128, 30), (128, 90), (256, 30)])
def test_many_rows_keep_their_precision(dtype, dim, new):
    # tiles of 128 and 256 rows x share: as precise as few rows are
    c = Case([(new + 6, new)], share=4, dim=dim, dtype=dtype, qscale=0.05, seed=dim + new)
    cache, batch, _ = c.dev(kq)
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, want_lse=True)
    want, wlse, size = K.attention(c.cache, c.batch, f64(c.q), dim ** -0.5)
    for r in range(c.rows):
        far, lfar = bounds(size[r], want[r], wlse[r], dtype, dim, new + 6)
        assert (np.abs(f64(out)[r] - want[r]) <= far).all(), r
        assert (np.abs(f64(lse)[r] - wlse[r]) <= lfar).all(), r


def half(x):
    """To fp16 under a factor that keeps all of x normal."""
    return (x * 2.0 ** 12).astype(np.float16).astype(np.float64) * 2.0 ** -12


def parts(c, b):
    """(key head -> keys, values, their scales) of a sequence's positions."""
    n = int(c.ctx[b])
    at = [K.place(c.cache, c.batch, b, j) for j in range(n)]
    for h in range(c.heads):
        x = {nm: np.stack([K.held(c.cache, c.batch, b, j, nm)[h] for j in range(n)]) for nm in "kv"}
        s = {nm: np.array([[K.word_scale(c.cache[nm + "_grid"][p, h, i])] for p, i in at]) for nm in "kv"}
        yield x["k"], x["v"], s["k"], s["v"]


def test_the_bounds_see_weights_in_one_part():
    c = case(torch.float16, 128, device="cpu", seed=5)
    want, wlse, size = K.attention(c.cache, c.batch, f64(c.q), 128 ** -0.5)
    lost = 0
    for b in range(2):
        for g, (k, v, _, vs) in enumerate(parts(c, b)):
            for h in range(4 * g, 4 * g + 4):
                far, _ = bounds(size[b][h], want[b][h], wlse[b, h], torch.float16, 128, 24)
                s = 128 ** -0.5 * k @ f64(c.q)[b, h]
                w = np.exp(s - s.max())[:, None]
                lost += bool((np.abs((half(w * vs) * (v / vs)).sum(0) / w.sum() - want[b][h]) > far).any())
    assert lost >= 14


def test_the_bounds_see_keys_that_carry_their_scales():
    c = case(torch.bfloat16, 64, keys=1, qscale=2.0, device="cpu", seed=5)
    want, wlse, size = K.attention(c.cache, c.batch, f64(c.q), 0.125)
    seen = 0
    for b in range(2):
        for g, (k, _, ks, _) in enumerate(parts(c, b)):
            for h in range(4 * g, 4 * g + 4):
                _, far = bounds(size[b][h], want[b][h], wlse[b, h], torch.bfloat16, 64, 24)
                s = 0.125 * half(half(ks) * (k / ks)) @ f64(c.q)[b, h]
                seen += bool(abs(np.log(np.exp(s).sum()) - wlse[b, h]) > far)
    assert seen >= 10
