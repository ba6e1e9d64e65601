"""Attention over packed prompts and its gradients on the device against 64 bits, and
a calibration pass of the operators together."""
import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import calib_oracle as C
from calib_helpers import (DEV, HALF, U, f64, near, prompt_case, prompt_grad_reference, prompt_reference, sequences_equal,
                           typed)

pytestmark = pytest.mark.gpu
DTYPES = (torch.float32, torch.bfloat16, torch.float16)

# lengths, query heads, key heads, dim, window
SHAPES = [
    ([1], 1, 1, 64, 0), ([1], 32, 8, 128, 0), ([2, 0, 3], 2, 1, 8, 0), ([33, 64, 65], 6, 2, 64, 0),
    ([127, 128, 129, 1, 0], 4, 4, 128, 0), ([300], 8, 1, 96, 0), ([257, 31], 3, 3, 256, 0), ([200, 90], 2, 1, 136, 70),
    ([150], 5, 1, 72, 1), ([400, 3], 2, 2, 128, 64), ([500], 2, 1, 64, 200), ([130], 2, 2, 16, 129), ([130], 2, 2, 128, 131),
]
# Enough workgroups of 128 rows for the ways that long calls take: many short sequences beside
# longer ones, many heads.  (lengths, query heads, key heads, dim, window)
SHORT = [5, 1, 33, 2] * 9
BUSY = [
    ([300, 1, 200, 0] + SHORT, 32, 32, 64, 0), ([300, 1, 200, 0] + SHORT, 32, 16, 128, 90),
    ([260, 129] + SHORT, 26, 26, 128, 0), ([290] + SHORT, 24, 24, 256, 150), ([260] + SHORT + [7] * 40, 24, 12, 64, 33),
    ([257] + SHORT, 64, 8, 96, 0),
]
IDS = ["%s-%d-%d-%d-%d" % ("+".join(map(str, s[0])), *s[1:]) for s in SHAPES]


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def check_forward(q, k, v, cu, out, lse, dtype, window, scale=None, before=7.0):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    want, wlse, tol, ltol = prompt_reference(f64(q), f64(k), f64(v), cu, np.float32(scale).astype(np.float64), window, dtype)
    sequences_equal(f64(out), want, tol, cu, before, "out")
    if lse is not None:
        sequences_equal(f64(lse), wlse, ltol, cu, before, "lse")
    return want, wlse


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,qh,kh,dim,window", SHAPES, ids=IDS)
def test_attention(lengths, qh, kh, dim, window, dtype):
    q, k, v, _, cu = prompt_case(lengths, qh, kh, dim, dtype, sum(lengths) + dim, before=2, behind=3)
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    kq.kronq_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), dev(cu), window=window, out=out, lse=lse)
    check_forward(q, k, v, cu, out, lse, dtype, window)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", range(len(BUSY)))
def test_busy_calls(shape, dtype):
    """Both directions where the chip is full."""
    lengths, qh, kh, dim, window = BUSY[shape]
    q, k, v, do, cu = prompt_case(lengths, qh, kh, dim, dtype, shape + 100, before=1, behind=2)
    args = [t.to(DEV) for t in (q, k, v)]
    out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    kq.kronq_prompt_attention(*args, dev(cu), window=window, out=out, lse=lse)
    check_forward(q, k, v, cu, out, lse, dtype, window)
    grads = [torch.full(t.shape, 7.0, dtype=dtype, device=DEV) for t in (q, k, v)]
    kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, dev(cu), window=window, dq=grads[0], dk=grads[1], dv=grads[2])
    check_backward(q, k, v, do, cu, out, lse, grads, dtype, window, before=7.0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_of_large_scores(dtype):
    """Weights that are nearly all one key's, maxima that rise along the row, another scale."""
    q, k, v, _, cu = prompt_case([200, 77], 4, 2, 64, dtype, 5, loud=6.0)
    k = (k.double() * torch.linspace(0.1, 3, k.shape[0], dtype=torch.float64)[:, None, None]).to(dtype)
    out, lse = kq.kronq_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), dev(cu), scale=0.31, want_lse=True)
    check_forward(q, k, v, cu, out, lse, dtype, 0, scale=0.31)


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_long_prompt(dtype):
    q, k, v, do, cu = prompt_case([2500, 700], 2, 1, 64, dtype, 11)
    args = [t.to(DEV) for t in (q, k, v)]
    for window in (0, 1100):
        out, lse = kq.kronq_prompt_attention(*args, dev(cu), window=window, want_lse=True)
        check_forward(q, k, v, cu, out, lse, dtype, window)
        got = kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, dev(cu), window=window)
        check_backward(q, k, v, do, cu, out, lse, got, dtype, window)


def odd_case(dtype, dim=64, kh=2):
    """NaN and infinities at late rows, which earlier rows do not see, and in rows of none."""
    lengths = [150, 70] + (SHORT if kh > 2 else [])
    q, k, v, do, cu = prompt_case(lengths, 2 * kh, kh, dim, dtype, 21, before=1, behind=2)
    nan, inf = float("nan"), float("inf")
    for t in (q, k, v, do):
        t[0], t[-2:] = nan, inf
    v[1 + 100, 0, 3] = nan
    v[1 + 120, 0, 5], v[1 + 130, 0, 5], v[1 + 121, 0, 7] = inf, -inf, -inf
    k[1 + 140, 1, 2] = nan
    v[1 + 149, 1] = inf
    return q, k, v, do, cu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window", (0, 20))
@pytest.mark.parametrize("dim,kh", [(64, 2), (128, 2), (200, 2), (64, 12), (128, 12), (200, 6), (64, 36), (128, 36), (200, 12)])
def test_what_a_row_does_not_see(dtype, window, dim, kh):
    """(Few heads, and as many as make a busy call.)"""
    q, k, v, _, cu = odd_case(dtype, dim, kh)
    out, lse = torch.full(q.shape, 7.0, dtype=dtype, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
    kq.kronq_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), dev(cu), window=window, out=out, lse=lse)
    with np.errstate(invalid="ignore"):
        want, wlse = C.prompt_attention(f64(q), f64(k), f64(v), cu, np.float64(np.float32(dim ** -0.5)), window)
    assert np.isnan(want[cu[0]:cu[-1]]).any() and np.isinf(want).any()
    fine = [np.where(np.isfinite(f64(t)), f64(t), 0) for t in (q, k, v)]
    _, _, tol, ltol = prompt_reference(*fine, cu, dim ** -0.5, window, dtype)
    sequences_equal(f64(out), want, tol, cu, 7.0, "out")
    sequences_equal(f64(lse), wlse, ltol, cu, 7.0, "lse")


def test_strides_stream_and_equal_bits():
    """q, k and v of one packed tensor, out and lse given, a stream of its own; twice the same bits."""
    dtype, qh, kh, dim = torch.bfloat16, 6, 2, 64
    q, k, v, do, cu = prompt_case([90, 61], qh, kh, dim, dtype, 31)
    rows = q.shape[0]
    whole = torch.zeros((rows, (qh + 2 * kh) * dim + 8), dtype=dtype, device=DEV)
    views = []
    at = 0
    for t in (q, k, v):
        n = t.shape[1] * dim
        whole[:, at:at + n] = t.view(rows, n).to(DEV)
        views.append(whole[:, at:at + n].view(rows, t.shape[1], dim))
        at += n
    plain = kq.kronq_prompt_attention(q.to(DEV), k.to(DEV), v.to(DEV), dev(cu), want_lse=True)
    grads = kq.kronq_prompt_attention_grad(do.to(DEV), q.to(DEV), k.to(DEV), v.to(DEV), *plain, dev(cu))
    c, d = dev(cu), do.to(DEV)
    g = torch.zeros_like(whole)
    gq, gk, gv = (g[:, a:b].view(rows, -1, dim) for a, b in ((0, qh * dim), (qh * dim, (qh + kh) * dim),
                                                             ((qh + kh) * dim, (qh + 2 * kh) * dim)))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = kq.kronq_prompt_attention(*views, c, want_lse=True, stream=s)
    kq.kronq_prompt_attention_grad(d, *views, out, lse, c, dq=gq, dk=gk, dv=gv, stream=s)
    s.synchronize()
    assert torch.equal(out, plain[0]) and torch.equal(lse, plain[1])
    assert torch.equal(gq, grads[0]) and torch.equal(gk, grads[1]) and torch.equal(gv, grads[2])
    assert not g[:, -8:].any()


def test_any_content_of_cu():
    """Sequences that decrease, overlap or lie outside are cut to the rows there are."""
    dtype = torch.float16
    q, k, v, do, _ = prompt_case([40], 2, 1, 64, dtype, 41)
    args = [t.to(DEV) for t in (q, k, v)]
    for cu in ([-5, 10, 60], [30, 10, 40], [50, 70, 90], [2 ** 31 - 1, -2 ** 31, 40], [0, 0, 0], [38, 2 ** 31 - 1, 39]):
        c = torch.tensor(cu, dtype=torch.int32, device=DEV)
        out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV)
        _, lse = kq.kronq_prompt_attention(*args, c, out=out, want_lse=True)
        lse = torch.nan_to_num(lse)
        dq, dk, dv = (torch.full(t.shape, 7.0, dtype=dtype, device=DEV) for t in (q, k, v))
        kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, c, dq=dq, dk=dk, dv=dv)
        torch.cuda.synchronize()
        inside = np.zeros(40, dtype=bool)
        for lo, hi in zip(cu, cu[1:]):
            inside[max(lo, 0):max(hi, 0)] = True
        for t in (out, dq, dk, dv):
            assert (t.cpu().numpy()[~inside] == 7).all()


# ---------------------------------------------------------------- gradients

def check_backward(q, k, v, do, cu, out, lse, got, dtype, window, before=None):
    scale = np.float64(np.float32(q.shape[2] ** -0.5))
    want, tol = prompt_grad_reference(f64(do), f64(q), f64(k), f64(v), f64(out), f64(lse), cu, scale, window, dtype)
    for g, w, t, nm in zip(got, want, tol, ("dq", "dk", "dv")):
        if before is None:
            near(f64(g), w, t, nm)
        else:
            sequences_equal(f64(g), w, t, cu, before, nm)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,qh,kh,dim,window", SHAPES, ids=IDS)
def test_grad(lengths, qh, kh, dim, window, dtype):
    q, k, v, do, cu = prompt_case(lengths, qh, kh, dim, dtype, sum(lengths) + dim, before=2, behind=3)
    args = [t.to(DEV) for t in (q, k, v)]
    out, lse = kq.kronq_prompt_attention(*args, dev(cu), window=window, want_lse=True)
    grads = [torch.full(t.shape, 7.0, dtype=dtype, device=DEV) for t in (q, k, v)]
    kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, dev(cu), window=window, dq=grads[0], dk=grads[1], dv=grads[2])
    check_backward(q, k, v, do, cu, out, lse, grads, dtype, window, before=7.0)


@pytest.mark.parametrize("size", (2.0 ** -14, 2.0 ** -20, 200.0))
def test_grad_of_small_and_large_gradients_in_fp16(size):
    """Gradients far from 1, and rows of very different ones, keep their precision."""
    dtype = torch.float16
    q, k, v, do, cu = prompt_case([180, 40], 4, 2, 64, dtype, 51)
    do = (do.double() * size * torch.logspace(0, -3, do.shape[0], dtype=torch.float64)[:, None, None]).to(dtype)
    args = [t.to(DEV) for t in (q, k, v)]
    out, lse = kq.kronq_prompt_attention(*args, dev(cu), want_lse=True)
    got = kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, dev(cu))
    check_backward(q, k, v, do, cu, out, lse, got, dtype, 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,kh", [(64, 2), (128, 2), (200, 2), (64, 18), (128, 18), (128, 28), (200, 12)])
def test_grad_of_what_a_row_does_not_see(dtype, dim, kh):
    """A late row's NaN reaches the rows and keys that it has to do with, and no others."""
    q, k, v, do, cu = prompt_case([150, 70] + (SHORT if kh > 2 else []), 2 * kh, kh, dim, dtype, 61)
    args = [t.to(DEV) for t in (q, k, v)]
    clean = kq.kronq_prompt_attention(*args, dev(cu), want_lse=True)
    # row 100: its query; row 130: its gradient; both of query head 1.  Keys behind 130 see neither
    q[100, 1, 4] = float("nan")
    do[130, 1, 9] = float("inf")
    # key 140 of key head 1: rows from 140 on see it
    k[140, 1, 2] = float("nan")
    v[145, 1, 2] = float("-inf")
    args = [t.to(DEV) for t in (q, k, v)]
    out, lse = kq.kronq_prompt_attention(*args, dev(cu), want_lse=True)
    dq, dk, dv = kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, dev(cu))
    bad = [np.isnan(f64(t)) | np.isinf(f64(t)) for t in (dq, dk, dv)]
    # head 1's rows 100 and 130 alone of key head 0's query heads; rows from 140 of heads 2 and 3
    rows = bad[0].any(-1)
    want = np.zeros_like(rows)
    want[[100, 130], 1] = True
    want[140:150, 2:4] = True
    assert np.array_equal(rows, want)
    keys = bad[1].any(-1)
    assert keys[:131, 0].all() and not keys[131:, 0].any()
    assert keys[:150, 1].all() and not keys[150:].any() and not keys[:, 2:].any()
    keys = bad[2].any(-1)
    assert keys[:131, 0].all() and not keys[131:, 0].any()
    assert not keys[150:].any() and not keys[:, 2:].any()
    # dv of keys 101 .. 130 sees only the gradient's one value
    assert not np.delete(bad[2][101:131, 0], 9, axis=-1).any()
    # and what has nothing to do with it is right
    fine = [torch.nan_to_num(t.double(), 0, 0, 0).to(dtype) for t in (q, k, v, do)]
    o2, l2 = kq.kronq_prompt_attention(*[t.to(DEV) for t in fine[:3]], dev(cu), want_lse=True)
    wanted, tol = prompt_grad_reference(f64(fine[3]), *(f64(t) for t in fine[:3]), f64(o2), f64(l2), cu,
                                        np.float64(np.float32(dim ** -0.5)), 0, dtype)
    near(f64(dq)[:100], wanted[0][:100], tol[0][:100], "dq")
    near(f64(dk)[131:, 0], wanted[1][131:, 0], tol[1][131:, 0], "dk")
    near(f64(dv)[131:, 0], wanted[2][131:, 0], tol[2][131:, 0], "dv")
    assert clean[0].isfinite().all()


def test_grad_by_differences():
    dtype = torch.float32
    q, k, v, w, cu = prompt_case([9, 20], 4, 2, 16, dtype, 71)
    args = [t.to(DEV) for t in (q, k, v)]
    out, lse = kq.kronq_prompt_attention(*args, dev(cu), window=6, want_lse=True)
    got = [f64(t) for t in kq.kronq_prompt_attention_grad(w.to(DEV), *args, out, lse, dev(cu), window=6)]
    rng = np.random.default_rng(1)
    host = [f64(t) for t in (q, k, v)]
    for n in range(3):
        for _ in range(4):
            at = tuple(rng.integers(0, s) for s in host[n].shape)
            both = []
            for sign in (1, -1):
                moved = [t.copy() for t in host]
                moved[n][at] += sign * 1e-5
                both.append((C.prompt_attention(*moved, cu, 0.25, 6)[0] * f64(w)).sum())
            want = (both[0] - both[1]) / 2e-5
            assert abs(want - got[n][at]) < 1e-5 * (1 + abs(want))


def test_captured_and_at_once():
    """A graph of both directions replayed over changing lengths, beside a call on another stream."""
    dtype = torch.bfloat16
    q, k, v, do, cu = prompt_case([300], 4, 2, 128, dtype, 81)
    args = [t.to(DEV) for t in (q, k, v)]
    d, c = do.to(DEV), torch.tensor([0, 300, 300, 300], dtype=torch.int32, device=DEV)

    def work(c, stream=None):
        out, lse = kq.kronq_prompt_attention(*args, c, want_lse=True, stream=stream)
        return (out, lse) + kq.kronq_prompt_attention_grad(d, *args, out, lse, c, stream=stream)

    work(c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(c)
    other = torch.cuda.Stream()
    for lengths in ([0, 300, 300, 300], [0, 17, 150, 300], [0, 0, 299, 300], [0, 100, 200, 300]):
        c.copy_(torch.tensor(lengths, dtype=torch.int32))
        c2 = c.clone()
        other.wait_stream(torch.cuda.current_stream())
        graph.replay()
        beside = work(c2, stream=other)
        torch.cuda.synchronize()
        want = work(c2)
        torch.cuda.synchronize()
        for a, b, w in zip(got, beside, want):
            assert torch.equal(a, w) and torch.equal(b, w)


# ---------------------------------------------------------------- together

def test_prompt_attention_is_the_caches():
    """What the 4-bit cache holds, read back, gives what attention over the cache gives."""
    rng = np.random.default_rng(5)
    lengths, qh, kh, dim = [70, 33], 4, 2, 64
    rows = sum(lengths)
    q, k, v, _, cu = prompt_case(lengths, qh, kh, dim, torch.float32, 91)
    cache = kq.KVCache.empty(8, kh, 16, dim)
    table = torch.from_numpy(rng.permutation(8)[:7].astype(np.int32)).to(DEV)
    tab = torch.full((2, 5), -1, dtype=torch.int32, device=DEV)
    tab[0, :5], tab[1, :2] = table[:5], table[5:7]
    # 33 rows need three pages
    tab[1, 2] = int(np.setdiff1d(np.arange(8), table.cpu().numpy())[0])
    batch = kq.KVBatch(tab, torch.tensor(lengths, dtype=torch.int32, device=DEV), dev(cu))
    rope = kq.kronq_rope_tables(100, dim)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lengths]).to(DEV)
    kq.kronq_kv_append(k.to(DEV), v.to(DEV), cache, batch, rope=rope)
    want, wlse = kq.kronq_kv_attention(q.to(DEV), cache, batch, rope=rope, want_lse=True)
    kk, vv = kq.kronq_kv_read(cache, batch, rows)        # keys as they are held: rotated
    turned, _ = kq.kronq_rotate(q.to(DEV), None, pos, rope)
    out, lse = kq.kronq_prompt_attention(turned, kk, vv, dev(cu), want_lse=True)
    # each within its own bound of the 64-bit result
    _, _, tol, ltol = prompt_reference(f64(turned), f64(kk), f64(vv), cu, dim ** -0.5, 0, torch.float32)
    near(f64(out), f64(want), 2 * tol + 2.0 ** -18, "out")
    near(f64(lse), f64(wlse), 2 * ltol + 2.0 ** -18, "lse")


@pytest.mark.parametrize("dtype,neighbours", [(torch.bfloat16, False), (torch.float32, True), (torch.float16, False)])
def test_calibration_pass(dtype, neighbours):
    """The Kronecker factors H_G of q, k and v projections and of the output head, from the
    loss of packed text: positions, attention, log probabilities, and back, then the Gram."""
    rng = np.random.default_rng(6)
    lengths, qh, kh, dim, vocab = [50, 78], 4, 2, 64, 999
    rows = sum(lengths)
    q, k, v, _, cu = prompt_case(lengths, qh, kh, dim, dtype, 95)
    head = typed(rng.normal(size=(qh * dim, vocab)) * 0.2, torch.float32)
    targets = rng.integers(0, vocab, rows).astype(np.int32)
    targets[[49, 127]] = -1                              # a text's last token has no next one
    pos = np.concatenate([np.arange(n) for n in lengths]).astype(np.int32)
    rope = kq.kronq_rope_tables(80, dim, scaling="parts", factor=4.0, original=40.0, neighbours=neighbours)
    c = dev(cu)
    tq, tk = kq.kronq_rotate(q.to(DEV), k.to(DEV), dev(pos), rope)
    vd = v.to(DEV)
    out, lse = kq.kronq_prompt_attention(tq, tk, vd, c, want_lse=True)
    hd = head.to(DEV)
    logits = (out.reshape(rows, -1).float() @ hd).to(dtype)
    got = kq.kronq_token_logprobs(logits, dev(targets), top=3, want_entropy=True)
    g = torch.full((rows,), -1.0 / (rows - 2), device=DEV)
    dlogits = kq.kronq_token_logprobs_grad(logits, dev(targets), got["lse"], g)
    dout = (dlogits.float() @ hd.t().contiguous()).to(dtype).view(rows, qh, dim)
    dq, dk, dv = kq.kronq_prompt_attention_grad(dout, tq, tk, vd, out, lse, c)
    gq, gk = kq.kronq_rotate(dq, dk, dev(pos), rope, back=True)
    grams = [kq.kronq_gram(x.reshape(rows, -1).to(torch.float32)) for x in (gq, gk, dv)]

    # the same in 64 bits
    cos, sin = f64(rope.cos), f64(rope.sin)
    rot = lambda x, back: np.stack(C.rotate(x, pos, cos, sin, neighbours, back))  # noqa: E731
    rq, rk = rot(f64(q), False), rot(f64(k), False)
    ro, _ = C.prompt_attention(rq, rk, f64(v), cu, dim ** -0.5)
    rl = ro.reshape(rows, -1) @ f64(head)
    want = C.token_logprobs(rl, targets, 0)
    rd, _ = C.token_logprobs_grad(rl, targets, want["lse"], d_logp=np.full(rows, -1.0 / (rows - 2)))
    rdo = (rd @ f64(head).T).reshape(rows, qh, dim)
    (rdq, rdk, rdv), _ = C.prompt_attention_grad(rdo, rq, rk, f64(v), cu, dim ** -0.5)
    exact = [(x.reshape(rows, -1).T @ x.reshape(rows, -1)) / rows for x in (rot(rdq, True), rot(rdk, True), rdv)]
    # Seven roundings to the type on the way (q and k, out, logits, dlogits, dout, dq or dk or dv,
    # turned back), each of half a step and largely their own, and those of weights and ds; a
    # logit of size 20 moves its probability by 20 half steps more.  Squared in the Gram: twice.
    bound = 2 * HALF[dtype] * (10 + 20) + 2000 * U
    loss, rloss = -float(got["logp"].double().sum()), -want["logp"].sum()
    assert abs(loss - rloss) < bound * (abs(rloss) + rows)
    for a, b in zip(grams, exact):
        assert np.linalg.norm(f64(a) - b) < bound * np.linalg.norm(b)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("lengths,dim,window", [([1, 1, 1], 64, 0), ([1] * 70, 128, 0), ([50, 3], 64, 1), ([40], 256, 1)])
def test_grad_of_rows_that_see_themselves(lengths, dim, window, dtype):
    """A weight of 1 whatever the scores are: nothing goes back to q and k, all of it to v."""
    q, k, v, do, cu = prompt_case(lengths, 4, 2, dim, dtype, 91)
    args = [t.to(DEV) for t in (q, k, v)]
    out, lse = kq.kronq_prompt_attention(*args, dev(cu), window=window, want_lse=True)
    dq, dk, dv = kq.kronq_prompt_attention_grad(do.to(DEV), *args, out, lse, dev(cu), window=window)
    assert not dq.any() and not dk.any()
    check_backward(q, k, v, do, cu, out, lse, (dq, dk, dv), dtype, window)
