"""Rotary positions and log probabilities of tokens on the device against 64 bits."""
import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import calib_oracle as C
from calib_helpers import DEV, U, check_logprobs, check_logprobs_grad, f64, near, rotate_bound, typed

pytestmark = pytest.mark.gpu
DTYPES = (torch.float32, torch.bfloat16, torch.float16)
INF = float("inf")


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).to(DEV)


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="parts", factor=8.0, original=8192.0),
    dict(scaling="index", factor=16.0, original=4096.0, high=32.0, magnitude=1.277),
    dict(scaling="parts", factor=0.5, original=300.0, low=0.5, high=0.75),
])
@pytest.mark.parametrize("positions,dim,first,base", [(1, 2, 0, 10000.0), (33, 64, 7, 10000.0), (1000, 128, 0, 500000.0),
                                                     (70, 512, 130000, 500000.0), (31, 96, 2 ** 31 - 31, 10000.0)])
def test_rope_tables(kw, positions, dim, first, base):
    rope = kq.kronq_rope_tables(positions, dim, base=base, first=first, **kw)
    args = {n: v for n, v in kw.items() if n != "magnitude"}
    mag = kw.get("magnitude", 1.0)
    f = C.frequencies(dim, base, **args)
    cos, sin = C.tables(first, positions, f, mag)
    # the result's rounding; fp64: the frequency (2^-50), its product with the position, 32 turns
    angle = np.arange(first, first + positions)[:, None] * f
    for got, want in ((rope.cos, cos), (rope.sin, sin)):
        want = want.astype(np.float64)
        near(f64(got), want, 1.01 * (np.abs(want) * U + mag * (angle * 2.0 ** -50 + 2.0 ** -46)), "table")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,qh,kh,dim,rot,neighbours,back", [
    (1, 1, 0, 16, 16, False, False), (1, 32, 8, 128, 128, False, False), (5, 3, 1, 64, 32, True, False),
    (257, 8, 2, 96, 96, False, True), (33, 5, 5, 256, 64, True, True), (2, 1, 1, 512, 512, False, False),
    (3000, 20, 4, 128, 64, False, True),
])
def test_rotate(dtype, rows, qh, kh, dim, rot, neighbours, back):
    rng = np.random.default_rng(rows + dim)
    n = 50
    rope = kq.kronq_rope_tables(n, rot, base=10000.0, neighbours=neighbours)
    pos = rng.integers(0, n, rows).astype(np.int32)
    if rows > 4:
        pos[1], pos[3], pos[4] = -1, n, n - 1            # no sequence; no row in the tables
    q, k = typed(rng.normal(size=(rows, qh, dim)), dtype), typed(rng.normal(size=(rows, kh, dim)), dtype)
    cos, sin = f64(rope.cos), f64(rope.sin)
    qo, ko = torch.full_like(q, 7).to(DEV), torch.full_like(k, 7).to(DEV)
    got = kq.kronq_rotate(q.to(DEV), k.to(DEV) if kh else None, dev(pos), rope, back=back, q_out=qo,
                          k_out=ko if kh else None)
    # in place gives the same bits
    q2, k2 = q.to(DEV), k.to(DEV)
    kq.kronq_rotate(q2, k2 if kh else None, dev(pos), rope, back=back, q_out=q2, k_out=k2 if kh else None)
    for x, y, z in ((q, got[0], q2), (k, got[1], k2)):
        if x.shape[1] == 0:
            continue
        want, tol = rotate_bound(f64(x), pos, cos, sin, neighbours, back, dtype)
        y, z, x = f64(y), f64(z), f64(x)
        for r in range(rows):
            if want[r] is None:
                assert (y[r] == 7).all() and np.array_equal(z[r], x[r])
                continue
            near(y[r], want[r], tol[r], "row %d" % r)
            assert np.array_equal(y[r], z[r], equal_nan=True)
            if pos[r] < n:
                assert np.array_equal(y[r][:, rot:], x[r][:, rot:])


def test_rotate_strides_and_streams():
    """q and k of one packed tensor, gradients into another one, on a stream of its own."""
    rng = np.random.default_rng(3)
    rows, qh, kh, dim = 40, 6, 2, 64
    qkv = typed(rng.normal(size=(rows, (qh + 2 * kh) * dim)), torch.bfloat16).to(DEV)
    q, k = qkv[:, :qh * dim].view(rows, qh, dim), qkv[:, qh * dim:(qh + kh) * dim].view(rows, kh, dim)
    rope = kq.kronq_rope_tables(rows, dim)
    pos = torch.arange(rows, dtype=torch.int32, device=DEV)
    plain = kq.kronq_rotate(q.contiguous(), k.contiguous(), pos, rope)
    out = torch.zeros_like(qkv)
    oq, ok = out[:, :qh * dim].view(rows, qh, dim), out[:, qh * dim:(qh + kh) * dim].view(rows, kh, dim)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kq.kronq_rotate(q, k, pos, rope, q_out=oq, k_out=ok, stream=s)
    s.synchronize()
    assert torch.equal(oq, plain[0]) and torch.equal(ok, plain[1])
    assert not out[:, (qh + kh) * dim:].any()


def test_rotate_back_is_the_gradient():
    """By differences: sum(w rotate(x)) has the gradient rotate_back(w)."""
    rng = np.random.default_rng(4)
    rows, dim = 3, 32
    rope = kq.kronq_rope_tables(9, dim, magnitude=1.5)
    pos = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    x, w = rng.normal(size=(rows, 1, dim)), rng.normal(size=(rows, 1, dim))
    g, _ = kq.kronq_rotate(typed(w, torch.float32).to(DEV), None, pos, rope, back=True)
    for r, d in ((0, 5), (1, 2), (1, 20), (2, 31)):
        step = np.zeros_like(x)
        step[r, 0, d] = 1.0                              # linear: any step will do
        both = [f64(kq.kronq_rotate(typed(x + s * step, torch.float32).to(DEV), None, pos, rope)[0]) for s in (1, -1)]
        assert abs((w * (both[0] - both[1])).sum() / 2 - f64(g)[r, 0, d]) < 64 * 40 * U


# ---------------------------------------------------------------- log probabilities

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 1), (3, 2, 0), (2, 7, 5), (5, 255, 64), (2, 2048, 20), (300, 1000, 3),
                                            (4, 32003, 20), (2, 128256, 64), (260, 20000, 0), (17, 16385, 1)])
def test_logprobs(dtype, rows, vocab, top):
    rng = np.random.default_rng(vocab + rows)
    x = typed(rng.normal(size=(rows, vocab)) * 4, dtype)
    targets = rng.integers(0, vocab, rows).astype(np.int32)
    targets[rows // 2] = -1 if rows > 1 else targets[0]
    got = kq.kronq_token_logprobs(x.to(DEV), dev(targets), top=top, want_entropy=True)
    check_logprobs(got, f64(x), targets, top)
    again = kq.kronq_token_logprobs(x.to(DEV), None, top=top)
    assert "logp" not in again and "entropy" not in again
    assert torch.equal(got["lse"], again["lse"])
    if top:
        assert torch.equal(got["top_ids"], again["top_ids"]) and torch.equal(got["top_logp"], again["top_logp"])


def odd_rows(vocab, dtype, rng):
    """Rows where it can go wrong."""
    low = float(torch.finfo(dtype).min)
    x = [np.full(vocab, 1.5), np.full(vocab, -INF), np.full(vocab, low), np.zeros(vocab)]
    x[3][::2] = -0.0                                     # zeros of both signs are one value
    few = np.full(vocab, -INF)
    few[[vocab - 1, vocab // 2, 3]] = 2.0, 5.0, 2.0
    x += [few, np.where(np.isinf(few), low, few)]
    one = rng.normal(size=vocab)
    one[vocab // 3] = np.nan
    x.append(one)
    one = rng.normal(size=vocab)
    one[5] = INF
    x.append(one)
    x += [np.sort(rng.normal(size=vocab)), np.sort(rng.normal(size=vocab))[::-1].copy()]
    x.append(rng.integers(0, 3, vocab).astype(np.float64))            # many equal ones
    x.append(rng.normal(size=vocab) * 1e-3 + 300)
    # a few threads hold nearly all large values: what reaches the bound does not fit the list
    per = 128 // torch.finfo(dtype).bits                   # values of sixteen bytes
    thread = np.arange(vocab) // per % 256
    x.append(np.where(thread < 60, 50 + rng.random(vocab) * 10, rng.normal(size=vocab)))
    x.append(np.where(thread < 60, 50 + rng.random(vocab) * 10, -INF))
    return np.stack(x)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,top,many", [(700, 64, False), (40001, 64, False), (40001, 5, True), (128256, 61, True)])
def test_logprobs_of_odd_rows(dtype, vocab, top, many):
    """The same rows in a call of a few (in segments) and of many."""
    rng = np.random.default_rng(vocab)
    x = typed(odd_rows(vocab, dtype, rng), dtype)
    rows = x.shape[0]
    targets = rng.integers(0, vocab, rows).astype(np.int32)
    targets[0], targets[4] = vocab, 0                    # out of range; one that is masked
    d, t = x.to(DEV), dev(targets)
    if many:
        d, t = d.repeat(260 // rows + 1, 1), t.repeat(260 // rows + 1)
    got = kq.kronq_token_logprobs(d, t, top=top, want_entropy=True)
    if many:
        # other borders of sixteen bytes than the first ones', so other orders of sums
        check_logprobs({n: v[-rows:] for n, v in got.items()}, f64(x), targets, top)
        got = {n: v[:rows] for n, v in got.items()}
    check_logprobs(got, f64(x), targets, top)


@pytest.mark.parametrize("dtype", DTYPES)
def test_logprobs_of_rows_at_any_border(dtype):
    """Odd leading dimensions and first columns: rows start at every place of sixteen bytes."""
    rng = np.random.default_rng(5)
    whole = typed(rng.normal(size=(20, 5011)), dtype)
    for at in range(0, 9):
        x = whole[:, at:at + 4097 + at]
        targets = rng.integers(0, x.shape[1], 20).astype(np.int32)
        got = kq.kronq_token_logprobs(whole.to(DEV)[:, at:at + 4097 + at], dev(targets), top=7, want_entropy=True)
        check_logprobs(got, f64(x), targets, 7)


def grad_case(rows, vocab, dtype, top, seed):
    rng = np.random.default_rng(seed)
    x = typed(rng.normal(size=(rows, vocab)) * 3, dtype)
    targets = rng.integers(0, vocab, rows).astype(np.int32)
    if rows > 2:
        targets[1] = -1
    want = C.token_logprobs(f64(x), targets, top)
    kw = dict(d_logp=rng.normal(size=rows), entropy=want["entropy"], d_entropy=rng.normal(size=rows))
    if top:
        ids = want["top_ids"].astype(np.int32)
        if top > 2:
            ids[0, 1], ids[0, 2] = -1, ids[0, 0]         # none, and the same twice
            ids[-1, 0] = max(targets[-1], 0)
        kw.update(top_ids=ids, d_top=rng.normal(size=(rows, top)))
    kw = {n: v.astype(np.float32) if v.dtype == np.float64 else v for n, v in kw.items()}
    return x, targets, want["lse"].astype(np.float32), kw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,top", [(1, 1, 0), (3, 2, 1), (4, 1000, 5), (5, 16385, 64), (3, 32003, 3), (2, 128256, 0),
                                            (300, 50, 7)])
def test_logprobs_grad(dtype, rows, vocab, top):
    x, targets, lse, kw = grad_case(rows, vocab, dtype, top, vocab + top)
    for names in ((), ("d_logp",), ("entropy", "d_entropy"), ("top_ids", "d_top"), tuple(kw)):
        part = {n: v for n, v in kw.items() if n in names}
        if "top_ids" in names and not top:
            continue
        got = kq.kronq_token_logprobs_grad(x.to(DEV), dev(targets), dev(lse), **{n: dev(v) for n, v in part.items()})
        check_logprobs_grad(f64(got), f64(x), dtype, targets, lse.astype(np.float64),
                            **{n: v.astype(np.float64) if v.dtype == np.float32 else v for n, v in part.items()})


@pytest.mark.parametrize("dtype", DTYPES)
def test_logprobs_grad_in_place_and_at_any_border(dtype):
    x, targets, lse, kw = grad_case(6, 20011, dtype, 4, 9)
    args = {n: dev(v) for n, v in kw.items()}
    plain = kq.kronq_token_logprobs_grad(x.to(DEV), dev(targets), dev(lse), **args)
    same = x.to(DEV)
    kq.kronq_token_logprobs_grad(same, dev(targets), dev(lse), out=same, **args)
    assert torch.equal(same, plain)
    for at in (0, 1, 3):
        out = torch.full((6, 20021), 9.0, dtype=dtype, device=DEV)
        kq.kronq_token_logprobs_grad(x.to(DEV), dev(targets), dev(lse), out=out[:, at:at + 20011], **args)
        assert torch.equal(out[:, at:at + 20011], plain)
        assert (out[:, :at] == 9).all() and (out[:, at + 20011:] == 9).all()


def test_logprobs_grad_of_odd_rows():
    rng = np.random.default_rng(6)
    dtype, vocab = torch.float32, 900
    x = odd_rows(vocab, dtype, rng)
    rows = x.shape[0]
    x = typed(x, dtype)
    targets = np.full(rows, 3, dtype=np.int32)
    targets[3] = vocab + 5
    want = C.token_logprobs(f64(x), targets, 2)
    lse, ent = want["lse"].astype(np.float32), want["entropy"].astype(np.float32)
    g, h, e = (rng.normal(size=s).astype(np.float32) for s in (rows, rows, (rows, 2)))
    ids = want["top_ids"].astype(np.int32)
    got = kq.kronq_token_logprobs_grad(x.to(DEV), dev(targets), dev(lse), dev(g), dev(ent), dev(h), dev(ids), dev(e))
    with np.errstate(invalid="ignore"):
        check_logprobs_grad(f64(got), f64(x), dtype, targets, lse.astype(np.float64), d_logp=g.astype(np.float64),
                            entropy=ent.astype(np.float64), d_entropy=h.astype(np.float64), top_ids=ids,
                            d_top=e.astype(np.float64))


def test_logprobs_grad_by_differences():
    """Of sum(g logp + h entropy + e top_logp), with the kernel's own forward in fp32."""
    rng = np.random.default_rng(8)
    rows, vocab, top = 3, 40, 4
    x = rng.normal(size=(rows, vocab)) * 2
    targets = np.array([3, -1, 39], dtype=np.int32)
    g, h, e = rng.normal(size=rows), rng.normal(size=rows), rng.normal(size=(rows, top))
    first = kq.kronq_token_logprobs(typed(x, torch.float32).to(DEV), dev(targets), top=top, want_entropy=True)
    ids = first["top_ids"]
    got = f64(kq.kronq_token_logprobs_grad(typed(x, torch.float32).to(DEV), dev(targets), first["lse"],
                                           dev(g.astype(np.float32)), first["entropy"], dev(h.astype(np.float32)),
                                           ids, dev(e.astype(np.float32))))
    ids = ids.cpu().numpy()

    def loss(y):
        w = C.token_logprobs(y, targets, 0)
        m = np.log(np.exp(y).sum(-1))
        tops = np.take_along_axis(y, ids, 1) - m[:, None]
        return (g * w["logp"]).sum() + (h * w["entropy"]).sum() + (e * tops).sum()

    for r, v in ((0, 3), (0, 7), (1, int(ids[1, 0])), (2, 39), (2, 0), (1, 1)):
        step = np.zeros_like(x)
        step[r, v] = 1e-5
        want = (loss(x + step) - loss(x - step)) / 2e-5
        assert abs(want - got[r, v]) < 1e-4 * (1 + abs(want))


def test_logprobs_captured():
    """Two captured calls with one graph each, replayed over changing logits."""
    rng = np.random.default_rng(10)
    rows, vocab = 12, 20000
    x = torch.zeros((rows, vocab), dtype=torch.bfloat16, device=DEV)
    targets = torch.zeros(rows, dtype=torch.int32, device=DEV)
    d = torch.ones(rows, dtype=torch.float32, device=DEV)

    def work():
        got = kq.kronq_token_logprobs(x, targets, top=5, want_entropy=True)
        return got, kq.kronq_token_logprobs_grad(x, targets, got["lse"], d)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, grad = work()
    for i in range(4):
        x.copy_(typed(rng.normal(size=(rows, vocab)) * (i + 1), torch.bfloat16))
        targets.copy_(torch.from_numpy(rng.integers(0, vocab, rows).astype(np.int32)))
        graph.replay()
        torch.cuda.synchronize()
        want, wgrad = work()
        torch.cuda.synchronize()
        assert all(torch.equal(got[n], want[n]) for n in want) and torch.equal(grad, wgrad)
