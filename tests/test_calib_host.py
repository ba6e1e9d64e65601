"""A calibration pass's operators without a GPU: the oracle against hand-worked values and
differences, the calls' refusals, and the kernels' index functions built for the host."""
import ctypes
import math
import os
import subprocess

import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import calib_oracle as C

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "post_quantization_02_amd", "csrc")


# ---------------------------------------------------------------- index functions

@pytest.fixture(scope="module")
def host(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("prompt") / "prompt_index.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-ftrapv", "-I", CSRC, os.path.join(HERE, "prompt_index_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def test_rows_stay_inside_for_any_cu(host):
    ends = (-2 ** 31, -2 ** 31 + 1, -5, -1, 0, 1, 39, 40, 41, 2 ** 22, 2 ** 31 - 2, 2 ** 31 - 1)
    for rows in (1, 40, 2 ** 22):
        for lo in ends:
            for hi in ends:
                assert host.rows_inside(lo, hi, rows) == 0, (lo, hi, rows)


@pytest.mark.parametrize("bm,kt", [(128, 64), (128, 32), (32, 32)])
def test_tiles_hold_every_visible_pair(host, bm, kt):
    for n in (1, 31, 32, 33, 127, 128, 129, 300):
        for window in (0, 1, 2, 31, 32, 33, 64, 127, 200, n, n + 1):
            assert host.tiles_cover(n, window, bm, kt) == 0, (n, window)


# ---------------------------------------------------------------- oracle

def test_frequencies_by_hand():
    assert list(C.frequencies(4, 100.0)) == [1.0, 0.1]
    assert list(C.frequencies(4, 100.0, "linear", factor=4.0)) == [0.25, 0.025]
    # turns over the original 20 pi positions: 10 and 1; kept whole from 4 on, not at all up to 1
    f = C.frequencies(4, 100.0, "parts", factor=4.0, original=20 * math.pi, low=1.0, high=4.0)
    assert np.allclose(f, [1.0, 0.025], rtol=1e-12)
    # half way between the two borders
    f = C.frequencies(4, 100.0, "parts", factor=4.0, original=20 * math.pi, low=0.5, high=1.5)
    assert np.allclose(f, [1.0, 0.1 * 0.5 + 0.025 * 0.5], rtol=1e-12)
    # places 4 log(10 / r) / (2 log 100): r = 10 at 0, r = 0.1 at 2; pair 1 is half way
    f = C.frequencies(4, 100.0, "index", factor=4.0, original=20 * math.pi, low=0.1, high=10.0)
    assert np.allclose(f, [1.0, 0.1 * 0.5 + 0.025 * 0.5], rtol=1e-9)


def test_rotation_by_hand_and_back():
    cos, sin = np.array([[1.0, 1.0], [0.0, -1.0]]), np.array([[0.0, 0.0], [1.0, 0.0]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]], [[1.0, 2.0, 3.0, 4.0, 5.0]]])
    y = C.rotate(x, [0, 1], cos, sin, False, False)
    assert y[0].tolist() == x[0].tolist() and y[1].tolist() == [[-3, -2, 1, -4, 5]]
    y = C.rotate(x, [1, -1], cos, sin, True, False)
    assert y[0].tolist() == [[-2, 1, -3, -4, 5]] and y[1] is None
    back = C.rotate(np.array([[[-2.0, 1, -3, -4, 5]]]), [1], cos, sin, True, True)
    assert back[0].tolist() == x[0].tolist()


def test_attention_by_hand():
    q = np.array([[[0.0]], [[1.0]], [[1.0]]])
    k = np.array([[[5.0]], [[0.0]], [[math.log(3.0)]]])
    v = np.array([[[1.0]], [[2.0]], [[10.0]]])
    out, lse = C.prompt_attention(q, k, v, [0, 1, 3], 1.0)
    assert out[0, 0, 0] == 1.0 and lse[0, 0] == 0.0
    assert out[1, 0, 0] == 2.0
    assert np.isclose(out[2, 0, 0], (2 + 30) / 4) and np.isclose(lse[2, 0], math.log(4))
    out, _ = C.prompt_attention(q, k, v, [0, 3], 1.0, window=1)
    assert out[:, 0, 0].tolist() == [1.0, 2.0, 10.0]


@pytest.mark.parametrize("window", (0, 3))
def test_attention_gradients_by_differences(window):
    rng = np.random.default_rng(0)
    cu = [0, 5, 5, 9]
    args = [rng.normal(size=(9, h, 8)) for h in (4, 2, 2)]
    w = rng.normal(size=(9, 4, 8))
    grads, size = C.prompt_attention_grad(w, *args, cu, 0.3, window)
    for n in range(3):
        assert (np.abs(grads[n]) <= size[n] * 2 + 1e-12).all()
        for _ in range(6):
            at = tuple(rng.integers(0, s) for s in args[n].shape)
            both = []
            for sign in (1, -1):
                moved = [t.copy() for t in args]
                moved[n][at] += sign * 1e-6
                both.append((C.prompt_attention(*moved, cu, 0.3, window)[0] * w).sum())
            assert np.isclose((both[0] - both[1]) / 2e-6, grads[n][at], rtol=1e-6, atol=1e-8)


def test_log_probabilities_by_hand_and_by_differences():
    x = np.log(np.array([[1.0, 2.0, 5.0, 2.0], [1.0, 1.0, 1.0, 1.0]]))
    got = C.token_logprobs(x, np.array([1, -1]), 3)
    assert np.allclose(got["logp"], [math.log(0.2), 0]) and np.allclose(got["lse"], [math.log(10), math.log(4)])
    assert got["top_ids"].tolist() == [[2, 1, 3], [0, 1, 2]]
    assert np.isclose(got["entropy"][1], math.log(4))
    rng = np.random.default_rng(1)
    x = rng.normal(size=(2, 6))
    t, ids = np.array([3, -1]), np.array([[0, 3], [5, 5]])
    g, h, e = rng.normal(size=2), rng.normal(size=2), rng.normal(size=(2, 2))
    first = C.token_logprobs(x, t, 0)
    grad, size = C.token_logprobs_grad(x, t, first["lse"], g, first["entropy"], h, ids, e)

    def loss(y):
        w = C.token_logprobs(y, t, 0)
        return (g * w["logp"] + h * w["entropy"]).sum() + (e * (np.take_along_axis(y, ids, 1) - w["lse"][:, None])).sum()

    for at in np.ndindex(*x.shape):
        step = np.zeros_like(x)
        step[at] = 1e-6
        assert np.isclose((loss(x + step) - loss(x - step)) / 2e-6, grad[at], rtol=1e-6, atol=1e-8)
    assert (np.abs(grad) <= size + 1e-12).all()


# ---------------------------------------------------------------- refusals

OK, EINVAL, EWORKSPACE, EUNSUPPORTED = 0, 1, 4, 5
P = 0x10000                                              # an aligned address: nothing is launched


def heads(data=P, row=512, head=64):
    return kq._Heads(data, row, head)


def rope(cos=P, sin=P, ld=32, positions=10, dim=64, neighbours=0):
    return kq._Rope(cos, sin, ld, positions, dim, neighbours)


def scaling(base=10000.0, factor=1.0, original=100.0, low=1.0, high=4.0, magnitude=1.0, kind=0):
    return kq._RopeScaling(base, factor, original, low, high, magnitude, kind)


@pytest.mark.parametrize("status,change", [
    (OK, dict(positions=0, cos=None)), (EINVAL, dict(cos=None)), (EINVAL, dict(sin=None)), (EINVAL, dict(dim=3)),
    (EINVAL, dict(dim=0)), (EINVAL, dict(dim=514)), (EINVAL, dict(ld=31)), (EINVAL, dict(first=-1)),
    (EINVAL, dict(positions=-1)), (EINVAL, dict(first=2 ** 31, positions=1)), (EINVAL, dict(first=2 ** 62, positions=2 ** 62)),
    (EINVAL, dict(c=None)), (EINVAL, dict(c=scaling(kind=4))), (EINVAL, dict(c=scaling(kind=-1))),
    (EINVAL, dict(c=scaling(base=1.0))), (EINVAL, dict(c=scaling(base=math.inf))), (EINVAL, dict(c=scaling(base=math.nan))),
    (EINVAL, dict(c=scaling(factor=0.0))), (EINVAL, dict(c=scaling(magnitude=math.nan))),
    (EINVAL, dict(c=scaling(kind=2, low=4.0))), (EINVAL, dict(c=scaling(kind=3, original=0.0))),
    (EINVAL, dict(c=scaling(kind=3, low=0.0))), (EINVAL, dict(c=scaling(kind=2, high=math.inf))),
    (EUNSUPPORTED, dict(positions=2 ** 31, dim=512, ld=256)),
])
def test_rope_tables_refusals(status, change):
    a = dict(cos=P, sin=P, ld=32, first=0, positions=5, dim=64, c=scaling())
    a.update(change)
    assert kq.load().kronq_rope_tables(a["cos"], a["sin"], a["ld"], a["first"], a["positions"], a["dim"],
                                       a["c"], None) == status


@pytest.mark.parametrize("status,change", [
    (OK, dict(rows=0, q=None, pos=None)), (EINVAL, dict(qh=0)), (EINVAL, dict(kh=-1)), (EINVAL, dict(dtype=7)),
    (EINVAL, dict(rows=-1)), (EUNSUPPORTED, dict(rows=2 ** 22 + 1)), (EUNSUPPORTED, dict(rows=2 ** 22, qh=8, kh=9)),
    (EINVAL, dict(dim=0)), (EUNSUPPORTED, dict(dim=72)), (EUNSUPPORTED, dict(dim=528)), (EINVAL, dict(rope=None)),
    (EINVAL, dict(rope=rope(cos=None))), (EINVAL, dict(rope=rope(dim=80, ld=40))), (EUNSUPPORTED, dict(rope=rope(dim=24))),
    (EINVAL, dict(rope=rope(ld=30))), (EINVAL, dict(pos=None)), (EINVAL, dict(q=None)), (EINVAL, dict(q=heads(P + 8))),
    (EINVAL, dict(q=heads(row=516))), (EINVAL, dict(qo=heads(head=32))), (EINVAL, dict(k=None)), (EINVAL, dict(ko=None)),
    (EINVAL, dict(qo=heads(row=1024))), (EINVAL, dict(ko=heads(2 * P, row=1024))),
    (EUNSUPPORTED, dict(rows=2 ** 22, qh=15, kh=1, dtype=0, dim=512, q=heads(row=8192, head=512), k=heads(2 * P, 8192, 512),
                        qo=heads(row=8192, head=512), ko=heads(2 * P, 8192, 512))),
])
def test_rotate_refusals(status, change):
    a = dict(q=heads(), qh=8, k=heads(2 * P), kh=2, dtype=1, rows=4, dim=64, pos=P, rope=rope(), back=0,
             qo=heads(), ko=heads(2 * P))
    a.update(change)
    assert kq.load().kronq_rotate(a["q"], a["qh"], a["k"], a["kh"], a["dtype"], a["rows"], a["dim"], a["pos"], a["rope"],
                                  a["back"], a["qo"], a["ko"], None) == status


PROMPT = [
    (OK, dict(rows=0, q=None, cu=None)), (OK, dict(seqs=0, q=None, cu=None)), (EINVAL, dict(dtype=3)), (EINVAL, dict(rows=-1)),
    (EINVAL, dict(heads=0)), (EINVAL, dict(qh=7)), (EINVAL, dict(qh=0)), (EINVAL, dict(dim=0)), (EUNSUPPORTED, dict(dim=60)),
    (EUNSUPPORTED, dict(dim=264)), (EINVAL, dict(seqs=-1)), (EUNSUPPORTED, dict(seqs=2 ** 14 + 1)), (EINVAL, dict(cu=None)),
    (EINVAL, dict(scale=0.0)), (EINVAL, dict(scale=-1.0)), (EINVAL, dict(scale=math.inf)), (EINVAL, dict(scale=math.nan)),
    (EINVAL, dict(window=-1)), (EUNSUPPORTED, dict(rows=2 ** 22 + 1)), (EUNSUPPORTED, dict(rows=2 ** 22, qh=32)),
    (EINVAL, dict(q=None)), (EINVAL, dict(k=None)), (EINVAL, dict(v=None)), (EINVAL, dict(out=None)),
    (EINVAL, dict(q=heads(P + 4))), (EINVAL, dict(v=heads(row=257))), (EINVAL, dict(k=heads(head=56))),
    (EUNSUPPORTED, dict(q=heads(row=2 ** 22 + 8))), (EUNSUPPORTED, dict(seqs=2 ** 14, qh=1024, heads=1024)),
]


def prompt_args(change):
    a = dict(q=heads(), k=heads(), v=heads(), out=heads(), dout=heads(), dtype=1, rows=5, qh=8, heads=2, dim=64, cu=P, seqs=2,
             scale=0.125, window=0, lse=P, dq=heads(), dk=heads(), dv=heads(), ws=P, bytes=1 << 40)
    a.update(change)
    return a


@pytest.mark.parametrize("status,change", PROMPT)
def test_prompt_attention_refusals(status, change):
    a = prompt_args(change)
    got = kq.load().kronq_prompt_attention(a["q"], a["k"], a["v"], a["dtype"], a["rows"], a["qh"], a["heads"], a["dim"], a["cu"],
                                           a["seqs"], a["scale"], a["window"], a["out"], a["lse"], None)
    assert got == status


@pytest.mark.parametrize("status,change", PROMPT + [
    (EINVAL, dict(lse=None)), (EINVAL, dict(dout=None)), (EINVAL, dict(dq=None)), (EINVAL, dict(dk=None)), (EINVAL, dict(dv=None)),
    (EINVAL, dict(dv=heads(P + 2))), (EWORKSPACE, dict(ws=None)), (EWORKSPACE, dict(bytes=5 * 8 * 8 - 1)), (EINVAL, dict(ws=P + 8)),
])
def test_prompt_attention_grad_refusals(status, change):
    a = prompt_args(change)
    got = kq.load().kronq_prompt_attention_grad(a["dout"], a["q"], a["k"], a["v"], a["out"], a["lse"], a["dtype"], a["rows"],
                                                a["qh"], a["heads"], a["dim"], a["cu"], a["seqs"], a["scale"], a["window"],
                                                a["dq"], a["dk"], a["dv"], a["ws"], a["bytes"], None)
    assert got == status


def test_prompt_attention_grad_ws():
    ws = kq.load().kronq_prompt_attention_grad_ws
    assert ws(5, 8) == 5 * 8 * 2 * 4
    assert [ws(0, 8), ws(5, 0), ws(2 ** 22 + 1, 1), ws(2 ** 22, 17), ws(1, 65536)] == [0] * 5


@pytest.mark.parametrize("status,change", [
    (OK, dict(rows=0, logits=None)), (EINVAL, dict(dtype=3)), (EINVAL, dict(rows=-1)), (EINVAL, dict(vocab=0)), (EINVAL, dict(ld=99)),
    (EINVAL, dict(top=-1)), (EINVAL, dict(vocab=50, ld=50, top=51)), (EUNSUPPORTED, dict(top=65)), (EUNSUPPORTED, dict(rows=2 ** 22 + 1)),
    (EUNSUPPORTED, dict(vocab=2 ** 24 + 1, ld=2 ** 25)), (EINVAL, dict(logits=None)), (EINVAL, dict(logits=P + 1)),
    (EINVAL, dict(targets=None)), (EINVAL, dict(logp=None)), (EINVAL, dict(top_logp=None)), (EINVAL, dict(top_ids=None)),
    (EWORKSPACE, dict(vocab=128256, ld=128256, ws=None)), (EWORKSPACE, dict(vocab=128256, ld=128256, bytes=100)),
    (EINVAL, dict(vocab=128256, ld=128256, ws=P + 4)),
])
def test_token_logprobs_refusals(status, change):
    a = dict(logits=P, dtype=1, rows=4, vocab=100, ld=100, targets=P, logp=P, lse=P, entropy=P, top=3, top_logp=P, top_ids=P, ws=P,
             bytes=1 << 40)
    a.update(change)
    assert kq.load().kronq_token_logprobs(a["logits"], a["dtype"], a["rows"], a["vocab"], a["ld"], a["targets"], a["logp"],
                                          a["lse"], a["entropy"], a["top"], a["top_logp"], a["top_ids"], a["ws"], a["bytes"],
                                          None) == status


@pytest.mark.parametrize("status,change", [
    (OK, dict(rows=0, logits=None, out=None)), (EINVAL, dict(dtype=-1)), (EINVAL, dict(ld=99)), (EINVAL, dict(ld_out=99)),
    (EINVAL, dict(lse=None)), (EINVAL, dict(out=None)), (EINVAL, dict(out=2 * P + 1)), (EINVAL, dict(out=P, ld_out=128)),
    (EINVAL, dict(targets=None)), (EINVAL, dict(entropy=None)), (EINVAL, dict(top_ids=None)), (EUNSUPPORTED, dict(top=65)),
    (EUNSUPPORTED, dict(rows=2 ** 22, vocab=2 ** 24, ld=2 ** 24, ld_out=2 ** 24)),
])
def test_token_logprobs_grad_refusals(status, change):
    a = dict(logits=P, dtype=1, rows=4, vocab=100, ld=100, targets=P, lse=P, entropy=P, d_logp=P, d_entropy=P, top=3, top_ids=P,
             d_top=P, out=2 * P, ld_out=100)
    a.update(change)
    assert kq.load().kronq_token_logprobs_grad(a["logits"], a["dtype"], a["rows"], a["vocab"], a["ld"], a["targets"], a["lse"],
                                               a["entropy"], a["d_logp"], a["d_entropy"], a["top"], a["top_ids"], a["d_top"],
                                               a["out"], a["ld_out"], None) == status


def test_the_binding_refuses():
    x = torch.zeros(3, 2, 64)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        kq.kronq_prompt_attention(x, x, x, cu)           # on the host
    with pytest.raises(ValueError):
        kq.kronq_prompt_attention(x.double(), x, x, cu)
    with pytest.raises(ValueError):
        kq.kronq_prompt_attention_grad(x, x[0], x, x, x, x, cu)
    with pytest.raises(ValueError):
        kq.kronq_token_logprobs(torch.zeros(3, 5))
    with pytest.raises(ValueError):
        kq.kronq_token_logprobs(torch.zeros(3, 5, dtype=torch.int32))
    with pytest.raises(ValueError):
        kq.kronq_token_logprobs_grad(torch.zeros(3, 5), None, torch.zeros(3))
    with pytest.raises(ValueError):
        kq.kronq_rope_tables(4, 64, scaling="more")
    with pytest.raises(ValueError):
        kq.kronq_rope_tables(4, 64, device="cpu")
    with pytest.raises(ValueError):
        kq.kronq_rotate(x, None, cu, None)
