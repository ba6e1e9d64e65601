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
