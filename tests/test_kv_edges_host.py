"""4-bit paged key/value cache without a GPU: batches at the edge of what the
calls allow, through the kernels' index functions (built for the host)."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from test_kv_host import Raw

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "post_quantization_02_amd", "csrc")


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("kv") / "edges.so")
    subprocess.run(["/opt/rocm/bin/hipcc", "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared",
                    "-ftrapv", "-I", CSRC, os.path.join(HERE, "kv_edges_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def test_attention_and_append_place_a_row_alike(index):
    rng = np.random.default_rng(2)
    big = 2 ** 31 - 1
    for n in range(400):
        seqs = int(rng.integers(1, 6))
        ctx = rng.integers(-5, 90, seqs).astype(np.int32)
        cu = np.concatenate([[rng.integers(-20, 3)], rng.integers(0, 30, seqs)]).cumsum().astype(np.int32)
        if n % 4 == 0:
            ctx[rng.integers(seqs)] = rng.choice([big, -big - 1])
            cu[-1] = big
        # as many rows as cu names, fewer, and more
        rows = max(0, min(int(cu[-1]), 150) + int(rng.integers(-40, 10)))
        assert index.places_differ(ptr(ctx), ptr(cu), seqs, rows) == 0, (ctx, cu, rows)


def test_attention_refuses_more_sequences_than_it_can_look_through():
    # each unit of work goes through all sequences: a call of 2^20 would hold the GPU for minutes
    for seqs in ((1 << 14) + 1, 1 << 20):
        a = Raw()
        a.batch.seqs, a.rows = seqs, seqs
        assert a.attention() == kq.KRONQ_EUNSUPPORTED and b"2^14" in kq.load().kronq_last_error()
        assert kq.load().kronq_kv_attention_ws(seqs, seqs, 8, 8, 128) == 0
    assert kq.load().kronq_kv_attention_ws(1 << 14, 1 << 14, 8, 8, 128) > 0


def test_a_stream_of_another_device_is_refused():
    # default streams of all devices have handle 0: the call would run beside the caller's work, not after it
    class Stream:
        device, cuda_stream = torch.device("cuda:1"), 0

    with pytest.raises(ValueError, match="stream"):
        kq._on_stream(torch.device("cuda:0"), Stream())
