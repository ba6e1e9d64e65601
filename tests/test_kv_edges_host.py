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


def places(index, ctx, cu, rows, share, bm, kt, units, aim, spare, least, sane):
    most = ctypes.c_int(0)
    st = index.places_suffice(ptr(ctx), ptr(cu), len(ctx), 1 << 13, rows, share, bm, kt, units, aim, spare, least,
                              int(sane), ctypes.byref(most))
    return st, most.value


@pytest.mark.parametrize("bm,kt", [(16, 32), (32, 32), (128, 64), (256, 64)])
def test_cut_sequences_have_places_for_their_chunks(index, bm, kt):
    rng = np.random.default_rng(bm + kt)
    for n in range(400):
        seqs, share = int(rng.integers(1, 120)), int(rng.choice([1, 3, 4, 16]))
        long = rng.random(seqs) < 0.05
        ctx = np.where(long, rng.integers(1, 60000, seqs), rng.integers(0, 700, seqs)).astype(np.int32)
        new = np.minimum(ctx, rng.integers(0, 400 if n % 3 == 0 else 3, seqs))
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rows = int(cu[-1])
        sane = n % 4 != 0
        if not sane:                       # any content: overlapping rows, ends before starts
            cu = rng.integers(-5, rows + 5, seqs + 1).astype(np.int32)
        tiles = (rows * share + (bm - 1) * min(rows, seqs)) // bm
        aim, least = int(rng.choice([1, 5, 23, 93, 744])), int(rng.choice([1, 4, 8]))
        spare = max(aim // 2, 1)
        st, _ = places(index, ctx, cu, rows, share, bm, kt, tiles + max(aim - tiles // 2, spare), aim, spare, least, sane)
        assert st == 0, (n, st)


def test_a_long_sequence_is_cut_however_many_there_are(index):
    # as 256 single tokens of 8 key heads are planned, one of them 131071 keys behind
    ctx = np.array([131071] + [500] * 255, np.int32)[np.random.default_rng(0).permutation(256)]
    cu = np.arange(257, dtype=np.int32)
    st, chunks = places(index, ctx, cu, 256, 4, 16, 32, 256 + 46, 93, 46, 8, True)
    assert st == 0 and chunks >= 10
    st, chunks = places(index, np.full(256, 4000, np.int32), cu, 256, 4, 16, 32, 256 + 46, 93, 46, 8, True)
    assert st == 0 and chunks == 1         # equal ones are not


@pytest.mark.parametrize("rows,seqs,q_heads,heads,dim", [(256, 256, 64, 8, 128), (200, 200, 64, 8, 128),
                                                         (48, 48, 32, 32, 128), (20000, 60, 32, 8, 128),
                                                         (1 << 14, 1 << 14, 8, 8, 64), (40000, 300, 16, 4, 256)])
def test_full_batches_leave_workspace_for_chunks(rows, seqs, q_heads, heads, dim):
    need = kq.load().kronq_kv_attention_ws(rows, seqs, q_heads, heads, dim)
    assert need >= 2 * 16 * (dim + 2) * 4  # two chunks of a row tile at least


def test_workspace_is_bounded():
    # both kernels' chunks of all key heads: twice 744 of 16 rows, twice 512 of 128 (or 256 of 256)
    for rows in (1, 10, 100, 500, 1000, 1100, 4000, 1 << 17, 1 << 20, 1 << 22):
        for seqs in (1, 2, 8, 64, 256, 1 << 14):
            for q_heads, heads in ((1, 1), (8, 8), (32, 8), (64, 8), (16, 4), (64, 1), (128, 128)):
                for dim in (64, 128, 256):
                    if rows * q_heads <= 1 << 26:
                        need = kq.load().kronq_kv_attention_ws(rows, seqs, q_heads, heads, dim)
                        assert 16 <= need <= (2 * 744 * 16 + 2 * 512 * 128) * (dim + 2) * 4 + 16
