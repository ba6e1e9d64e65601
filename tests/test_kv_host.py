"""4-bit paged key/value cache without a GPU: the oracle against hand-worked
values, the calls' refusals, and the kernels' index functions (built for the
host) on valid batches and on any content of the batch arrays."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import kv_oracle as K
from kv_helpers import Case, attention_bound, f64

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "post_quantization_02_amd", "csrc")


# ---------------------------------------------------------------- oracle

def test_grid_by_hand():
    # -7 .. 8: a scale of 1, a zero point of 7
    x = np.array([-7.0, 8.0, 0.0, 0.5, 1.5, -0.5, 7.9, -6.6])
    codes, word = K.to_grid(x)
    assert K.word_scale(word) == 1.0 and word & 15 == 7
    assert list(codes) == [0, 15, 7, 8, 8, 6, 15, 0]       # 7.5 -> 8, 8.5 -> 8, 6.5 -> 6
    assert list(K.from_grid(codes, word)) == [-7, 8, 0, 1, 1, -1, 8, -7]


def test_grid_of_nothing_and_of_what_is_not_finite():
    codes, word = K.to_grid(np.zeros(4))
    # 2 / 15 is 0x3E088889 in fp32 and 0x3E088890 in 20 bits: a little more, so 1 / s is below 7.5
    assert word == 0x3E088890 | 7 and list(codes) == [7] * 4
    assert list(K.from_grid(codes, word)) == [0.0] * 4
    for bad in (np.nan, np.inf, -np.inf):
        codes, word = K.to_grid(np.array([1.0, bad]))
        assert word == K.NAN_WORD and np.isnan(K.from_grid(codes, word)).all()


def test_scale_has_twenty_bits_ties_to_even():
    one = 0x3F800000
    for low, up in ((0, 0), (7, 0), (8, 0), (9, 16), (15, 16), (16, 16), (24, 32), (25, 32), (23, 16)):
        x = float(np.uint32(one + low).view(np.float32))
        assert K.scale_word(x) == one + up
    assert K.word_scale(K.scale_word(0.0)) == 2.0 ** -126


def test_grid_error_is_half_a_step():
    rng = np.random.default_rng(0)
    for _ in range(50):
        x = rng.normal(size=64) * 10.0 ** rng.integers(-20, 20)
        codes, word = K.to_grid(x)
        s = K.word_scale(word)
        # the zero point's rounding moves the grid by up to half a step, where an end is cut off
        assert np.abs(K.from_grid(codes, word) - x).max() <= s * 1.0001
        inside = (codes > 0) & (codes < 15)
        assert np.abs(K.from_grid(codes, word) - x)[inside].max() <= s * 0.50001
        # the library's quantizer on the same group: same zero point, scale to 20 bits
        from oracle import kronq_oracle as O
        scale, zero = O.quant_params(x[None], 4)
        assert abs(scale[0] / s - 1) < 2.0 ** -19 and zero[0] == word & 15


def test_rotation_by_hand():
    rope = (np.array([[1, 1], [0, -1]], np.float32), np.array([[0, 0], [1, 0]], np.float32), False)
    x = np.array([1.0, 2.0, 3.0, 4.0, 5.0])
    assert list(K.rotate(x, 0, rope)) == [1, 2, 3, 4, 5]
    assert list(K.rotate(x, 1, rope)) == [-3, -2, 1, -4, 5]          # pairs (0, 2), (1, 3)
    assert list(K.rotate(x, 1, rope[:2] + (True,))) == [-2, 1, -3, -4, 5]


def test_visibility_by_hand():
    assert list(K.visible(5, 0, 3)) == [0, 1, 2, 3, 4, 5]
    assert list(K.visible(5, 2, 0)) == [4, 5]
    assert list(K.visible(5, 2, 1)) == [0, 4, 5]
    assert list(K.visible(1, 9, 4)) == [0, 1]
    assert list(K.visible(-1, 0, 4)) == []


def test_attention_equals_a_dense_softmax():
    c = Case([(20, 6), (7, 7)], heads=2, share=3, dim=64, rot=64, device="cpu")
    out, lse, _ = K.attention(c.cache, c.batch, f64(c.q), 0.125, 5, 2, c.rope)
    k = np.stack([K.held(c.cache, c.batch, 0, j, "k") for j in range(20)])
    v = np.stack([K.held(c.cache, c.batch, 0, j, "v") for j in range(20)])
    for r in range(6):
        for h in range(6):
            s = 0.125 * k[:, h // 3] @ K.rotate(f64(c.q)[r, h], 14 + r, c.rope)
            j = np.arange(20)
            s[(j > 14 + r) | ((j <= 14 + r - 5) & (j >= 2))] = -np.inf
            w = np.exp(s)
            assert np.allclose(out[r][h], (w / w.sum()) @ v[:, h // 3], rtol=1e-12)
            assert np.isclose(lse[r, h], np.log(w.sum()), rtol=1e-12)


def test_append_then_read_returns_the_grid_points():
    c = Case([(20, 6), (7, 7), (4, 0)], heads=2, dim=64, rot=32, device="cpu")
    K.append(c.cache, c.batch, f64(c.k), f64(c.v), c.rope)
    rows = K.rows_of(c.batch, c.rows)
    for r, x in enumerate(K.read(c.cache, c.batch, c.rows, "k")):
        for h in range(2):
            y = K.rotate(f64(c.k)[r, h], rows[r][1], c.rope)
            assert np.array_equal(x[h], K.from_grid(*K.to_grid(y)))


def test_the_bound_is_tight_enough_to_see_a_wrong_key():
    # leaving out one of 60 keys is outside the bound in most rows
    c = Case([(60, 3)], heads=2, share=2, dim=64, dtype=torch.float16, device="cpu")
    out, _, size = K.attention(c.cache, c.batch, f64(c.q), 0.125)
    p, slot = K.place(c.cache, c.batch, 0, 31)
    c.cache["v_grid"][p, :, slot] &= 15
    less, _, _ = K.attention(c.cache, c.batch, f64(c.q), 0.125)
    caught = [np.abs(less[r][h] - out[r][h]).max() >
              attention_bound(size[r], out[r], torch.float16, 64, 60, False)[h].min()
              for r in range(3) for h in range(4)]
    assert sum(caught) >= 10


# ---------------------------------------------------------------- refusals

class Raw:
    """Valid host arguments (addresses that are never followed) to spoil one at a time."""

    def __init__(self):
        a = 1 << 20
        self.cache = kq._Cache(a, 2 * a, 3 * a, 4 * a, 4 * 16 * 32, 4 * 16 * 32, 4 * 16, 4 * 16, 8, 4, 16, 64)
        self.batch = kq._Batch(5 * a, 6 * a, 7 * a, 10, 3, 10)
        self.rope = kq._Rope(8 * a, 9 * a, 16, 100, 32, 0)
        self.x = kq._Heads(10 * a, 256, 64)
        self.y = kq._Heads(11 * a, 512, 64)
        self.dtype, self.rows, self.qheads, self.scale, self.window, self.sinks = kq.KRONQ_BF16, 5, 8, 0.125, 0, 0
        self.ws, self.ws_bytes = 12 * a, 1 << 40

    def append(self):
        return kq.load().kronq_kv_append(self.x, self.x, self.dtype, self.rows, self.cache, self.batch, self.rope, None)

    def read(self):
        return kq.load().kronq_kv_read(self.x, self.x, self.dtype, self.rows, self.cache, self.batch, None)

    def attention(self):
        return kq.load().kronq_kv_attention(self.y, self.dtype, self.rows, self.qheads, self.cache, self.batch, self.rope,
                                            self.scale, self.window, self.sinks, self.y, None, self.ws, self.ws_bytes,
                                            None)


CACHE_BAD = [("cache.k_codes", None, 1), ("cache.v_grid", None, 1), ("cache.dim", 96, 5), ("cache.dim", 0, 1),
             ("cache.page", 24, 5), ("cache.page", 8, 5), ("cache.page", 2048, 5), ("cache.heads", 0, 1),
             ("cache.pages", 0, 1), ("cache.pages", 1 << 31, 1), ("cache.k_codes_stride", 2032, 1),
             ("cache.v_grid_stride", 60, 1), ("cache.v_codes_stride", 2056, 1), ("cache.k_grid_stride", 66, 1),
             ("cache.k_codes", (1 << 20) + 8, 1), ("cache.k_grid", (1 << 20) + 4, 1), ("batch.table", None, 1),
             ("batch.ctx", None, 1), ("batch.cu", None, 1), ("batch.seqs", -1, 1), ("batch.seqs", (1 << 20) + 1, 5),
             ("batch.columns", -1, 1), ("batch.ld_table", 9, 1), ("batch.columns", 1 << 27, 1), ("dtype", 3, 1),
             ("dtype", -1, 1), ("rows", -1, 1), ("rows", (1 << 22) + 1, 5)]
ROPE_BAD = [("rope.cos", None, 1), ("rope.sin", None, 1), ("rope.dim", 0, 1), ("rope.dim", 80, 1), ("rope.dim", 24, 5),
            ("rope.positions", 0, 1), ("rope.ld", 15, 1), ("rope.ld", 18, 1), ("rope.cos", (1 << 20) + 4, 1)]
X_BAD = [("x.data", None, 1), ("x.data", (1 << 20) + 2, 1), ("x.row_stride", 257, 1), ("x.head_stride", 68, 1),
         ("x.row_stride", 32, 1), ("x.head_stride", 0, 1)]
Y_BAD = [(n.replace("x.", "y."), v, s) for n, v, s in X_BAD]
ATTN_BAD = [("qheads", 6, 1), ("qheads", 0, 1), ("qheads", 1 << 17, 5), ("scale", 0.0, 1), ("scale", float("nan"), 1),
            ("scale", float("inf"), 1), ("scale", -1.0, 1), ("window", -1, 1), ("sinks", -1, 1), ("ws", None, 4),
            ("ws", (1 << 20) + 8, 1), ("ws_bytes", 100, 4)]


@pytest.mark.parametrize("call,bad", [("append", CACHE_BAD + ROPE_BAD + X_BAD), ("read", CACHE_BAD + X_BAD),
                                      ("attention", CACHE_BAD + ROPE_BAD + Y_BAD + ATTN_BAD)])
def test_refused_before_any_launch(call, bad):
    # KRONQ_EINVAL 1, KRONQ_EWORKSPACE 4, KRONQ_EUNSUPPORTED 5; no GPU is here to launch on
    for name, value, status in bad:
        a = Raw()
        if name == "batch.columns" and value > 1:
            a.batch.ld_table = value
            status = kq.KRONQ_EUNSUPPORTED
        at = a
        *path, last = name.split(".")
        for p in path:
            at = getattr(at, p)
        setattr(at, last, value)
        assert getattr(a, call)() == status, (name, value)
        assert kq.load().kronq_last_error()


@pytest.mark.parametrize("stride", ["k_codes_stride", "v_codes_stride", "k_grid_stride", "v_grid_stride"])
def test_page_strides_fit_32_bits(stride):
    for call in ("append", "read", "attention"):
        a = Raw()
        setattr(a.cache, stride, 1 << 32)
        assert getattr(a, call)() == kq.KRONQ_EUNSUPPORTED


def test_nothing_to_do_is_fine_without_operands():
    for call in ("append", "read", "attention"):
        a = Raw()
        a.rows, a.x.data, a.y.data, a.ws, a.ws_bytes = 0, None, None, None, 0
        assert getattr(a, call)() == 0
        a = Raw()
        a.batch.seqs, a.batch.table, a.batch.ctx, a.batch.cu = 0, None, None, None
        assert getattr(a, call)() == 0


def test_workspace_query():
    ws = kq.load().kronq_kv_attention_ws
    assert ws(1, 1, 32, 8, 128) > 0 and ws(1, 1, 32, 8, 128) % 16 == 0
    for bad in ((0, 1, 32, 8, 128), (1, 0, 32, 8, 128), (1, 1, 31, 8, 128), (1, 1, 4, 8, 128), (1, 1, 32, 0, 128),
                (1 << 23, 1, 32, 8, 128)):
        assert ws(*bad) == 0


def test_binding_refuses_what_is_not_on_a_device_or_misshapen():
    z = torch.zeros
    with pytest.raises(ValueError, match="device"):
        kq.KVCache(z((2, 1, 16, 32), dtype=torch.uint8), z((2, 1, 16, 32), dtype=torch.uint8),
                   z((2, 1, 16), dtype=torch.int32), z((2, 1, 16), dtype=torch.int32))
    with pytest.raises(ValueError, match="4|pages"):
        kq.KVCache(z((2, 16, 32), dtype=torch.uint8), *[None] * 3)
    with pytest.raises(ValueError, match="device"):
        kq.KVBatch(z((1, 2), dtype=torch.int32), z(1, dtype=torch.int32), z(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="device"):
        kq.Rope(z((4, 8)), z((4, 8)))


# ---------------------------------------------------------------- index functions

@pytest.fixture(scope="module")
def index(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("kv") / "index.so")
    subprocess.run(["/opt/rocm/bin/hipcc", "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-fPIC", "-shared",
                    "-ftrapv", "-I", CSRC, os.path.join(HERE, "kv_index_host.cpp"), "-o", out], check=True)
    return ctypes.CDLL(out)


def ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def cover(index, table, ctx, cu, pages, lgp, rows, share, window, sinks, bm, kt, units, least, sane):
    used = ctypes.c_int(0)
    t = np.ascontiguousarray(table, np.int32)
    st = index.units_cover(ptr(t), ptr(ctx), ptr(cu), len(ctx), t.shape[1], pages, lgp, rows, share, window, sinks, bm,
                           kt, units, least, int(sane), ctypes.byref(used))
    return st, used.value


@pytest.mark.parametrize("bm,kt", [(16, 32), (128, 64)])
def test_units_cover_each_visible_key_once(index, bm, kt):
    rng = np.random.default_rng(bm)
    for n in range(200):
        seqs = int(rng.integers(1, 9))
        share = int(rng.choice([1, 2, 3, 4, 7, 16, 20]))
        lengths = []
        for _ in range(seqs):
            ctx = int(rng.integers(0, 700))
            lengths.append((ctx, int(rng.integers(0, min(ctx, 300 if n % 3 else 3) + 1))))
        ctx = np.array([c for c, _ in lengths], np.int32)
        cu = np.concatenate([[0], np.cumsum([k for _, k in lengths])]).astype(np.int32)
        rows, columns = int(cu[-1]), 50
        table = rng.integers(0, 9, (seqs, columns))
        window, sinks = int(rng.choice([0, 1, 5, 64, 200])), int(rng.choice([0, 1, 33, 500]))
        least = int(rng.choice([1, 2, 8]))
        bound = (rows * share + (bm - 1) * min(rows, seqs)) // bm
        units = bound + int(rng.choice([1, 3, 40, 500]))
        st, used = cover(index, table, ctx, cu, 9, 4, rows, share, window, sinks, bm, kt, units, least, True)
        assert st == 0, (n, st, lengths, share, window, sinks, units)
        if bound and units > 2 * bound + 100:
            assert used >= sum(k > 0 for _, k in lengths)


@pytest.mark.parametrize("bm,kt", [(16, 32), (32, 32), (128, 64), (256, 64)])
def test_where_nothing_may_be_cut_no_unit_is_a_chunk(index, bm, kt):
    # units for every sequence's rows, of which few have any
    for lengths in ([(1000, 3)] * 20 + [(7, 0)] * 40, [(800, 780)] + [(7, 0)] * 11, [(0, 0), (64, 1)]):
        ctx = np.array([c for c, _ in lengths], np.int32)
        cu = np.concatenate([[0], np.cumsum([k for _, k in lengths])]).astype(np.int32)
        table = np.zeros((len(lengths), 70), np.int32)
        rows = int(cu[-1])
        st, used = cover(index, table, ctx, cu, 9, 4, rows, 2, 0, 0, bm, kt, rows + 100, 2 ** 31 - 1, True)
        assert st == 0 and used == sum(-(-2 * k // bm) for _, k in lengths)


def test_any_batch_content_stays_in_bounds(index):
    rng = np.random.default_rng(1)
    big = 2 ** 31 - 1
    for n in range(300):
        seqs, columns, pages, rows = int(rng.integers(1, 7)), int(rng.integers(0, 5)), int(rng.integers(1, 5)), 40
        lgp = int(rng.integers(4, 11))
        wild = lambda k: np.where(rng.random(k) < 0.3, rng.integers(-big - 1, big, k), rng.integers(-50, 90, k)).astype(np.int32)  # noqa: E731
        table, ctx, cu = wild((seqs, max(columns, 1)))[:, :columns], wild(seqs), wild(seqs + 1)
        if n % 5 == 0:
            ctx[0] = big
            cu[:2] = 0, rows
        t = np.ascontiguousarray(table)
        assert index.rows_in_bounds(ptr(t), ptr(ctx), ptr(cu), seqs, columns, pages, lgp, rows) == 0
        for bm, kt in ((16, 32), (128, 64)):
            room = max(columns << lgp, 1)
            window, sinks = int(rng.integers(0, room)), int(rng.integers(0, room + 1))
            st, _ = cover(index, t, ctx, cu, pages, lgp, rows, 4, window, sinks, bm, kt, 1 << 20, 1, False)
            assert st == 0
