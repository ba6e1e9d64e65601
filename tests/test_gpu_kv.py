"""4-bit paged key/value cache on the GPU against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import kv_oracle as K
from gpu_helpers import say
from kv_helpers import DEV, Case, cache_equal, check_attention, f64

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
ids = [str(t).replace("torch.", "") for t in TYPES]


def append_both(c, k=None, v=None):
    k, v = c.k if k is None else k, c.v if v is None else v
    cache, batch, rope = c.dev(kq)
    kq.kronq_kv_append(k.to(DEV), v.to(DEV), cache, batch, rope=rope)
    K.append(c.cache, c.batch, f64(k), f64(v), c.rope)
    return cache, batch


# ---------------------------------------------------------------- append, read

@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,page,rot,neighbours", [(64, 16, 64, False), (64, 32, 32, True), (128, 16, 128, True),
                                                     (128, 64, 48, False), (256, 16, 256, False), (256, 1024, 16, True),
                                                     (128, 32, 0, False)])
def test_append_equals_the_oracle_bit_for_bit(dtype, dim, page, rot, neighbours):
    say("append", dtype, dim, page, rot, neighbours)
    c = Case([(1, 1), (17, 17), (40, 3), (64, 0), (33, 16)], heads=3, dim=dim, page=page, dtype=dtype, rot=rot,
             neighbours=neighbours, padding=2, seed=dim + page)
    cache, _ = append_both(c)
    cache_equal(cache, c.cache)          # the tokens, and every slot left as it was


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_append_special_values(dtype):
    c = Case([(9, 9)], heads=2, dim=64, dtype=dtype, rot=32)
    big = torch.finfo(dtype).max
    c.k[0], c.v[0] = 0, 0                                  # nothing to scale by
    c.k[1], c.v[1] = float("nan"), 1
    c.k[2, :, 5], c.v[2, :, 60] = float("inf"), -float("inf")
    c.k[3], c.v[3] = big, -big
    c.k[4], c.v[4] = torch.finfo(dtype).smallest_normal, torch.finfo(dtype).smallest_normal / 4
    c.v[5] = torch.linspace(-3, 12, 64).to(dtype)          # ties: a scale of 1
    c.v[6] = torch.linspace(0, 7.5, 64).to(dtype)
    c.k[7], c.v[7] = 1, -1                                 # one side of zero
    c.v[8] = 0
    c.v[8, :, 3] = 1e-7
    cache, batch = append_both(c)
    cache_equal(cache, c.cache)
    k, v = kq.kronq_kv_read(cache, batch, c.rows)
    for nm, got in (("k", f64(k)), ("v", f64(v))):
        want = np.stack(K.read(c.cache, c.batch, c.rows, nm))
        with np.errstate(over="ignore"):
            assert np.array_equal(got, want.astype(np.float32), equal_nan=True)


def test_append_values_at_borders_take_the_even_side():
    # a scale of 1 and a zero point of 0 or 7: every half is a border
    c = Case([(2, 2)], heads=1, dim=64)
    c.v[0, 0] = torch.arange(64) % 31 / 2.0
    c.v[1, 0] = torch.arange(64) % 31 / 2.0 - 7
    cache, _ = append_both(c)
    cache_equal(cache, c.cache)
    assert K.word_scale(c.cache["v_grid"][c.table[0, 0], 0, 0]) == 1.0


def test_append_takes_strided_projections_and_leaves_padding():
    c = Case([(20, 4), (7, 7)], heads=2, share=3, dim=128, dtype=torch.bfloat16, rot=128, padding=3)
    cache, batch, rope = c.dev(kq)
    fused = torch.full((c.rows, 10, 128), float("nan"), dtype=torch.bfloat16, device=DEV)   # q k v of one product
    fused[:, 6:8], fused[:, 8:10] = c.k.to(DEV), c.v.to(DEV)
    kq.kronq_kv_append(fused[:, 6:8], fused[:, 8:10], cache, batch, rope=rope)
    heads_first = c.k.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)
    other, _, _ = c.dev(kq)
    kq.kronq_kv_append(heads_first, fused[:, 8:10], other, batch, rope=rope)
    K.append(c.cache, c.batch, f64(c.k), f64(c.v), c.rope)
    cache_equal(cache, c.cache)
    cache_equal(other, c.cache)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_read_rounds_the_held_values_once(dtype, dim, page):
    c = Case([(5, 5), (70, 33), (16, 0), (90, 1)], heads=3, dim=dim, page=page, dtype=dtype, padding=2)
    cache, batch, _ = c.dev(kq)
    k = torch.full((c.rows, 3, dim), 7.0, dtype=dtype, device=DEV)
    v = k.clone()
    kq.kronq_kv_read(cache, batch, c.rows, dtype=dtype, k=k, v=v)
    for nm, got in (("k", k), ("v", v)):
        want = torch.full((c.rows, 3, dim), 7.0, dtype=dtype)
        for r, x in enumerate(K.read(c.cache, c.batch, c.rows, nm)):
            if x is not None:
                want[r] = torch.from_numpy(x).to(torch.float32).to(dtype)     # exact in fp32
        assert torch.equal(got.cpu(), want)


def test_places_out_of_range_are_not_written_and_read_as_nan():
    c = Case([(40, 40), (30, 4), (10, 12), (8, 2)], heads=2, dim=64, rot=64, columns=2)   # room for 32 positions
    c.table[1, 1] = c.pages              # a page that is not there
    c.table[3, 0] = -1
    c.rope = (c.rope[0][:31], c.rope[1][:31], False)     # position 31 has no angle
    cache, batch = append_both(c)
    cache_equal(cache, c.cache)
    k, _ = kq.kronq_kv_read(cache, batch, c.rows)
    want = np.stack(K.read(c.cache, c.batch, c.rows, "k"))
    assert np.isnan(want[32:44]).all() and np.isnan(want[44:46]).all() and not np.isnan(want[46:56]).any()
    assert np.array_equal(f64(k), want.astype(np.float32), equal_nan=True)


def test_many_sequences():
    rng = np.random.default_rng(3)
    lengths = [(int(rng.integers(1, 40)), int(rng.integers(0, 2))) for _ in range(1100)]
    c = Case(lengths, heads=1, dim=64, dtype=torch.float16)
    cache, batch = append_both(c)
    cache_equal(cache, c.cache)
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, want_lse=True)
    check_attention(c, out, lse)


@pytest.mark.parametrize("heads,dim,new", [(11, 64, 1900), (3, 256, 9), (130, 64, 1), (8, 128, 2100)])
def test_append_and_read_of_head_blocks(heads, dim, new):
    # lane groups that take eight, fewer and one head each, and a last block of fewer
    c = Case([(new + 5, new), (40, min(new, 40)), (3, 0), (1, 1)], heads=heads, dim=dim, page=32,
             dtype=torch.bfloat16, rot=32, neighbours=True, padding=3, seed=heads)
    cache, batch = append_both(c)
    cache_equal(cache, c.cache)
    k, v = kq.kronq_kv_read(cache, batch, c.rows, k=torch.full((c.rows, heads, dim), 7.0, device=DEV),
                            v=torch.full((c.rows, heads, dim), 7.0, device=DEV))
    for t, nm in ((k, "k"), (v, "v")):
        rows = K.read(c.cache, c.batch, c.rows, nm)
        want = np.stack([np.full((heads, dim), 7.0) if r is None else r for r in rows])
        assert np.array_equal(f64(t), want.astype(np.float32))


@pytest.mark.parametrize("dim,dtype", [(64, torch.float16), (128, torch.bfloat16), (256, torch.float32)])
def test_append_groups_with_an_entry_that_is_not_finite(dim, dtype):
    # in the rotated part, behind it, and in the values: that group alone is lost
    c = Case([(20, 20)], heads=3, dim=dim, dtype=dtype, rot=dim // 2)
    for row, head, d, x in ((0, 0, 0, np.inf), (3, 1, dim // 4 - 1, -np.inf), (5, 2, dim - 1, np.nan), (6, 0, dim // 2, np.inf)):
        c.k[row, head, d] = x
        c.v[row + 1, head, d] = x
    cache, batch = append_both(c)
    cache_equal(cache, c.cache)
    k, v = kq.kronq_kv_read(cache, batch, c.rows)
    assert int(torch.isnan(k).any(-1).sum()) == 4 and int(torch.isnan(v).any(-1).sum()) == 4


# ---------------------------------------------------------------- attention

def attend(c, window=0, sinks=0, scale=None):
    cache, batch, rope = c.dev(kq)
    before = torch.full((c.rows, c.heads * c.share, c.dim), 3.0, dtype=c.dtype, device=DEV)
    out = before.clone()
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, scale=scale, window=window, sinks=sinks, rope=rope,
                                     out=out, want_lse=True)
    torch.cuda.synchronize()
    check_attention(c, out, lse, scale, window, sinks, f64(before))
    return out


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,share", [(1, 1), (3, 4), (2, 7), (1, 20)])
def test_one_token(dtype, dim, heads, share):
    say("one token", dtype, dim, heads, share)
    c = Case([(1, 1), (16, 1), (33, 1), (500, 1), (0, 0), (257, 1)], heads=heads, share=share, dim=dim, dtype=dtype,
             seed=dim + share)
    attend(c)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("page", [16, 32, 128, 1024])
def test_lengths_around_tiles(dtype, page):
    c = Case([(n, 1) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129)], heads=2, share=4, dim=128,
             page=page, dtype=dtype, rot=128, seed=page)
    attend(c)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rot,neighbours", [(0, False), (64, True), (32, False), (16, True)])
def test_several_rows_of_a_sequence(dtype, rot, neighbours):
    c = Case([(5, 5), (40, 3), (9, 0), (130, 17), (64, 1)], heads=2, share=3, dim=64, dtype=dtype, rot=rot,
             neighbours=neighbours, padding=3, seed=rot)
    attend(c)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,share", [(64, 5), (128, 4), (256, 2)])
def test_many_rows(dtype, dim, share):
    c = Case([(150, 150), (200, 77), (300, 1), (90, 40)], heads=1, share=share, dim=dim, page=32, dtype=dtype,
             rot=dim, padding=5, seed=dim)
    attend(c)


@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 1), (32, 4), (33, 40), (100, 0), (64, 1000), (5000, 2)])
@pytest.mark.parametrize("new", [1, 4, 90])
def test_window_and_first_tokens(window, sinks, new):
    c = Case([(1, 1), (130, min(new, 130)), (333, new), (96, min(new, 96))], heads=2, share=2, dim=64,
             dtype=torch.float16, rot=64, seed=window + sinks + new)
    attend(c, window, sinks)


def test_rows_that_see_nothing_are_zero():
    # more rows than positions: the first rows are before the sequence's start
    c = Case([(3, 5), (0, 2), (20, 1)], heads=2, share=2, dim=64)
    out = attend(c)
    assert not out[:2].any() and not out[5:7].any() and out[2:5].any()


@pytest.mark.parametrize("new", [2, 70])
def test_what_is_not_seen_does_not_matter(new):
    c = Case([(100, new), (200, new)], heads=2, share=2, dim=64, dtype=torch.bfloat16, seed=new)
    out = attend(c, 24, 3)
    # every slot that no row sees holds NaN and infinite scales now
    seen = np.zeros((c.pages, c.page), dtype=bool)
    for r, at in enumerate(K.rows_of(c.batch, c.rows)):
        for j in K.visible(at[1], 24, 3):
            p, slot = K.place(c.cache, c.batch, at[0], int(j))
            seen[p, slot] = True
    for nm in "kv":
        w = c.cache[nm + "_grid"]
        w[np.broadcast_to(~seen[:, None], w.shape)] = 0x7FC00003
        w[:, 1][~seen] = 0x7F800001
    # and the pages that hold none of them need no entry
    for i, (ctx, n) in enumerate(c.lengths):
        for col in range(-(-ctx // c.page)):
            if not seen[c.table[i, col]].any():
                c.table[i, col] = 1 << 30
    assert torch.equal(attend(c, 24, 3), out)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_values_that_are_not_numbers_reach_the_rows_that_see_them(dtype):
    c = Case([(100, 40), (50, 2)], heads=2, share=2, dim=64, dtype=dtype)
    p, slot = K.place(c.cache, c.batch, 0, 80)
    c.cache["v_grid"][p, 0, slot] = K.NAN_WORD
    p, slot = K.place(c.cache, c.batch, 1, 49)
    c.cache["k_grid"][p, 1, slot] = K.NAN_WORD
    c.q[5, 1, 7] = float("inf")
    c.q[6, 0, 0] = float("nan")
    attend(c)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_places_out_of_range_give_nan_to_the_rows_that_see_them(dtype):
    c = Case([(60, 40), (30, 3), (45, 1), (20, 2)], heads=2, share=2, dim=64, dtype=dtype, rot=64, columns=3)  # 48 positions
    c.table[1, 0] = -5
    c.table[3, 1] = c.pages
    c.rope = (c.rope[0][:44], c.rope[1][:44], True)
    attend(c)
    attend(c, 4, 0)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_scales_far_apart(dtype):
    # sharp weights, and value scales over thirteen orders of magnitude, largest last
    c = Case([(300, 2), (290, 2)], heads=2, share=2, dim=64, dtype=dtype, qscale=6.0)
    w = c.cache["v_grid"]
    for i in range(2):
        for j in range(c.lengths[i][0]):
            p, slot = K.place(c.cache, c.batch, i, j)
            s = np.float32(10.0 ** (-4 + 4 * j / 300)) if i == 0 else np.float32(10.0 ** (9 - 13 * j / 300))
            w[p, :, slot] = (s.view(np.uint32) & np.uint32(0xFFFFFFF0)) | (w[p, :, slot] & 15)
    attend(c)
    attend(c, scale=0.002)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("new", [2, 60])
def test_scales_far_apart_within_a_tile(dtype, new):
    # every few keys another magnitude; and one key that only later rows see is
    # beyond all others, which must not cost the earlier rows their precision
    c = Case([(250, new)], heads=2, share=2, dim=64, dtype=dtype)
    for nm, decades in (("k", 2), ("v", 12)):
        w = c.cache[nm + "_grid"]
        for j in range(250):
            p, slot = K.place(c.cache, c.batch, 0, j)
            s = np.float32(0.1 * 10.0 ** (-decades * (j % 5) / 4))
            if j == 248:
                s = np.float32(0.1 if nm == "k" else 1e3)
            w[p, :, slot] = (s.view(np.uint32) & np.uint32(0xFFFFFFF0)) | (w[p, :, slot] & 15)
    attend(c)
    attend(c, 30, 2)


def test_small_and_large_queries():
    c = Case([(80, 3)], heads=2, share=2, dim=64)
    c.q[0] *= 1e-30
    c.q[1] *= 2.0 ** 12
    c.q[2] = 0
    attend(c)


def test_long_context_is_cut_and_joined():
    c = Case([(9000, 2), (700, 1), (4100, 1)], heads=1, share=3, dim=64, page=64, dtype=torch.float32, rot=64)
    attend(c)
    attend(c, 2500, 5)


def test_many_rows_of_a_long_context_are_cut_and_joined():
    c = Case([(3500, 30), (200, 1), (1000, 90)], heads=1, share=2, dim=64, page=64, dtype=torch.bfloat16, rot=64)
    attend(c)
    attend(c, 700, 5)


@pytest.mark.parametrize("new", [1, 100])
def test_equal_calls_give_equal_bits(new):
    c = Case([(5000, new), (300, 2)], heads=2, share=4, dim=128, page=32, dtype=torch.bfloat16, rot=128)
    cache, batch, rope = c.dev(kq)
    q = c.q.to(DEV)
    first = kq.kronq_kv_attention(q, cache, batch, rope=rope)
    for _ in range(5):
        assert torch.equal(kq.kronq_kv_attention(q, cache, batch, rope=rope), first)


def test_strided_queries_and_outputs():
    c = Case([(50, 4), (33, 2)], heads=2, share=2, dim=128, dtype=torch.float16)
    cache, batch, _ = c.dev(kq)
    wide = torch.full((c.rows, 9, 128), float("nan"), dtype=torch.float16, device=DEV)
    wide[:, 2:6] = c.q.to(DEV)
    heads_first = torch.zeros((4, c.rows, 128), dtype=torch.float16, device=DEV).transpose(0, 1)
    out = kq.kronq_kv_attention(wide[:, 2:6], cache, batch, out=heads_first)
    assert out is heads_first
    check_attention(c, out, None)


def test_layers_share_a_buffer_past_32_bit_offsets():
    # pages of one layer 1.5 GB apart: the last ones begin past 2^32 bytes
    c = Case([(100, 3)], heads=2, share=2, dim=128, page=64, dtype=torch.bfloat16, rot=128)
    c.table[0, :2] = 3, 2
    own, batch, rope = c.dev(kq)
    per, stride = 2 * 64 * 64, 1500 << 20
    views = []
    pool = torch.empty((c.pages - 1) * stride + 4 * per, dtype=torch.uint8, device=DEV)
    for n, nm in enumerate(("k_codes", "v_codes")):
        t = pool.as_strided((c.pages, 2, 64, 64), (stride, 64 * 64, 64, 1), n * per)
        t.copy_(getattr(own, nm))
        views.append(t)
    words = pool[:4 * (pool.numel() // 4)].view(torch.int32)
    for n, nm in enumerate(("k_grid", "v_grid")):
        t = words.as_strided((c.pages, 2, 64), (stride // 4, 64, 1), (2 + n) * per // 4)
        t.copy_(getattr(own, nm))
        views.append(t)
    cache = kq.KVCache(*views)
    assert c.pages == 4 and 3 * stride > 1 << 32
    kq.kronq_kv_append(c.k.to(DEV), c.v.to(DEV), cache, batch, rope=rope)
    K.append(c.cache, c.batch, f64(c.k), f64(c.v), c.rope)
    cache_equal(cache, c.cache)
    out = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, rope=rope)
    check_attention(c, out, None)


def test_nothing_to_do():
    c = Case([(5, 0), (9, 0)], heads=2, dim=64)
    cache, batch, _ = c.dev(kq)
    empty = torch.empty((0, 2, 64), device=DEV)
    kq.kronq_kv_append(empty, empty, cache, batch)
    assert kq.kronq_kv_read(cache, batch, 0)[0].shape == (0, 2, 64)
    assert kq.kronq_kv_attention(torch.empty((0, 4, 64), device=DEV), cache, batch).shape == (0, 4, 64)
    none = kq.KVBatch(torch.empty((0, 3), dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV),
                      torch.zeros(1, dtype=torch.int32, device=DEV))
    out = torch.ones((2, 4, 64), device=DEV)
    kq.kronq_kv_attention(torch.ones((2, 4, 64), device=DEV), cache, none, out=out)
    assert bool((out == 1).all())
    cache_equal(cache, c.cache)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("page,window,sinks", [(16, 0, 0), (64, 0, 0), (32, 150, 3), (128, 40, 70)])
def test_prompts_among_single_tokens(dtype, page, window, sinks):
    # tiles of 256 rows for the prompts, 16 for the others, in one call
    c = Case([(520, 400), (33, 1), (470, 470), (7, 7), (300, 0), (900, 351)], heads=2, share=3, dim=64, page=page,
             dtype=dtype, rot=64, padding=2, seed=page)
    attend(c, window, sinks)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim", [128, 256])
def test_prompts_of_wide_heads(dtype, dim):
    c = Case([(300, 300), (411, 290)], heads=1, share=2, dim=dim, page=16, dtype=dtype, rot=dim // 2, neighbours=True,
             spread=2.0, seed=dim)
    attend(c)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("dim,page,window", [(64, 16, 0), (128, 16, 0), (128, 64, 700), (256, 32, 300), (64, 64, 5)])
def test_short_drafts(dtype, dim, page, window):
    # 17 to 32 rows x share on average, some sequences of fewer and of more
    c = Case([(1500, 6), (40, 6), (900, 1), (6, 6), (333, 9)], heads=2, share=4, dim=dim, page=page, dtype=dtype,
             rot=64, padding=1, seed=dim + page)
    attend(c, window, 3 if window else 0)


def test_chunks_of_uneven_rows_are_all_joined():
    # more rows than one a sequence, of so many query heads that 32 / share is one
    c = Case([(2600, 1), (2500, 4), (30, 1), (2700, 1), (2600, 1), (2600, 1), (2600, 1)], heads=1, share=20, dim=64,
             page=64, dtype=torch.float32)
    attend(c)


def test_sequences_that_share_pages():
    c = Case([(200, 1), (200, 4), (200, 90)], heads=2, share=2, dim=64, page=32, dtype=torch.float32, rot=64)
    c.table[1:] = c.table[0]
    attend(c)


# ---------------------------------------------------------------- streams, graphs, together

def test_two_calls_at_once():
    one = Case([(3000, 2), (700, 600)], heads=2, share=2, dim=128, page=64, dtype=torch.bfloat16, rot=128, seed=1)
    two = Case([(2000, 600), (2500, 1)], heads=2, share=2, dim=128, page=16, dtype=torch.float16, rot=64, seed=2)
    ready = [(c.dev(kq), c.q.to(DEV), torch.cuda.Stream()) for c in (one, two)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(3):
        for (cache, batch, rope), q, stream in ready:
            outs.append(kq.kronq_kv_attention(q, cache, batch, rope=rope, stream=stream))
    torch.cuda.synchronize()
    for i, c in enumerate((one, two)):
        check_attention(c, outs[i], None)
        assert torch.equal(outs[i], outs[i + 2]) and torch.equal(outs[i], outs[i + 4])


def test_two_captured_calls_with_workspaces_of_their_own():
    c = Case([(3000, 2), (700, 300), (90, 1)], heads=2, share=2, dim=64, page=32, dtype=torch.float16, rot=64)
    cache, batch, rope = c.dev(kq)
    qs = [c.q.to(DEV), c.q.to(DEV) * 0.5]
    need = kq.load().kronq_kv_attention_ws(c.rows, 3, 4, 2, 64)
    outs, graphs, side = [torch.empty_like(q) for q in qs], [], torch.cuda.Stream()
    spaces = [torch.empty(need, dtype=torch.uint8, device=DEV) for _ in qs]
    torch.cuda.synchronize()
    for q, out, ws in zip(qs, outs, spaces):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            kq.kronq_kv_attention(q, cache, batch, rope=rope, out=out, ws=ws)
    other = torch.cuda.Stream()
    for _ in range(4):
        for out in outs:
            out.fill_(float("nan"))
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for q, out in zip(qs, outs):
            assert torch.equal(out, kq.kronq_kv_attention(q, cache, batch, rope=rope))
        torch.cuda.synchronize()
        for q in qs:
            q.copy_(torch.randn_like(q))


@pytest.mark.parametrize("lengths", [[(1000, 3)] * 20 + [(7, 0)] * 40, [(800, 780)] + [(7, 0)] * 11],
                         ids=["few rows", "many rows"])
def test_row_tiles_enough_are_not_cut(lengths):
    # rows of few of the sequences: row tiles are less than the bound the launch is made for
    c = Case(lengths, heads=32, share=1, dim=64, page=64, dtype=torch.bfloat16, rot=64)
    cache, batch, rope = c.dev(kq)
    need = kq.load().kronq_kv_attention_ws(c.rows, len(lengths), 32, 32, 64)
    space = torch.full((need + (1 << 24),), 7, dtype=torch.uint8, device=DEV)
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, rope=rope, want_lse=True, ws=space[:need])
    check_attention(c, out, lse)
    assert bool((space[need:] == 7).all())


def test_a_workspace_that_is_too_small_is_replaced_and_a_wrong_one_refused():
    c = Case([(3000, 2)], heads=2, share=2, dim=64, page=32, dtype=torch.float32)
    cache, batch, _ = c.dev(kq)
    q = c.q.to(DEV)
    want = kq.kronq_kv_attention(q, cache, batch)
    assert torch.equal(kq.kronq_kv_attention(q, cache, batch, ws=torch.empty(16, dtype=torch.uint8, device=DEV)), want)
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, dtype=torch.int32, device=DEV)):
        with pytest.raises(ValueError):
            kq.kronq_kv_attention(q, cache, batch, ws=ws)


def test_another_stream():
    c = Case([(3000, 2), (40, 1)], heads=2, share=2, dim=128, page=16, dtype=torch.bfloat16, rot=128)
    cache, batch, rope = c.dev(kq)
    q, k, v = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kq.kronq_kv_append(k, v, cache, batch, rope=rope, stream=side)
    out = kq.kronq_kv_attention(q, cache, batch, rope=rope, stream=side)
    # memory that the call's workspace must not be lost to
    torch.full((1 << 22,), float("nan"), device=DEV)
    side.synchronize()
    K.append(c.cache, c.batch, f64(c.k), f64(c.v), c.rope)
    check_attention(c, out, None)


def test_a_captured_step_follows_the_batch():
    c = Case([(2900, 1), (60, 1), (17, 1)], heads=2, share=4, dim=128, page=16, dtype=torch.bfloat16, rot=128,
             columns=200)
    for i in range(3):                   # pages for the tokens to come
        c.table[i] = np.where(c.table[i] == -7, c.table[i, 0], c.table[i])
    c.rope = tuple(np.concatenate([x, x[:8]]) for x in c.rope[:2]) + (False,)
    cache, batch, rope = c.dev(kq)
    eager, _, _ = c.dev(kq)
    q, k, v = c.q.to(DEV), c.k.to(DEV), c.v.to(DEV)
    out = torch.empty_like(q)
    need = kq.load().kronq_kv_attention_ws(c.rows, 3, 8, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    ws2 = torch.empty(need, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kq.kronq_kv_append(k, v, cache, batch, rope=rope)
        kq.kronq_kv_attention(q, cache, batch, rope=rope, out=out, ws=ws)
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        kq.kronq_kv_append(k, v, eager, batch, rope=rope)
        want = kq.kronq_kv_attention(q, eager, batch, rope=rope, ws=ws2)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        cache_equal(cache, {n: getattr(eager, n).cpu().numpy().view(np.uint32 if n.endswith("grid") else np.uint8)
                            for n in ("k_codes", "v_codes", "k_grid", "v_grid")})
        batch.ctx.add_(1)                # the next token
        q.copy_(torch.randn_like(q))
        k.copy_(torch.randn_like(k))
        v.copy_(torch.randn_like(v))


def test_a_decoded_token_through_packed_weights():
    """q, k, v by packed products, the cache, and the output product: as a
    quantized layer decodes a token, twice in a row."""
    rng = np.random.default_rng(5)
    n, heads, share, dim = 256, 2, 2, 64
    qh = heads * share

    def layer(m, n_in):
        codes = torch.from_numpy(rng.integers(0, 16, (m, n_in), dtype=np.uint8)).to(DEV)
        scales = torch.from_numpy(rng.uniform(0.01, 0.02, (m, n_in // 128)).astype(np.float32)).to(DEV)
        zeros = torch.from_numpy(rng.integers(6, 10, (m, n_in // 128)).astype(np.float32)).to(DEV)
        dense = (f64(codes) - np.repeat(f64(zeros), 128, 1)) * np.repeat(f64(scales), 128, 1)
        packed = kq.kronq_pack_codes(codes, 4)
        call = lambda x: kq.kronq_decode_matvec(packed, n_in, 4, 128, scales, zeros, None, 1, None, 1, None, x)  # noqa: E731
        return call, dense

    (wq, dq), (wk, dk), (wv, dv), (wo, do) = layer(qh * dim, n), layer(heads * dim, n), layer(heads * dim, n), layer(n, qh * dim)
    c = Case([(60, 1)], heads=heads, share=share, dim=dim, rot=dim)
    c.rope = tuple(np.concatenate([x, x[:4]]) for x in c.rope[:2]) + (False,)
    cache, batch, rope = c.dev(kq)
    for step in range(2):
        x = torch.from_numpy(rng.normal(size=n).astype(np.float32)).to(DEV)
        q, k, v = wq(x).view(1, qh, dim), wk(x).view(1, heads, dim), wv(x).view(1, heads, dim)
        kq.kronq_kv_append(k, v, cache, batch, rope=rope)
        a = kq.kronq_kv_attention(q, cache, batch, rope=rope)
        y = wo(a.view(-1))
        # products in fp32: sums of 256 terms, each off by at most 256 half steps of its size
        for got, dense in ((q, dq), (k, dk), (v, dv)):
            far = np.abs(f64(got).reshape(-1) - dense @ f64(x))
            assert (far <= (np.abs(dense) @ np.abs(f64(x))) * 256 * 2.0 ** -24).all()
        c.q = q.cpu()
        K.append(c.cache, c.batch, f64(k), f64(v), c.rope)
        cache_equal(cache, c.cache)
        check_attention(c, a, None)
        far = np.abs(f64(y) - do @ f64(a).reshape(-1))
        assert (far <= (np.abs(do) @ np.abs(f64(a).reshape(-1))) * 256 * 2.0 ** -24).all()
        c.ctx += 1
        batch.ctx.add_(1)
