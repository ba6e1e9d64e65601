"""4-bit paged key/value cache on the GPU: contents and batches at the edge of
what the calls allow, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

import post_quantization_02_amd as kq
from oracle import kv_oracle as K
from kv_helpers import DEV, HALF, Case, cache_equal, check_attention, f64
from test_gpu_kv import TYPES, attend, ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("new", [2, 100])
@pytest.mark.parametrize("which", ["all", "some"])
def test_negative_scales(dtype, new, which):
    # a grid word is the bits of a scale, of either sign
    c = Case([(200, new), (150, new)], heads=2, share=2, dim=64, dtype=dtype, seed=new)
    rng = np.random.default_rng(new)
    for nm in "kv":
        w = c.cache[nm + "_grid"]
        w[rng.random(w.shape) < (1.0 if which == "all" else 0.5)] |= np.uint32(1 << 31)
    attend(c)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("lengths,rows", [([(100, 40), (90, 30)], 55), ([(300, 150), (260, 120)], 200),
                                          ([(900, 500), (50, 3)], 77), ([(5, 9), (20, 20)], 8)])
@pytest.mark.parametrize("window", [0, 20])
def test_rows_of_a_batch_cut_short_keep_their_positions(dtype, lengths, rows, window):
    # cu names more rows than the call has: those that it has are what they are in the whole call
    c = Case(lengths, heads=2, share=2, dim=64, dtype=dtype, rot=64, seed=rows)
    cache, batch, rope = c.dev(kq)
    q = c.q.to(DEV)
    got, lse = kq.kronq_kv_attention(q, cache, batch, rope=rope, window=window, sinks=2, want_lse=True)
    got[:rows], lse[:rows] = kq.kronq_kv_attention(q[:rows], cache, batch, rope=rope, window=window, sinks=2,
                                                   want_lse=True)
    check_attention(c, got, lse, None, window, 2)


def test_as_many_sequences_as_a_call_takes():
    rng = np.random.default_rng(4)
    lengths = [(int(rng.integers(0, 4)), 1) for _ in range(1 << 14)]
    c = Case(lengths, heads=1, share=1, dim=64, dtype=torch.bfloat16)
    attend(c)


def test_dimensions_of_one_entry_have_any_stride():
    c = Case([(14, 3)], heads=1, share=2, dim=64, dtype=torch.float16, rot=64)
    own, batch, rope = c.dev(kq)
    head = [t.as_strided(t.shape, (t.stride(0), 7) + t.stride()[2:]) for t in (own.k_codes, own.v_codes, own.k_grid, own.v_grid)]
    q = c.q.to(DEV)
    out = kq.kronq_kv_attention(q, kq.KVCache(*head), batch, rope=rope)
    check_attention(c, out, None)
    page = int(c.table[0, 0])
    one = kq.KVCache(*(t[page:page + 1].as_strided((1,) + t.shape[1:], (1,) + t.stride()[1:]) for t in head))
    at_0 = kq.KVBatch(torch.zeros_like(batch.table), batch.ctx, batch.cu)
    assert torch.equal(kq.kronq_kv_attention(q, one, at_0, rope=rope), out)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("heads,lengths,padding", [
    (32, [(60, 1)] * 30 + [(2500, 1)] + [(40, 1)] * 40, 0),          # one long among many short, one row each
    (8, [(30, 1)] * 290 + [(2600, 1)] + [(20, 1)] * 230 + [(2000, 1)], 0),   # more than a workgroup looks through at once
    (32, [(0, 0)] * 60 + [(2500, 1), (100, 1)], 60),                 # mostly empty places of a padded batch
    (32, [(200, 200)] * 7 + [(1500, 70), (300, 1)], 3),              # row tiles of prompts, and one behind a long context
], ids=["single rows", "hundreds", "padded", "prompts"])
def test_a_long_sequence_among_many_is_cut(dtype, heads, lengths, padding):
    c = Case(lengths, heads=heads, share=1, dim=64, page=64, dtype=dtype, rot=64, padding=padding, seed=len(lengths))
    cache, batch, rope = c.dev(kq)
    need = kq.load().kronq_kv_attention_ws(c.rows, len(lengths), heads, heads, 64)
    assert need > 1 << 16
    space = torch.full((need + (1 << 24),), 7, dtype=torch.uint8, device=DEV)
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, rope=rope, want_lse=True, ws=space[:need])
    check_attention(c, out, lse)
    assert bool((space[need:] == 7).all()) and not bool((space[:need] == 7).all())


def test_a_captured_call_of_many_sequences_follows_the_batch():
    # which sequence is long, and so cut, changes from replay to replay
    n, heads = 100, 32
    c = Case([(1600, 1)] * n, heads=heads, share=1, dim=64, page=64, dtype=torch.bfloat16, rot=64)
    c.table[:] = c.table[0]
    cache, batch, rope = c.dev(kq)
    q = c.q.to(DEV)
    out, side, graph = torch.empty_like(q), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    ws = torch.empty(kq.load().kronq_kv_attention_ws(n, n, heads, heads, 64), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        kq.kronq_kv_attention(q, cache, batch, rope=rope, out=out, ws=ws)
    rng = np.random.default_rng(1)
    for step in range(4):
        ctx = rng.integers(0, 20, n).astype(np.int32)
        ctx[rng.integers(n, size=2)] = 1600, 1300 if step % 2 else 3
        batch.ctx.copy_(torch.from_numpy(ctx))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, kq.kronq_kv_attention(q, cache, batch, rope=rope))
        c.ctx = ctx
        check_attention(c, out, None)


def test_a_cache_of_no_pages_is_refused_by_the_calls():
    c = Case([(3, 1)], heads=2, dim=64)
    _, batch, _ = c.dev(kq)
    with pytest.raises(kq.KronqError):
        kq.kronq_kv_read(kq.KVCache.empty(0, 2, 16, 64, DEV), batch, c.rows)


def test_tables_of_one_column_and_of_none_have_any_stride():
    c = Case([(14, 3), (9, 1)], heads=2, share=2, dim=64, rot=64)
    cache, batch, rope = c.dev(kq)
    q = c.q.to(DEV)
    one = kq.KVBatch(batch.table.as_strided((2, 1), (1, 5)), batch.ctx, batch.cu)
    check_attention(c, kq.kronq_kv_attention(q, cache, one, rope=rope), None)
    none = kq.KVBatch(batch.table.as_strided((2, 0), (3, 5)), batch.ctx, batch.cu)
    assert bool(torch.isnan(kq.kronq_kv_attention(q, cache, none, rope=rope)).all())
    assert bool(torch.isnan(kq.kronq_kv_read(cache, none, c.rows)[0]).all())
    kq.kronq_kv_append(c.k.to(DEV), c.v.to(DEV), cache, none, rope=rope)
    cache_equal(cache, c.cache)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("new", [2, 90])
@pytest.mark.parametrize("power", [12, 20, 27, 28, 30, 34, 60, 90])
def test_scores_of_any_size(dtype, new, power):
    # scores so large that a unit of them is less than their last place: one key has all the weight
    c = Case([(200, new), (150, 2)], heads=2, share=2, dim=64, dtype=dtype, seed=power)
    if dtype == torch.float16:                       # queries do not reach so far; keys do
        c.cache["k_grid"] += np.uint32(power - 12 << 23)
    c.q[:] = torch.sign(c.q.float()) * 2.0 ** (12 if dtype == torch.float16 else power)
    cache, batch, _ = c.dev(kq)
    out, lse = kq.kronq_kv_attention(c.q.to(DEV), cache, batch, want_lse=True)
    assert bool(torch.isfinite(out).all() and torch.isfinite(lse).all())
    # the other tests' bound takes scores' errors to be small; here they are not, and what
    # is sure is where one score is beyond all others' errors
    got, glse, sure = f64(out), f64(lse), 0
    for r, (b, pos) in enumerate(K.rows_of(c.batch, c.rows)):
        k = np.stack([K.held(c.cache, c.batch, b, j, "k") for j in range(pos + 1)])
        v = np.stack([K.held(c.cache, c.batch, b, j, "v") for j in range(pos + 1)])
        for h in range(4):
            s = 0.125 * k[:, h // 2] @ f64(c.q)[r, h]
            size = 0.125 * np.abs(k[:, h // 2]) @ np.abs(f64(c.q)[r, h])
            order = np.argsort(s)
            # a score is off by 72 half steps of fp32, and 2 2^-11 where keys carry their scales
            off = size.max() * (72 * 2.0 ** -24 + (2 * 2.0 ** -11 if dtype == torch.bfloat16 else 0))
            top = s[order[-1]]
            assert abs(glse[r, h] - top - np.log(np.exp(s - top).sum())) <= off + 2.0 ** -20 * (1 + abs(top)), (r, h)
            if top - s[order[-2]] > 2 * off + 40:
                # the value, in bf16 with its scale rounded, and the result's own rounding
                want = v[order[-1], h // 2]
                tol = np.abs(want) * (HALF[dtype] + (3 * 2.0 ** -11 if dtype != torch.float32 else 2.0 ** -20)) + 1e-6
                assert (np.abs(got[r, h] - want) <= tol).all(), (r, h)
                sure += 1
    assert sure > c.rows
