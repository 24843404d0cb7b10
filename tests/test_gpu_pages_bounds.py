"""kvs_attend_pages: what the batch's bounds (rows of the tensors, longest
sequence) must not change, and numbers at the ends of int32."""
import numpy as np
import pytest

from pages_testlib import PAIR_IDS, PAIRS, Q4_0, Q8_0, Batch, torch
from test_gpu_pages_attend import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
def test_padding_does_not_change_a_short_sequence(types):
    """One sequence of a few rows in tensors of many, its rows not stated: the same
    results, to the bit, as in tensors of its own rows."""
    t = torch()
    for new in (1, 3):
        b = Batch([new], [700], 8, 2, types, pad=64 - new, seed=61, outliers=False).device(max_new=0)
        q = t.from_numpy(b.q).half().cuda()
        _, out, lse = run(b, "float16", "float32", q=q)
        one = b.kvs.make_page_batch(b.d["start"], b.d["lens"], b.d["table"], new, max_new=new)
        want, wl = t.zeros(new, 8, 128, device="cuda"), t.zeros(new, 8, device="cuda")
        b.kvs.kvs_attend_pages(b.c_pool, one, q, want, wl, None, None, b.workspace())
        t.cuda.synchronize()
        assert t.equal(out[:new], want) and t.equal(lse[:new], wl)
        assert bool((out[new:] == 3).all()) and bool((lse[new:] == 3).all())


def test_one_sequence_with_fewer_rows_than_stated():
    """One sequence is taken to have the rows that max_new states: fewer are right,
    with the bounds of many rows."""
    for new in (1, 3, 20):
        b = Batch([new], [700], 8, 2, (Q8_0, Q4_0), pad=64 - new, seed=65).device(max_new=64)
        check(b, *run(b, "float16", "float32"), wide=True)


def test_a_short_sequence_replayed_where_a_long_one_was_captured():
    """The rows change between replays of a captured call of one sequence."""
    t = torch()
    b = Batch([64], [400], 4, 2, (Q8_0, Q4_0), prefix=30, seed=66).device(max_new=0)
    work, s = b.workspace(), t.cuda.Stream()
    q = t.from_numpy(b.q).half().cuda()
    out, lse = t.zeros(64, 4, 128, device="cuda"), t.zeros(64, 4, device="cuda")
    s.wait_stream(t.cuda.current_stream())
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g, stream=s):
        b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, out, lse, None, b.c_prefix, work, s)
    for new, length in ((64, 400), (1, 400), (16, 333), (17, 17), (0, 400), (2, 1)):
        b.new, b.lens, b.start = [new], [length], np.array([0, new], np.int32)
        b.d["start"].copy_(t.from_numpy(b.start))
        b.d["lens"].fill_(length)
        out.fill_(3.0), lse.fill_(3.0)
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        check(b, q.double().cpu().numpy(), out, lse, wide=True)


def test_batches_without_rows():
    """Tensors of no rows (null addresses) are the smallest batch: nothing is done."""
    t = torch()
    b = Batch([0, 0], [300, 0], 4, 2, (Q8_0, Q4_0), prefix=40, seed=64).device(status=True)
    before = b.d_pool.clone()
    kv, q = t.empty(0, 2, 128, dtype=t.float16, device="cuda"), t.empty(0, 4, 128, dtype=t.float16, device="cuda")
    f = t.ones(64, device="cuda")
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, kv, kv, q, t.empty_like(q), b.kvs.make_rope(f))
    b.kvs.kvs_read_pages(b.c_pool, b.c_batch, kv, t.empty_like(kv))
    b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, t.empty_like(q), t.empty(0, 4, device="cuda"), None, b.c_prefix, b.workspace())
    t.cuda.synchronize()
    assert t.equal(b.d_pool, before) and int(b.status) == 0


@pytest.mark.parametrize("new", [6, 40], ids=["few-rows", "many-rows"])
@pytest.mark.parametrize("prefix", [0, 20])
def test_largest_window_at_negative_positions(new, prefix):
    """Rows before position -1 whose end_key lies past them, with the largest window:
    its lower bound is below int32."""
    b = Batch([new], [3], 2, 1, (Q8_0, Q4_0), prefix=prefix, seed=62).device()
    end = np.full(new, prefix + 3, np.int32)
    score = b.kvs.make_score(window=2 ** 31 - 1, end_key=torch().from_numpy(end).cuda())
    check(b, *run(b, "float16", "float32", score=score), wide=new > 16, window=2 ** 31 - 1, end=end)


@pytest.mark.parametrize("new", [3, 40], ids=["few-rows", "many-rows"])
@pytest.mark.parametrize("prefix", [0, 300])
def test_largest_length(new, prefix):
    """A length of 2^31 - 1, far beyond the table: NaN and the status bit, with a
    prefix before it too."""
    b = Batch([new, 1], [400, 100], 2, 1, (Q8_0, Q4_0), prefix=prefix, seed=63).device(status=True)
    b.d["lens"][0] = 2 ** 31 - 1
    q64, out, lse = run(b, "float16", "float32")
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    assert bool(out[:new].isnan().all()) and bool(lse[:new].isnan().all())
    assert not bool(out[new:].isnan().any()) and not bool(lse[new:].isnan().any())
