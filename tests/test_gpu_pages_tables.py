"""kvs_attend_pages and page numbers that are not in the pool: a row is NaN, and
*status says so, exactly if the row sees a key of such a page or beyond the page
table; released pages (entries -1) that no row sees count for nothing.  Bounds
as derived in test_gpu_pages_attend.py."""
import numpy as np
import pytest

from pages_testlib import F16, PAIR_IDS, PAIRS, Q4_0, Q8_0, Batch, torch
from test_gpu_pages_attend import check, run

pytestmark = pytest.mark.gpu


def ints(a):
    return torch().tensor(a, dtype=torch().int32, device="cuda")


def check_where(b, bad, q64, out, lse, wide, **how):
    """Rows `bad` are NaN, the others follow the plain form."""
    t = torch()
    bad = sorted(bad)
    assert bool(out[bad].isnan().all()) and bool(lse[bad].isnan().all())
    want, wlse = b.plain_attention(q64, **how)
    out, lse = out.clone(), lse.clone()
    out[bad], lse[bad] = t.from_numpy(want[bad]).to(out), t.from_numpy(wlse[bad]).to(lse)
    check(b, q64, out, lse, wide=wide, **how)


# more than 32 rows per kv head in all: the prefix goes to the tensor cores; own
# pages too where one sequence has the rows
@pytest.mark.parametrize("new,lens", [([40], [400]), ([1] * 20, [400] * 20), ([30, 1, 9], [400, 390, 500])], ids=["chunk", "decode", "mixed"])
@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
def test_window_past_a_released_prefix(new, lens, types):
    """Every row's window has passed the prefix and each sequence's first page:
    their entries are -1, and nothing of them counts."""
    b = Batch(new, lens, 4, 2, types, prefix=300, pad=1, seed=51).device(status=True)
    b.d["ptable"].fill_(-1)
    b.d["table"][:, 0] = -1
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(window=90))
    assert int(b.status) == 0
    check(b, q64, out, lse, wide=True, window=90)


@pytest.mark.parametrize("new", [6, 40], ids=["few-rows", "many-rows"])
def test_intervals_that_end_inside_the_prefix(new):
    """Own pages released where all intervals end inside the prefix; the first
    rows see nothing at all."""
    b = Batch([new, new], [300, 270], 2, 1, (Q8_0, Q4_0), prefix=200, pad=1, seed=52).device(status=True)
    b.d["table"].fill_(-1)
    first, end = np.zeros(b.rows, np.int32), np.full(b.rows, 190, np.int32)
    first[:3] = 190
    end[new:] = 200
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(first_key=ints(first), end_key=ints(end)))
    assert int(b.status) == 0
    check(b, q64, out, lse, wide=new > 16, first=first, end=end)
    # nothing is seen and nothing is there
    b.d["ptable"].fill_(-1)
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(first_key=ints(end), end_key=ints(end)))
    assert int(b.status) == 0
    check(b, q64, out, lse, wide=new > 16, first=end, end=end)


@pytest.mark.parametrize("new,group,over", [(40, 1, 3), (40, 1, 1), (70, 1, 33), (17, 2, 1)])
def test_status_of_rows_beyond_the_page_table(new, group, over):
    """The last rows end behind the table's last entry: NaN and the status bit,
    whichever lanes and warps hold them."""
    b = Batch([new], [512], group, 1, (Q8_0, Q4_0), pad=1, seed=56, extra_cols=0).device(status=True)
    b.d["lens"].fill_(512 + over)
    q64, out, lse = run(b, "float16", "float32")
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    end = np.minimum(512 + over - new + 1 + np.arange(b.rows), 600)
    check_where(b, range(new - over, new), q64, out, lse, new * group > 32, end=end)


@pytest.mark.parametrize("new", [6, 40], ids=["few-rows", "many-rows"])
@pytest.mark.parametrize("types", [(Q8_0, Q4_0), (F16, F16)], ids=["q8-q4_0", "f16-f16"])
def test_only_rows_that_see_a_bad_page_are_nan(new, types):
    """Bad own pages and a bad prefix page, seen by some rows of a tile only."""
    b = Batch([new, new], [600, 530], 2, 1, types, prefix=600, pad=1, seed=53).device(status=True)
    b.d["ptable"][1] = b.n_pages               # keys 256..511
    b.d["table"][0, 0] = -1                    # keys 600..855 of sequence 0
    b.d["table"][1, 1] = 2 ** 31 - 1           # keys 856..1111 of sequence 1
    first, end = np.full(b.rows, 856, np.int32), np.full(b.rows, 10 ** 6, np.int32)
    first[0] = 511                             # the bad prefix page's last key
    first[1], end[1] = 512, 600                # the prefix behind it
    first[2], end[2] = 0, 256                  # and before it
    first[3] = 855                             # the bad own page's last key
    first[4], end[4] = 700, 700                # nothing, inside the bad page
    first[new:], end[new:] = 600, 856          # sequence 1 before its bad page
    first[new], end[new] = 300, 601
    end[new + 1] = 857
    first[new + 2] = 1112
    bad = [0, 3, new, new + 1]
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(first_key=ints(first), end_key=ints(end)))
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    check_where(b, bad, q64, out, lse, new > 16, first=first, end=end)


@pytest.mark.parametrize("new", [2, 40], ids=["few-rows", "many-rows"])
def test_a_bad_page_between_the_rows_intervals(new):
    """Two rows of one tile with a page between their intervals that neither sees."""
    b = Batch([new], [900], 2, 1, (Q8_0, Q4_0), seed=54).device(status=True)
    b.d["table"][0, 1:3] = -1
    first, end = np.zeros(new, np.int32), np.full(new, 256, np.int32)
    first[new // 2:], end[new // 2:] = 768, 900
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(first_key=ints(first), end_key=ints(end)))
    assert int(b.status) == 0
    check(b, q64, out, lse, wide=new > 16, first=first, end=end)


@pytest.mark.parametrize("new", [3, 40], ids=["few-rows", "many-rows"])
def test_a_window_that_leaves_the_bad_page_out(new):
    b = Batch([new, new], [700, 650], 2, 1, (Q8_0, Q4_0), seed=55).device(status=True)
    b.d["table"][:, 0] = b.n_pages + 3
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(window=340))
    assert int(b.status) == 0
    check(b, q64, out, lse, wide=new > 16, window=340)
    # the first rows of the second sequence see the page's last key again
    window = 650 - new + 1 - 255
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(window=window))
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    check_where(b, [new], q64, out, lse, new > 16, window=window)


def test_length_hint_below_the_truth():
    """max_new says one row a sequence, two have more: right, by the few-row kernel."""
    for n in (20, 70):
        b = Batch([n, 1, 12], [500, 300, 20], 4, 2, (Q8_0, Q4_0), prefix=60, pad=3, seed=57).device(max_new=1)
        check(b, *run(b, "float16", "float32"), wide=True)
        b = Batch([n, 1, 12], [500, 300, 20], 4, 2, (Q8_0, Q4_0), pad=3, seed=58).device(max_new=1)
        check(b, *run(b, "float16", "float32"))


def test_status_of_few_rows_beyond_the_page_table():
    """The same by the few-row kernel: the rows inside the table keep their values."""
    b = Batch([6, 1], [512, 300], 2, 1, (Q8_0, Q4_0), pad=1, seed=59, extra_cols=0).device(status=True)
    b.d["lens"][0] = 514
    q64, out, lse = run(b, "float16", "float32")
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    end = np.array([509 + i for i in range(6)] + [300, 0])
    check_where(b, [4, 5], q64, out, lse, False, end=end)
