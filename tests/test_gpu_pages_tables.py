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
