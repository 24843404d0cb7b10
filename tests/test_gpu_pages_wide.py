"""kvs_attend_pages with more than 32 rows per kv head: the tensor-core kernel,
alone, for a shared prefix, and beside short sequences.  Bounds as derived in
test_gpu_pages_attend.py, with K, V and weights rounded to fp16 once each."""
import numpy as np
import pytest

from pages_testlib import F16, PAIR_IDS, PAIRS, Q4_0, Q4_1, Q8_0, Batch, field_rows, torch
from test_gpu_pages_attend import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("dtypes", [("float16", "float32"), ("bfloat16", "bfloat16")], ids=["f16-f32", "bf16"])
def test_prompt_chunk(types, dtypes):
    """One sequence, 90 rows x 3 heads: two tiles and a ragged second one."""
    b = Batch([90], [400], 6, 2, types, pad=2, seed=31).device()
    check(b, *run(b, *dtypes), wide=True)


@pytest.mark.parametrize("new,length,group", [(33, 33, 1), (128, 128, 1), (129, 300, 1), (17, 1000, 2), (64, 200, 4), (100, 100, 5), (40, 700, 16)])
def test_tiles(new, length, group):
    """One tile, exactly one, two, several groups; from the first token on."""
    b = Batch([new], [length], group, 1, (Q8_0, Q4_0), pad=1, seed=32).device()
    check(b, *run(b, "bfloat16", "float32"), wide=True)


def test_ragged_mixed_batch():
    """Long and short sequences in one call, without and with the length hint."""
    for hint in (None, 0):
        b = Batch([70, 1, 0, 12, 1, 40, 9], [500, 300, 20, 12, 1, 41, 700], 4, 1, (Q8_0, Q4_0), prefix=60, pad=3, seed=33).device(max_new=hint)
        check(b, *run(b, "float16", "float32"), wide=True)


@pytest.mark.parametrize("prefix", [1, 200, 256, 700])
@pytest.mark.parametrize("types", [(Q8_0, Q4_0), (F16, F16), (Q8_0, Q4_1)])
def test_prefix_of_many_sequences(prefix, types):
    b = Batch([1, 2, 1, 1, 3, 1, 1, 1, 0, 1], [1, 200, 0, 129, 3, 5, 64, 256, 9, 300], 8, 2, types, prefix=prefix, pad=2, seed=34).device()
    check(b, *run(b, "float16", "float32"), wide=True)


def test_more_rows_than_tokens():
    """Rows at negative positions see the prefix up to their position, or nothing."""
    for prefix in (0, 50):
        b = Batch([60, 2], [20, 1], 2, 1, (Q8_0, Q4_0), prefix=prefix, seed=35).device()
        check(b, *run(b, "float16", "float32"), wide=True)


def test_score_forms():
    t = torch()
    for how in (dict(softcap=3.0), dict(window=50), dict(window=1), dict(scale=0.2), dict(slopes=np.array([0.5, 0.01, 1.0, 0.0], np.float32)),
                dict(softcap=8.0, window=200, slopes=np.array([0.25, 0.125, 0.5, 2.0], np.float32))):
        b = Batch([50, 30], [300, 30], 4, 1, (Q8_0, Q4_0), prefix=150, pad=1, seed=36).device()
        kw = dict(how)
        if "slopes" in kw:
            kw["alibi_slopes"] = t.from_numpy(kw.pop("slopes")).cuda()
        q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(**kw))
        check(b, q64, out, lse, wide=True, **how)


def test_documents_and_empty_rows():
    """Packed documents with a bidirectional head each, and rows that see nothing."""
    t = torch()
    b = Batch([300], [300], 4, 2, (F16, F16), pad=1, seed=37).device()
    cut = [0, 1, 60, 190, 300]
    first, end = np.zeros(301, np.int32), np.zeros(301, np.int32)
    for a, z in zip(cut, cut[1:]):
        for p in range(a, z):
            first[p], end[p] = a, max(p + 1, a + (z - a) // 3)
    first[100:110], end[100:110] = 90, 90
    end[200] = -5
    first[201] = 2 ** 31 - 1
    first[250], end[250] = -10, 2 ** 31 - 1
    score = b.kvs.make_score(first_key=t.from_numpy(first).cuda(), end_key=t.from_numpy(end).cuda())
    q64, out, lse = run(b, "float16", "float32", score=score)
    check(b, q64, out, lse, wide=True, first=first, end=end)


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
def test_unseen_keys_do_not_count(types):
    t = torch()
    b = Batch([40], [300], 2, 1, types, prefix=40, seed=38)
    fields, _ = field_rows(*types)

    def poison(page, tok, value):
        for name in ("kq" if types[0] == F16 else "kd", "vq" if types[1] == F16 else "vd"):
            w, off = fields[name]
            b.pool[page, :, off + tok * w:off + (tok + 1) * w].view(np.float16)[...] = value
    for tok in range(44, 256):
        poison(int(b.table[0, 1]), tok, np.float16(np.nan) if tok % 2 else np.float16(np.inf))
    for tok in range(40, 256):
        poison(int(b.prefix_table[0]), tok, np.float16(np.nan))
    poison(int(b.table[0, 1]), 43, np.float16(np.inf))       # the last token: only the last row sees it
    b.device()
    q64, out, lse = run(b, "float16", "float32")
    assert bool(out[39].isnan().all())
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    want, wlse = b.plain_attention(q64)
    assert np.all(np.abs(got[:39] - want[:39]) <= 0.05) and np.all(np.abs(glse[:39] - wlse[:39]) <= 0.02)


def test_bad_pages_give_nan_and_status():
    t = torch()
    b = Batch([40, 40], [600, 600], 2, 1, (Q8_0, Q4_0), seed=39)
    b.table[0, 1] = -3
    b.device(status=True)
    q64, out, lse = run(b, "float16", "float32")
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    assert bool(out[:40].isnan().all()) and bool(lse[:40].isnan().all()) and not bool(out[40:].isnan().any())
    b.status.zero_()
    b.d["lens"][1] = 256 * b.table.shape[1] + 20       # 20 rows end beyond the page table
    q64, out, lse = run(b, "float16", "float32")
    assert bool(out[60:].isnan().all()) and int(b.status) == b.kvs.KVS_ERR_BAD_PAGE


def test_shared_units_are_joined_in_order():
    """A few units spread over all SMs; calls repeat bit for bit, one workspace."""
    b = Batch([80], [6000], 4, 1, (Q8_0, Q4_0), seed=40, outliers=False).device()
    work = b.workspace()
    first = run(b, "bfloat16", "float32", work=work)
    for _ in range(3):
        again = run(b, "bfloat16", "float32", work=work)
        assert b.t.equal(first[1], again[1]) and b.t.equal(first[2], again[2])
    b.q = b.q[::1]
    rows = [0, 1, 40, 79]
    want, wlse = [], []
    k, v = b.values(0)
    q64 = first[0]
    for r in rows:
        n = 6000 - 80 + r + 1
        for h in range(4):
            s = k[:n, 0] @ q64[r, h] / np.sqrt(128)
            e = np.exp(s - s.max())
            want.append(e @ v[:n, 0] / e.sum())
            wlse.append(s.max() + np.log(e.sum()))
    got = first[1].double().cpu().numpy()[rows].reshape(-1, 128)
    # K rounding moves a score by at most 2^-11 A (A < 25 here), V and weights 2^-11 each, |v| <= 5
    assert np.abs(got - np.array(want)).max() <= 5 * (2 * 25 + 2) * 2.0 ** -11 / 4
    assert np.abs(first[2].double().cpu().numpy()[rows].reshape(-1) - np.array(wlse)).max() <= 25 * 2.0 ** -11


def test_graph_follows_the_batch():
    t = torch()
    b = Batch([40, 50], [400, 513], 4, 2, (Q8_0, Q4_0), prefix=300, seed=41).device()
    work = b.workspace()
    q = t.from_numpy(b.q).half().cuda()
    out, lse = t.zeros(b.rows, 4, 128, device="cuda"), t.zeros(b.rows, 4, device="cuda")
    s = t.cuda.Stream()
    call = lambda: b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, out, lse, None, b.c_prefix, work, s)  # noqa: E731
    with t.cuda.stream(s):
        call()
        s.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=s):
            call()
    for new, lens in (([40, 50], [400, 513]), ([89, 1], [100, 256]), ([3, 87], [400, 87])):
        b.new, b.lens = new, lens
        b.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        b.d["start"].copy_(t.from_numpy(b.start))
        b.d["lens"].copy_(t.tensor(lens, dtype=t.int32))
        q.normal_()
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        check(b, q.double().cpu().numpy(), out, lse, wide=True)
