"""kvs_attend_pages on the GPU against the plain binary64 implementation.

Tolerances, derived (q, page values as given; A = |scale| max_j sum_d |q_d k_jd|
(a magnitude: a negative scale turns scores round, not their size),
n keys, V = max |v|):
  scores: 128 exact products summed in fp32 (at most 2^-23 each step, the
    tensor cores may truncate), a few more roundings: 140 * 2^-23 A; the wide
    kernel rounds K to fp16 first: + 2^-11 A (half a step, relative).
  weights: 2^x to 2^-22, plus the score's error; a softmax mean moves by at most
    twice the weights' relative error times V.
  sums over keys in fp32: (n / 16 + 32) * 2^-23.
  few rows: weights are hi + lo fp16 terms (2^-21) unless out is bf16, where
    they are rounded twice (2 * 2^-11); wide rows round them once (2^-11), and
    V once (2^-11).  Q4_1 / Q5_1 values are rounded once (2^-11) always.
  fp16 weights below 2^-14 are subnormal: 2^-25 against a largest weight of 2^6,
    2^-31 n in all, and through the V scale the same of V.
  out: half a step of its type.
"""
import math

import numpy as np
import pytest

from pages_testlib import F16, PAIR_IDS, PAIRS, Q4_0, Q4_1, Q5_1, Q8_0, Batch, torch

pytestmark = pytest.mark.gpu

EPS = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}


def run(b, q_dtype="float16", out_dtype=None, work=None, lse=True, score=None, fill=3.0, stream=None, q=None):
    t = b.t
    q = t.from_numpy(b.q).to(getattr(t, q_dtype)).cuda() if q is None else q
    out = t.full((b.rows, b.n_qh, 128), fill, dtype=getattr(t, out_dtype or q_dtype), device="cuda")
    l = t.full((b.rows, b.n_qh), fill, dtype=t.float32, device="cuda") if lse else None
    work = b.workspace() if work is None else work
    b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, out, l, score, b.c_prefix, work, stream)
    t.cuda.synchronize()
    return q.double().cpu().numpy(), out, l


def check(b, q64, out, lse, wide=False, **how):
    """out and lse against the plain form within the derived bounds; padding untouched."""
    want, wlse = b.plain_attention(q64, **how)
    n_real = int(b.start[-1])
    dt = str(out.dtype).split(".")[-1]
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    G = b.n_qh // b.n_kv
    scale = abs(how.get("scale") or 1 / math.sqrt(128))
    for i in range(len(b.new)):
        k, v = b.values(i)
        n, V = k.shape[0], np.abs(v).max() if v.size else 0.0
        for row in range(b.start[i], b.start[i + 1]):
            for h in range(b.n_qh):
                A = scale * (np.abs(k[:, h // G]) @ np.abs(q64[row, h])).max() if n else 0.0
                es = 140 * 2.0 ** -23 * A + (2.0 ** -11 * A if wide and b.types[0] != F16 else 0.0)
                es += 2.0 ** -22 + (2.0 ** -22 * how["softcap"] if how.get("softcap") else 0.0)
                if how.get("slopes") is not None:
                    es += 2.0 ** -23 * float(how["slopes"][h]) * (n + b.prefix + 64)
                ew = es + (n / 16 + 32) * 2.0 ** -23 + (2.0 ** -11 if wide else 2.0 ** -10 if dt == "bfloat16" else 2.0 ** -21)
                ev = 2.0 ** -11 if wide or b.types[1] in (Q4_1, Q5_1) else 0.0
                tol = EPS[dt] * np.abs(want[row, h]) + V * (2 * ew + ev + n * 2.0 ** -31) + 1e-30
                if dt == "float16":
                    tol = tol + 2.0 ** -25
                d = np.abs(got[row, h] - want[row, h])
                assert not bool((~(d <= tol)).any()), (i, row, h, d.max(), tol.min())
                if np.isinf(wlse[row, h]):
                    assert glse[row, h] == wlse[row, h]
                else:
                    assert abs(glse[row, h] - wlse[row, h]) <= es + (n / 16 + 32) * 2.0 ** -23 + 2.0 ** -22 * (1 + abs(wlse[row, h])), (i, row, h)
    assert np.all(got[n_real:] == 3.0) and np.all(glse[n_real:] == 3.0)


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("dtypes", [("float16", "float32"), ("bfloat16", "bfloat16")], ids=["f16-f32", "bf16"])
def test_decode_batch(types, dtypes):
    """One token a sequence, lengths around the stage and page borders, an empty
    sequence, one without rows, padding behind the last."""
    lens = [1, 2, 127, 128, 129, 255, 256, 257, 640, 0, 33, 1030]
    new = [1] * 12
    new[10] = 0
    b = Batch(new, lens, 8, 2, types, pad=3, seed=11).device()
    check(b, *run(b, *dtypes))


@pytest.mark.parametrize("group,new", [(1, 1), (3, 2), (5, 3), (8, 2), (4, 8), (7, 1), (16, 2)])
def test_rows_and_groups(group, new):
    """Every unit width (8, 16, 32 rows) and partly filled ones."""
    b = Batch([new, new, 1], [new + 300, new, 513], 2 * group, 2, (Q8_0, Q4_0), pad=1, seed=12).device()
    check(b, *run(b, "float16"))


@pytest.mark.parametrize("prefix", [1, 128, 256, 300, 1000])
@pytest.mark.parametrize("types", [(Q8_0, Q4_0), (F16, F16), (Q8_0, Q5_1)])
def test_shared_prefix(prefix, types):
    """A prefix that ends anywhere in a page; sequences with no tokens of their own."""
    b = Batch([1, 1, 2, 1, 1], [1, 300, 2, 0, 129], 4, 2, types, prefix=prefix, pad=2, seed=13).device()
    check(b, *run(b, "float16", "float32"))


def test_score_forms():
    t = torch()
    for how in (dict(softcap=2.0), dict(softcap=30.0), dict(window=1), dict(window=100), dict(window=5000), dict(scale=0.3),
                dict(scale=-0.05), dict(slopes=np.array([2.0 ** -(i + 1) for i in range(6)], np.float32)),
                dict(softcap=5.0, window=140, slopes=np.array([0.0, 0.5, 0.01, 1.0, 0.1, 0.25], np.float32))):
        b = Batch([1, 4, 2], [400, 260, 5], 6, 2, (Q8_0, Q4_0), prefix=200, pad=1, seed=14).device()
        kw = dict(how)
        if "slopes" in kw:
            kw["alibi_slopes"] = t.from_numpy(kw.pop("slopes")).cuda()
        q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(**kw))
        check(b, q64, out, lse, **how)


def test_document_and_prefix_masks_and_empty_rows():
    """Key intervals per row: documents, bidirectional parts, rows that see
    nothing (first >= end, intervals outside the keys), ends past the last key."""
    t = torch()
    b = Batch([9, 3], [300, 700], 4, 2, (Q8_0, Q4_0), prefix=130, pad=2, seed=15).device()
    first = np.array([0, 5, 140, 129, 130, 400, 0, 250, 2**31 - 1, -50, 600, 131] + [0] * 2, np.int32)
    end = np.array([1, 5, 141, 131, 430, 430, -3, 10000, 9, 2**31 - 1, 829, 140] + [5] * 2, np.int32)
    for f, e in ((first, end), (first, None), (None, end)):
        score = b.kvs.make_score(first_key=None if f is None else t.from_numpy(f).cuda(), end_key=None if e is None else t.from_numpy(e).cuda())
        q64, out, lse = run(b, "float16", "float32", score=score)
        check(b, q64, out, lse, first=f, end=e)


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
def test_unseen_keys_do_not_count(types):
    """Infinities and NaN in K and V of keys that some rows do not see, in what
    lies behind the last token, and in other documents: only rows that see them
    are affected."""
    t = torch()
    b = Batch([3, 1], [300, 200], 4, 2, types, prefix=40, seed=16)
    fields, _ = __import__("pages_testlib").field_rows(*types)
    nan, inf = np.float16(np.nan), np.float16(np.inf)

    def poison(page, tok, value):
        for name in ("kq" if types[0] == F16 else "kd", "vq" if types[1] == F16 else "vd"):
            w, off = fields[name]
            b.pool[page, :, off + tok * w:off + (tok + 1) * w].view(np.float16)[...] = value
    for tok in (44, 45, 60, 127, 255):          # behind the last token of sequence 0 (page 1: tokens 256..299)
        poison(int(b.table[0, 1]), tok, nan if tok % 2 else inf)
    for tok in range(200, 256):
        poison(int(b.table[1, 0]), tok, nan)
    for tok in range(40, 256):
        poison(int(b.prefix_table[0]), tok, inf)
    poison(int(b.table[0, 1]), 43, inf)          # the last row's own key: rows 0 and 1 do not see it
    poison(int(b.table[0, 0]), 7, nan)           # a key of another document for row 0 only
    b.device()
    first = np.array([40 + 8, 0, 0, 0], np.int32)
    q64, out, lse = run(b, "float16", "float32", score=b.kvs.make_score(first_key=t.from_numpy(first).cuda()))
    assert bool(out[1].isnan().all()) and bool(out[2].isnan().all()), "rows that see the bad keys are NaN"
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    want, wlse = b.plain_attention(q64, first=first)
    V = 80.0
    for row in (0, 3):
        assert np.all(np.abs(got[row] - want[row]) <= V * 2.0 ** -9) and np.all(np.abs(glse[row] - wlse[row]) <= 1e-4)


def test_large_scales_stay_finite():
    """V scales whose product with a weight passes fp16's range."""
    b = Batch([1, 1], [150, 400], 4, 2, (Q8_0, Q8_0), seed=17, scale=3000.0, outliers=False)
    b.q = b.q * 1e-4
    b.device()
    check(b, *run(b, "float16", "float32"))


def test_far_and_tiny_queries_in_bf16():
    """bf16 rows keep their own power of two: 1e30 and 1e-30 rows beside each other."""
    b = Batch([1, 1, 1], [300, 300, 5], 2, 1, (Q8_0, Q4_0), seed=18)
    b.q[0] *= 1e-30
    b.q[1] *= 1e3
    b.q[2] = 0.0
    b.device()
    q64, out, lse = run(b, "bfloat16", "float32")
    check(b, q64, out, lse)


def test_bad_pages_give_nan_and_status():
    t = torch()
    b = Batch([1, 1, 1], [600, 600, 600], 4, 2, (Q8_0, Q4_0), seed=19)
    b.table[0, 2] = b.n_pages + 5
    good = b.table[1].copy()
    b.device(status=True)
    q64, out, lse = run(b, "float16", "float32")
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    assert bool(out[0].isnan().all()) and bool(lse[0].isnan().all()) and not bool(out[1:].isnan().any())
    # a window that leaves the bad page out, and a length beyond the table
    b.status.zero_()
    b.d["lens"][1] = 256 * b.table.shape[1] + 1
    q64, out, lse = run(b, "float16", "float32")
    assert bool(out[1].isnan().all()) and not bool(out[2].isnan().any()) and int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    assert np.array_equal(good, b.table[1])


def test_same_results_whatever_the_split():
    """Repeated calls are bit-equal, and a workspace is ready for the next call."""
    b = Batch([1] * 6, [3000, 5, 1200, 700, 64, 2500], 8, 2, (Q8_0, Q4_0), prefix=700, seed=20).device()
    work = b.workspace()
    first = run(b, "bfloat16", work=work)
    for _ in range(3):
        again = run(b, "bfloat16", work=work)
        assert b.t.equal(first[1], again[1]) and b.t.equal(first[2], again[2])


def test_graph_follows_the_batch():
    """A captured call replayed after lengths, tables and queries changed."""
    t = torch()
    b = Batch([1, 1, 1], [900, 256, 513], 4, 2, (Q8_0, Q4_0), prefix=300, seed=21).device()  # every token of the replays below is written
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
    for lens in ([900, 200, 513], [3, 256, 400], [700, 0, 1]):
        b.lens = lens
        b.d["lens"].copy_(t.tensor(lens, dtype=t.int32))
        q.normal_()
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        check(b, q.double().cpu().numpy(), out, lse)


def test_strided_tensors_and_another_stream():
    t = torch()
    b = Batch([2, 1], [100, 300], 4, 2, (Q8_0, Q4_0), pad=1, seed=22).device()
    big = t.zeros(b.rows, 9, 256, dtype=t.float16, device="cuda")
    q = big[:, 3:7, 128:]
    q.copy_(t.from_numpy(b.q))
    store = t.full((4, b.rows, 128), 3.0, device="cuda")
    out = store.transpose(0, 1)  # head-major rows
    lse = t.full((b.rows, 4), 3.0, device="cuda")
    s = t.cuda.Stream()
    s.wait_stream(t.cuda.current_stream())
    b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, out, lse, None, None, b.workspace(), s)
    s.synchronize()
    check(b, q.double().cpu().numpy(), out, lse)


def test_append_then_attend_as_a_serving_loop():
    """Prompt, then decode steps: append with rotation, attention with the rotated
    queries, read-back, all from one pool, against binary64 over what the pages
    hold."""
    t = torch()
    types = (Q8_0, Q5_1)
    b = Batch([60, 200], [60, 200], 4, 2, types, prefix=270, seed=23, extra_cols=1)
    b.table[:, 1] = [b.n_pages - 1, b.n_pages - 2]
    b.device()
    f = t.tensor([10000.0 ** (-i / 64) for i in range(64)], device="cuda")
    work = t.zeros(b.kvs.kvs_attend_pages_workspace(b.c_batch, 4, 2), dtype=t.uint8, device="cuda")
    for step, (new, lens) in enumerate([([60, 200], [60, 200]), ([1, 1], [61, 201]), ([3, 1], [64, 202]), ([1, 60], [65, 262])]):
        b.new, b.lens = new, lens
        b.start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        b.rows = sum(new)
        start, length = t.from_numpy(b.start).cuda(), t.tensor(lens, dtype=t.int32, device="cuda")
        batch = b.kvs.make_page_batch(start, length, b.d["table"], b.rows, max_new=max(new))
        qkv = t.randn(b.rows, 8, 128, device="cuda").half()
        rope = b.kvs.make_rope(f, pos_offset=b.prefix)
        q = t.empty(b.rows, 4, 128, dtype=t.float16, device="cuda")
        out, lse = t.zeros(b.rows, 4, 128, device="cuda"), t.zeros(b.rows, 4, device="cuda")
        b.kvs.kvs_append_pages(b.c_pool, batch, qkv[:, 4:6], qkv[:, 6:], qkv[:, :4], q, rope)
        b.kvs.kvs_attend_pages(b.c_pool, batch, q, out, lse, None, b.c_prefix, work)
        t.cuda.synchronize()
        b.pool = b.d_pool.cpu().numpy()
        check(b, q.double().cpu().numpy(), out, lse, wide=max(new) * 2 > 32)


def test_many_short_sequences_and_an_empty_batch():
    """More sequences than a warp scans at once, most without rows or tokens."""
    t = torch()
    rng = np.random.default_rng(24)
    new = [int(x) for x in rng.choice([0, 0, 1, 2], 300)]
    lens = [max(n, int(x)) for n, x in zip(new, rng.choice([0, 1, 40, 130], 300))]
    b = Batch(new, lens, 2, 1, (Q8_0, Q4_0), pad=2, seed=24).device()
    check(b, *run(b, "float16", "float32"))
    none = b.kvs.make_page_batch(b.d["start"][:1], b.d["lens"][:0], b.d["table"][:0], 4)
    out = t.full((4, 2, 128), 5.0, device="cuda")
    q = t.zeros(4, 2, 128, dtype=t.float16, device="cuda")
    b.kvs.kvs_attend_pages(b.c_pool, none, q, out, None, None, None, b.workspace())
    b.kvs.kvs_read_pages(b.c_pool, none, out[:, :1])
    t.cuda.synchronize()
    assert bool((out == 5).all())


def test_two_streams_with_a_workspace_each():
    """Two calls in flight at once do not disturb each other."""
    t = torch()
    pair = [Batch([1] * 4, [2000, 300, 5, 900], 8, 2, (Q8_0, Q4_0), prefix=p, seed=25 + p).device() for p in (0, 500)]
    alone = [run(b, "bfloat16") for b in pair]
    streams = [t.cuda.Stream() for _ in pair]
    works = [b.workspace() for b in pair]
    qs = [t.from_numpy(b.q).bfloat16().cuda() for b in pair]
    outs = [t.zeros(b.rows, 8, 128, dtype=t.bfloat16, device="cuda") for b in pair]
    t.cuda.synchronize()
    for _ in range(10):
        for b, s, w, q, o in zip(pair, streams, works, qs, outs):
            b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, o, None, None, b.c_prefix, w, s)
    t.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert t.equal(a[1], o)


def test_first_call_of_a_process_may_be_captured():
    """No lazy set-up of the calls needs a run outside a capture."""
    import os
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = ['tests', '.']
import torch as t
from pages_testlib import Batch
b = Batch([1, 40], [300, 200], 4, 2, (8, 2), prefix=100, seed=26).device()
q = t.from_numpy(b.q).half().cuda(); out = t.zeros(b.rows, 4, 128, device='cuda'); kv = t.zeros(b.rows, 2, 128, device='cuda')
w = b.workspace(); s = t.cuda.Stream(); t.cuda.synchronize()
g = t.cuda.CUDAGraph()
with t.cuda.graph(g, stream=s):
    b.kvs.kvs_read_pages(b.c_pool, b.c_batch, kv, stream=s)
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, kv, kv, stream=s)
    b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, out, None, None, b.c_prefix, w, s)
g.replay(); t.cuda.synchronize()
first = out.clone(); out.zero_()
b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, q, out, None, None, b.c_prefix, w); t.cuda.synchronize()
assert t.equal(first, out) and float(out.abs().sum()) > 0
print('captured')
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_binding_refuses_wrong_tensors():
    t = torch()
    b = Batch([2, 1], [100, 300], 4, 2, (Q8_0, Q4_0), seed=27).device()
    q = t.zeros(b.rows, 4, 128, dtype=t.float16, device="cuda")
    w = b.workspace()
    bad = [dict(q=q[:2]), dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q.cpu()), dict(out=q.to(t.int32)),
           dict(q=t.zeros(b.rows, 128, 4, dtype=t.float16, device="cuda").transpose(1, 2)), dict(lse=t.zeros(2, 4, device="cuda")),
           dict(workspace=None), dict(workspace=w[:1000]), dict(score=b.kvs.make_score(alibi_slopes=t.ones(3, device="cuda"))),
           dict(score=b.kvs.make_score(first_key=t.zeros(2, dtype=t.int32, device="cuda")))]
    for kw in bad:
        args = dict(q=q, out=t.zeros_like(q), lse=None, score=None, prefix=None, workspace=w)
        args.update(kw)
        with pytest.raises(b.kvs.KvsError):
            b.kvs.kvs_attend_pages(b.c_pool, b.c_batch, **args)
    for make in (lambda: b.kvs.make_page_pool(b.d_pool.flatten()[:-1], 2), lambda: b.kvs.make_page_prefix(b.d["lens"][:1], 300),
                 lambda: b.kvs.make_page_batch(b.d["start"][:2], b.d["lens"], b.d["table"], 3),
                 lambda: b.kvs.make_page_batch(b.d["start"].long(), b.d["lens"], b.d["table"], 3),
                 lambda: b.kvs.make_rope(t.ones(10, device="cuda"), 64)):
        with pytest.raises(b.kvs.KvsError):
            make()


@pytest.mark.parametrize("new", [3, 40], ids=["few-rows", "many-rows"])
def test_extreme_intervals_beside_a_prefix(new):
    """Ends at the lowest int32 and starts at the highest see nothing, also where
    the prefix is subtracted from them."""
    t = torch()
    b = Batch([new], [200], 2, 1, (Q8_0, Q4_0), prefix=150, seed=28).device()
    first, end = np.zeros(new, np.int32), np.full(new, 2 ** 31 - 1, np.int32)
    end[0], first[1] = -2 ** 31, 2 ** 31 - 1
    first[2], end[2] = -2 ** 31, 151
    score = b.kvs.make_score(first_key=t.from_numpy(first).cuda(), end_key=t.from_numpy(end).cuda())
    q64, out, lse = run(b, "float16", "float32", score=score)
    check(b, q64, out, lse, wide=new > 16, first=first, end=end)
    assert bool((out[:2] == 0).all()) and bool((lse[:2] == -math.inf).all())
