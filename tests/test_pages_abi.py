"""The batch operators over caller-owned pages, without a GPU: every refusal of
the C entry points is made on the host before any CUDA call, and the workspace
size is a pure function of the batch's bounds."""
import ctypes

import pytest

from host_streamed_paged_kvs_b200 import build as B


@pytest.fixture(scope="module")
def kvs():
    B.build()
    from host_streamed_paged_kvs_b200 import kvs as K
    return K


A = 1 << 20  # an address that nothing dereferences: every call below is refused


def pool(kvs, **kw):
    p = dict(pages=A, n_pages=4, n_kv_heads=2, type_k=kvs.KVS_TYPE_Q8_0, type_v=kvs.KVS_TYPE_Q4_0)
    p.update(kw)
    return kvs.kvs_page_pool(*(p[n] for n, _ in kvs.kvs_page_pool._fields_))


def batch(kvs, **kw):
    b = dict(n_seqs=2, n_rows=4, max_new=0, q_start=A, seq_len=A, page_table=A, table_stride=2, status=None)
    b.update(kw)
    return kvs.kvs_page_batch(*(b[n] for n, _ in kvs.kvs_page_batch._fields_))


def rows(kvs, data=A, row=512, head=128):
    return kvs.kvs_page_rows(data, row, head)


def refused(kvs, rc, text):
    assert rc == kvs.KVS_E_INVAL, rc
    assert text in kvs.kvs_last_error(), kvs.kvs_last_error()


POOLS = [(dict(pages=None), "null pool"), (dict(pages=A + 8), "16-byte"), (dict(n_pages=0), "at least one page"),
         (dict(n_kv_heads=0), "at least one page"), (dict(type_k=2), "type pair"), (dict(type_k=1, type_v=2), "type pair"),
         (dict(type_v=30), "type pair"), (dict(n_pages=1 << 30, n_kv_heads=2), "2^31")]
BATCHES = [(dict(n_seqs=-1), "negative"), (dict(n_rows=-1), "negative"), (dict(table_stride=-1), "negative"), (dict(max_new=-2), "negative"),
           (dict(q_start=None), "null q_start"), (dict(seq_len=None), "null q_start"), (dict(page_table=None), "null page_table"),
           (dict(q_start=A + 2), "4-byte"), (dict(status=A + 1), "4-byte"), (dict(page_table=A + 3), "4-byte")]
ROWS = [(dict(data=None), "null"), (dict(data=A + 8), "16 bytes"), (dict(row=514), "16 bytes"), (dict(head=130), "16 bytes")]


@pytest.mark.parametrize("what,text", POOLS + BATCHES)
def test_pool_and_batch_are_checked_by_every_call(kvs, what, text):
    p = pool(kvs, **what) if set(what) <= {n for n, _ in kvs.kvs_page_pool._fields_} else pool(kvs)
    b = batch(kvs, **what) if set(what) <= {n for n, _ in kvs.kvs_page_batch._fields_} else batch(kvs)
    r = rows(kvs)
    refused(kvs, kvs.lib.kvs_append_pages(p, b, kvs.KVS_DT_F16, r, r, 0, None, None, None, None), text)
    refused(kvs, kvs.lib.kvs_read_pages(p, b, kvs.KVS_DT_F16, r, r, None), text)
    refused(kvs, kvs.lib.kvs_attend_pages(p, b, kvs.KVS_DT_F16, 4, r, kvs.KVS_DT_F16, r, None, None, None, A, 1 << 40, None), text)


def test_null_descriptors(kvs):
    r = rows(kvs)
    refused(kvs, kvs.lib.kvs_append_pages(None, batch(kvs), 0, r, r, 0, None, None, None, None), "null pool")
    refused(kvs, kvs.lib.kvs_read_pages(pool(kvs), None, 0, r, r, None), "null batch")
    refused(kvs, kvs.lib.kvs_attend_pages(pool(kvs), batch(kvs), 0, 4, None, 0, r, None, None, None, A, 1 << 40, None), "null q")


@pytest.mark.parametrize("what,text", ROWS)
def test_rows_are_checked(kvs, what, text):
    p, b, r, x = pool(kvs), batch(kvs), rows(kvs), rows(kvs, **what)
    for args in ((x, r, 0, None, None), (r, x, 0, None, None), (r, r, 4, x, r), (r, r, 4, r, x)):
        k, v, h, q, qo = args
        refused(kvs, kvs.lib.kvs_append_pages(p, b, kvs.KVS_DT_BF16, k, v, h, q, qo, None, None), text)
    refused(kvs, kvs.lib.kvs_read_pages(p, b, kvs.KVS_DT_F32, x, None, None), text)
    refused(kvs, kvs.lib.kvs_read_pages(p, b, kvs.KVS_DT_F32, r, x, None), text)
    for q, o in ((x, r), (r, x)):
        refused(kvs, kvs.lib.kvs_attend_pages(p, b, 0, 4, q, 0, o, None, None, None, A, 1 << 40, None), text)


def test_append_refusals(kvs):
    p, b, r = pool(kvs), batch(kvs), rows(kvs)

    def call(dtype=0, heads=0, q=None, qo=None, rope=None):
        return kvs.lib.kvs_append_pages(p, b, dtype, r, r, heads, q, qo, rope, None)
    refused(kvs, call(dtype=3), "dtype")
    refused(kvs, call(heads=4, q=r), "go together")
    refused(kvs, call(heads=4, qo=r), "go together")
    refused(kvs, call(heads=0, q=r, qo=r), "n_q_heads")
    refused(kvs, call(heads=65534, q=r, qo=r), "65535")
    for rope, text in ((kvs.kvs_rope(A, 3, 0, None, 0, 1.0), "rot_dim"), (kvs.kvs_rope(A, 130, 0, None, 0, 1.0), "rot_dim"),
                       (kvs.kvs_rope(A, -2, 0, None, 0, 1.0), "rot_dim"), (kvs.kvs_rope(None, 64, 0, None, 0, 1.0), "inv_freq"),
                       (kvs.kvs_rope(A + 2, 64, 0, None, 0, 1.0), "inv_freq"), (kvs.kvs_rope(A, 64, 0, A + 1, 0, 1.0), "inv_freq"),
                       (kvs.kvs_rope(A, 64, 0, None, 0, float("nan")), "mscale")):
        refused(kvs, call(rope=rope), text)


def test_read_refusals(kvs):
    p, b, r = pool(kvs), batch(kvs), rows(kvs)
    refused(kvs, kvs.lib.kvs_read_pages(p, b, 5, r, r, None), "dtype")
    refused(kvs, kvs.lib.kvs_read_pages(p, b, 0, None, None, None), "neither")


def test_attend_refusals(kvs):
    p, b, r = pool(kvs), batch(kvs), rows(kvs)
    size = kvs.lib.kvs_attend_pages_workspace(b, 4, 2)

    def call(q_dtype=0, heads=4, out_dtype=0, lse=None, score=None, prefix=None, work=A, bytes=size):
        return kvs.lib.kvs_attend_pages(p, b, q_dtype, heads, r, out_dtype, r, lse, score, prefix, work, bytes, None)
    refused(kvs, call(heads=3), "multiple")
    refused(kvs, call(heads=0), "multiple")
    refused(kvs, call(q_dtype=kvs.KVS_DT_F32), "F16 or BF16")
    refused(kvs, call(out_dtype=7), "out_dtype")
    refused(kvs, call(lse=A + 2), "lse")
    refused(kvs, call(work=None), "workspace")
    refused(kvs, call(work=A + 128), "workspace")
    refused(kvs, call(bytes=size - 1), "workspace")
    for score in (kvs.kvs_score(float("inf")), kvs.kvs_score(0.0, -1.0), kvs.kvs_score(0.0, float("nan")), kvs.kvs_score(0.0, 0.0, -1)):
        refused(kvs, call(score=score), "score")
    for at in (3, 4, 5):
        arrays = [None, None, None]
        arrays[at - 3] = A + 2
        refused(kvs, call(score=kvs.kvs_score(0.0, 0.0, 0, *arrays)), "score arrays")
    refused(kvs, call(prefix=kvs.kvs_page_prefix(A, -1)), "prefix")
    refused(kvs, call(prefix=kvs.kvs_page_prefix(None, 5)), "prefix")
    refused(kvs, call(prefix=kvs.kvs_page_prefix(A + 1, 5)), "prefix")


def test_workspace_size(kvs):
    f = kvs.lib.kvs_attend_pages_workspace
    small, big = f(batch(kvs, n_rows=1), 8, 2), f(batch(kvs, n_rows=4096), 8, 2)
    assert 0 < small < big and big >= 4096 * 8 * 130 * 4
    assert f(batch(kvs), 3, 2) == 0 and f(None, 4, 2) == 0 and f(batch(kvs, n_rows=-1), 4, 2) == 0 and f(batch(kvs), 4, 0) == 0
    with pytest.raises(kvs.KvsError):
        kvs.kvs_attend_pages_workspace(batch(kvs), 3, 2)


def test_struct_sizes_match_the_header(kvs):
    """The header's structs, compiled, have the binding's sizes."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ["kvs_page_pool", "kvs_page_batch", "kvs_page_rows", "kvs_rope", "kvs_score", "kvs_page_prefix"]
    src = '#include <stdio.h>\n#include "kvs.h"\nint main(void) {\n' + "".join(f'printf("%zu\\n", sizeof({n}));\n' for n in names) + "return 0;}\n"
    with tempfile.TemporaryDirectory() as d:
        with open(os.path.join(d, "s.c"), "w") as f:
            f.write(src)
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), "-o", os.path.join(d, "s"), os.path.join(d, "s.c")], check=True)
        out = subprocess.run([os.path.join(d, "s")], check=True, capture_output=True, text=True).stdout.split()
    assert [int(x) for x in out] == [ctypes.sizeof(getattr(kvs, n)) for n in names]
