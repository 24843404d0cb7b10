"""The batch operators' host side beyond their refusals, without a GPU."""
import pytest

from test_pages_abi import A, batch, kvs, pool, rows  # noqa: F401  (kvs: the fixture)


def test_tensors_of_no_rows_may_have_null_addresses(kvs):  # noqa: F811
    """n_rows 0: a null address is not refused (here the calls end at the device
    check, as there is no device behind A)."""
    p, b, r = pool(kvs), batch(kvs, n_rows=0), rows(kvs, data=None)
    for call in (lambda: kvs.lib.kvs_append_pages(p, b, kvs.KVS_DT_F16, r, r, 4, r, r, None, None),
                 lambda: kvs.lib.kvs_read_pages(p, b, kvs.KVS_DT_F32, r, r, None),
                 lambda: kvs.lib.kvs_attend_pages(p, b, kvs.KVS_DT_F16, 4, r, kvs.KVS_DT_F32, r, None, None, None, A, 1 << 40, None)):
        assert call() != kvs.KVS_OK
        assert "device" in kvs.kvs_last_error(), kvs.kvs_last_error()


@pytest.mark.parametrize("bad", [dict(row=514), dict(head=130)])
def test_strides_are_checked_without_rows_too(kvs, bad):  # noqa: F811
    r = rows(kvs, data=None, **bad)
    assert kvs.lib.kvs_read_pages(pool(kvs), batch(kvs, n_rows=0), kvs.KVS_DT_F16, r, None, None) == kvs.KVS_E_INVAL
    assert "16 bytes" in kvs.kvs_last_error()
