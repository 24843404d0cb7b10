"""The binding of the batch operators refuses host tensors and tensors of another
device before any address reaches the library.  Without a GPU: stand-ins with a
tensor's attributes, on devices that need not exist.  A call that is let through
ends at the library's check of the pool's address, with a message of its own."""
import pytest
import torch

from test_pages_abi import A, kvs  # noqa: F401  (kvs: the fixture)


class Tensor:
    def __init__(self, *shape, dtype=torch.float16, device=0, strides=None):
        self.shape, self.dtype, self.at = shape, dtype, device
        step, at = [], 1
        for n in reversed(shape):
            step.insert(0, at)
            at *= n
        self.steps, self.flat = strides or tuple(step), strides is None
        self.is_cuda = device >= 0

    def get_device(self):
        return self.at

    def stride(self):
        return self.steps

    def dim(self):
        return len(self.shape)

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    def is_contiguous(self):
        return self.flat

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def data_ptr(self):
        return A


def ints(*shape, **kw):
    return Tensor(*shape, dtype=torch.int32, **kw)


def parts(kvs, other=0):  # noqa: F811
    """Descriptors on device 0, and those that may be on `other`."""
    head = kvs.kvs_page_bytes(kvs.make_config(1, 2, 2, 256, 1))
    pool = kvs.make_page_pool(Tensor(4 * head, dtype=torch.uint8), 2)
    batch = kvs.make_page_batch(ints(3, device=other), ints(2, device=other), ints(2, 4, device=other), 5, status=ints(1, device=other))
    return pool, batch


def refuser(kvs, call):  # noqa: F811
    with pytest.raises(kvs.KvsError) as e:
        call()
    late = "pool pages must be device memory" in str(e.value) or e.value.code == kvs.KVS_E_CUDA
    assert late or e.value.code == kvs.KVS_E_INVAL
    return "library" if late else "binding"


def attend(kvs, pool, batch, **kw):  # noqa: F811
    n = kvs.kvs_attend_pages_workspace(batch, 4, 2)
    a = dict(q=Tensor(5, 4, 128), out=Tensor(5, 4, 128), lse=Tensor(5, 4, dtype=torch.float32), workspace=Tensor(n, dtype=torch.uint8))
    a.update(kw)
    return refuser(kvs, lambda: kvs.kvs_attend_pages(pool, batch, **a))


@pytest.mark.parametrize("device", [-1, 1], ids=["host", "another-device"])
def test_attend_refuses_tensors_elsewhere(kvs, device):  # noqa: F811
    pool, batch = parts(kvs)
    n = kvs.kvs_attend_pages_workspace(batch, 4, 2)
    assert attend(kvs, pool, batch) == "library"  # all as it should be but for the address
    for kw in (dict(q=Tensor(5, 4, 128, device=device)), dict(out=Tensor(5, 4, 128, device=device)),
               dict(lse=Tensor(5, 4, dtype=torch.float32, device=device)), dict(workspace=Tensor(n, dtype=torch.uint8, device=device)),
               dict(workspace=Tensor(n, dtype=torch.uint8, strides=(2,)))):
        assert attend(kvs, pool, batch, **kw) == "binding", kw


@pytest.mark.parametrize("device", [-1, 1], ids=["host", "another-device"])
def test_append_and_read_refuse_tensors_elsewhere(kvs, device):  # noqa: F811
    pool, batch = parts(kvs)
    k, q, far = Tensor(5, 2, 128), Tensor(5, 4, 128), Tensor(5, 2, 128, device=device)
    for args in ((far, k), (k, far), (k, k, Tensor(5, 4, 128, device=device), q), (k, k, q, Tensor(5, 4, 128, device=device))):
        assert refuser(kvs, lambda: kvs.kvs_append_pages(pool, batch, *args)) == "binding"
    for args in ((far, None), (None, far), (k, far)):
        assert refuser(kvs, lambda: kvs.kvs_read_pages(pool, batch, *args)) == "binding"


def test_descriptors_of_another_device(kvs):  # noqa: F811
    pool, batch = parts(kvs)
    _, far = parts(kvs, other=1)
    assert attend(kvs, pool, far) == "binding"
    for kw in (dict(score=kvs.make_score(first_key=ints(5, device=1))), dict(prefix=kvs.make_page_prefix(ints(2, device=1), 300))):
        assert attend(kvs, pool, batch, **kw) == "binding"
    k = Tensor(5, 2, 128)
    rope = kvs.make_rope(Tensor(64, dtype=torch.float32, device=1))
    assert refuser(kvs, lambda: kvs.kvs_append_pages(pool, batch, k, k, rope=rope)) == "binding"
    for make in (lambda: kvs.make_page_batch(ints(3), ints(2), ints(2, 4, device=1), 5), lambda: kvs.make_page_batch(ints(3), ints(2, device=-1), ints(2, 4), 5),
                 lambda: kvs.make_score(first_key=ints(5), end_key=ints(5, device=1)),
                 lambda: kvs.make_rope(Tensor(64, dtype=torch.float32), positions=ints(5, device=1))):
        with pytest.raises(kvs.KvsError):
            make()
