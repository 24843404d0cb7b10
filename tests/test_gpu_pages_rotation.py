"""kvs_append_pages: rotated Q is rounded once, from the binary64 rotation."""
import numpy as np
import pytest

from pages_testlib import F16, Batch, torch
from test_gpu_pages_append import inv_freq, rotate64

pytestmark = pytest.mark.gpu


def nearest(x, bits, least):
    """x (binary64) as its nearest number of `bits` significant bits, ties to even,
    with exponents from 2^least on (below it the grid stays)."""
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e, least) - bits)
    return np.rint(x / step) * step


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,bits,least", [("float16", 11, -13), ("bfloat16", 8, -125)])
@pytest.mark.parametrize("rot", [128, 20])
def test_q_is_rounded_once(dtype, bits, least, inter, rot):
    """A value whose binary32 rounding falls on the middle of two numbers of the
    type must still go to its own side: about one in 2^13 fp16 values, 2^16 bf16
    values does.  Binary64 itself is off by 2^-50, which no value here is near a
    border by (the check leaves out those that are)."""
    t = torch()
    b = Batch([600], [600], 16, 1, (F16, F16), seed=71 + rot + inter).device()
    dt = getattr(t, dtype)
    f = inv_freq(rot)
    q = t.from_numpy(b.rng.standard_normal((600, 16, 128))).to(dt).cuda()
    k = t.zeros(600, 1, 128, dtype=dt, device="cuda")
    out = t.zeros_like(q)
    pos = np.arange(600) + 7000
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k, q, out, b.kvs.make_rope(t.from_numpy(f).cuda(), rot, interleaved=inter, pos_offset=7000))
    x = rotate64(q.double().cpu().numpy(), pos, f, rot, inter)
    got = out.double().cpu().numpy()
    lo, hi = nearest(x * (1 - 2.0 ** -48), bits, least), nearest(x * (1 + 2.0 ** -48), bits, least)
    sure = lo == hi
    assert sure.mean() > 0.999
    assert np.array_equal(got[sure], lo[sure])
