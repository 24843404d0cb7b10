"""kvs_append_pages and kvs_read_pages on the GPU: page bytes against the CPU
oracle's blocks, rotation against binary64, read-back exact, padding and bad
pages left alone."""
import numpy as np
import pytest

from pages_testlib import F16, PAIR_IDS, PAIRS, Q4_0, Q8_0, Batch, field_rows, put_rows, row_values, torch

pytestmark = pytest.mark.gpu


def rotate64(x, pos, inv_freq, rot, inter, mscale=1.0):
    """Rows [n, h, 128] turned in binary64."""
    x = x.astype(np.float64).copy()
    a = pos[:, None].astype(np.float64) * inv_freq.astype(np.float64)[None]
    c, s = (mscale * np.cos(a))[:, None], (mscale * np.sin(a))[:, None]
    lo, hi = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if inter else (np.arange(rot // 2), np.arange(rot // 2, rot))
    u, v = x[..., lo].copy(), x[..., hi].copy()
    x[..., lo], x[..., hi] = u * c - v * s, v * c + u * s
    return x


def inv_freq(rot, base=10000.0):
    return (base ** (-np.arange(rot // 2) / (rot // 2))).astype(np.float32)


def expected_pool(b, k, v):
    """b's pool with the new rows stored: K and V rows are fp16-representable."""
    pool = b.pool.copy()
    pages, toks, rows = [], [], []
    for row in range(int(b.start[-1])):
        i = b.seq_of(row)
        p = b.position(row, i)
        if p >= 0:
            pages.append(int(b.table[i, p // 256]))
            toks.append(p % 256)
            rows.append(row)
    put_rows(pool, b.types, pages, toks, np.ascontiguousarray(k[rows]), np.ascontiguousarray(v[rows]))
    return pool


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_append_bytes_are_the_oracles(types, dtype):
    """No rotation: the stored bytes are the oracle's blocks of the same values,
    and nothing else in the pool changes (bf16 and fp32 inputs hold
    fp16-representable values so that the oracle takes them)."""
    t = torch()
    b = Batch([1, 5, 0, 300, 3], [1, 260, 40, 513, 2], 4, 2, types, pad=3, seed=1).device()
    x = b.rng.standard_normal((2, b.rows, 2, 128))
    x = np.where(b.rng.random(x.shape) < 0.01, 8 * x, x)
    x[0, 0, 0, :32] = 0.0                      # a zero block, ties, a single value
    x[1, 0, 1, 32:64] = 1.0
    x[1, 0, 1, 64:96] = 0.0
    x[1, 0, 1, 70] = -3.0
    src = t.from_numpy(x).to(getattr(t, dtype)).cuda()
    x16 = src.half().cpu().numpy()
    if dtype == "bfloat16":                    # small bf16 values may lie below fp16's grid: take those it holds
        src = t.from_numpy(x16).to(t.bfloat16).half().to(t.bfloat16).cuda()
        x16 = src.half().cpu().numpy()
        assert (t.from_numpy(x16).to(t.bfloat16).cuda() == src).all()
    if dtype == "float32":
        src = t.from_numpy(x16).float().cuda()
    # rows 1 past the tensor's own: strided views of one buffer, K and V side by side
    both = t.cat([src[0], src[1]], dim=1)
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, both[:, :2], both[:, 2:])
    # sequence 4 has 3 new rows and 2 tokens: its first row is at -1 and stored nowhere
    want = expected_pool(b, x16[0], x16[1])
    got = b.d_pool.cpu().numpy()
    assert np.array_equal(got, want)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [128, 64, 20, 2])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_rotation(rot, inter, dtype):
    """Q's rounding is the only one (half a step of its type); K comes out as the
    oracle's blocks of the rotated rows, far positions and an offset among them."""
    t = torch()
    b = Batch([2, 1, 7], [700, 1, 300], 3, 1, (F16, F16), seed=rot + inter).device()
    f = inv_freq(rot)
    pos = np.array([700 - 2, 700 - 1, 0] + list(range(293, 300))) + 1000000
    dt = getattr(t, dtype)
    k, v, q = (t.from_numpy(b.rng.standard_normal((b.rows, h, 128))).to(dt).cuda() for h in (1, 1, 3))
    q_out = t.full_like(q, 7.0)
    rope = b.kvs.make_rope(t.from_numpy(f).cuda(), rot, interleaved=inter, pos_offset=1000000, mscale=1.25)
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, v, q, q_out, rope)
    want = rotate64(q.double().cpu().numpy(), pos, f, rot, inter, 1.25)
    got = q_out.double().cpu().numpy()
    eps = t.finfo(dt).eps / 2
    # products and sum in binary64 add far less than the 1e-9 kept here
    assert np.all(np.abs(got - want) <= eps * np.abs(want) + 1e-7)
    assert np.array_equal(got[..., rot:], q.double().cpu().numpy()[..., rot:])
    kw = rotate64(k.double().cpu().numpy(), pos, f, rot, inter, 1.25)
    pages = [int(b.table[b.seq_of(r), (p - 1000000) // 256]) for r, p in enumerate(pos)]
    kp, vp = row_values(b.d_pool.cpu().numpy(), b.types, pages, [int(p - 1000000) % 256 for p in pos])
    assert np.array_equal(kp.astype(np.float16), kw.astype(np.float32).astype(np.float16))
    assert np.array_equal(vp, v.half().double().cpu().numpy())


def test_rotated_codes_are_those_of_the_binary32_values():
    """Quantized K decided from the binary32 rounding of the binary64 rotation."""
    t = torch()
    b = Batch([400, 33], [900, 33], 2, 2, (Q8_0, Q4_0), seed=5).device()
    f = inv_freq(128, 500000.0)
    k, v = (t.from_numpy(b.rng.standard_normal((b.rows, 2, 128))).bfloat16().cuda() for _ in range(2))
    pos = np.concatenate([np.arange(500, 900), np.arange(33)])
    explicit = t.from_numpy((pos * 3 + 5).astype(np.int32)).cuda()
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, v, rope=b.kvs.make_rope(t.from_numpy(f).cuda(), 128, positions=explicit))
    x = rotate64(k.double().cpu().numpy(), pos * 3 + 5, f, 128, False).astype(np.float32).reshape(-1, 2, 4, 32)
    d = np.abs(x).max(-1, keepdims=True) / np.float32(127)
    r = (x / d).astype(np.float64)
    codes = np.sign(r) * np.floor(np.abs(r) + 0.5)
    want = (codes * d.astype(np.float16).astype(np.float64)).reshape(-1, 2, 128)
    pages = [int(b.table[b.seq_of(row), p // 256]) for row, p in enumerate(pos)]
    got, _ = row_values(b.d_pool.cpu().numpy(), b.types, pages, [int(p % 256) for p in pos])
    assert np.array_equal(got, want)


def test_q_in_place_and_without_rotation():
    t = torch()
    b = Batch([3], [3], 5, 1, (Q8_0, Q4_0), seed=9).device()
    q = t.randn(3, 5, 128, device="cuda").half()
    before = q.clone()
    k = t.randn(3, 1, 128, device="cuda").half()
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k, q, q)
    assert t.equal(q, before)
    f = t.from_numpy(inv_freq(128)).cuda()
    out = t.empty_like(q)
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k, q, out, b.kvs.make_rope(f))
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k, q, q, b.kvs.make_rope(f))
    assert t.equal(q, out) and not t.equal(q, before)


@pytest.mark.parametrize("types", PAIRS, ids=PAIR_IDS)
@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_read_back(types, dtype):
    """fp32 is exact; fp16 and bf16 are its nearest values; rows at negative
    positions are zeros, padding stays."""
    t = torch()
    b = Batch([257, 0, 4, 1], [700, 3, 2, 1], 4, 3, types, pad=5, seed=3).device(status=True)
    dt = getattr(t, dtype)
    wide = t.full((b.rows, 3, 256), 9.0, dtype=dt, device="cuda")
    k, v = wide[..., :128], t.full((b.rows, 3, 128), 9.0, dtype=dt, device="cuda")
    b.kvs.kvs_read_pages(b.c_pool, b.c_batch, k, v)
    n = int(b.start[-1])
    kw, vw = np.zeros((n, 3, 128)), np.zeros((n, 3, 128))
    for row in range(n):
        i = b.seq_of(row)
        p = b.position(row, i)
        if p >= 0:
            a, c = row_values(b.pool, types, [int(b.table[i, p // 256])], [p % 256])
            kw[row], vw[row] = a[0], c[0]
    for got, want in ((k, kw), (v, vw)):
        # d q + m rounds once to binary32 for the types with a minimum
        assert t.equal(got[:n].cpu(), t.from_numpy(want).float().to(dt))
        assert bool((got[n:] == 9).all())
    assert bool((wide[..., 128:] == 9).all()) and int(b.status) == 0
    only = t.zeros_like(v)
    b.kvs.kvs_read_pages(b.c_pool, b.c_batch, v=only)
    assert t.equal(only[:n], v[:n])


def test_bad_pages_are_not_followed():
    """Page numbers outside the pool and positions beyond the page table: no
    write, NaN on reading, the status bit set, every other row as usual."""
    t = torch()
    b = Batch([2, 2, 2], [300, 300, 300], 2, 1, (Q8_0, Q4_0), seed=4)
    b.table[0, 1] = b.n_pages       # one past the pool
    b.table[1, 1] = -1
    b.device(status=True)
    k = t.randn(b.rows, 1, 128, device="cuda").half()
    b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k)
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    want = b.pool.copy()
    k16 = k.cpu().numpy()
    put_rows(want, b.types, [int(b.table[2, 1])] * 2, [42, 43], k16[4:], k16[4:])
    assert np.array_equal(b.d_pool.cpu().numpy(), want)
    b.status.zero_()
    out = t.zeros(b.rows, 1, 128, device="cuda")
    b.kvs.kvs_read_pages(b.c_pool, b.c_batch, out)
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE
    assert bool(out[:4].isnan().all()) and not bool(out[4:].isnan().any())
    # a length beyond the table
    b.d["lens"].fill_(256 * b.table.shape[1] + 2)
    b.status.zero_()
    b.kvs.kvs_read_pages(b.c_pool, b.c_batch, out)
    assert int(b.status) == b.kvs.KVS_ERR_BAD_PAGE and bool(out.isnan().all())


def test_captured_append_follows_the_lengths():
    """A captured append replayed after the lengths moved writes the new slots."""
    t = torch()
    b = Batch([1, 1], [255, 10], 2, 2, (Q8_0, Q4_0), seed=6, extra_cols=2)
    b.table[0, 1] = b.n_pages - 1
    b.device()
    k = t.randn(2, 2, 128, device="cuda").half()
    s = t.cuda.Stream()
    with t.cuda.stream(s):
        b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k, stream=s)
        s.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=s):
            b.kvs.kvs_append_pages(b.c_pool, b.c_batch, k, k, stream=s)
    want = b.pool.copy()
    for step in range(3):
        lens = [255 + step, 10 + step]
        b.d["lens"].copy_(t.tensor(lens, dtype=t.int32))
        k.normal_()
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        k16 = k.cpu().numpy()
        put_rows(want, b.types, [int(b.table[i, (n - 1) // 256]) for i, n in enumerate(lens)], [(n - 1) % 256 for n in lens], k16, k16)
    if True:  # the call before the capture wrote the first step's slots with other rows, overwritten by step 0
        assert np.array_equal(b.d_pool.cpu().numpy(), want)


def test_page_geometry_of_the_helpers_is_the_librarys():
    from host_streamed_paged_kvs_b200 import kvs
    for types in PAIRS:
        cfg = kvs.make_config(1, 2, 2, 256, 1, type_k=types[0], type_v=types[1])
        assert kvs.kvs_page_bytes(cfg) == 2 * field_rows(*types)[1]
