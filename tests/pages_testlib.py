"""Helpers of the tests of the batch operators over caller-owned pages.

The plain implementation works on canonical blocks made by the CPU oracle and
in binary64; page bytes are laid out here from the documented page format, so
nothing below shares code with the kernels.
"""
import math

import numpy as np

import oracle

F16, Q4_0, Q4_1, Q5_0, Q5_1, Q8_0 = 1, 2, 3, 6, 7, 8
PAIRS = [(Q8_0, Q4_0), (Q8_0, Q8_0), (Q8_0, Q5_0), (Q8_0, Q4_1), (Q8_0, Q5_1), (Q8_0, F16), (F16, F16)]
PAIR_IDS = ["q8-q4_0", "q8-q8", "q8-q5_0", "q8-q4_1", "q8-q5_1", "q8-f16", "f16-f16"]


def torch():
    import torch as t
    return t


def field_rows(type_k, type_v):
    """[(name, bytes per token, offset in the page head)], page head bytes."""
    rows = [("kq", 256 if type_k == F16 else 128), ("kd", 0 if type_k == F16 else 8),
            ("vq", {F16: 256, Q8_0: 128}.get(type_v, 64)), ("vh", 16 if type_v in (Q5_0, Q5_1) else 0),
            ("vd", 0 if type_v == F16 else 8), ("vm", 8 if type_v in (Q4_1, Q5_1) else 0)]
    out, at = {}, 0
    for name, b in rows:
        out[name] = (b, at)
        at += 256 * b
    return out, at


def split_blocks(kb, vb, type_k, type_v):
    """Canonical block bytes [..., 4, bytes] -> the page fields' bytes per row."""
    flat = lambda a: a.reshape(*a.shape[:-2], -1)  # noqa: E731
    f = {}
    if type_k == F16:
        f["kq"] = flat(kb)
    else:
        f["kd"], f["kq"] = flat(kb[..., :2]), flat(kb[..., 2:])
    if type_v == F16:
        f["vq"] = flat(vb)
        return f
    f["vd"] = flat(vb[..., :2])
    at = 2
    if type_v in (Q4_1, Q5_1):
        f["vm"] = flat(vb[..., 2:4])
        at = 4
    if type_v in (Q5_0, Q5_1):
        f["vh"] = flat(vb[..., at:at + 4])
        at += 4
    f["vq"] = flat(vb[..., at:])
    return f


def put_rows(pool, types, pages, toks, k16, v16):
    """Quantize fp16 rows [n, n_kv, 128] (oracle) into host page bytes pool
    [n_pages, n_kv, head bytes] at (pages[i], toks[i])."""
    fields, _ = field_rows(*types)
    kb, vb = oracle.quantize_rows(k16, v16, types[1], types[0])
    for name, a in split_blocks(kb, vb, *types).items():
        b, off = fields[name]
        for i, (p, t) in enumerate(zip(pages, toks)):
            pool[p, :, off + t * b:off + (t + 1) * b] = a[i]


def row_values(pool, types, pages, toks):
    """The binary64 values of K and V rows [n, n_kv, 128] held in page bytes."""
    fields, _ = field_rows(*types)
    n, H = len(pages), pool.shape[1]

    def get(name, dtype):
        b, off = fields[name]
        if not b:
            return None
        rows = np.stack([pool[p, :, off + t * b:off + (t + 1) * b] for p, t in zip(pages, toks)]) if n else \
            np.zeros((0, H, b), np.uint8)
        return np.ascontiguousarray(rows).view(dtype)
    half = lambda x: x.view(np.float16).astype(np.float64)  # noqa: E731
    kq = get("kq", np.uint8)
    k = half(kq) if types[0] == F16 else (kq.view(np.int8).astype(np.float64).reshape(n, H, 4, 32) *
                                          half(get("kd", np.uint8))[..., None]).reshape(n, H, 128)
    vq = get("vq", np.uint8)
    if types[1] == F16:
        return k, half(vq)
    d = half(get("vd", np.uint8))[..., None]
    if types[1] == Q8_0:
        return k, (vq.view(np.int8).astype(np.float64).reshape(n, H, 4, 32) * d).reshape(n, H, 128)
    c = vq.reshape(n, H, 4, 16)
    c = np.concatenate([c & 15, c >> 4], -1).astype(np.int64)
    if types[1] in (Q5_0, Q5_1):
        w = get("vh", np.uint32).astype(np.int64)[..., None]
        c += ((w >> np.arange(32)) & 1) << 4
    if types[1] in (Q4_0, Q5_0):
        return k, ((c - (8 if types[1] == Q4_0 else 16)) * d).reshape(n, H, 128)
    return k, (c * d + half(get("vm", np.uint8))[..., None]).reshape(n, H, 128)


class Batch:
    """A batch over a host-made pool: `new` and `lens` per sequence, random page
    numbers, `pad` rows behind the last sequence, an optional shared prefix."""

    def __init__(self, new, lens, n_qh, n_kv, types, prefix=0, pad=0, seed=0, spare=2, scale=1.0, outliers=True, extra_cols=1):
        t = torch()
        rng = self.rng = np.random.default_rng([seed, 77])
        self.new, self.lens, self.n_qh, self.n_kv, self.types, self.prefix = list(new), list(lens), n_qh, n_kv, types, prefix
        self.rows = sum(self.new) + pad
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        need = [-(-max(n, 0) // 256) for n in self.lens]
        pp = -(-prefix // 256)
        self.n_pages = sum(need) + pp + spare
        order = rng.permutation(self.n_pages).astype(np.int32)
        self.prefix_table = order[:pp].copy()
        cols = max(need + [0]) + extra_cols
        self.table = np.full((len(self.lens), cols), -7, np.int32)  # entries past the last page are never read
        at = pp
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        _, head = field_rows(*types)
        self.pool = rng.integers(0, 256, (self.n_pages, n_kv, head), dtype=np.uint8)  # what nobody wrote holds anything

        def rows(n, h):
            x = rng.standard_normal((n, h, 128)) * scale
            if outliers:
                x = np.where(rng.random(x.shape) < 0.01, 8 * x, x)
            return x.astype(np.float16)
        for length, table in [(prefix, self.prefix_table)] + [(n, self.table[i]) for i, n in enumerate(self.lens)]:
            p = np.arange(max(length, 0))
            if p.size:
                put_rows(self.pool, types, [int(table[x // 256]) for x in p], [int(x % 256) for x in p], rows(p.size, n_kv),
                         rows(p.size, n_kv))
        self.q = (rng.standard_normal((self.rows, n_qh, 128)) * 1.5).astype(np.float32)
        self.t = t

    # ---- device side ----
    def device(self, status=False, max_new=None):
        from host_streamed_paged_kvs_b200 import kvs
        t = self.t
        self.kvs = kvs
        self.d_pool = t.from_numpy(self.pool).cuda()
        self.d = dict(start=t.from_numpy(self.start).cuda(), lens=t.tensor(self.lens, dtype=t.int32, device="cuda"),
                      table=t.from_numpy(self.table).cuda(), ptable=t.from_numpy(self.prefix_table).cuda())
        self.status = t.zeros(1, dtype=t.int32, device="cuda") if status else None
        self.c_pool = kvs.make_page_pool(self.d_pool, self.n_kv, *self.types)
        self.c_batch = kvs.make_page_batch(self.d["start"], self.d["lens"], self.d["table"], self.rows,
                                           max_new=max(self.new + [0]) if max_new is None else max_new, status=self.status)
        self.c_prefix = kvs.make_page_prefix(self.d["ptable"], self.prefix) if self.prefix else None
        return self

    def workspace(self):
        n = self.kvs.kvs_attend_pages_workspace(self.c_batch, self.n_qh, self.n_kv)
        return self.t.zeros(n, dtype=self.t.uint8, device="cuda")

    # ---- plain implementation ----
    def seq_of(self, row):
        for i in range(len(self.new)):
            if self.start[i] <= row < self.start[i + 1]:
                return i
        return -1

    def position(self, row, i):
        """Own position of a row of sequence i."""
        return self.lens[i] - int(self.start[i + 1]) + row

    def values(self, i):
        """K, V values of the prefix and sequence i, binary64."""
        parts = []
        for length, table in ((self.prefix, self.prefix_table), (max(self.lens[i], 0), self.table[i])):
            p = np.arange(length)
            parts.append(row_values(self.pool, self.types, [int(table[x // 256]) for x in p], [int(x % 256) for x in p]))
        return [np.concatenate(x) for x in zip(*parts)]

    def plain_attention(self, q, scale=None, softcap=0.0, window=0, slopes=None, first=None, end=None):
        """(out, lse) in binary64 for q [rows, n_qh, 128] (its values as given); NaN rows for padding."""
        G = self.n_qh // self.n_kv
        out = np.full((self.rows, self.n_qh, 128), np.nan)
        lse = np.full((self.rows, self.n_qh), np.nan)
        scale = 1 / math.sqrt(128) if scale is None else scale
        for i in range(len(self.new)):
            k, v = self.values(i)
            total = k.shape[0]
            j = np.arange(total)
            for row in range(self.start[i], self.start[i + 1]):
                p = self.prefix + self.position(row, i)
                lo = max(0, p - window + 1) if window and first is None else (0 if first is None else max(0, int(first[row])))
                hi = min(total, p + 1 if end is None else int(end[row]))
                sel = (j >= lo) & (j < hi)
                for h in range(self.n_qh):
                    if not sel.any():
                        out[row, h], lse[row, h] = 0.0, -np.inf
                        continue
                    s = scale * (k[sel, h // G] @ q[row, h].astype(np.float64))
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    if slopes is not None:
                        s = s - float(slopes[h]) * np.abs(p - j[sel])
                    m = s.max()
                    e = np.exp(s - m)
                    out[row, h] = e @ v[sel, h // G] / e.sum()
                    lse[row, h] = m + np.log(e.sum())
        return out, lse
