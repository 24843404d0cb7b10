"""Operators over caller-owned device pages: what is measured, and their plain forms.

Three operators work on one pool of quantized pages that a batch of sequences
shares through page tables:

  append   K/V rows of every sequence's new tokens are rotated by position (Q
           rows too), quantized and written to the pages; Q comes back rotated
  read     the new tokens' rows are read back from the pages as values
  attend   the new tokens attend their sequence's pages, with a causal bound,
           capped scores, a distance bias, a window, and document and prefix
           masks as key intervals; with a prefix whose pages all sequences share

A page is 256 tokens of all kv heads, [n_kv][page head]; a page head holds its
fields one after another (K codes, K scales, V codes, V fifth bits, V scales, V
minima).  Pool, page tables and lengths are what a serving loop has in hand.
"""
import math
import random

import torch

own = False

D, T, NB = 128, 256, 4                     # head dim, tokens a page, 32-value blocks a row
F16, Q4_0, Q4_1, Q5_0, Q5_1, Q8_0 = 1, 2, 3, 6, 7, 8
KINDS = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step's append for 64 sequences, f16 pages: a small batch's latency
        dict(name="append_decode_64", op="append", seqs=64, new_lo=1, new_hi=1, len_lo=100, len_hi=1000, n_qh=32, n_kv=8,
             type_k=F16, type_v=F16, dtype="bf16", rot=128, inter=False, packed=True),
        # prompts of 5 sequences brought in at once, quantized pages, half of each head rotated, values read back
        dict(name="append_prompts_8k", op="append", seqs=5, new_lo=301, new_hi=2999, len_lo=300, len_hi=3100, n_qh=32, n_kv=8,
             type_k=Q8_0, type_v=Q4_0, dtype="bf16", rot=64, inter=True, packed=True),
        # one short sequence handed to another engine as fp32 values
        dict(name="read_4k", op="read", seqs=1, new_lo=4096, new_hi=4096, len_lo=4096, len_hi=4096, n_qh=8, n_kv=2,
             type_k=Q8_0, type_v=Q5_1, dtype="f32"),
        # 16 ragged sequences as bf16 values
        dict(name="read_16_ragged", op="read", seqs=16, new_lo=1, new_hi=8191, len_lo=8191, len_hi=8191, n_qh=32, n_kv=8,
             type_k=Q8_0, type_v=Q4_0, dtype="bf16"),
        # the smallest decode call: one token of one 4K sequence
        dict(name="decode_1x4k", op="attend", seqs=1, new_lo=1, new_hi=1, len_lo=4096, len_hi=4096, n_qh=8, n_kv=2,
             type_k=Q8_0, type_v=Q4_0, dtype="f16"),
        # a serving batch: 64 sequences of every length up to 8K, scores capped
        dict(name="decode_64_ragged_capped", op="attend", seqs=64, new_lo=1, new_hi=1, len_lo=1, len_hi=8191, n_qh=32, n_kv=8,
             type_k=Q8_0, type_v=Q4_0, dtype="bf16", cap=30.0),
        # one very long sequence
        dict(name="decode_1x256k", op="attend", seqs=1, new_lo=1, new_hi=1, len_lo=262144, len_hi=262144, n_qh=40, n_kv=8,
             type_k=Q8_0, type_v=Q4_0, dtype="bf16"),
        # a 256-token prompt chunk at the end of 64K
        dict(name="chunk_256_at_64k", op="attend", seqs=1, new_lo=256, new_hi=256, len_lo=65536, len_hi=65536, n_qh=40, n_kv=8,
             type_k=Q8_0, type_v=Q4_0, dtype="bf16"),
        # documents packed into one row, each with a prefix that sees itself whole, and a distance bias
        dict(name="documents_4k", op="attend", seqs=1, new_lo=4096, new_hi=4096, len_lo=4096, len_hi=4096, n_qh=32, n_kv=8,
             type_k=F16, type_v=F16, dtype="bf16", alibi=True, docs=5),
        # 4 sequences that share a short system prompt ending inside a page
        dict(name="prefix_4x1000", op="attend", seqs=4, new_lo=1, new_hi=1, len_lo=1, len_hi=300, n_qh=8, n_kv=2,
             type_k=Q8_0, type_v=Q4_0, dtype="f16", prefix=1000),
        # 64 sequences on one 32K document
        dict(name="prefix_64x32k", op="attend", seqs=64, new_lo=1, new_hi=1, len_lo=1, len_hi=2048, n_qh=32, n_kv=8,
             type_k=Q8_0, type_v=Q4_0, dtype="bf16", prefix=32768),
        # 256 verify steps of 1 to 4 tokens on one 8K prompt, q8_0 pages
        dict(name="prefix_256x8k_verify", op="attend", seqs=256, new_lo=1, new_hi=4, len_lo=4, len_hi=512, n_qh=40, n_kv=8,
             type_k=Q8_0, type_v=Q8_0, dtype="bf16", prefix=8200),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    n_qh, n_kv = rng.choice([(8, 2), (32, 8), (40, 8)])
    type_k, type_v = rng.choice([(Q8_0, Q4_0), (Q8_0, Q4_0), (Q8_0, Q8_0), (Q8_0, Q5_0), (Q8_0, Q5_1), (Q8_0, Q4_1), (Q8_0, F16), (F16, F16)])
    c = dict(n_qh=n_qh, n_kv=n_kv, type_k=type_k, type_v=type_v, dtype="bf16")
    kind = rng.choice(["append", "read", "decode", "decode", "chunk", "documents", "prefix", "prefix"])
    if kind == "append":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 8000 // seqs))
        c.update(op="append", seqs=seqs, new_lo=max(1, new // 3), new_hi=new, len_lo=new, len_hi=new + 500, dtype=rng.choice(["bf16", "f16"]),
                 rot=rng.choice([128, 128, 64, 96, 20]), inter=rng.random() < 0.4, packed=rng.random() < 0.5)
    elif kind == "read":
        seqs = _log(rng, 1, 16)
        n = _log(rng, 16, 60000 // seqs)
        c.update(op="read", seqs=seqs, new_lo=1 + n // 2, new_hi=n, len_lo=n, len_hi=n + 300, dtype=rng.choice(["bf16", "f16", "f32"]))
    elif kind == "decode":
        seqs = _log(rng, 1, 64)
        n = _log(rng, 200, 400000 // seqs)
        c.update(op="attend", seqs=seqs, new_lo=1, new_hi=1, len_lo=1 if seqs > 3 else n // 2, len_hi=n)
        c.update(rng.choice([{}, {"cap": 30.0}, {"window": 1 + n // 3}, {"alibi": True}]))
    elif kind == "chunk":
        new, seqs = _log(rng, 16, 500), rng.randint(1, 3)
        n = _log(rng, 600, 9000000 // (new * seqs) if new > 150 else 60000 // seqs)
        c.update(op="attend", seqs=seqs, new_lo=max(1, new // 2), new_hi=new, len_lo=max(new, n // 2), len_hi=max(new, n))
        c.update(rng.choice([{}, {}, {"cap": 50.0}, {"window": 1 + n // 3}]))
    elif kind == "documents":
        n = _log(rng, 300, 4000)
        c.update(op="attend", seqs=1, new_lo=n, new_hi=n, len_lo=n, len_hi=n, docs=rng.randint(1, 9), alibi=rng.random() < 0.5)
    else:
        seqs = _log(rng, 2, 200)
        c.update(op="attend", seqs=seqs, new_lo=1, new_hi=rng.choice([1, 1, 4]), len_lo=4, len_hi=_log(rng, 16, 60000 // seqs),
                 prefix=_log(rng, 300, 32000 if seqs < 80 else 8000))
        c["len_hi"] = min(c["len_hi"], 2048)
    return c


def _lengths(case):
    """New tokens and lengths after the append of every sequence, from the case's own numbers."""
    r = random.Random("%(seqs)d %(new_lo)d %(new_hi)d %(len_lo)d %(len_hi)d" % case)
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
    new[0] = case["new_hi"]
    lens = [max(n, r.randint(case["len_lo"], case["len_hi"])) for n in new]
    lens[-1] = max(new[-1], case["len_hi"])
    return new, lens


def _intervals(case):
    """For every new token its position and the keys first..end-1 that it sees."""
    new, lens = _lengths(case)
    P, W, docs = case.get("prefix", 0), case.get("window", 0), case.get("docs", 0)
    pos, first, end = [], [], []
    for n, length in zip(new, lens):
        for p in range(P + length - n, P + length):
            pos.append(p)
            first.append(max(0, p - W + 1) if W else 0)
            end.append(p + 1)
    if docs:  # one sequence of `docs` documents; the first quarter of each sees itself whole
        r = random.Random("docs %d %d" % (docs, lens[0]))
        cut = sorted({0, lens[0]} | {r.randint(1, lens[0]) for _ in range(docs - 1)})
        for a, b in zip(cut, cut[1:]):
            for p in range(a, b):
                first[p], end[p] = a, max(p + 1, a + (b - a) // 4)
    return pos, first, end


# ---------------------------------------------------------------- pages

def _fields(type_k, type_v):
    """(bytes a token, byte offset in the page head) of K codes, K scales, V codes, V fifth bits, V scales, V minima; page head bytes."""
    rows = [256 if type_k == F16 else 128, 0 if type_k == F16 else 8, {F16: 256, Q8_0: 128}.get(type_v, 64), 16 if type_v in (Q5_0, Q5_1) else 0,
            0 if type_v == F16 else 8, 8 if type_v in (Q4_1, Q5_1) else 0]
    out, at = [], 0
    for b in rows:
        out.append((b, at))
        at += b * T
    return out, at


def _views(pool, type_k, type_v):
    """The pool's fields as [page, kv head, token, ...] views; None for a field that the types lack."""
    pages, n_kv, _ = pool.shape

    def view(field, dtype):
        size, at = field
        return pool[:, :, at:at + size * T].view(dtype).view(pages, n_kv, T, -1) if size else None
    kq, kd, vq, vh, vd, vm = _fields(type_k, type_v)[0]
    return (view(kq, torch.float16 if type_k == F16 else torch.int8), view(kd, torch.float16),
            view(vq, torch.float16 if type_v == F16 else torch.int8 if type_v == Q8_0 else torch.uint8), view(vh, torch.int32),
            view(vd, torch.float16), view(vm, torch.float16))


def _over(a, b):
    """a / b in 32 bits, 0 where b is 0 (a divisor held in a tensor: a true division)."""
    return torch.where(b == 0, torch.zeros_like(a), a / torch.where(b == 0, torch.ones_like(b), b))


def _codes(x, kind):
    """Rows of 128 values in 32 bits as block codes: (codes, scales, minima), codes as whole numbers from the type's zero on."""
    x = x.reshape(*x.shape[:-1], NB, 32)
    full = lambda v: torch.full(x.shape[:-1] + (1,), float(v), device=x.device)  # noqa: E731
    if kind == Q8_0:
        d = x.abs().amax(-1, keepdim=True) / full(127)
        r = _over(x, d.expand_as(x)).double()
        return (r.sign() * torch.floor(r.abs() + 0.5)).int(), d.half(), None
    if kind in (Q4_0, Q5_0):
        half = 8 if kind == Q4_0 else 16
        top = x.gather(-1, x.abs().argmax(-1, keepdim=True))
        d = top / full(-half)
        q = (_over(x, d.expand_as(x)) + (half + 0.5)).int().clamp(max=2 * half - 1)
        return torch.where(d == 0, half, q), d.half(), None
    top = 15 if kind == Q4_1 else 31
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    d = (hi - lo) / full(top)
    q = (_over(x - lo, d.expand_as(x)) + 0.5).int().clamp(max=top)
    return torch.where(d == 0, 0, q), d.half(), lo.half()


def _store(pool, type_k, type_v, page, tok, k, v):
    """K and V rows [n, n_kv, 128] in 32 bits into tokens tok[n] of pages page[n]."""
    kq, kd, vq, vh, vd, vm = _views(pool, type_k, type_v)
    if type_k == F16:
        kq[page, :, tok] = k.half()
    else:
        q, d, _ = _codes(k, Q8_0)
        kq[page, :, tok], kd[page, :, tok] = q.to(torch.int8).flatten(-2), d.squeeze(-1)
    if type_v == F16:
        vq[page, :, tok] = v.half()
        return
    q, d, m = _codes(v, type_v)
    vd[page, :, tok] = d.squeeze(-1)
    if type_v == Q8_0:
        vq[page, :, tok] = q.to(torch.int8).flatten(-2)
        return
    vq[page, :, tok] = ((q[..., :16] & 15) | ((q[..., 16:] & 15) << 4)).to(torch.uint8).flatten(-2)
    if vh is not None:
        vh[page, :, tok] = ((q >> 4).long() << torch.arange(32, device=q.device)).sum(-1).to(torch.int32)
    if vm is not None:
        vm[page, :, tok] = m.squeeze(-1)


def _load(pool, type_k, type_v, page, tok):
    """K and V values in 32 bits, [..., n_kv, 128], of tokens tok of pages page."""
    kq, kd, vq, vh, vd, vm = _views(pool, type_k, type_v)
    block = lambda a: a[page, :, tok].float().unsqueeze(-1)  # noqa: E731
    k = kq[page, :, tok].float()
    if type_k != F16:
        k = (k.unflatten(-1, (NB, 32)) * block(kd)).flatten(-2)
    q = vq[page, :, tok]
    if type_v == F16:
        return k, q.float()
    if type_v == Q8_0:
        q = q.float().unflatten(-1, (NB, 32))
    else:
        q = q.unflatten(-1, (NB, 16))
        q = torch.cat([q & 15, q >> 4], -1).float()
        if vh is not None:
            q += 16.0 * ((vh[page, :, tok].unsqueeze(-1) >> torch.arange(32, device=q.device, dtype=torch.int32)) & 1)
        q -= {Q4_0: 8.0, Q5_0: 16.0}.get(type_v, 0.0)
    v = q * block(vd)
    return k, (v + block(vm) if vm is not None else v).flatten(-2)


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    new, lens = _lengths(case)
    rows, P, n_qh, n_kv = sum(new), case.get("prefix", 0), case["n_qh"], case["n_kv"]
    kinds = case["type_k"], case["type_v"]
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    need = [-(-n // T) for n in lens]
    p_pages = -(-P // T)
    order = torch.randperm(sum(need) + p_pages + 1, device="cuda", generator=g).to(torch.int32)
    table = torch.zeros(len(new), max(need), dtype=torch.int32, device="cuda")
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), torch.tensor(need, device="cuda"))
    nth = torch.cat([torch.arange(n, device="cuda") for n in need])
    table[seq, nth] = order[p_pages:p_pages + sum(need)]
    pool = torch.zeros(order.numel(), n_kv, _fields(*kinds)[1], dtype=torch.uint8, device="cuda")
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s = dict(case=case, pool=pool, table=table, start=ints(start), lens=ints(lens), rows=rows, prefix=order[:p_pages].contiguous())
    if case["op"] != "append":  # the pages hold K and V rows of N(0, 1), as the cache's own workloads do
        for a in range(0, pool.shape[0], 64):
            b = min(pool.shape[0], a + 64)
            page = torch.arange(a, b, device="cuda").repeat_interleave(T)
            tok = torch.arange(T, device="cuda").repeat(b - a)
            _store(pool, *kinds, page, tok, rand(page.numel(), n_kv, D), rand(page.numel(), n_kv, D))
    if case["op"] == "read":
        kind = KINDS.get(case["dtype"], torch.float32)
        s["k_out"], s["v_out"] = (torch.zeros(rows, n_kv, D, dtype=kind, device="cuda") for _ in range(2))
        return s
    kind = KINDS[case["dtype"]]
    if case["op"] == "append":
        if case["packed"]:  # one projection's output, split by views
            qkv = rand(rows, n_qh + 2 * n_kv, D).to(kind)
            s["q"], s["k"], s["v"] = qkv[:, :n_qh], qkv[:, n_qh:n_qh + n_kv], qkv[:, n_qh + n_kv:]
        else:
            s["q"], s["k"], s["v"] = (rand(rows, h, D).to(kind) for h in (n_qh, n_kv, n_kv))
        half = case["rot"] // 2
        s["inv_freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        s["q_out"] = torch.zeros(rows, n_qh, D, dtype=kind, device="cuda")
        if case["type_k"] != F16 or case["type_v"] != F16:
            s["k_out"], s["v_out"] = (torch.zeros(rows, n_kv, D, dtype=torch.float32, device="cuda") for _ in range(2))
        return s
    s["q"] = (2 * rand(rows, n_qh, D)).to(kind)
    s["out"] = torch.zeros_like(s["q"])
    if case.get("docs"):
        _, first, end = _intervals(case)
        s["first"], s["end"] = ints(first), ints(end)
    if case.get("alibi"):
        s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, n_qh + 1, dtype=torch.float64, device="cuda") / n_qh)).float()
    return s


# ---------------------------------------------------------------- the framework's calls

def _handles(s):
    """What a serving loop builds once from its buffers: descriptors and a workspace."""
    from host_streamed_paged_kvs_b200 import kvs
    c = s["case"]
    h = dict(kvs=kvs, pool=kvs.make_page_pool(s["pool"], c["n_kv"], c["type_k"], c["type_v"]),
             batch=kvs.make_page_batch(s["start"], s["lens"], s["table"], s["rows"], max_new=max(_lengths(c)[0])))
    if c["op"] == "append":
        h["rope"] = kvs.make_rope(s["inv_freq"], c["rot"], interleaved=c["inter"])
    if c["op"] == "attend":
        h["score"] = kvs.make_score(softcap=c.get("cap", 0.0), window=c.get("window", 0), alibi_slopes=s.get("slopes"), first_key=s.get("first"),
                                    end_key=s.get("end"))
        h["prefix"] = kvs.make_page_prefix(s["prefix"], c["prefix"]) if c.get("prefix") else None
        h["work"] = torch.zeros(kvs.kvs_attend_pages_workspace(h["batch"], c["n_qh"], c["n_kv"]), dtype=torch.uint8, device="cuda")
    return h


def _own(s):
    h = s.get("handles") or s.setdefault("handles", _handles(s))
    kvs, op, stream = h["kvs"], s["case"]["op"], torch.cuda.current_stream()
    if op == "attend":
        kvs.kvs_attend_pages(h["pool"], h["batch"], s["q"], s["out"], None, h["score"], h["prefix"], h["work"], stream)
        return s["out"]
    if op == "append":
        kvs.kvs_append_pages(h["pool"], h["batch"], s["k"], s["v"], s["q"], s["q_out"], h["rope"], stream)
        if "k_out" not in s:
            return s["q_out"], s["pool"].view(torch.float16)
    kvs.kvs_read_pages(h["pool"], h["batch"], s["k_out"], s["v_out"], stream)
    return (s["q_out"], s["k_out"], s["v_out"]) if op == "append" else (s["k_out"], s["v_out"])


# ---------------------------------------------------------------- the plain forms

def _rows(s):
    """Sequence and own position of every new token."""
    count = s["start"].diff()
    seq = torch.repeat_interleave(torch.arange(count.numel(), device="cuda"), count, output_size=s["rows"])
    t = torch.arange(s["rows"], device="cuda") - s["start"][seq]
    return seq, (s["lens"] - count)[seq] + t


def _rotate(x, pos, inv_freq, rot, inter):
    """Rows [n, heads, 128] turned by their positions, in 64 bits: the angles of far positions need them, and so do values next to a code's border."""
    a = pos.double()[:, None, None] * inv_freq.double()
    x, c, s = x.double(), a.cos(), a.sin()
    u, v = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = u * c - v * s, v * c + u * s
    return torch.cat([torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1), x[..., rot:]], -1)


def _append(s):
    c = s["case"]
    seq, pos = _rows(s)
    page, tok = s["table"][seq, pos // T].long(), pos % T
    turn = lambda x: _rotate(x, pos, s["inv_freq"], c["rot"], c["inter"])  # noqa: E731
    _store(s["pool"], c["type_k"], c["type_v"], page, tok, turn(s["k"]).float(), s["v"].float())
    s["q_out"].copy_(turn(s["q"]).to(s["q"].dtype))


def _read(s):
    c = s["case"]
    seq, pos = _rows(s)
    k, v = _load(s["pool"], c["type_k"], c["type_v"], s["table"][seq, pos // T].long(), pos % T)
    s["k_out"].copy_(k)
    s["v_out"].copy_(v)


def _attend(s):
    c = s["case"]
    n_qh, n_kv, P = c["n_qh"], c["n_kv"], c.get("prefix", 0)
    G, B, L = n_qh // n_kv, s["table"].shape[0], s["table"].shape[1] * T
    new, lens = _lengths(c)
    N = max(new)
    count = s["start"].diff()
    t = torch.arange(N, device="cuda")
    row = (s["start"][:-1, None] + t).clamp(max=s["rows"] - 1).long()                       # [B, N], padded
    q = s["q"][row].float().view(B, N, n_kv, G, D).permute(0, 2, 1, 3, 4)                    # [B, kv, N, G, D]
    at = torch.arange(L, device="cuda")
    k, v = _load(s["pool"], c["type_k"], c["type_v"], s["table"][:, at // T].long(), (at % T).expand(B, L))  # [B, L, kv, D]
    k, v = k.transpose(1, 2), v.transpose(1, 2)
    q = q.reshape(B, n_kv, N * G, D)
    x = q @ k.transpose(-1, -2)
    if P:
        at = torch.arange(P, device="cuda")
        pk, pv = (a.transpose(0, 1) for a in _load(s["pool"], c["type_k"], c["type_v"], s["prefix"][at // T].long(), at % T))
        flat = q.transpose(0, 1).reshape(n_kv, -1, D)
        x = torch.cat([(flat @ pk.transpose(-1, -2)).view(n_kv, B, N * G, P).transpose(0, 1), x], -1)
    x = x.view(B, n_kv, N, G, P + L) / math.sqrt(D)
    if c.get("cap"):
        x = c["cap"] * torch.tanh(x / c["cap"])
    key = torch.arange(P + L, device="cuda")
    pos = P + (s["lens"] - count)[:, None] + t                                               # [B, N]
    if "slopes" in s:
        x = x - s["slopes"].view(n_kv, 1, G, 1) * (pos[..., None] - key).abs()[:, None, :, None]
    first = s["first"][row] if "first" in s else (pos + 1 - c["window"] if c.get("window") else torch.zeros_like(pos))
    end = s["end"][row] if "end" in s else pos + 1
    seen = (key >= first[..., None]) & (key < torch.minimum(end, P + s["lens"][:, None])[..., None])
    x = x.masked_fill(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = p.sum(-1, keepdim=True)
    p = p.view(B, n_kv, N * G, P + L)
    o = p[..., P:] @ v
    if P:
        o = o + (p[..., :P].transpose(0, 1).reshape(n_kv, -1, P) @ pv).view(n_kv, B, N * G, D).transpose(0, 1)
    o = o.view(B, n_kv, N, G, D) / torch.where(total == 0, torch.ones_like(total), total)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, N, n_qh, D)
    s["out"].copy_(o[t < count[:, None]])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "attend":
        _attend(state)
        return state["out"]
    if op == "append":
        _append(state)
        if "k_out" not in state:
            return state["q_out"], state["pool"].view(torch.float16)
    _read(state)
    return (state["q_out"], state["k_out"], state["v_out"]) if op == "append" else (state["k_out"], state["v_out"])


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    new, lens = _lengths(case)
    n_qh, n_kv, rows, P = case["n_qh"], case["n_kv"], sum(new), case.get("prefix", 0)
    token = sum(f[0] for f in _fields(case["type_k"], case["type_v"])[0]) * n_kv
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "read":
        return {"bytes": rows * (token + 2 * n_kv * D * size), "flops": rows * 4 * n_kv * D}
    if case["op"] == "append":
        values = rows * (n_qh + 2 * n_kv) * D
        back = 0 if case["type_k"] == F16 and case["type_v"] == F16 else rows * (token + 2 * n_kv * D * 4)
        return {"bytes": values * size + rows * (n_qh * D * size + token) + back, "flops": 6 * values}
    pos, first, end = _intervals(case)
    keys = max(0, P - min(first)) if P else 0
    at, pairs = 0, sum(max(0, e - f) for f, e in zip(first, end))
    for n, length in zip(new, lens):
        keys += P + length - max(P, min(first[at:at + n]))
        at += n
    return {"bytes": keys * token + 2 * rows * n_qh * D * size, "flops": 4 * D * n_qh * pairs}


# ---------------------------------------------------------------- 64 bits

def _exact_values(raw, kind, codes_at, scales_at, fifth_at, least_at, tok):
    """Values in 64 bits of tokens tok [n] from page heads raw [n, bytes], byte by byte."""
    n = raw.shape[0]
    pick = lambda at, size: raw.gather(1, at + size * tok[:, None] + torch.arange(size, device=raw.device))  # noqa: E731
    halves = lambda at, size: pick(at, size).contiguous().view(torch.float16).double()  # noqa: E731
    if kind == F16:
        return halves(codes_at, 256)
    d = halves(scales_at, 8)
    if kind == Q8_0:
        return (pick(codes_at, 128).view(torch.int8).double().view(n, 4, 32) * d[..., None]).view(n, 128)
    low = pick(codes_at, 64).long().view(n, 4, 16)
    code = torch.empty(n, 4, 32, dtype=torch.int64, device=raw.device)
    code[..., :16], code[..., 16:] = low % 16, low // 16
    if fifth_at is not None:
        bits = pick(fifth_at, 16).long().view(n, 4, 4)
        code += 16 * ((bits[..., None] // (2 ** torch.arange(8, device=raw.device))) % 2).view(n, 4, 32)
    zero = {Q4_0: 8, Q5_0: 16}.get(kind, 0)
    value = (code - zero).double() * d[..., None]
    if least_at is not None:
        value = value + halves(least_at, 8)[..., None]
    return value.view(n, 128)


def _exact_kv(pool, kinds, page, tok, head):
    f, _ = _fields(*kinds)
    raw = pool[page.long(), head]
    k = _exact_values(raw, kinds[0], f[0][1], f[1][1], None, None, tok)
    v = _exact_values(raw, kinds[1], f[2][1], f[4][1], f[3][1] if f[3][0] else None, f[5][1] if f[5][0] else None, tok)
    return k, v


def _exact_quantized(x, kind):
    """The values that 64-bit rows [..., 128] stand for once stored: code decisions in 32 bits, scales in 16, as the formats define."""
    x = x.float()
    if kind == F16:
        return x.half().double()
    b = x.view(*x.shape[:-1], 4, 32)
    div = lambda p, q: torch.div(p, q.expand_as(p).contiguous())  # noqa: E731
    big = b.abs().max(-1, keepdim=True).values
    if kind == Q8_0:
        d = div(big, torch.tensor([127.0], device=x.device))
        r = div(b, d).nan_to_num(0.0, 0.0, 0.0).double()
        code = torch.trunc(r + 0.5 * torch.sign(r))
        return (code * d.half().double()).view(x.shape)
    if kind in (Q4_0, Q5_0):
        z = {Q4_0: 8, Q5_0: 16}[kind]
        ranks = torch.arange(32, device=x.device).expand_as(b)
        at = torch.where(b.abs() == big, ranks, 32).min(-1, keepdim=True).values
        d = div(b.gather(-1, at), torch.tensor([-float(z)], device=x.device))
        code = torch.minimum(torch.trunc(div(b, d) + (z + 0.5)), torch.tensor(2.0 * z - 1, device=x.device))
        return torch.where(d == 0, 0.0, (code - z).double() * d.half().double()).view(x.shape)
    top = {Q4_1: 15.0, Q5_1: 31.0}[kind]
    lo = b.min(-1, keepdim=True).values
    d = div(b.max(-1, keepdim=True).values - lo, torch.tensor([top], device=x.device))
    code = torch.minimum(torch.trunc(div(b - lo, d) + 0.5), torch.tensor(top, device=x.device))
    return (torch.where(d == 0, 0.0, code.double() * d.half().double()) + lo.half().double()).view(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    new, lens = _lengths(case)
    kinds, n_qh, n_kv, P = (case["type_k"], case["type_v"]), case["n_qh"], case["n_kv"], case.get("prefix", 0)
    G = n_qh // n_kv
    if case["op"] == "append":
        pos = torch.cat([torch.arange(b - n, b, device="cuda") for n, b in zip(new, lens)]).double()
        z = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), pos[:, None] * s["inv_freq"].double())[:, None]

        def turned(x):
            x = x.double()
            pair = x[..., :case["rot"]]
            pair = pair.unflatten(-1, (-1, 2)) if case["inter"] else pair.unflatten(-1, (2, -1)).transpose(-1, -2)
            w = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * z)
            return torch.cat([(w if case["inter"] else w.transpose(-1, -2)).flatten(-2), x[..., case["rot"]:]], -1)
        k, v = _exact_quantized(turned(s["k"]), kinds[0]), _exact_quantized(s["v"].double(), kinds[1])
        if "k_out" in s:
            return turned(s["q"]), k, v
        pool = torch.zeros(s["pool"].shape[0], n_kv, 2, T, D, dtype=torch.float64, device="cuda")
        row = 0
        for i, (n, b) in enumerate(zip(new, lens)):
            for p in range(b - n, b):
                at = int(s["table"][i, p // T]), slice(None)
                pool[at[0], :, 0, p % T], pool[at[0], :, 1, p % T] = k[row], v[row]
                row += 1
        return turned(s["q"]), pool.view(pool.shape[0], n_kv, -1)
    if case["op"] == "read":
        k, v = (torch.empty(s["rows"], n_kv, D, dtype=torch.float64, device="cuda") for _ in range(2))
        row = 0
        for i, (n, b) in enumerate(zip(new, lens)):
            for a in range(b - n, b, 4096):
                at = torch.arange(a, min(b, a + 4096), device="cuda")
                for h in range(n_kv):
                    k[row:row + at.numel(), h], v[row:row + at.numel(), h] = _exact_kv(s["pool"], kinds, s["table"][i, at // T], at % T, h)
                row += at.numel()
        return k, v
    pos, first, end = (torch.tensor(a, device="cuda") for a in _intervals(case))
    out = torch.zeros(s["rows"], n_qh, D, dtype=torch.float64, device="cuda")

    def values(table, length, h):
        parts = []
        for a in range(0, length, 8192):
            at = torch.arange(a, min(length, a + 8192), device="cuda")
            parts.append(_exact_kv(s["pool"], kinds, table[at // T], at % T, h))
        return [torch.cat(x) for x in zip(*parts)] if parts else [torch.zeros(0, D, dtype=torch.float64, device="cuda")] * 2
    for h in range(n_kv):
        shared = values(s["prefix"], P, h)
        row = 0
        for i, (n, length) in enumerate(zip(new, lens)):
            k, v = (torch.cat(x) for x in zip(shared, values(s["table"][i], length, h)))
            key = torch.arange(P + length, device="cuda")
            at = slice(row, row + n)
            hide = (key < first[at, None]) | (key >= end[at, None])
            for g in range(G):
                x = s["q"][at, h * G + g].double() @ k.T * D ** -0.5
                if case.get("cap"):
                    x = torch.tanh(x / case["cap"]) * case["cap"]
                if "slopes" in s:
                    x -= s["slopes"][h * G + g].double() * (pos[at, None] - key).abs()
                x[hide] = -math.inf
                out[at, h * G + g] = torch.softmax(x, -1) @ v
            row += n
    return out
