"""Thin Python binding of libkvs (include/kvs.h).

Argument marshalling only: every step of the path runs in the CUDA library.
Tensors are passed by address (torch CUDA tensors, pinned or plain CPU tensors,
numpy arrays); streams by their cudaStream_t handle.  There is no fallback:
importing this module fails loudly if libkvs.so has not been built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvs.so")

KVS_OK = 0
KVS_E_INVAL = -1
KVS_E_ARENA = -2
KVS_E_WIDTH = -3
KVS_E_ORDER = -4
KVS_E_CUDA = -5
KVS_E_TIMEOUT = -6
KVS_E_NOMEM = -7
KVS_TYPE_F16 = 1
KVS_TYPE_Q4_0 = 2
KVS_TYPE_Q4_1 = 3
KVS_TYPE_Q5_0 = 6
KVS_TYPE_Q5_1 = 7
KVS_TYPE_Q8_0 = 8
KVS_PAGE_ABSENT = -1
KVS_PAGE_RESIDENT = 1
KVS_PAGE_STREAMED = 2
KVS_FLAG_PROFILE = 1
KVS_FLAG_PHASE_ARENA = 2
KVS_PHASE_PREFILL = 0
KVS_PHASE_DECODE = 1
KVS_DT_F16 = 0
KVS_DT_BF16 = 1
KVS_DT_F32 = 2

ERROR_NAMES = {0: "KVS_OK", -1: "KVS_E_INVAL", -2: "KVS_E_ARENA", -3: "KVS_E_WIDTH",
               -4: "KVS_E_ORDER", -5: "KVS_E_CUDA", -6: "KVS_E_TIMEOUT", -7: "KVS_E_NOMEM"}

# every symbol the header declares
EXPORTS = ["kvs_resolve_config", "kvs_page_bytes", "kvs_plan_page", "kvs_plan_ring", "kvs_create", "kvs_destroy",
           "kvs_append", "kvs_attend", "kvs_export_page", "kvs_page_location", "kvs_layer_length",
           "kvs_get_config", "kvs_get_stats", "kvs_reset_stats", "kvs_set_profiling",
           "kvs_set_zero_copy_pct", "kvs_sync",
           "kvs_measure_h2d", "kvs_attend_pages_static", "kvs_selftest_bounded_wait",
           "kvs_last_error", "kvs_eject_init", "kvs_eject_step", "kvs_draft_capacity_pages",
           "kvs_phase_layout", "kvs_set_phase", "kvs_pin", "kvs_draft_eject", "kvs_draft_restore",
           "kvs_get_arena", "kvs_append_pages", "kvs_read_pages", "kvs_attend_pages", "kvs_attend_pages_workspace"]


class kvs_config(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int), ("n_q_heads", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("max_ctx", ctypes.c_int),
                ("n_resident_pages", ctypes.c_int), ("n_ring_slots", ctypes.c_int),
                ("max_q_tokens", ctypes.c_int), ("type_k", ctypes.c_int),
                ("type_v", ctypes.c_int), ("chunk_pages", ctypes.c_int),
                ("flags", ctypes.c_int), ("zero_copy_pct", ctypes.c_int),
                ("arena_bytes", ctypes.c_size_t), ("n_aux_layers", ctypes.c_int),
                ("aux_resident_pages", ctypes.c_int), ("zero_copy_pct_wide", ctypes.c_int)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class kvs_arena_status(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int) for n in ("phase", "width", "n_resident_pages", "aux_resident_pages",
                                             "draft_active", "phase_arena")] +
                [(n, ctypes.c_size_t) for n in ("arena_bytes", "compute_bytes", "resident_bytes", "ring_bytes",
                                                "aux_bytes", "pinned_bytes", "free_bytes")])

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class kvs_stats(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_uint64) for n in
                 ("appends", "attends", "tokens_appended", "pages_streamed", "bytes_h2d",
                  "bytes_resident_read", "h2d_copies", "kernel_launches")] +
                [(n, ctypes.c_double) for n in
                 ("ms_decode_resident", "ms_decode_ring", "ms_merge", "ms_append", "ms_chunk_mma",
                  "ms_decode_zc")] +
                [(n, ctypes.c_uint64) for n in
                 ("n_decode_resident", "n_decode_ring", "n_merge", "n_append", "n_chunk_mma",
                  "n_decode_zc", "bytes_decode_resident", "bytes_decode_ring", "bytes_decode_zc")] +
                [("ms_chunk_zc", ctypes.c_double), ("n_chunk_zc", ctypes.c_uint64),
                 ("bytes_chunk_zc", ctypes.c_uint64)])

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class kvs_eject_params(ctypes.Structure):
    _fields_ = [("keep_pages", ctypes.c_int), ("reenable_pages", ctypes.c_int),
                ("stable_decodes", ctypes.c_int), ("capacity_pages", ctypes.c_int)]


class kvs_eject_state(ctypes.Structure):
    _fields_ = [("draft_active", ctypes.c_int), ("streak", ctypes.c_int)]


class kvs_page_pool(ctypes.Structure):
    device = None  # of its tensors, where make_* made it
    _fields_ = [("pages", ctypes.c_void_p), ("n_pages", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("type_k", ctypes.c_int), ("type_v", ctypes.c_int)]


class kvs_page_batch(ctypes.Structure):
    device = None  # of its tensors, where make_* made it
    _fields_ = [("n_seqs", ctypes.c_int), ("n_rows", ctypes.c_int), ("max_new", ctypes.c_int),
                ("q_start", ctypes.c_void_p), ("seq_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int), ("status", ctypes.c_void_p)]


class kvs_page_rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_longlong), ("head_stride", ctypes.c_longlong)]


class kvs_rope(ctypes.Structure):
    device = None  # of its tensors, where make_* made it
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int),
                ("positions", ctypes.c_void_p), ("pos_offset", ctypes.c_int), ("mscale", ctypes.c_float)]


class kvs_score(ctypes.Structure):
    device = None  # of its tensors, where make_* made it
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int),
                ("alibi_slopes", ctypes.c_void_p), ("first_key", ctypes.c_void_p), ("end_key", ctypes.c_void_p)]


class kvs_page_prefix(ctypes.Structure):
    device = None  # of its tensors, where make_* made it
    _fields_ = [("page_table", ctypes.c_void_p), ("n_tokens", ctypes.c_int)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libkvs.so not found at {LIB_PATH}: build it with "
            "`python -m host_streamed_paged_kvs_b200.build` (there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i, cp = ctypes.c_void_p, ctypes.c_int, ctypes.POINTER
    L.kvs_resolve_config.argtypes = [cp(kvs_config), cp(kvs_config), cp(ctypes.c_size_t)]
    L.kvs_page_bytes.restype = ctypes.c_size_t
    L.kvs_page_bytes.argtypes = [cp(kvs_config)]
    L.kvs_plan_page.argtypes = [cp(kvs_config), i, i, cp(i), cp(i)]
    L.kvs_plan_ring.argtypes = [cp(kvs_config), i, i, ctypes.c_longlong, cp(i), cp(i), cp(i), i]
    L.kvs_create.argtypes = [cp(kvs_config), i, cp(vp)]
    L.kvs_destroy.argtypes = [vp]
    L.kvs_destroy.restype = None
    L.kvs_append.argtypes = [vp, i, i, i, vp, vp, vp]
    L.kvs_attend.argtypes = [vp, i, i, i, vp, vp, vp, vp]
    L.kvs_export_page.argtypes = [vp, i, i, i, vp]
    L.kvs_page_location.argtypes = [vp, i, i, cp(i), cp(i)]
    L.kvs_layer_length.argtypes = [vp, i, cp(i)]
    L.kvs_get_config.argtypes = [vp, cp(kvs_config)]
    L.kvs_get_stats.argtypes = [vp, cp(kvs_stats)]
    L.kvs_reset_stats.argtypes = [vp]
    L.kvs_set_profiling.argtypes = [vp, i]
    L.kvs_set_zero_copy_pct.argtypes = [vp, i, i]
    L.kvs_sync.argtypes = [vp, vp, ctypes.c_double]
    L.kvs_measure_h2d.argtypes = [vp, ctypes.c_size_t, ctypes.c_size_t, i, cp(ctypes.c_double)]
    L.kvs_attend_pages_static.argtypes = [vp, i, i, i, i, i, i, vp, vp, vp, vp]
    L.kvs_selftest_bounded_wait.argtypes = [i, ctypes.c_double, cp(i)]
    L.kvs_last_error.restype = ctypes.c_char_p
    L.kvs_last_error.argtypes = [vp]
    L.kvs_eject_init.argtypes = [cp(kvs_eject_params), cp(kvs_eject_state)]
    L.kvs_eject_step.argtypes = [cp(kvs_eject_params), cp(kvs_eject_state), i]
    L.kvs_draft_capacity_pages.argtypes = [cp(kvs_config), ctypes.c_size_t, cp(i)]
    L.kvs_phase_layout.argtypes = [cp(kvs_config), i, ctypes.c_size_t, i, cp(kvs_arena_status)]
    L.kvs_set_phase.argtypes = [vp, i, i, vp]
    L.kvs_pin.argtypes = [vp, ctypes.c_size_t, cp(vp), vp]
    L.kvs_draft_eject.argtypes = [vp, vp]
    L.kvs_draft_restore.argtypes = [vp, vp]
    L.kvs_get_arena.argtypes = [vp, cp(kvs_arena_status)]
    pool, batch, rows = cp(kvs_page_pool), cp(kvs_page_batch), cp(kvs_page_rows)
    L.kvs_append_pages.argtypes = [pool, batch, i, rows, rows, i, rows, rows, cp(kvs_rope), vp]
    L.kvs_read_pages.argtypes = [pool, batch, i, rows, rows, vp]
    L.kvs_attend_pages.argtypes = [pool, batch, i, i, rows, i, rows, vp, cp(kvs_score), cp(kvs_page_prefix), vp,
                                   ctypes.c_size_t, vp]
    L.kvs_attend_pages_workspace.argtypes = [batch, i, i]
    L.kvs_attend_pages_workspace.restype = ctypes.c_size_t
    return L


lib = _load()


class KvsError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


def _addr(x) -> Optional[int]:
    """Address of a tensor / array / raw int (None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)}")


def _stream(s) -> Optional[int]:
    if s is None:
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream  # torch.cuda.Stream


def _check(rc: int, handle=None):
    if rc != KVS_OK:
        raise KvsError(rc, lib.kvs_last_error(handle).decode())


def make_config(n_layers, n_q_heads, n_kv_heads, max_ctx, n_resident_pages=0, n_ring_slots=0,
                max_q_tokens=1, chunk_pages=0, flags=0, arena_bytes=0, head_dim=128,
                page_tokens=256, type_k=KVS_TYPE_Q8_0, type_v=KVS_TYPE_Q4_0,
                zero_copy_pct=0, n_aux_layers=0, aux_resident_pages=0,
                zero_copy_pct_wide=0) -> kvs_config:
    return kvs_config(n_layers, n_q_heads, n_kv_heads, head_dim, page_tokens, max_ctx,
                      n_resident_pages, n_ring_slots, max_q_tokens, type_k, type_v, chunk_pages,
                      flags, zero_copy_pct, arena_bytes, n_aux_layers, aux_resident_pages,
                      zero_copy_pct_wide)


# ---- functions with the C names ------------------------------------------

def kvs_resolve_config(cfg: kvs_config):
    out = kvs_config()
    hb = ctypes.c_size_t()
    _check(lib.kvs_resolve_config(ctypes.byref(cfg), ctypes.byref(out), ctypes.byref(hb)))
    return out, hb.value


def kvs_page_bytes(cfg: kvs_config) -> int:
    return lib.kvs_page_bytes(ctypes.byref(cfg))


def kvs_plan_page(cfg: kvs_config, n_tokens: int, page: int):
    k, i = ctypes.c_int(), ctypes.c_int()
    _check(lib.kvs_plan_page(ctypes.byref(cfg), n_tokens, page, ctypes.byref(k), ctypes.byref(i)))
    return k.value, i.value


def kvs_plan_ring(cfg: kvs_config, n_q: int, s_ring: int, ring_ctr0: int = 0):
    """The ring schedule of one attend call: [(page0, pages, slot0), ...]."""
    n = lib.kvs_plan_ring(ctypes.byref(cfg), n_q, s_ring, ring_ctr0, None, None, None, 0)
    _check(n if n < 0 else 0)
    p0, pg, sl = (ctypes.c_int * max(1, n))(), (ctypes.c_int * max(1, n))(), (ctypes.c_int * max(1, n))()
    _check(min(0, lib.kvs_plan_ring(ctypes.byref(cfg), n_q, s_ring, ring_ctr0, p0, pg, sl, n)))
    return [(p0[k], pg[k], sl[k]) for k in range(n)]


def kvs_create(cfg: kvs_config, device: int = 0) -> int:
    h = ctypes.c_void_p()
    _check(lib.kvs_create(ctypes.byref(cfg), device, ctypes.byref(h)))
    return h.value


def kvs_destroy(h: int) -> None:
    lib.kvs_destroy(h)


def kvs_append(h, layer, pos0, n_tok, k, v, stream=None) -> None:
    _check(lib.kvs_append(h, layer, pos0, n_tok, _addr(k), _addr(v), _stream(stream)), h)


def kvs_attend(h, layer, pos0, n_q, q, out, lse=None, stream=None) -> None:
    _check(lib.kvs_attend(h, layer, pos0, n_q, _addr(q), _addr(out), _addr(lse), _stream(stream)), h)


def kvs_export_page(h, layer, page, from_device, dst) -> None:
    _check(lib.kvs_export_page(h, layer, page, int(from_device), _addr(dst)), h)


def kvs_page_location(h, layer, page):
    k, i = ctypes.c_int(), ctypes.c_int()
    _check(lib.kvs_page_location(h, layer, page, ctypes.byref(k), ctypes.byref(i)), h)
    return k.value, i.value


def kvs_layer_length(h, layer) -> int:
    n = ctypes.c_int()
    _check(lib.kvs_layer_length(h, layer, ctypes.byref(n)), h)
    return n.value


def kvs_get_config(h) -> kvs_config:
    c = kvs_config()
    _check(lib.kvs_get_config(h, ctypes.byref(c)), h)
    return c


def kvs_get_stats(h) -> dict:
    s = kvs_stats()
    _check(lib.kvs_get_stats(h, ctypes.byref(s)), h)
    return s.as_dict()


def kvs_reset_stats(h) -> None:
    _check(lib.kvs_reset_stats(h), h)


def kvs_set_profiling(h, enable: bool) -> None:
    _check(lib.kvs_set_profiling(h, int(bool(enable))), h)


def kvs_set_zero_copy_pct(h, pct: int = -1, pct_wide: int = -1) -> None:
    """In-place shares for decode calls and wider calls; -1 leaves one unchanged."""
    _check(lib.kvs_set_zero_copy_pct(h, int(pct), int(pct_wide)), h)


def kvs_phase_layout(cfg: kvs_config, width: int, pinned_bytes: int = 0, draft_active: bool = True) -> dict:
    st = kvs_arena_status()
    _check(lib.kvs_phase_layout(ctypes.byref(cfg), int(width), int(pinned_bytes), int(bool(draft_active)),
                                ctypes.byref(st)))
    return st.as_dict()


def kvs_set_phase(h, phase: int, width: int = 0, stream=None) -> None:
    _check(lib.kvs_set_phase(h, int(phase), int(width), _stream(stream)), h)


def kvs_pin(h, nbytes: int, stream=None) -> int:
    p = ctypes.c_void_p()
    _check(lib.kvs_pin(h, int(nbytes), ctypes.byref(p), _stream(stream)), h)
    return p.value


def kvs_draft_eject(h, stream=None) -> None:
    _check(lib.kvs_draft_eject(h, _stream(stream)), h)


def kvs_draft_restore(h, stream=None) -> None:
    _check(lib.kvs_draft_restore(h, _stream(stream)), h)


def kvs_get_arena(h) -> dict:
    st = kvs_arena_status()
    _check(lib.kvs_get_arena(h, ctypes.byref(st)), h)
    return st.as_dict()


def kvs_sync(h, stream=None, timeout_s: float = 60.0) -> None:
    _check(lib.kvs_sync(h, _stream(stream), timeout_s), h)


def kvs_measure_h2d(h, chunk_bytes: int, total_bytes: int, reps: int = 10) -> float:
    g = ctypes.c_double()
    _check(lib.kvs_measure_h2d(h, chunk_bytes, total_bytes, reps, ctypes.byref(g)), h)
    return g.value


def kvs_attend_pages_static(pages, n_pages, n_tokens, n_q_heads, n_kv_heads, pos0, n_q, q, out,
                            lse=None, stream=None) -> None:
    """No-allocation attention over caller-owned device pages (see include/kvs.h)."""
    _check(lib.kvs_attend_pages_static(_addr(pages), n_pages, n_tokens, n_q_heads, n_kv_heads, pos0,
                                       n_q, _addr(q), _addr(out), _addr(lse), _stream(stream)))


KVS_ERR_WAIT_TIMEOUT = 1
KVS_ERR_BAD_PAGE = 2


# ---- batches over caller-owned pages (include/kvs.h) ----------------------
# The make_* functions describe buffers once; the descriptors keep the tensors
# alive and can be used for any number of calls, captured ones too.

_DTYPE_NAMES = {"torch.float16": KVS_DT_F16, "torch.bfloat16": KVS_DT_BF16, "torch.float32": KVS_DT_F32}
_dtype_codes = {}  # dtype objects seen, by identity of the type itself


def _dtype(x) -> Optional[int]:
    try:
        return _dtype_codes[x.dtype]
    except KeyError:
        return _dtype_codes.setdefault(x.dtype, _DTYPE_NAMES.get(str(x.dtype)))


def _bad(msg: str):
    raise KvsError(KVS_E_INVAL, msg)


def _int32(x, what: str, least: int = 0) -> Optional[int]:
    """Address of a contiguous int32 device tensor of at least `least` values (None -> NULL)."""
    if x is None:
        return None
    if str(x.dtype) != "torch.int32" or not x.is_contiguous() or x.numel() < least or not x.is_cuda:
        _bad(f"{what}: a contiguous int32 device tensor of at least {least} values is wanted")
    return x.data_ptr()


def _float32(x, what: str, least: int) -> Optional[int]:
    if x is None:
        return None
    if str(x.dtype) != "torch.float32" or not x.is_contiguous() or x.numel() < least or not x.is_cuda:
        _bad(f"{what}: a contiguous float32 device tensor of at least {least} values is wanted")
    return x.data_ptr()


def _device(what: str, *tensors) -> Optional[int]:
    """The one device of the tensors given (None: none is)."""
    at = {x.get_device() for x in tensors if x is not None}
    if len(at) > 1:
        _bad(f"{what}: tensors of one device are wanted")
    return at.pop() if at else None


def _beside(pool, d) -> None:
    """Refuses a descriptor whose tensors are not on the pool's device (structs filled from
    addresses have none)."""
    if None not in (pool.device, d.device):
        _bad(f"{type(d).__name__}: its tensors must be on the pool's device")


def make_page_pool(pages, n_kv_heads: int, type_k: int = KVS_TYPE_Q8_0, type_v: int = KVS_TYPE_Q4_0) -> kvs_page_pool:
    """A pool of pages: a contiguous uint8 device tensor of whole pages."""
    head = kvs_page_bytes(make_config(1, n_kv_heads, n_kv_heads, 256, 1, type_k=type_k, type_v=type_v))
    if not head:
        _bad("unsupported K/V type pair or heads")
    if not pages.is_contiguous() or not pages.is_cuda or pages.element_size() != 1 or pages.numel() % head or not pages.numel():
        _bad(f"pages: a contiguous uint8 device tensor of whole pages of {head} bytes is wanted")
    p = kvs_page_pool(pages.data_ptr(), pages.numel() // head, n_kv_heads, type_k, type_v)
    p.keep = pages
    p.device = pages.get_device()
    return p


def make_page_batch(q_start, seq_len, page_table, n_rows: int, max_new: int = 0, status=None) -> kvs_page_batch:
    """q_start int32 [n_seqs + 1], seq_len int32 [n_seqs], page_table int32 [n_seqs, entries], all on the device."""
    n = seq_len.numel()
    if page_table.dim() != 2 or page_table.shape[0] != n:
        _bad("page_table: [n_seqs, entries] is wanted")
    b = kvs_page_batch(n, n_rows, max_new, _int32(q_start, "q_start", n + 1), _int32(seq_len, "seq_len"),
                       _int32(page_table, "page_table"), page_table.shape[1], _int32(status, "status", 1))
    b.keep = (q_start, seq_len, page_table, status)
    b.device = _device("page batch", *b.keep)
    return b


def make_rope(inv_freq, rot_dim: int = 128, interleaved: bool = False, positions=None, pos_offset: int = 0,
              mscale: float = 1.0) -> kvs_rope:
    """inv_freq float32 [rot_dim / 2]; positions int32 [n_rows] or None (own position + pos_offset)."""
    r = kvs_rope(_float32(inv_freq, "inv_freq", rot_dim // 2), rot_dim, int(interleaved), _int32(positions, "positions"),
                 pos_offset, mscale)
    r.keep = (inv_freq, positions)
    r.device = _device("rope", *r.keep)
    return r


def make_score(scale: float = 0.0, softcap: float = 0.0, window: int = 0, alibi_slopes=None, first_key=None,
               end_key=None) -> kvs_score:
    """alibi_slopes float32 [n_q_heads]; first_key, end_key int32 [n_rows]."""
    s = kvs_score(scale, softcap, window, _float32(alibi_slopes, "alibi_slopes", 1), _int32(first_key, "first_key"),
                  _int32(end_key, "end_key"))
    s.keep = (alibi_slopes, first_key, end_key)
    s.device = _device("score", *s.keep)
    return s


def make_page_prefix(page_table, n_tokens: int) -> kvs_page_prefix:
    """page_table int32 [pages of n_tokens]."""
    p = kvs_page_prefix(_int32(page_table, "prefix page_table", -(-n_tokens // 256)), n_tokens)
    p.keep = page_table
    p.device = _device("page prefix", page_table)
    return p


def _rows(x, batch, heads: int, what: str, at: Optional[int]):
    """(descriptor, dtype code) of a [rows, heads, 128] tensor on device `at`, strides as they are."""
    dt = _dtype(x)
    shape, stride, on = x.shape, x.stride(), x.get_device()
    if dt is None or len(shape) != 3 or shape[0] < batch.n_rows or shape[1] != heads or shape[2] != 128 or \
            stride[2] != 1 or on < 0 or (on != at and at is not None):
        _bad(f"{what}: a float16, bfloat16 or float32 tensor [rows >= {batch.n_rows}, {heads}, 128] with "
             "contiguous heads on the pool's device is wanted")
    return kvs_page_rows(x.data_ptr(), stride[0], stride[1]), dt


def _same(a: int, b: int, what: str) -> int:
    if a != b:
        _bad(f"{what} must have the same dtype")
    return a


def kvs_append_pages(pool, batch, k, v, q=None, q_out=None, rope=None, stream=None) -> None:
    """Rotate K (and Q into q_out), quantize K and V and write them to the batch's pages."""
    at = pool.device
    if batch.device != at:
        _beside(pool, batch)
    if rope is not None and rope.device != at:
        _beside(pool, rope)
    kr, dt = _rows(k, batch, pool.n_kv_heads, "k", at)
    vr, dv = _rows(v, batch, pool.n_kv_heads, "v", at)
    _same(dt, dv, "k and v")
    qr = qo = None
    heads = 0
    if q is not None or q_out is not None:
        if q is None or q_out is None or q.dim() != 3:
            _bad("q and q_out go together, [rows, heads, 128]")
        heads = q.shape[1]
        (qr, d0), (qo, d1) = _rows(q, batch, heads, "q", at), _rows(q_out, batch, heads, "q_out", at)
        _same(_same(dt, d0, "k and q"), d1, "k and q_out")
    if rope is not None and rope.keep[1] is not None and rope.keep[1].numel() < batch.n_rows:
        _bad("positions: one per row is wanted")
    _check(lib.kvs_append_pages(pool, batch, dt, kr, vr, heads, qr, qo, rope, _stream(stream)))


def kvs_read_pages(pool, batch, k=None, v=None, stream=None) -> None:
    """Write the values of the batch's rows, read from its pages, to k and / or v."""
    at = pool.device
    if batch.device != at:
        _beside(pool, batch)
    kr, dk = _rows(k, batch, pool.n_kv_heads, "k", at) if k is not None else (None, None)
    vr, dv = _rows(v, batch, pool.n_kv_heads, "v", at) if v is not None else (None, None)
    if dk is None and dv is None:
        _bad("neither k nor v is wanted")
    dt = _same(dk, dv, "k and v") if dk is not None and dv is not None else (dk if dv is None else dv)
    _check(lib.kvs_read_pages(pool, batch, dt, kr, vr, _stream(stream)))


def kvs_attend_pages_workspace(batch, n_q_heads: int, n_kv_heads: int) -> int:
    """Bytes of workspace (a zero-filled device buffer) for calls up to this batch's size."""
    n = lib.kvs_attend_pages_workspace(batch, n_q_heads, n_kv_heads)
    if not n:
        _bad(kvs_last_error())
    return n


def kvs_attend_pages(pool, batch, q, out, lse=None, score=None, prefix=None, workspace=None, stream=None) -> None:
    """Attention of the batch's rows over their pages (after a shared prefix); see include/kvs.h."""
    if q.dim() != 3:
        _bad("q: [rows, heads, 128] is wanted")
    heads = q.shape[1]
    at = pool.device
    for d in (batch, score, prefix):
        if d is not None and d.device != at:
            _beside(pool, d)
    (qr, dq), (orow, do) = _rows(q, batch, heads, "q", at), _rows(out, batch, heads, "out", at)
    qat = q.get_device()  # the pool's, where that is known
    if workspace is None or workspace.get_device() != qat or not workspace.is_contiguous():
        _bad("a workspace is wanted (kvs_attend_pages_workspace bytes, zero-filled, contiguous, on the pool's device)")
    if lse is not None and (_dtype(lse) != KVS_DT_F32 or not lse.is_contiguous() or lse.numel() < batch.n_rows * heads or
                            lse.get_device() != qat):
        _bad("lse: a contiguous float32 tensor [n_rows, heads] on the pool's device is wanted")
    if score is not None:
        slopes, first, end = score.keep
        if (slopes is not None and slopes.numel() < heads) or any(x is not None and x.numel() < batch.n_rows
                                                                  for x in (first, end)):
            _bad("score: alibi_slopes has one value a head, first_key and end_key one a row")
    _check(lib.kvs_attend_pages(pool, batch, dq, heads, qr, do, orow, _addr(lse), score, prefix, workspace.data_ptr(),
                                workspace.numel() * workspace.element_size(), _stream(stream)))


def kvs_selftest_bounded_wait(device: int = 0, limit_s: float = 0.2) -> int:
    bits = ctypes.c_int()
    _check(lib.kvs_selftest_bounded_wait(device, limit_s, ctypes.byref(bits)))
    return bits.value


def kvs_last_error(h=None) -> str:
    return lib.kvs_last_error(h).decode()


def kvs_eject_init(keep_pages=0, reenable_pages=0, stable_decodes=0, capacity_pages=0):
    """Returns (params with defaults filled, state with the draft active)."""
    p = kvs_eject_params(keep_pages, reenable_pages, stable_decodes, capacity_pages)
    s = kvs_eject_state()
    _check(lib.kvs_eject_init(ctypes.byref(p), ctypes.byref(s)))
    return p, s


def kvs_eject_step(params: kvs_eject_params, state: kvs_eject_state, working_pages: int) -> bool:
    """One decode batch; True when the draft was ejected or re-enabled."""
    rc = lib.kvs_eject_step(ctypes.byref(params), ctypes.byref(state), int(working_pages))
    _check(rc if rc < 0 else 0)
    return rc == 1


def kvs_draft_capacity_pages(cfg: kvs_config, pinned_bytes: int) -> int:
    n = ctypes.c_int()
    _check(lib.kvs_draft_capacity_pages(ctypes.byref(cfg), int(pinned_bytes), ctypes.byref(n)))
    return n.value


class KVS:
    """Owning handle with the same calls as methods."""

    def __init__(self, cfg: kvs_config, device: int = 0):
        self.h = kvs_create(cfg, device)
        self.cfg = kvs_get_config(self.h)

    def append(self, layer, pos0, n_tok, k, v, stream=None):
        kvs_append(self.h, layer, pos0, n_tok, k, v, stream)

    def attend(self, layer, pos0, n_q, q, out, lse=None, stream=None):
        kvs_attend(self.h, layer, pos0, n_q, q, out, lse, stream)

    def export_page(self, layer, page, from_device, dst):
        kvs_export_page(self.h, layer, page, from_device, dst)

    def page_location(self, layer, page):
        return kvs_page_location(self.h, layer, page)

    def layer_length(self, layer):
        return kvs_layer_length(self.h, layer)

    def stats(self):
        return kvs_get_stats(self.h)

    def reset_stats(self):
        kvs_reset_stats(self.h)

    def sync(self, stream=None, timeout_s=60.0):
        kvs_sync(self.h, stream, timeout_s)

    def measure_h2d(self, chunk_bytes, total_bytes, reps=10):
        return kvs_measure_h2d(self.h, chunk_bytes, total_bytes, reps)

    def close(self):
        if self.h:
            kvs_destroy(self.h)
            self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
