"""ctypes binding of libdbsa.so (see include/dbsa.h for the contract).

Argument marshalling only: torch tensors are passed as raw device pointers,
host arrays as numpy int32 buffers, and the current torch CUDA stream as the
call's stream.  Every step of the computation runs in the library's CUDA
kernels; there is no fallback.  If the library is missing, the first call
raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libdbsa.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CAPACITY, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(7)
BF16, F32 = 0, 1
PATTERN_SINK_PREV_SELF, PATTERN_FULL, PATTERN_SINK_SELF, PATTERN_SELF = range(4)

SYMBOLS = (
    "dbsa_group_blocks", "dbsa_encode_workspace_size", "dbsa_encode_blocks",
    "dbsa_append_workspace_size", "dbsa_append_block", "dbsa_gather_workspace_size",
    "dbsa_gather_rope_attend", "dbsa_last_error", "dbsa_read_status", "dbsa_stage1_plan",
    "dbsa_stage1_tile_count", "dbsa_version", "dbsa_kernel_launches", "dbsa_set_profile_events",
    "dbsa_gather_rope_attend_noalloc", "dbsa_block_keys_size", "dbsa_block_keys",
    "dbsa_gather_rope_attend_prepared", "dbsa_noalloc_read_status", "dbsa_test_wait_expiry",
    "dbsa_host_allocation_calls", "dbsa_rope_tables_size", "dbsa_rope_tables",
    "dbsa_paged_append", "dbsa_shared_prefix_workspace_size", "dbsa_shared_prefix_attend",
)


class DbsaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("dbsa status %d: %s" % (status, msg))
        self.status = status


class Config(ctypes.Structure):
    _fields_ = [("n_q_heads", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("rope_theta", ctypes.c_double), ("window_j", ctypes.c_int32),
                ("pattern", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class TileItem(ctypes.Structure):
    _fields_ = [("head", ctypes.c_int32), ("q_row0", ctypes.c_int32), ("q_pos0", ctypes.c_int32),
                ("n_rows", ctypes.c_int32), ("n_ranges", ctypes.c_int32), ("block", ctypes.c_int32),
                ("k_row0", ctypes.c_int32 * 2), ("v_row0", ctypes.c_int32 * 2),
                ("pos0", ctypes.c_int32 * 2), ("len", ctypes.c_int32 * 2)]


class PagedCache(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("n_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32)]


class PagedBatch(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("n_rows", ctypes.c_int32),
                ("row_ptr", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("page_table", ctypes.c_void_p), ("table_width", ctypes.c_int32),
                ("table_stride", ctypes.c_int32)]


@dataclass(frozen=True)
class DbsaConfig:
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    dtype: str = "bf16"          # "bf16" or "f32"
    rope_theta: float = 1e4
    window_j: int = 2
    pattern: int = PATTERN_SINK_PREV_SELF
    softmax_scale: float = 0.0

    def c(self) -> Config:
        return Config(self.n_q_heads, self.n_kv_heads, self.head_dim,
                      F32 if self.dtype == "f32" else BF16, float(self.rope_theta),
                      self.window_j, self.pattern, float(self.softmax_scale), 0)


_lib = None


def load(path: str = LIB_PATH):
    """Load libdbsa.so (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libdbsa.so not found at %s: build it with "
                           "`python -m many_shot_icl_b200.build`" % path)
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    cfgp = ctypes.POINTER(Config)
    lib.dbsa_group_blocks.argtypes = [vp, i32, i32, vp]
    lib.dbsa_group_blocks.restype = i32
    lib.dbsa_encode_workspace_size.argtypes = [cfgp, i64, i32]
    lib.dbsa_encode_workspace_size.restype = sz
    lib.dbsa_encode_blocks.argtypes = [cfgp, vp, vp, vp, vp, i32, vp, vp, i64, vp, vp, sz, vp]
    lib.dbsa_encode_blocks.restype = ctypes.c_int
    lib.dbsa_append_workspace_size.argtypes = [cfgp, vp, i32, i32]
    lib.dbsa_append_workspace_size.restype = sz
    lib.dbsa_append_block.argtypes = [cfgp, vp, vp, vp, i32, vp, i32, vp, vp, i64, vp, vp, sz, vp]
    lib.dbsa_append_block.restype = ctypes.c_int
    lib.dbsa_gather_workspace_size.argtypes = [cfgp, vp, i32, i32, vp, vp, i32, i32]
    lib.dbsa_gather_workspace_size.restype = sz
    lib.dbsa_gather_rope_attend.argtypes = [cfgp, vp, vp, i64, vp, i32, i32, vp, vp, vp, i32, vp,
                                            vp, i32, i32, vp, vp, i64, vp, sz, vp]
    lib.dbsa_gather_rope_attend.restype = ctypes.c_int
    lib.dbsa_gather_rope_attend_noalloc.argtypes = [cfgp, vp, vp, i64, vp, i32, i32, vp, vp, vp,
                                                    i32, vp, vp, i32, i32, vp, vp, i64, vp]
    lib.dbsa_gather_rope_attend_noalloc.restype = ctypes.c_int
    lib.dbsa_block_keys_size.argtypes = [cfgp, vp, i32]
    lib.dbsa_block_keys_size.restype = sz
    lib.dbsa_block_keys.argtypes = [cfgp, vp, vp, i64, vp, i32, vp, sz, vp]
    lib.dbsa_block_keys.restype = ctypes.c_int
    lib.dbsa_gather_rope_attend_prepared.argtypes = [cfgp, vp, vp, i64, vp, i32, i32, vp, vp, vp,
                                                     i32, vp, vp, i32, i32, vp, vp, i64, vp, sz,
                                                     vp, sz, vp]
    lib.dbsa_gather_rope_attend_prepared.restype = ctypes.c_int
    lib.dbsa_last_error.argtypes = []
    lib.dbsa_last_error.restype = ctypes.c_char_p
    lib.dbsa_read_status.argtypes = [vp, vp]
    lib.dbsa_read_status.restype = ctypes.c_int
    lib.dbsa_stage1_plan.argtypes = [cfgp, vp, i32, vp, i64]
    lib.dbsa_stage1_plan.restype = i64
    lib.dbsa_stage1_tile_count.argtypes = [cfgp, vp, i32]
    lib.dbsa_stage1_tile_count.restype = i64
    lib.dbsa_version.argtypes = []
    lib.dbsa_version.restype = ctypes.c_char_p
    lib.dbsa_kernel_launches.argtypes = []
    lib.dbsa_kernel_launches.restype = i64
    lib.dbsa_set_profile_events.argtypes = [vp, vp]
    lib.dbsa_set_profile_events.restype = None
    lib.dbsa_noalloc_read_status.argtypes = [vp]
    lib.dbsa_noalloc_read_status.restype = ctypes.c_int
    lib.dbsa_test_wait_expiry.argtypes = [ctypes.c_uint64]
    lib.dbsa_test_wait_expiry.restype = None
    lib.dbsa_host_allocation_calls.argtypes = []
    lib.dbsa_host_allocation_calls.restype = i64
    lib.dbsa_rope_tables_size.argtypes = [cfgp, i64]
    lib.dbsa_rope_tables_size.restype = sz
    lib.dbsa_rope_tables.argtypes = [cfgp, i64, vp, sz, vp]
    lib.dbsa_rope_tables.restype = ctypes.c_int
    cachep, batchp = ctypes.POINTER(PagedCache), ctypes.POINTER(PagedBatch)
    lib.dbsa_paged_append.argtypes = [cfgp, vp, i64, i64, vp, i64, i64, cachep, batchp, i64, vp,
                                      sz, vp]
    lib.dbsa_paged_append.restype = ctypes.c_int
    lib.dbsa_shared_prefix_workspace_size.argtypes = [cfgp, i32, i32, i64]
    lib.dbsa_shared_prefix_workspace_size.restype = sz
    lib.dbsa_shared_prefix_attend.argtypes = [cfgp, vp, i64, cachep, vp, i64, batchp, vp, sz, vp,
                                              vp, sz, vp]
    lib.dbsa_shared_prefix_attend.restype = ctypes.c_int
    _lib = lib
    return lib


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _hp(a: np.ndarray):
    return a.ctypes.data_as(ctypes.c_void_p)


def _dp(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(status: int):
    if status != OK:
        raise DbsaError(status, load().dbsa_last_error().decode())


def last_error() -> str:
    return load().dbsa_last_error().decode()


def version() -> str:
    return load().dbsa_version().decode()


def group_blocks(demo_len, k: int) -> np.ndarray:
    dl = _i32(demo_len)
    offs = np.zeros((len(dl) + k - 1) // k + 1, dtype=np.int32)
    nb = load().dbsa_group_blocks(_hp(dl), len(dl), k, _hp(offs))
    if nb < 0:
        raise DbsaError(ERR_INVALID_ARG, last_error())
    return offs


def stage1_plan(cfg: DbsaConfig, offs) -> list:
    o = _i32(offs)
    c = cfg.c()
    lib = load()
    n = lib.dbsa_stage1_plan(ctypes.byref(c), _hp(o), len(o) - 1, None, 0)
    if n < 0:
        raise DbsaError(ERR_INVALID_ARG, last_error())
    arr = (TileItem * max(n, 1))()
    lib.dbsa_stage1_plan(ctypes.byref(c), _hp(o), len(o) - 1, ctypes.cast(arr, ctypes.c_void_p), n)
    return list(arr[:n])


def stage1_tile_count(cfg: DbsaConfig, offs) -> int:
    o = _i32(offs)
    c = cfg.c()
    return int(load().dbsa_stage1_tile_count(ctypes.byref(c), _hp(o), len(o) - 1))


def encode_workspace_size(cfg: DbsaConfig, n_tokens: int, nb: int) -> int:
    c = cfg.c()
    return int(load().dbsa_encode_workspace_size(ctypes.byref(c), n_tokens, nb))


def append_workspace_size(cfg: DbsaConfig, offs, L: int) -> int:
    o = _i32(offs)
    c = cfg.c()
    return int(load().dbsa_append_workspace_size(ctypes.byref(c), _hp(o), len(o) - 1, L))


def gather_workspace_size(cfg: DbsaConfig, offs, sel_ptr, sel_blocks, n_new: int,
                          tail_len: int) -> int:
    o, sp, sb = _i32(offs), _i32(sel_ptr), _i32(sel_blocks)
    c = cfg.c()
    return int(load().dbsa_gather_workspace_size(ctypes.byref(c), _hp(o), len(o) - 1,
                                                 len(sp) - 1, _hp(sp), _hp(sb), n_new, tail_len))


def encode_blocks(cfg: DbsaConfig, q, k, v, offs, k_cache, v_cache, out, workspace, stream=None):
    """Stage 1 over all blocks: fills k_cache/v_cache rows [0, T) and out."""
    o = _i32(offs)
    c = cfg.c()
    _check(load().dbsa_encode_blocks(
        ctypes.byref(c), _dp(q), _dp(k), _dp(v), _hp(o), len(o) - 1, _dp(k_cache), _dp(v_cache),
        k_cache.shape[1], _dp(out), _dp(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))


def append_block(cfg: DbsaConfig, q, k, v, offs, k_cache, v_cache, out, workspace, stream=None):
    """Encode one new block after the blocks of `offs` (its length = q.shape[0])."""
    o = _i32(offs)
    c = cfg.c()
    _check(load().dbsa_append_block(
        ctypes.byref(c), _dp(q), _dp(k), _dp(v), q.shape[0], _hp(o), len(o) - 1, _dp(k_cache),
        _dp(v_cache), k_cache.shape[1], _dp(out), _dp(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


def gather_rope_attend(cfg: DbsaConfig, k_cache, v_cache, offs, sel_ptr, sel_blocks, q_new,
                       k_tail, v_tail, tail_len: int, out, workspace, dbg_map=None, stream=None,
                       block_keys=None):
    """Stage 2 for a batch of queries (see dbsa_gather_rope_attend); with
    block_keys (from block_keys()), dbsa_gather_rope_attend_prepared."""
    o, sp, sb = _i32(offs), _i32(sel_ptr), _i32(sel_blocks)
    c = cfg.c()
    args = [ctypes.byref(c), _dp(k_cache), _dp(v_cache), k_cache.shape[1], _hp(o), len(o) - 1,
            len(sp) - 1, _hp(sp), _hp(sb), _dp(q_new), q_new.shape[1], _dp(k_tail), _dp(v_tail),
            tail_len, k_tail.shape[1], _dp(out), _dp(dbg_map),
            0 if dbg_map is None else dbg_map.shape[1]]
    ws = [_dp(workspace), workspace.numel() * workspace.element_size(), _stream(stream)]
    if block_keys is None:
        _check(load().dbsa_gather_rope_attend(*args, *ws))
    else:
        _check(load().dbsa_gather_rope_attend_prepared(
            *args, _dp(block_keys), block_keys.numel() * block_keys.element_size(), *ws))


def block_keys_size(cfg: DbsaConfig, offs) -> int:
    o = _i32(offs)
    c = cfg.c()
    return int(load().dbsa_block_keys_size(ctypes.byref(c), _hp(o), len(o) - 1))


def block_keys(cfg: DbsaConfig, k_cache, v_cache, offs, buf, stream=None):
    """Keys of every cache row rotated at their position inside their block,
    into buf (uint8 device tensor of block_keys_size() bytes)."""
    o = _i32(offs)
    c = cfg.c()
    _check(load().dbsa_block_keys(
        ctypes.byref(c), _dp(k_cache), _dp(v_cache), k_cache.shape[1], _hp(o), len(o) - 1,
        _dp(buf), buf.numel() * buf.element_size(), _stream(stream)))


def kernel_launches() -> int:
    return int(load().dbsa_kernel_launches())


def set_profile_events(start, stop):
    """Record torch.cuda.Event objects around the next call's main kernel."""
    def handle(ev):
        if ev is None:
            return None
        if not ev.cuda_event:   # torch creates the CUDA event on its first record()
            ev.record()
        return ev.cuda_event
    load().dbsa_set_profile_events(handle(start), handle(stop))


def gather_rope_attend_noalloc(cfg: DbsaConfig, k_cache, v_cache, offs, sel_ptr, sel_blocks,
                               q_new, k_tail, v_tail, tail_len: int, out, dbg_map=None,
                               stream=None):
    """Stage 2 without a workspace: for callers that cannot allocate device
    memory.  Scratch is the library's fixed 16 MiB per-device array, shared
    by every call (serialise calls that would overlap on the GPU)."""
    o, sp, sb = _i32(offs), _i32(sel_ptr), _i32(sel_blocks)
    c = cfg.c()
    _check(load().dbsa_gather_rope_attend_noalloc(
        ctypes.byref(c), _dp(k_cache), _dp(v_cache), k_cache.shape[1], _hp(o), len(o) - 1,
        len(sp) - 1, _hp(sp), _hp(sb), _dp(q_new), q_new.shape[1], _dp(k_tail), _dp(v_tail),
        tail_len, k_tail.shape[1], _dp(out), _dp(dbg_map),
        0 if dbg_map is None else dbg_map.shape[1], _stream(stream)))


def read_status(workspace, stream=None) -> int:
    return int(load().dbsa_read_status(_dp(workspace), _stream(stream)))


def noalloc_read_status(stream=None) -> int:
    return int(load().dbsa_noalloc_read_status(_stream(stream)))


def test_wait_expiry(limit_ns: int):
    """Test hook: the next call on this thread loads no tile, so its device
    waits run out after limit_ns nanoseconds (see dbsa_test_wait_expiry)."""
    load().dbsa_test_wait_expiry(int(limit_ns))


def host_allocation_calls() -> int:
    return int(load().dbsa_host_allocation_calls())


def selection_csr(selections) -> tuple[np.ndarray, np.ndarray]:
    """CSR (sel_ptr, sel_blocks) from a list of per-query block-id arrays."""
    ptr = np.zeros(len(selections) + 1, dtype=np.int32)
    ptr[1:] = np.cumsum([len(s) for s in selections])
    return ptr, (np.concatenate(selections).astype(np.int32) if selections else
                 np.zeros(0, np.int32))


def _refuse(msg: str):
    raise DbsaError(ERR_INVALID_ARG, msg)


# torch and what the paged calls use of it, taken by the first of them: the
# host-only functions above and the size queries do without.
torch = _DTYPES = _current_device = _raw_stream = None


def _with_torch():
    """The library, with torch imported."""
    global torch, _DTYPES, _current_device, _raw_stream
    lib = load()
    if torch is None:
        import torch as t
        _DTYPES = {"f32": t.float32, "bf16": t.bfloat16}
        _current_device = t.cuda.current_device
        # (the public stream object costs 2 us, a quarter of a short call)
        _raw_stream = getattr(t._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: t.cuda.current_stream(index).cuda_stream)
        torch = t
    return lib


def _run(fn, index: int, stream, *args):
    """Call fn(*args, stream) with device `index` current, on its current
    stream unless one is given."""
    st = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        status = fn(*args, st)
    else:
        with torch.cuda.device(index):
            status = fn(*args, st)
    if status:
        _check(status)


def _config_ref(cfg: DbsaConfig):
    """byref() of the config's struct, which is made once per config (the library
    only reads it)."""
    c = cfg.__dict__.get("_c")
    if c is None:
        c = cfg.c()
        object.__setattr__(cfg, "_c", c)
    return ctypes.byref(c)


def _paged_args(cfg: DbsaConfig, k_pages, v_pages, page_table, row_ptr, seq_lens, tables, n_rows,
                pos0, index):
    """The cache and batch structs of a call on device `index`, after checking
    the tensors (and the position of the sequences' first tokens)."""
    shape, st, dtype = k_pages.shape, k_pages.stride(), _DTYPES[cfg.dtype]
    if len(shape) != 4 or v_pages.shape != shape:
        _refuse("pages must be [n_pages][n_kv_heads][page_size][head_dim], keys and values alike")
    n_pages, hkv, page_size, d = shape
    if hkv != cfg.n_kv_heads or d != cfg.head_dim:
        _refuse("pages of %d heads of %d elements; cfg has %d of %d"
                % (hkv, d, cfg.n_kv_heads, cfg.head_dim))
    page = page_size * d
    vst = v_pages.stride()
    stride = st[0]
    if n_pages == 1:
        stride = hkv * page
        st, vst = (stride, *st[1:]), (stride, *vst[1:])
    if hkv == 1:
        st, vst = (st[0], page, *st[2:]), (vst[0], page, *vst[2:])
    if (k_pages.dtype != dtype or v_pages.dtype != dtype or st != vst or st[3] != 1 or st[2] != d
            or st[1] != page):
        _refuse("pages must be %s, contiguous inside a page, with one page stride" % dtype)
    n_seqs, table, pt, i32 = seq_lens.numel(), page_table.shape, page_table.stride(), torch.int32
    if (row_ptr.dtype != i32 or seq_lens.dtype != i32 or page_table.dtype != i32
            or len(table) != 2 or table[0] != n_seqs or row_ptr.numel() != n_seqs + 1):
        _refuse("row_ptr [n_seqs + 1], seq_lens [n_seqs] and page_table [n_seqs][width] must be "
                "int32")
    width = table[1]
    if (not row_ptr.is_contiguous() or not seq_lens.is_contiguous()
            or (width > 1 and pt[1] != 1) or not tables.is_contiguous()):
        _refuse("row_ptr, seq_lens and tables must be contiguous, and the rows of page_table")
    # (ctypes cuts a number that its C type cannot hold)
    if max(n_rows, n_seqs, width, pt[0], n_pages) > 0x7FFFFFFF:
        _refuse("more than 2^31 - 1 pages, rows, sequences, table entries or entries between "
                "table rows")
    if not 0 <= pos0 <= 1 << 30:
        _refuse("positions must start at 0..2^30")
    if index < 0 or not (index == v_pages.get_device() == page_table.get_device()
                         == row_ptr.get_device() == seq_lens.get_device() == tables.get_device()):
        _refuse("pages, page_table, row_ptr, seq_lens and tables must be on one CUDA device")
    return (PagedCache(k_pages.data_ptr(), v_pages.data_ptr(), stride, n_pages, page_size),
            PagedBatch(n_seqs, n_rows, row_ptr.data_ptr(), seq_lens.data_ptr(),
                       page_table.data_ptr(), width, pt[0] if n_seqs > 1 else width))


def _count(n: int) -> int:
    """n, or -1, which the library refuses, where its C type might not hold it (no
    count may be larger)."""
    return n if 0 <= n <= 1 << 31 else -1


def rope_tables_size(cfg: DbsaConfig, n_pos: int) -> int:
    c = cfg.c()
    return int(load().dbsa_rope_tables_size(ctypes.byref(c), _count(n_pos)))


def rope_tables(cfg: DbsaConfig, n_pos: int, buf, stream=None):
    """Angle tables for positions [0, n_pos) into buf (uint8 device tensor of
    rope_tables_size() bytes, or more: all of it is filled), for paged_append and
    shared_prefix_attend, which may be given any part from its start that covers
    their positions."""
    if buf.get_device() < 0 or not buf.is_contiguous():
        _refuse("buf must be a contiguous CUDA tensor")
    c = cfg.c()
    _run(_with_torch().dbsa_rope_tables, buf.get_device(), stream, ctypes.byref(c), _count(n_pos),
         _dp(buf), buf.numel() * buf.element_size())


def paged_append(cfg: DbsaConfig, k, v, k_pages, v_pages, page_table, row_ptr, seq_lens, tables,
                 pos0: int = 0, stream=None):
    """Append the rows k, v [n_rows][n_kv_heads][head_dim] (any row and head
    stride) of a batch to their sequences' pages, keys rotated at pos0 + their
    index in the sequence (see dbsa_paged_append)."""
    if torch is None:
        _with_torch()
    shape, ks, vs, index = k.shape, k.stride(), v.stride(), k_pages.get_device()
    cache, batch = _paged_args(cfg, k_pages, v_pages, page_table, row_ptr, seq_lens, tables,
                               shape[0], pos0, index)
    dtype = _DTYPES[cfg.dtype]
    if (k.dtype != dtype or v.dtype != dtype or len(shape) != 3 or v.shape != shape
            or shape[1] != cfg.n_kv_heads or shape[2] != cfg.head_dim or ks[2] != 1 or vs[2] != 1):
        _refuse("k and v must be %s [n_rows][n_kv_heads][head_dim] with contiguous elements"
                % dtype)
    if k.get_device() != index or v.get_device() != index:
        _refuse("k and v must be on the CUDA device of the pages")
    if (ks[0] | ks[1] | vs[0] | vs[1]) & 7:   # the stride of a dimension of one means nothing
        ks, vs = ([x if n > 1 else 0 for x, n in zip(t, shape)] for t in (ks, vs))
    _run(_lib.dbsa_paged_append, index, stream, _config_ref(cfg), k.data_ptr(), ks[0], ks[1],
         v.data_ptr(), vs[0], vs[1], ctypes.byref(cache), ctypes.byref(batch), pos0,
         tables.data_ptr(), tables.nbytes)


def shared_prefix_workspace_size(cfg: DbsaConfig, n_seqs: int, n_rows: int,
                                 prefix_len: int) -> int:
    c = cfg.c()
    return int(load().dbsa_shared_prefix_workspace_size(ctypes.byref(c), _count(n_seqs),
                                                        _count(n_rows), _count(prefix_len)))


def shared_prefix_attend(cfg: DbsaConfig, q, k_pages, v_pages, prefix_pages, prefix_len: int,
                         page_table, row_ptr, seq_lens, tables, out, workspace, stream=None):
    """Attention of the rows q [n_rows][n_q_heads][head_dim] (any row stride)
    over a shared prefix and, causally, each row's own sequence, into out of
    the same shape, contiguous (see dbsa_shared_prefix_attend).  prefix_pages
    may be None when prefix_len is 0."""
    if torch is None:
        _with_torch()
    shape, st, index, d = q.shape, q.stride(), k_pages.get_device(), cfg.head_dim
    cache, batch = _paged_args(cfg, k_pages, v_pages, page_table, row_ptr, seq_lens, tables,
                               shape[0], prefix_len, index)
    dtype = _DTYPES[cfg.dtype]
    if (q.dtype != dtype or len(shape) != 3 or shape[1] != cfg.n_q_heads or shape[2] != d
            or st[2] != 1 or (st[1] != d and shape[1] > 1)):
        _refuse("q must be %s [n_rows][n_q_heads][head_dim], each row contiguous" % dtype)
    if out.dtype != dtype or out.shape != shape or not out.is_contiguous():
        _refuse("out must be %s, contiguous, of q's shape" % dtype)
    if not workspace.is_contiguous():
        _refuse("workspace must be contiguous")
    if not (index == q.get_device() == out.get_device() == workspace.get_device()):
        _refuse("q, out and workspace must be on the CUDA device of the pages")
    prefix = None
    if prefix_len > 0:
        if (prefix_pages is None or prefix_pages.dtype != torch.int32
                or not prefix_pages.is_contiguous() or prefix_pages.get_device() != index
                or prefix_pages.numel() * cache.page_size < prefix_len):
            _refuse("prefix_pages must be contiguous int32 on the CUDA device of the pages, one "
                    "entry per page of the prefix")
        prefix = prefix_pages.data_ptr()
    _run(_lib.dbsa_shared_prefix_attend, index, stream, _config_ref(cfg), q.data_ptr(),
         st[0] if shape[0] > 1 else 0, ctypes.byref(cache), prefix, prefix_len,
         ctypes.byref(batch), tables.data_ptr(), tables.nbytes, out.data_ptr(),
         workspace.data_ptr(), workspace.nbytes)
