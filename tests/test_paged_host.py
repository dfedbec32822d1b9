"""Argument checks of the paged append and the shared-prefix attention, CPU
only: every refusal comes before any device work."""
import ctypes

import pytest
import torch

from many_shot_icl_b200 import dbsa

FAKE = 1 << 20      # aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from many_shot_icl_b200 import build
    build.build()
    return dbsa.load()


CFG = dbsa.DbsaConfig(8, 2, 128)
TABLES = 1 << 24


def cache(**kw):
    c = dict(k_pages=FAKE, v_pages=FAKE, page_stride=2 * 64 * 128, n_pages=10, page_size=64)
    c.update(kw)
    return dbsa.PagedCache(*c.values())


def batch(**kw):
    b = dict(n_seqs=3, n_rows=5, row_ptr=FAKE, seq_lens=FAKE, page_table=FAKE, table_width=4,
             table_stride=4)
    b.update(kw)
    return dbsa.PagedBatch(*b.values())


def append(lib, cfg=CFG, k=FAKE, v=FAKE, strides=(256, 128, 256, 128), pos0=0, tables=FAKE,
           tables_bytes=TABLES, c=None, b=None, null=()):
    cc = cfg.c()
    return lib.dbsa_paged_append(
        None if "cfg" in null else ctypes.byref(cc), k, *strides[:2], v, *strides[2:],
        None if "cache" in null else ctypes.byref(c or cache()),
        None if "batch" in null else ctypes.byref(b or batch()), pos0, tables, tables_bytes, None)


def attend(lib, cfg=CFG, q=FAKE, q_stride=1024, prefix=FAKE, prefix_len=100, tables=FAKE,
           tables_bytes=TABLES, out=FAKE, ws=FAKE, ws_bytes=1 << 40, c=None, b=None):
    cc = cfg.c()
    return lib.dbsa_shared_prefix_attend(
        ctypes.byref(cc), q, q_stride, ctypes.byref(c or cache()), prefix, prefix_len,
        ctypes.byref(b or batch()), tables, tables_bytes, out, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [append, attend])
@pytest.mark.parametrize("bad,status", [
    (dict(c=cache(page_size=48, page_stride=1 << 20)), dbsa.ERR_UNSUPPORTED),
    (dict(c=cache(page_size=8)), dbsa.ERR_UNSUPPORTED),
    (dict(c=cache(page_size=512, page_stride=1 << 20)), dbsa.ERR_UNSUPPORTED),
    (dict(c=cache(page_size=0)), dbsa.ERR_UNSUPPORTED),
    (dict(c=cache(page_stride=2 * 64 * 128 - 8)), dbsa.ERR_INVALID_ARG),
    (dict(c=cache(page_stride=2 * 64 * 128 + 4)), dbsa.ERR_INVALID_ARG),
    (dict(c=cache(page_stride=1 << 40)), dbsa.ERR_INVALID_ARG),
    (dict(c=cache(n_pages=0)), dbsa.ERR_INVALID_ARG),
    (dict(c=cache(k_pages=None)), dbsa.ERR_INVALID_ARG),
    (dict(c=cache(v_pages=FAKE + 8)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(n_seqs=0)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(n_seqs=65536)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(n_rows=0)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(n_rows=(1 << 30) + 1)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(row_ptr=None)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(seq_lens=FAKE + 2)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(table_width=0)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(table_stride=3)), dbsa.ERR_INVALID_ARG),
    (dict(b=batch(table_width=1 << 26, table_stride=1 << 26)), dbsa.ERR_INVALID_ARG),
    (dict(tables=None), dbsa.ERR_INVALID_ARG),
    (dict(tables_bytes=0), dbsa.ERR_INVALID_ARG),
    (dict(cfg=dbsa.DbsaConfig(8, 3, 128)), dbsa.ERR_UNSUPPORTED),
    (dict(cfg=dbsa.DbsaConfig(8, 2, 96)), dbsa.ERR_UNSUPPORTED),
])
def test_bad_caches_and_batches(lib, call, bad, status):
    assert call(lib, **bad) == status
    assert dbsa.last_error()


def test_tables_must_reach_the_last_position(lib):
    # four pages of 64 tokens behind position 1000: positions below 1256
    enough = dbsa.rope_tables_size(CFG, 1256)
    short = dbsa.rope_tables_size(CFG, 1240)
    assert append(lib, pos0=1000, tables_bytes=short) == dbsa.ERR_INVALID_ARG
    assert "1256" in dbsa.last_error()
    assert attend(lib, prefix_len=1000, tables_bytes=short) == dbsa.ERR_INVALID_ARG
    assert attend(lib, prefix_len=1000, tables_bytes=enough, ws=None) == dbsa.ERR_WORKSPACE


def test_append_refusals(lib):
    assert append(lib, null=("cfg",)) == dbsa.ERR_INVALID_ARG
    assert append(lib, null=("cache",)) == dbsa.ERR_INVALID_ARG
    assert append(lib, null=("batch",)) == dbsa.ERR_INVALID_ARG
    assert append(lib, k=None) == dbsa.ERR_INVALID_ARG
    assert append(lib, v=FAKE + 4) == dbsa.ERR_INVALID_ARG
    assert append(lib, strides=(256, 128, 256, 100)) == dbsa.ERR_INVALID_ARG
    assert append(lib, pos0=-1) == dbsa.ERR_INVALID_ARG


def test_attend_refusals(lib):
    assert attend(lib, q=None) == dbsa.ERR_INVALID_ARG
    assert attend(lib, out=FAKE + 8) == dbsa.ERR_INVALID_ARG
    assert attend(lib, q_stride=1028) == dbsa.ERR_INVALID_ARG
    assert attend(lib, prefix=None) == dbsa.ERR_INVALID_ARG
    assert attend(lib, prefix_len=-1) == dbsa.ERR_INVALID_ARG
    assert attend(lib, b=batch(n_rows=(1 << 25) + 1)) == dbsa.ERR_INVALID_ARG
    need = dbsa.shared_prefix_workspace_size(CFG, 3, 5, 100)
    assert need > 0
    assert attend(lib, ws_bytes=need - 1) == dbsa.ERR_WORKSPACE
    assert attend(lib, ws=FAKE + 16) == dbsa.ERR_WORKSPACE
    assert attend(lib, ws=None) == dbsa.ERR_WORKSPACE


def test_sizes(lib):
    assert dbsa.rope_tables_size(CFG, 0) == 0 and dbsa.rope_tables_size(CFG, (1 << 31) + 1) == 0
    # cos and sin, 64 frequencies, fp32: a row per 16 positions and 16 fine rows
    assert dbsa.rope_tables_size(CFG, 16) == 2 * (1 + 16) * 64 * 4
    assert dbsa.rope_tables_size(CFG, 17) == 2 * (2 + 16) * 64 * 4
    size = dbsa.shared_prefix_workspace_size
    assert size(CFG, 0, 5, 100) == 0 and size(CFG, 3, 0, 100) == 0 and size(CFG, 3, 5, -1) == 0
    assert size(dbsa.DbsaConfig(8, 3, 128), 3, 5, 100) == 0
    # grows with the rows, and with the prefix only up to a full set of ranges
    assert size(CFG, 3, 5, 0) < size(CFG, 3, 500, 0) < size(CFG, 3, 500, 100000)
    assert size(CFG, 64, 64, 1 << 20) == size(CFG, 64, 64, 1 << 24)
    c = CFG.c()
    bad = dbsa.DbsaConfig(8, 2, 96).c()
    call = lib.dbsa_rope_tables
    assert call(ctypes.byref(bad), 16, FAKE, 1 << 20, None) == dbsa.ERR_UNSUPPORTED
    assert call(ctypes.byref(c), 0, FAKE, 1 << 20, None) == dbsa.ERR_INVALID_ARG
    assert call(ctypes.byref(c), 16, None, 1 << 20, None) == dbsa.ERR_INVALID_ARG
    assert call(ctypes.byref(c), 16, FAKE + 4, 1 << 20, None) == dbsa.ERR_INVALID_ARG
    assert call(ctypes.byref(c), 16, FAKE, 100, None) == dbsa.ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(32, 8, 128), (32, 32, 128), (5, 1, 64)])
def test_a_workspace_for_the_largest_call_serves_the_smaller_ones(lib, dtype, heads):
    cfg = dbsa.DbsaConfig(*heads, dtype)
    for prefix in (0, 1, 100, 4001, 90223):
        sizes = [dbsa.shared_prefix_workspace_size(cfg, 64, n, prefix) for n in range(1, 700)]
        assert sizes == sorted(sizes)
    for rows in (1, 3, 64, 641):
        sizes = [dbsa.shared_prefix_workspace_size(cfg, n, rows, 1000) for n in range(1, 300)]
        assert sizes == sorted(sizes)
        sizes = [dbsa.shared_prefix_workspace_size(cfg, 8, rows, n) for n in range(0, 9000, 17)]
        assert sizes == sorted(sizes)


def test_binding_refuses_tensors_it_cannot_pass(lib):
    """Types, shapes and strides are checked before the device is asked for."""
    i32 = dict(dtype=torch.int32)
    pages = torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16)
    good = dict(k=torch.zeros(3, 2, 128, dtype=torch.bfloat16),
                v=torch.zeros(3, 2, 128, dtype=torch.bfloat16), k_pages=pages, v_pages=pages,
                page_table=torch.zeros(3, 1, **i32), row_ptr=torch.zeros(4, **i32),
                seq_lens=torch.zeros(3, **i32), tables=torch.zeros(1 << 16, dtype=torch.uint8))

    def refused(what, **kw):
        with pytest.raises(dbsa.DbsaError) as e:
            dbsa.paged_append(CFG, **{**good, **kw})
        assert e.value.status == dbsa.ERR_INVALID_ARG and what in str(e.value)

    refused("CUDA device")                                       # all on the CPU
    refused("pages must be", k_pages=pages.float(), v_pages=pages.float())
    refused("alike", v_pages=pages[:2])
    refused("heads", k_pages=pages[:, :1], v_pages=pages[:, :1])
    refused("one page stride", k_pages=pages[::2], v_pages=pages[:2])
    refused("contiguous inside", k_pages=pages.transpose(1, 2).contiguous().transpose(1, 2))
    refused("int32", row_ptr=torch.zeros(4, dtype=torch.int64))
    refused("int32", row_ptr=torch.zeros(3, **i32))
    refused("int32", page_table=torch.zeros(2, 1, **i32))
    refused("contiguous", row_ptr=torch.zeros(8, **i32)[::2])
    refused("contiguous", tables=torch.zeros(1 << 16, dtype=torch.uint8)[::2])


def test_binding_refuses_counts_beyond_32_bits(lib):
    """A row that is repeated by a stride of 0 makes such a count without the memory."""
    i32 = dict(dtype=torch.int32)
    pages = torch.zeros(4, 2, 64, 128, dtype=torch.bfloat16)
    row = torch.zeros(1, 2, 128, dtype=torch.bfloat16)
    for n in (2**31, 2**32 + 1):
        rows = row.expand(n, 2, 128)
        with pytest.raises(dbsa.DbsaError) as e:
            dbsa.paged_append(CFG, rows, rows, pages, pages, torch.zeros(1, 1, **i32),
                              torch.zeros(2, **i32), torch.zeros(1, **i32),
                              torch.zeros(1 << 16, dtype=torch.uint8))
        assert e.value.status == dbsa.ERR_INVALID_ARG and "rows" in str(e.value)
