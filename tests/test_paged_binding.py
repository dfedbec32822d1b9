"""What the binding of the paged calls passes on to C and what it refuses,
CPU only."""
import pytest
import torch

from many_shot_icl_b200 import dbsa

I32 = dict(dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from many_shot_icl_b200 import build
    build.build()


def call(name, cfg, **kw):
    """The message that the call of that name is refused with, on CPU tensors
    that are right but for what `kw` replaces."""
    hkv, d = cfg.n_kv_heads, cfg.head_dim
    pages = torch.zeros(4, hkv, 64, d, dtype=torch.bfloat16)
    a = dict(k_pages=pages, v_pages=pages, page_table=torch.zeros(3, 1, **I32),
             row_ptr=torch.zeros(4, **I32), seq_lens=torch.zeros(3, **I32),
             tables=torch.zeros(1 << 16, dtype=torch.uint8))
    if name == "append":
        a.update(k=torch.zeros(3, hkv, d, dtype=torch.bfloat16),
                 v=torch.zeros(3, hkv, d, dtype=torch.bfloat16))
    else:
        q = torch.zeros(3, cfg.n_q_heads, d, dtype=torch.bfloat16)
        a.update(q=q, out=torch.zeros_like(q), prefix_pages=None, prefix_len=0,
                 workspace=torch.zeros(1 << 16, dtype=torch.uint8))
        kw = {"prefix_len" if k == "pos0" else k: v for k, v in kw.items()}
    a.update(kw)
    with pytest.raises(dbsa.DbsaError) as e:
        (dbsa.paged_append if name == "append" else dbsa.shared_prefix_attend)(cfg, **a)
    assert e.value.status == dbsa.ERR_INVALID_ARG
    return str(e.value)


CFG = dbsa.DbsaConfig(8, 2, 128)


@pytest.mark.parametrize("name", ["append", "attend"])
def test_numbers_beyond_their_c_types(name):
    """ctypes would cut them to 32 or 64 bits without a word."""
    assert "CUDA device" in call(name, CFG)      # nothing else is wrong with the rest
    wide = torch.empty(3, 2 ** 32 + 1, device="meta", **I32)
    assert "2^31 - 1" in call(name, CFG, page_table=wide)
    one = dict(row_ptr=torch.zeros(2, **I32), seq_lens=torch.zeros(1, **I32))
    assert "2^31 - 1" in call(name, CFG, page_table=wide[:1].as_strided((1, 2 ** 32 + 1), (8, 1)),
                              **one)
    pool = torch.empty(2 ** 32 + 4, 2, 64, 128, device="meta", dtype=torch.bfloat16)
    assert "2^31 - 1" in call(name, CFG, k_pages=pool, v_pages=pool)
    for pos0 in (2 ** 64, 2 ** 64 + 7, -2 ** 64, -1, 2 ** 30 + 1):
        assert "2^30" in call(name, CFG, pos0=pos0)


def test_sizes_beyond_their_c_types():
    assert dbsa.rope_tables_size(CFG, 2 ** 64 + 16) == 0
    assert dbsa.rope_tables_size(CFG, 2 ** 31) > 0
    size = dbsa.shared_prefix_workspace_size
    assert size(CFG, 2 ** 32 + 3, 5, 100) == 0
    assert size(CFG, 3, 2 ** 32 + 5, 100) == 0
    assert size(CFG, 3, 5, 2 ** 64 + 100) == 0
    assert size(CFG, 3, 5, -2 ** 64) == 0
    assert size(CFG, 3, 5, 100) > 0


@pytest.mark.parametrize("name", ["append", "attend"])
def test_the_stride_of_a_dimension_of_one_means_nothing(name):
    """One KV head, its pages taken from [page][token][head][d] pools: the strides
    of keys and values differ only where there is nothing to step over."""
    cfg = dbsa.DbsaConfig(8, 1, 128)
    k = torch.zeros(4, 64, 1, 128, dtype=torch.bfloat16).transpose(1, 2)
    v = torch.zeros(4, 1, 64, 128, dtype=torch.bfloat16)
    assert k.stride() != v.stride()
    assert "CUDA device" in call(name, cfg, k_pages=k, v_pages=v)
    assert "CUDA device" in call(name, cfg, k_pages=v, v_pages=k)
    assert "CUDA device" in call(name, cfg, k_pages=k[:1], v_pages=v[:1])
    # what does mean something still has to be alike
    assert "page stride" in call(name, cfg, k_pages=k,
                                 v_pages=torch.zeros(8, 1, 64, 128, dtype=torch.bfloat16)[::2])
    two = torch.zeros(4, 64, 2, 128, dtype=torch.bfloat16).transpose(1, 2)
    assert "contiguous inside" in call(name, CFG, k_pages=two, v_pages=two)
