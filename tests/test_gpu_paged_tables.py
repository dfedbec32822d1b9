"""The angle tables of the paged calls: any byte count that covers the
positions reads the same angles, whatever count they were filled with."""
import pytest
import torch

from many_shot_icl_b200 import dbsa
from tests.paged_ref import Batch, check, rotate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from many_shot_icl_b200 import build
    build.build()
    dbsa.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 1, 64)])
@pytest.mark.parametrize("filled,used", [("exact", "whole"), ("whole", "exact"),
                                         ("exact", "one more row"), ("whole", "whole")])
def test_filled_with_one_size_and_used_with_another(dtype, heads, filled, used):
    """The bytes behind those that were filled hold NaN, and no position of the
    batch lies there."""
    cfg = dbsa.DbsaConfig(*heads, dtype=dtype, rope_theta=5e5)
    b = Batch(cfg, 32, 500, [1, 7], [70, 33], seed=2).fill()
    n_pos = b.prefix_len + b.width * b.page
    exact = dbsa.rope_tables_size(cfg, n_pos)
    whole = torch.full((3 * exact + 4096,), 0xFF, dtype=torch.uint8, device="cuda")
    size = {"exact": exact, "whole": whole.numel(),
            "one more row": dbsa.rope_tables_size(cfg, n_pos + 16)}
    dbsa.rope_tables(cfg, n_pos, whole[:size[filled]])
    tables = whole[:size[used]]

    k, v = b.randn(b.rows, heads[1], heads[2]), b.randn(b.rows, heads[1], heads[2])
    b.append(k, v, tables=tables)
    row, half = 0, torch.finfo(b.dtype).eps / 2
    for s, (n, ln) in enumerate(zip(b.n_new, b.lens)):
        for i in range(n):
            t = ln - n + i
            got = b.k_pages[int(b.page_table[s, t // 32]), :, t % 32].double()
            want = rotate(k[row + i].double()[None], torch.tensor([500 + t], device="cuda"),
                          5e5)[0]
            # one rounding of the rotated pair; angles good to ~1e-6, products to 2^-23
            assert ((got - want).abs() <= half * want.abs()
                    + 2 * k.float().abs().max().item() * 2e-6).all()
        row += n
    q = b.randn(b.rows, heads[0], heads[2])
    want, tol = b.attention(q)
    check(b.attend(q, tables=tables), want, tol, dtype, "%s, then %s" % (filled, used))
