"""Shared-prefix attention with pieces of several key tiles whose running
maximum moves, against the plain fp64 reference (tests/paged_ref.py, which
derives the tolerances).  tests/paged_plan.py says how a call is cut."""
import pytest
import torch

from many_shot_icl_b200 import dbsa
from tests.paged_plan import Plan
from tests.paged_ref import Batch, check

pytestmark = pytest.mark.gpu

HEADS = {128: (32, 8, 128), 64: (16, 4, 64)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from many_shot_icl_b200 import build
    build.build()
    dbsa.load()
    assert torch.cuda.is_available()


# One dimension of the keys, of a pair that RoPE hardly turns (theta^-(1 - 2/D)
# radians a position: below 0.2 at the furthest one here), rises by STEP from
# each 64-key tile to the next, eight tiles long, and starts again.  A query with A
# there has scores that rise by A * STEP * SCALE = 7 (10 in log2 units, a rescale
# every tile), half of that (one every second tile), fall, or stay.
SCALE, STEP = 0.125, 7.0
A = (8.0, 4.0, -8.0, 0.0)


class Rising(Batch):
    def fill(self, scale=1.0):
        super().fill(scale)
        dim = self.cfg.head_dim // 2 - 1
        lists = [(self.prefix_pages, self.prefix_len)] + list(zip(self.page_table, self.lens))
        for pages, n in lists:
            t = torch.arange(n, device=self.device)
            p = pages.long()[t // self.page]
            self.k_pages[p, :, t % self.page, dim] = (STEP * (t // 64 % 8).to(self.dtype))[:, None]
            self.v_pages[p, :, t % self.page] += 2.0     # a lost factor moves every sum
        return self

    def queries(self, a):
        """N(0, 1) queries with the given values at the rising dimension, heads in turn."""
        cfg = self.cfg
        q = self.randn(self.rows, cfg.n_q_heads, cfg.head_dim)
        q[..., cfg.head_dim // 2 - 1] = torch.tensor(a, dtype=self.dtype, device=self.device)[
            torch.arange(cfg.n_q_heads, device=self.device) % len(a)]
        q[..., -1] = 0
        return q


def config(d, dtype):
    return dbsa.DbsaConfig(*HEADS[d], dtype=dtype, rope_theta=5e5, softmax_scale=SCALE)


def run(b, q):
    want, tol = b.attention(q)
    got = b.attend(q)
    assert not torch.isnan(got).any()
    over = (got.double() - want).abs() > tol
    assert not over.any(), "%d of %d elements beyond their bound" % (int(over.sum()), over.numel())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("rows", [4, 10, 70])
def test_maximum_rises_along_the_prefix(dtype, d, rows):
    """Pieces of up to 16 packed rows, of up to 64, and of more."""
    cfg = config(d, dtype)
    prefix = (6000 if rows == 70 else 20001) * (2 if d == 64 else 1)
    lens = [9 + 13 * i % 90 for i in range(rows)]
    plan = Plan(cfg, prefix, [1] * rows, lens)
    assert (16 if rows == 4 else 64 if rows == 10 else 1 << 30) >= plan.rows
    pieces = plan.prefix_pieces()
    assert sum(e - b >= 5 for b, e in pieces) > len(pieces) // 2
    b = Rising(cfg, 64, prefix, [1] * rows, lens, seed=rows + d).fill()
    run(b, b.queries(A))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("n_new,lens", [([1], [30000]), ([10], [9000]), ([40, 3], [8000, 5000])])
def test_maximum_rises_along_own_tokens(dtype, d, n_new, lens):
    cfg = config(d, dtype)
    lens = [n * (2 if d == 64 else 1) for n in lens]
    pieces = Plan(cfg, 0, n_new, lens).own_pieces()
    assert sum(e - b >= 3 for b, e, _ in pieces) > len(pieces) // 2
    b = Rising(cfg, 128, 0, n_new, lens, seed=sum(n_new) + d).fill()
    run(b, b.queries(A))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_maximum_rises_along_ranges_of_decreasing_length(dtype):
    cfg = config(64, dtype)
    n_new, lens = [1] * 9, [36000 + 700 * i for i in range(9)]
    plan = Plan(cfg, 0, n_new, lens)
    assert plan.guided and max(e - b for b, e, _ in plan.own_pieces()) > 8
    b = Rising(cfg, 256, 0, n_new, lens, seed=19).fill()
    run(b, b.queries(A))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [4, 70])
def test_maximum_starts_at_nothing(dtype, rows):
    """Pieces that begin with tiles on missing pages, and some that hold nothing else."""
    cfg = config(128, dtype)
    prefix = 6000 if rows == 70 else 20001
    lens = [500] * rows
    b = Rising(cfg, 64, prefix, [1] * rows, lens, seed=rows).fill()
    gone = torch.arange(len(b.prefix_pages), device="cuda")
    b.prefix_pages[(gone % 5 < 2) | (gone // 20 % 3 == 1)] = -1
    b.page_table[:, 0] = len(b.k_pages)
    missing = b.prefix_pages.cpu().numpy() < 0
    pieces = Plan(cfg, prefix, [1] * rows, lens).prefix_pieces()
    assert any(missing[s:e].all() for s, e in pieces)
    assert any(missing[s] and not missing[s:e].all() for s, e in pieces)
    run(b, b.queries(A))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 64])
def test_a_row_keeps_its_bits_whatever_the_other_rows_ask(dtype, d):
    """The other rows' maxima rise by more than a rescale's threshold, this row's do not."""
    cfg = config(d, dtype)
    prefix, n_new, lens = 20001 * (128 // d), [1] * 9, [30 * i + 1 for i in range(9)]
    assert min(e - b for b, e in Plan(cfg, prefix, n_new, lens).prefix_pieces()) > 4
    b = Rising(cfg, 64, prefix, n_new, lens, seed=12).fill()
    q = b.queries((0.0,))
    got = b.attend(q)
    want, tol = b.attention(q)
    check(got, want, tol, dtype, "level")
    for other in ((8.0,), A, (-8.0,)):
        loud = b.queries(other)
        loud[3] = q[3]
        assert torch.equal(b.attend(loud)[3], got[3])
