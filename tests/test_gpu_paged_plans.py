"""Shared-prefix attention in the plans that only large or unusual batches
get: more items than CTAs, several ranges per CTA, tens of thousands of
sequences, key counts beyond 32-bit products, and row_ptr contents that leave
rows to no sequence."""
import copy

import pytest
import torch

from many_shot_icl_b200 import dbsa
from tests.paged_plan import N_CTAS, Plan
from tests.paged_ref import Batch, check, rotate

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from many_shot_icl_b200 import build
    build.build()
    dbsa.load()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("dtype,rows,prefix,groups", [
    ("bf16", 600, 500, 1),      # one range, more row tiles than CTAs
    ("bf16", 200, 6000, 5),     # five ranges of 100 row tiles: more than one each to a CTA
    ("f32", 150, 1500, 3),
    ("f32", 80, 6000, 7),
])
def test_more_prefix_items_than_ctas(dtype, rows, prefix, groups):
    cfg = dbsa.DbsaConfig(64, 1, 64, dtype, 5e5)
    n_new, lens = [rows - 3, 3], [rows + 40, 3]
    plan = Plan(cfg, prefix, n_new, lens)
    assert plan.groups == groups and plan.prefix_items > N_CTAS
    b = Batch(cfg, 32, prefix, n_new, lens, seed=rows).fill()
    q = b.randn(b.rows, 64, 64)
    want, tol = b.attention(q)
    check(b.attend(q), want, tol, dtype, "%d items" % plan.prefix_items)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("long_one", [0, 100])
def test_the_most_sequences_a_batch_may_have(dtype, long_one):
    """One own token each, or none: the output is that token's value, or 0.  One
    sequence may have many tokens, all of one value."""
    hkv, d, page, n_seqs = 2, 64, 16, 65535
    cfg = dbsa.DbsaConfig(2 * hkv, hkv, d, dtype, 1e4)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    g = torch.Generator().manual_seed(3)
    n_pages = 1009
    k = torch.full((n_pages + 7, hkv, page, d), float("nan"), dtype=dt, device="cuda")
    v = torch.full_like(k, float("nan"))
    k[:n_pages, :, 0] = torch.randn(n_pages, hkv, d, generator=g).to(dt).cuda()
    v[:n_pages, :, 0] = torch.randn(n_pages, hkv, d, generator=g).to(dt).cuda()
    k[n_pages:] = torch.randn(7, hkv, page, d, generator=g).to(dt).cuda()
    v[n_pages:] = v[5, :, :1]
    i32 = dict(dtype=torch.int32, device="cuda")
    s = torch.arange(n_seqs, device="cuda")
    lens = (s % 11 != 3).int()
    table = torch.full((n_seqs, 7), -1, **i32)
    table[:, 0] = (s % n_pages).int()
    n_new = torch.ones(n_seqs, **i32)
    at = n_seqs // 3
    if long_one:
        n_new[at], lens[at] = long_one, long_one
        table[at] = torch.arange(n_pages, n_pages + 7, **i32)
    row_ptr = torch.zeros(n_seqs + 1, **i32)
    row_ptr[1:] = torch.cumsum(n_new, 0)
    rows = int(row_ptr[-1])
    q = torch.randn(rows, 2 * hkv, d, generator=g).to(dt).cuda()
    tables = torch.empty(dbsa.rope_tables_size(cfg, 7 * page), dtype=torch.uint8, device="cuda")
    dbsa.rope_tables(cfg, 7 * page, tables)
    ws = torch.full((dbsa.shared_prefix_workspace_size(cfg, n_seqs, rows, 0),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    dbsa.shared_prefix_attend(cfg, q, k, v, None, 0, table, row_ptr, lens, tables, out, ws)
    assert dbsa.read_status(ws) == dbsa.OK
    value = torch.where(lens.bool()[:, None, None], v[s % n_pages, :, 0], 0.0)
    want = value.repeat_interleave(n_new, 0, output_size=rows).repeat_interleave(2, 1)
    exact = torch.ones(rows, dtype=torch.bool, device="cuda")
    if long_one:
        # probabilities rounded, their sum not; sums of up to 100 terms; the output
        here = slice(int(row_ptr[at]), int(row_ptr[at + 1]))
        exact[here] = False
        want[here] = v[5, :, 0].repeat_interleave(2, 0)
        half = torch.finfo(dt).eps / 2 if dtype == "bf16" else 0.0
        tol = 2 * half + 240 * 2.0 ** -24
        w = want[here].double()
        assert ((out[here].double() - w).abs() <= tol * w.abs()).all()
    assert torch.equal(out[exact], want[exact].to(dt))


def test_key_counts_beyond_32_bit_products():
    """16.8 million prefix tokens of 64 KV heads (262 148 key tiles each, 296
    ranges), which name eight pages again and again; every head has a level of
    its own, so that another head's partial shows."""
    cfg = dbsa.DbsaConfig(64, 64, 64, "bf16", 5e5)
    hkv, d, page, many = 64, 64, 256, 8
    n_prefix = 65537
    prefix_len, lens = n_prefix * page, [1, 1, 200, 1]
    plan = Plan(cfg, prefix_len, [1] * 4, lens)
    assert plan.groups == N_CTAS and plan.units * plan.groups >= 1 << 32
    g = torch.Generator().manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=g)

    level = (torch.arange(hkv) % 7 - 3.0)[None, :, None, None]
    k = randn(many + 4, hkv, page, d).to(torch.bfloat16).cuda()
    v = (0.25 * randn(many + 4, hkv, page, d) + level).to(torch.bfloat16).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    prefix = torch.arange(n_prefix, **i32) % many
    table = torch.arange(many, many + 4, **i32).view(4, 1)
    q = randn(4, hkv, d).to(torch.bfloat16).cuda()
    n_pos = prefix_len + page
    tables = torch.empty(dbsa.rope_tables_size(cfg, n_pos), dtype=torch.uint8, device="cuda")
    dbsa.rope_tables(cfg, n_pos, tables)
    ws = torch.full((dbsa.shared_prefix_workspace_size(cfg, 4, 4, prefix_len),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, float("nan"))
    dbsa.shared_prefix_attend(cfg, q, k, v, prefix, prefix_len, table,
                              torch.arange(5, **i32), torch.tensor(lens, **i32), tables, out, ws)
    assert dbsa.read_status(ws) == dbsa.OK
    times = torch.bincount(prefix.long(), minlength=many).double()
    for r, ln in enumerate(lens):
        pos = torch.tensor([prefix_len + ln - 1], device="cuda")
        for c in range(hkv):
            qr = rotate(q[r, c].double()[None, None], pos, 5e5)[0, 0]
            kk = torch.cat((k[:many, c].reshape(-1, d), k[many + r, c, :ln])).double()
            vv = torch.cat((v[:many, c].reshape(-1, d), v[many + r, c, :ln])).double()
            w = torch.cat((times.repeat_interleave(page),
                           torch.ones(ln, dtype=torch.double, device="cuda")))
            sc = kk @ qr / d ** 0.5 + w.log()
            p = torch.softmax(sc, 0)
            o = p @ vv
            # rounded query and probabilities as in paged_ref; angles of positions this
            # far (2^24, to 1e-6) and their use; sums in fp32 of a piece's tiles, four
            # additions of 16 keys each, every one off by at most a whole step
            half = 2.0 ** -8
            e = kk.abs() @ qr.abs() / d ** 0.5 * (half + 4e-6)
            dev = (vv - o).abs()
            move = (p * torch.expm1(e)) @ dev * e.max().exp()
            steps = 4 * max(b - a for a, b in plan.prefix_pieces()) + 64
            tol = move + (p @ vv.abs()) * (half + steps * 2.0 ** -23) + o.abs() * half
            assert ((out[r, c].double() - o).abs() <= tol).all(), (r, c)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("row_ptr,rows_of,none", [
    ([-4, 2, 4, 9], [2, 2, 5], slice(0, 2)),     # sequence 0 starts before the batch
    ([0, 4, 8, 100], [4, 4, 1], slice(8, 9)),    # sequence 2 ends behind it
    ([0, 0, 9, 9], [0, 9, 0], slice(0, 0)),      # two without rows
    ([2, 5, 5, 7], [5, 0, 4], None),             # rows before the first and behind the last
    ([7, 7, 7, 7], [3, 3, 3], slice(0, 9)),      # rows of nobody
])
def test_sequences_beside_rows_of_nobody(dtype, row_ptr, rows_of, none):
    """Where row_ptr leaves rows out, the other sequences' results are theirs, and
    the rows of nobody keep what they held."""
    cfg = dbsa.DbsaConfig(32, 8, 128, dtype, 5e5)
    b = Batch(cfg, 16, 33, [3, 3, 3], [3, 30, 8], width=4, seed=7).fill()
    k, v, q = b.randn(9, 8, 128), b.randn(9, 8, 128), b.randn(9, 32, 128)
    b.row_ptr.copy_(torch.tensor(row_ptr, dtype=torch.int32))
    before = b.v_pages.clone()
    b.append(k, v)
    want_v = before.clone()
    for s in range(3):
        r0, r1 = row_ptr[s], row_ptr[s + 1]
        if r0 < 0 or r1 > 9:
            continue
        for r in range(r0, r1):
            t = b.lens[s] - (r1 - r)
            if t >= 0:
                want_v[int(b.page_table[s, t // 16]), :, t % 16] = v[r]
    assert torch.equal(torch.nan_to_num(b.v_pages.float(), nan=77.0),
                       torch.nan_to_num(want_v.float(), nan=77.0))
    got = b.attend(q)
    ref = copy.copy(b)
    if none is None:      # the reference walks rows from 0: shift them
        ref.n_new = [3, 0, 2]
        want, tol = ref.attention(q[2:7])
        pad = torch.full((9, 32, 128), float("nan"), dtype=torch.float64, device="cuda")
        want, tol = pad.index_copy(0, torch.arange(2, 7, device="cuda"), want), torch.zeros_like(
            pad).index_copy(0, torch.arange(2, 7, device="cuda"), tol)
    else:
        ref.n_new = rows_of
        want, tol = ref.attention(q)
        want[none] = float("nan")
    check(got, want, tol, dtype, str(row_ptr))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_the_prefix_of_the_moment(dtype, captured):
    """Calls without a wait between them, each right after its prefix was changed
    in the stream (its page list, then its pages by an append): every one sees what
    was written last, eagerly and replayed."""
    cfg = dbsa.DbsaConfig(32, 8, 128, dtype, 5e5)
    prefix_len, page = 6001, 64
    b = Batch(cfg, page, prefix_len, [1] * 6, [9, 1, 70, 130, 5, 64], seed=41).fill()
    q, tables, ws = b.randn(6, 32, 128), b.tables(), b.workspace()
    n = len(b.prefix_pages)
    gen = torch.Generator().manual_seed(8)
    lists = [b.prefix_pages[torch.randperm(n, generator=gen).cuda()].contiguous()
             for _ in range(3)]
    for x in lists:             # any order of pages: the last one is not whole
        tail = b.prefix_pages[-1]
        at = (x == tail).nonzero()[0, 0]
        x[at] = x[-1]
        x[-1] = tail
    prefixes = [(b.randn(prefix_len, 8, 128), b.randn(prefix_len, 8, 128)) for _ in range(3)]
    i32 = dict(dtype=torch.int32, device="cuda")
    row_ptr, lens = torch.tensor([0, prefix_len], **i32), torch.tensor([prefix_len], **i32)
    k, v = b.randn(prefix_len, 8, 128), b.randn(prefix_len, 8, 128)
    out = torch.empty_like(q)

    def attend():
        b.attend(q, out=out, tables=tables, workspace=ws)

    def refill():
        dbsa.paged_append(cfg, k, v, b.k_pages, b.v_pages, b.prefix_pages.view(1, -1), row_ptr,
                          lens, tables)
        attend()

    refill()                    # before capture, as callers do
    steps = [attend, refill]
    if captured:
        graphs = []
        for f in steps:
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                f()
        steps = [g.replay for g in graphs]

    def run(i, wait):
        b.prefix_pages.copy_(lists[i % 3])
        if wait:
            torch.cuda.synchronize()
        steps[0]()
        first = out.clone()
        k.copy_(prefixes[i % 3][0])
        v.copy_(prefixes[i % 3][1])
        if wait:
            torch.cuda.synchronize()
        steps[1]()
        return first, out.clone()

    run(2, True)
    want = [run(i, True) for i in range(3)]
    assert not torch.equal(want[0][0], want[1][0]) and not torch.equal(want[0][1], want[1][1])
    run(2, True)
    got = [run(i, False) for i in range(30)]
    for i, (first, second) in enumerate(got):
        assert torch.equal(first, want[i % 3][0]), i
        assert torch.equal(second, want[i % 3][1]), i
    ref, tol = b.attention(q)
    check(out, ref, tol, dtype, "the last")
