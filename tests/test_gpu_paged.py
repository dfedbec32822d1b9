"""Paged append and shared-prefix attention on a B200, against the plain fp64
reference (tests/paged_ref.py, which derives the tolerances)."""
import numpy as np
import pytest
import torch

import oracle
from many_shot_icl_b200 import dbsa
from tests.paged_ref import Batch, check, rotate

pytestmark = pytest.mark.gpu

HEADS = {
    "gqa4": dict(n_q_heads=32, n_kv_heads=8, head_dim=128),
    "mha": dict(n_q_heads=4, n_kv_heads=4, head_dim=128),
    "g3": dict(n_q_heads=12, n_kv_heads=4, head_dim=128),
    "g5": dict(n_q_heads=5, n_kv_heads=1, head_dim=64),
    "g64": dict(n_q_heads=64, n_kv_heads=1, head_dim=64),
}


def config(heads, dtype):
    return dbsa.DbsaConfig(**HEADS[heads], dtype=dtype, rope_theta=5e5)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from many_shot_icl_b200 import build
    build.build()
    dbsa.load()
    assert torch.cuda.is_available()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", ["gqa4", "g5"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("source", ["dense", "fused", "cache"])
def test_append_writes_the_tokens_and_nothing_else(dtype, heads, page, source):
    cfg = config(heads, dtype)
    # a sequence without rows, one starting mid page, one padding, a long one
    b = Batch(cfg, page, 1000, [1, 0, 17, 2, 300], [41, 9, 17, 0, 613], seed=page, spare_rows=2,
              interleaved=source == "fused")
    n, hq, hkv, d = b.rows, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim
    if source == "dense":
        k, v = b.randn(n, hkv, d), b.randn(n, hkv, d)
    elif source == "fused":
        qkv = b.randn(n, hq + 2 * hkv, d)
        k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        k, v = b.randn(hkv, n + 3, d)[:, :n].transpose(0, 1), b.randn(hkv, n, d).transpose(0, 1)
    want_k, want_v = b.k_pages.double(), b.v_pages.clone()
    row = 0
    for s, (m, ln) in enumerate(zip(b.n_new, b.lens)):
        for i in range(m):
            t = ln - m + i
            if t >= 0:
                page_id, slot = int(b.page_table[s, t // page]), t % page
                pos = torch.tensor([1000 + t], device="cuda")
                want_k[page_id, :, slot] = rotate(k[row + i].double()[None], pos, 5e5)[0]
                want_v[page_id, :, slot] = v[row + i]
        row += m
    b.append(k, v)
    assert torch.equal(torch.nan_to_num(b.v_pages.float(), nan=77.0),
                       torch.nan_to_num(want_v.float(), nan=77.0))
    written = ~torch.isnan(want_k)
    assert torch.equal(written, ~torch.isnan(b.k_pages))
    # one rounding of the rotated pair; angles good to ~1e-6, products to 2^-23
    x = torch.cat((k.float().abs().flatten(), v.float().abs().flatten())).max().item()
    half = torch.finfo(b.dtype).eps / 2
    err = torch.where(written, (b.k_pages.double() - want_k), 0.0).abs()
    assert (err <= half * torch.where(written, want_k.abs(), 0.0) + 2 * x * 2e-6).all()


def test_append_drops_what_has_no_page():
    cfg = config("g5", "bf16")
    b = Batch(cfg, 16, 5, [40, 20, 3], [40, 20, 3], width=4)
    table = b.page_table.clone()
    n_pages = len(b.k_pages)
    b.page_table[0, 1] = -1
    b.page_table[0, 2] = n_pages            # one past the pool
    b.page_table[1, 0] = 2 ** 31 - 1
    b.seq_lens[2] = 4 * 16 + 1              # longer than its table: counts as no length
    k, v = b.randn(b.rows, 1, 64), b.randn(b.rows, 1, 64)
    b.append(k, v)
    filled = (~torch.isnan(b.v_pages)).all(-1).sum().item()
    assert filled == 16 + 4                 # page 0 of sequence 0, tokens 16..19 of sequence 1
    assert torch.equal(b.v_pages[table[1, 1].long(), 0, :4], v[40 + 16:40 + 20, 0])


@pytest.mark.parametrize("row_ptr", [[0, 5, 3, 9], [-4, 2, 4, 9], [0, 4, 8, 100], [7, 7, 7, 7],
                                     [0, 9, 0, 9]])
def test_rows_outside_the_batch_belong_to_no_sequence(row_ptr):
    """Contents of row_ptr that no batch has stay inside the buffers: whatever
    is written is a row of the batch."""
    cfg = config("gqa4", "bf16")
    b = Batch(cfg, 16, 33, [3, 3, 3], [3, 30, 8], width=4).fill()
    guard = torch.full((2 * b.rows, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = guard[b.rows // 2:b.rows // 2 + b.rows]
    b.row_ptr.copy_(torch.tensor(row_ptr, dtype=torch.int32))
    b.append(b.randn(b.rows, 8, 128), b.randn(b.rows, 8, 128))
    b.attend(b.randn(b.rows, 32, 128), out=out)
    torch.cuda.synchronize()
    assert torch.isnan(guard[:b.rows // 2]).all() and torch.isnan(guard[b.rows // 2 + b.rows:]).all()


# --------------------------------------------------------------- attention

def run_attention(cfg, page, prefix_len, n_new, lens, seed=0, scale=1.0, **kw):
    b = Batch(cfg, page, prefix_len, n_new, lens, seed=seed, **kw).fill(scale)
    q = b.randn(b.rows, cfg.n_q_heads, cfg.head_dim)
    want, tol = b.attention(q)
    got = b.attend(q)
    check(got, want, tol, cfg.dtype, "prefix %d page %d" % (prefix_len, page))
    return b, q, got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("prefix_len", [0, 1, 127, 128, 129, 777])
def test_decode_step(dtype, heads, prefix_len):
    run_attention(config(heads, dtype), 64, prefix_len, [1] * 7, [1, 2, 63, 64, 65, 130, 300],
                  seed=prefix_len, spare_rows=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_that_end_inside_a_tile(dtype, page):
    run_attention(config("g3", dtype), page, 5 * page // 2 + 3, [1, 1, 9], [page + 1, 3 * page, 9],
                  seed=page, interleaved=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", ["gqa4", "g5", "g64"])
def test_ragged_prompts(dtype, heads):
    # rows of one sequence over several tiles, sequences of one row, none, and
    # padding; some with tokens of their own before the prompt
    run_attention(config(heads, dtype), 32, 300, [45, 1, 0, 70, 2, 5], [45, 90, 11, 200, 0, 3],
                  seed=3, spare_rows=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_long_prompt_alone(dtype):
    run_attention(config("mha", dtype), 64, 0, [400], [700], seed=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_row_one_key(dtype):
    run_attention(config("mha", dtype), 16, 0, [1], [1], seed=6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sharp_scores(dtype):
    """Scores spread over +-40: the running maximum moves along the keys.
    (REL_FRO assumes scores of spread one: the worst case alone is checked.)"""
    cfg = config("gqa4", dtype)
    b = Batch(cfg, 64, 1500, [1] * 5, [1, 40, 200, 400, 65], seed=8).fill(scale=10.0)
    q = b.randn(b.rows, cfg.n_q_heads, cfg.head_dim)
    want, tol = b.attention(q)
    err = (b.attend(q).double() - want).abs()
    assert (err <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences_and_a_long_prefix(dtype):
    cfg = dbsa.DbsaConfig(8, 2, 128, dtype, 5e5)
    rng = np.random.default_rng(4)
    run_attention(cfg, 64, 6000, [1] * 70, rng.integers(1, 500, 70).tolist(), seed=9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_missing_pages_and_rows_that_see_nothing(dtype):
    cfg = config("g3", dtype)
    b = Batch(cfg, 16, 90, [1, 20, 1, 4], [50, 20, 16, 4], seed=10)
    b.fill()
    b.prefix_pages[2] = -1
    b.prefix_pages[3] = len(b.k_pages)
    b.page_table[0, 1] = -1
    b.page_table[1, 0] = -7
    q = b.randn(b.rows, 12, 128)
    want, tol = b.attention(q)
    check(b.attend(q), want, tol, dtype, "holes")
    b.prefix_pages.fill_(-1)
    b.page_table[2].fill_(-1)
    want, tol = b.attention(q)
    assert (want[21] == 0).all()
    got = b.attend(q)
    check(got, want, tol, dtype, "no prefix")
    assert (got[21] == 0).all()
    b.page_table.fill_(2 ** 31 - 1)
    assert (b.attend(q) == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pages_shared_between_tables(dtype):
    """Two sequences forked from one, a page twice in one table, and prefix pages
    as own pages: reads only, each as often as it is named."""
    cfg = config("g3", dtype)
    b = Batch(cfg, 32, 100, [1, 1, 2], [70, 70, 96], seed=20).fill()
    b.page_table[1, :2] = b.page_table[0, :2]
    b.page_table[2, 1] = b.page_table[2, 0]
    b.page_table[2, 2] = b.prefix_pages[0]
    q = b.randn(b.rows, 12, 128)
    want, tol = b.attention(q)
    check(b.attend(q), want, tol, dtype, "shared pages")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_queries_a_wide_table_and_a_scale(dtype):
    cfg = dbsa.DbsaConfig(8, 2, 128, dtype, 1e4, softmax_scale=0.2)
    b = Batch(cfg, 32, 100, [3, 1], [70, 40], seed=11, width=3).fill()
    wide = torch.full((2, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:5] = b.page_table
    b.page_table = wide[:, 2:5]
    q = b.randn(b.rows, 8 + 4, 128)[:, :8]
    want, tol = b.attention(q)
    check(b.attend(q, out=torch.full((4, 8, 128), float("nan"), dtype=b.dtype, device="cuda")),
          want, tol, dtype, "strided")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_repeats_bit_for_bit_and_a_row_does_not_depend_on_the_batch_values(dtype):
    cfg = config("gqa4", dtype)
    b, q, got = run_attention(cfg, 64, 900, [1] * 9, [30 * i + 1 for i in range(9)], seed=12)
    assert torch.equal(got, b.attend(q))
    other = q.clone()
    other[1:] = 3e4                         # the other sequences' queries
    assert torch.equal(b.attend(other)[0], got[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("long_one", [0, 70])
def test_more_sequences_than_one_scan_of_the_plan(dtype, long_one):
    """Over 256 sequences, with rows of one tile each, or one with several."""
    cfg = dbsa.DbsaConfig(4, 2, 64, dtype, 5e5)
    n_new = [i % 3 for i in range(300)]
    lens = [n + (i * 7) % 40 for i, n in enumerate(n_new)]
    if long_one:
        n_new[271], lens[271] = long_one, long_one + 5
    run_attention(cfg, 16, 150, n_new, lens, seed=30, spare_rows=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ranges_of_decreasing_length(dtype):
    """Enough own tokens for ranges of several lengths per CTA."""
    cfg = dbsa.DbsaConfig(16, 8, 64, dtype, 5e5)
    rng = np.random.default_rng(6)
    lens = rng.integers(3000, 6000, 48).tolist()
    units = sum(-(-n // 64) for n in lens) * 8
    assert units >= 64 * 296
    run_attention(cfg, 256, 300, [1] * 48, lens, seed=31)


def test_repeats_over_long_ragged_sequences():
    """Ragged ends in most tiles (V rows zeroed while later loads are in
    flight), several pieces per CTA: the same bits every time."""
    cfg = config("gqa4", "bf16")
    rng = np.random.default_rng(2)
    b = Batch(cfg, 128, 1511, [1] * 48, rng.integers(100, 3000, 48).tolist(), seed=18).fill()
    q = b.randn(b.rows, 32, 128)
    tables, ws = b.tables(), b.workspace()
    first = b.attend(q, tables=tables, workspace=ws)
    want, tol = b.attention(q)
    check(first, want, tol, "bf16", "long")
    out = torch.empty_like(first)
    for _ in range(30):
        assert torch.equal(b.attend(q, out=out, tables=tables, workspace=ws), first)


def test_offsets_beyond_32_bits():
    """Pages 2^31 elements apart (a view of one allocation)."""
    cfg = config("g5", "bf16")
    stride = 2 ** 31 + 64
    flat = torch.empty(2 * stride + 2 * 16 * 64, dtype=torch.bfloat16, device="cuda")
    b = Batch(cfg, 16, 16, [1], [16], seed=13)
    order = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    b.k_pages = flat.as_strided((3, 1, 16, 64), (stride, 1024, 64, 1), 0)
    b.v_pages = flat.as_strided((3, 1, 16, 64), (stride, 1024, 64, 1), 1024)
    b.prefix_pages, b.page_table = order[:1].contiguous(), order[1:].view(1, 1).contiguous()
    b.fill()
    b.append(b.randn(1, 1, 64), b.randn(1, 1, 64))
    q = b.randn(1, 5, 64)
    want, tol = b.attention(q)
    check(b.attend(q), want, tol, "bf16", "far pages")


def test_other_stream_and_two_calls_at_once():
    cfg = config("gqa4", "bf16")
    b = Batch(cfg, 64, 2000, [1] * 8, [20 * i + 5 for i in range(8)], seed=14).fill()
    q1, q2 = b.randn(8, 32, 128), b.randn(8, 32, 128)
    tables = b.tables()
    want1, want2 = b.attend(q1), b.attend(q2)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws1, ws2 = b.workspace(), b.workspace()
    o1, o2 = torch.empty_like(q1), torch.empty_like(q2)
    torch.cuda.synchronize()
    for _ in range(5):
        b.attend(q1, out=o1, tables=tables, workspace=ws1, stream=s1)
        b.attend(q2, out=o2, tables=tables, workspace=ws2, stream=s2)
    torch.cuda.synchronize()
    assert torch.equal(o1, want1) and torch.equal(o2, want2)


def test_captured_decode_step_follows_the_device_arrays():
    """append + attention captured once, replayed for lengths that grow and for
    a slot that goes idle."""
    cfg = config("gqa4", "bf16")
    n = 4
    b = Batch(cfg, 16, 500, [1] * n, [33, 70, 90, 16], seed=15, width=8)
    b.page_table.copy_(torch.arange(n * 8, dtype=torch.int32).view(n, 8))
    pool = torch.zeros((n * 8 + 40, 8, 16, 128), dtype=torch.bfloat16, device="cuda")
    b.k_pages, b.v_pages = pool.clone(), pool.clone()
    b.prefix_pages = torch.arange(n * 8, n * 8 + 32, dtype=torch.int32, device="cuda")
    b.fill()
    q, k, v = b.randn(n, 32, 128), b.randn(n, 8, 128), b.randn(n, 8, 128)
    tables, ws, out = b.tables(), b.workspace(), torch.empty_like(q)
    step = lambda: (b.append(k, v, tables=tables),
                    b.attend(q, out=out, tables=tables, workspace=ws))
    step()                                   # before capture, as callers do
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        b.lens = [x + 1 for x in b.lens]
        if i == 2:
            b.lens[1] = 0
        b.seq_lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        q.copy_(b.randn(n, 32, 128))
        k.copy_(b.randn(n, 8, 128))
        v.copy_(b.randn(n, 8, 128))
        graph.replay()
        want, tol = b.attention(q)
        check(out, want, tol, "bf16", "replay %d" % i)
        for s, ln in enumerate(b.lens):
            if ln:
                page, slot = int(b.page_table[s, (ln - 1) // 16]), (ln - 1) % 16
                assert torch.equal(b.v_pages[page, :, slot], v[s])


def test_fixed_icl_from_the_stage1_cache():
    """The demonstrations' contiguous pre-RoPE cache moved into pages, the
    prompts of three queries appended and attended to, then decode steps:
    each pass against the oracle's Stage 2 with every block selected."""
    cfg = dbsa.DbsaConfig(8, 2, 128, "bf16", 5e5)
    offs = np.array([0, 300, 410, 900], np.int32)
    T, page, hkv, d = 900, 64, 2, 128
    gen = torch.Generator().manual_seed(21)

    def randn(*shape):
        return torch.randn(shape, generator=gen).to(torch.bfloat16).cuda()

    kc, vc = randn(hkv, T + 20, d), randn(hkv, T + 20, d)     # cap > T
    prompts, n_seqs, width = [5, 17, 1], 3, 2
    n_prefix = -(-T // page)
    k_pages = torch.full((n_prefix + n_seqs * width, hkv, page, d), float("nan"),
                         dtype=torch.bfloat16, device="cuda")
    v_pages = torch.full_like(k_pages, float("nan"))
    i32 = dict(dtype=torch.int32, device="cuda")
    ids = torch.randperm(len(k_pages), generator=gen).to(torch.int32).cuda()
    prefix_pages, table = ids[:n_prefix].contiguous(), ids[n_prefix:].view(n_seqs, width).contiguous()
    n_pos = max(T + width * page, n_prefix * page)
    tables = torch.empty(dbsa.rope_tables_size(cfg, n_pos), dtype=torch.uint8, device="cuda")
    dbsa.rope_tables(cfg, n_pos, tables)
    # the prefix: rows of the head-major cache, appended as one sequence
    dbsa.paged_append(cfg, kc.transpose(0, 1)[:T], vc.transpose(0, 1)[:T], k_pages, v_pages,
                      prefix_pages.view(1, -1), torch.tensor([0, T], **i32),
                      torch.tensor([T], **i32), tables)
    lens = [0] * n_seqs
    k_own, v_own = [[] for _ in prompts], [[] for _ in prompts]
    for step in range(4):
        new = prompts if step == 0 else [1] * n_seqs
        lens = [a + b for a, b in zip(lens, new)]
        rows = sum(new)
        q, k, v = randn(rows, 8, d), randn(rows, hkv, d), randn(rows, hkv, d)
        row_ptr = torch.tensor([0] + list(np.cumsum(new)), **i32)
        seq_lens = torch.tensor(lens, **i32)
        out = torch.empty_like(q)
        ws = torch.empty(dbsa.shared_prefix_workspace_size(cfg, n_seqs, rows, T),
                         dtype=torch.uint8, device="cuda")
        dbsa.paged_append(cfg, k, v, k_pages, v_pages, table, row_ptr, seq_lens, tables, pos0=T)
        dbsa.shared_prefix_attend(cfg, q, k_pages, v_pages, prefix_pages, T, table, row_ptr,
                                  seq_lens, tables, out, ws)
        assert dbsa.read_status(ws) == dbsa.OK
        at = 0
        for s, n in enumerate(new):
            k_own[s].append(k[at:at + n])
            v_own[s].append(v[at:at + n])
            f = lambda x: x.float().cpu().numpy()
            want = oracle.stage2_all(f(kc[:, :T]), f(vc[:, :T]), offs, np.arange(3),
                                     f(q[at:at + n]), f(torch.cat(k_own[s])),
                                     f(torch.cat(v_own[s])), 5e5)
            got = out[at:at + n].float().cpu().numpy()
            # this reference holds unrotated keys: the cache's rounding of the
            # rotated keys is one more independent rounding of the scores
            rel = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert rel <= 8e-3, (step, s, rel)
            at += n



def test_expired_waits_are_reported_and_the_next_call_is_right():
    cfg = config("gqa4", "bf16")
    b = Batch(cfg, 64, 700, [1] * 5, [1, 40, 200, 400, 65], seed=17).fill()
    q = b.randn(b.rows, 32, 128)
    want, tol = b.attention(q)
    ws, tables = b.workspace(), b.tables()
    dbsa.test_wait_expiry(1_000_000)
    b.attend(q, tables=tables, workspace=ws)
    assert dbsa.read_status(ws) == dbsa.ERR_TIMEOUT
    out = b.attend(q, tables=tables, workspace=ws)
    assert dbsa.read_status(ws) == dbsa.OK
    check(out, want, tol, "bf16", "after an expired call")
