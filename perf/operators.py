"""Two operators of many-shot serving, measured: appending keys and values to
a paged cache with RoPE applied on the way, and attention for a batch of
sequences that share one long prefix (the encoded demonstrations) and keep
their own tokens in pages of the same cache.

A pool holds pages [n_pages][Hkv][page][D] of keys (rotated) and values.  A
sequence's own tokens sit at positions prefix, prefix + 1, ...; entry j of its
row of the page table names the page of its tokens [j * page, (j + 1) * page).
Row r of the batch belongs to sequence s with row_ptr[s] <= r < row_ptr[s + 1]
and is the token seq_lens[s] - (row_ptr[s + 1] - r) of it; rows for which that
is negative are padding (nothing is appended for them, their output is 0).
Rows behind row_ptr[n_seqs] are left as they were.

Each case is one call of one operator.  `run` computes it with elementary
torch operations, or, with `own`, by the library's entry points.
"""
import math

import torch

own = False

LLAMA31 = dict(hq=32, hkv=8, d=128, dtype="bf16", theta=5e5)
LLAMA2 = dict(hq=32, hkv=32, d=128, dtype="bf16", theta=1e4)
TINY = dict(hq=2, hkv=1, d=64, dtype="f32", theta=1e4)


def _case(name, op, heads, prefix, seqs, new, have, page, source="projection", idle=0, spare=0):
    """new, have: (lowest, highest) count of new rows and of tokens already
    present per sequence; idle: every idle-th sequence is padding; spare: rows
    behind the last sequence."""
    return dict(name=name, op=op, **heads, prefix=prefix, seqs=seqs, new_lo=new[0], new_hi=new[1],
                have_lo=have[0], have_hi=have[1], page=page, source=source, idle=idle, spare=spare)


def listed():
    return [
        # one generated token of one query: latency
        _case("append decode 1", "append", LLAMA31, 90223, 1, (1, 1), (40, 40), 64),
        # a decode step of a batch, each sequence at its own length
        _case("append decode 64", "append", LLAMA31, 90223, 64, (1, 1), (15, 700), 64, spare=3),
        # the prompts of a batch of short test questions
        _case("append prompt 64", "append", LLAMA31, 90223, 64, (15, 45), (0, 0), 64),
        # the encoded demonstrations moved from the contiguous cache into pages
        _case("append prefix 90k", "append", LLAMA31, 0, 1, (90223, 90223), (0, 0), 64, "cache"),
        # fp32, a few tokens of the smallest workload
        _case("append tiny f32", "append", TINY, 397, 3, (8, 16), (0, 9), 16),
        # the smallest attention: one short fp32 prompt over a few demonstrations
        _case("attend tiny f32", "attend", TINY, 397, 1, (16, 16), (0, 0), 16),
        # one query generating after 90k tokens of demonstrations
        _case("attend decode 1", "attend", LLAMA31, 90223, 1, (1, 1), (40, 40), 64),
        # a decode step of the headline batch, some slots of the batch idle
        _case("attend decode 64", "attend", LLAMA31, 90223, 64, (1, 1), (15, 160), 64, idle=13),
        # a decode step of the stress batch
        _case("attend decode 256", "attend", LLAMA31, 128364, 256, (1, 1), (15, 45), 64),
        # the prompt pass of the headline batch: the largest case
        _case("attend prompt 64", "attend", LLAMA31, 90223, 64, (15, 45), (0, 0), 64, spare=5),
        # long private histories behind a prefix of one block of demonstrations
        _case("attend decode 48 long", "attend", LLAMA31, 1511, 48, (1, 1), (500, 8000), 128),
        # multi-head attention (no shared heads), small pages
        _case("attend decode 16 mha", "attend", LLAMA2, 30074, 16, (1, 1), (15, 300), 16),
    ]


_LARGEST = dict(hq=32, d=128, rows=1920, keys=90300)


def draw(rng):
    """One call somewhere in the range the listed cases span."""
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attend", "attend"])
    hq, hkv, d = rng.choice([(32, 8, 128), (32, 32, 128), (8, 2, 128), (2, 1, 64), (16, 2, 64),
                             (12, 4, 128), (5, 1, 64)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    page = rng.choice([16, 32, 64, 128, 256])
    seqs = log_int(1, 256)
    prefix = 0 if rng.random() < 0.1 else log_int(1, 128364)
    new_lo = new_hi = 1
    if rng.random() < 0.4:
        new_lo = log_int(1, 64)
        new_hi = new_lo + rng.randrange(0, 64)
    have_lo = 0 if rng.random() < 0.3 else log_int(1, 2000)
    have_hi = have_lo + log_int(1, 6000)
    source, idle = rng.choice(["projection", "cache"]), 0
    if op == "append":
        if rng.random() < 0.3:   # a long prefix or chunk into one or two tables
            seqs, prefix = rng.choice([1, 2]), 0
            new_lo = new_hi = log_int(1000, 45000)
            have_lo, have_hi = 0, rng.randrange(0, 2000)
    else:
        idle = rng.choice([0, 0, 7])
    # no dearer than the largest listed case, in operations and in memory
    most = 4.0 * _LARGEST["hq"] * _LARGEST["d"] * _LARGEST["rows"] * _LARGEST["keys"]
    if dtype == "f32":
        most /= 64
    while (op == "attend" and 4.0 * hq * d * seqs * new_hi * (prefix + have_hi + new_hi) > most
           or 4.0 * seqs * hkv * (have_hi + new_hi + page) * d > 2e9
           or op == "attend" and 4.0 * seqs * hq * new_hi * (have_hi + new_hi + page) > 8e9):
        if seqs > 1:
            seqs = (seqs + 1) // 2
        else:
            prefix, have_hi = prefix // 2, max(have_lo, have_hi // 2)
    return dict(op=op, hq=hq, hkv=hkv, d=d, dtype=dtype, theta=5e5, prefix=prefix, seqs=seqs,
                new_lo=new_lo, new_hi=new_hi, have_lo=have_lo, have_hi=have_hi, page=page,
                source=source, idle=idle, spare=rng.choice([0, 0, 1, 6]))


def _lengths(case):
    """Per sequence: its rows in the batch and its length with them."""
    new, lens = [], []
    for i in range(case["seqs"]):
        n = case["new_lo"] + (i * 7919 + 13) % (case["new_hi"] - case["new_lo"] + 1)
        have = case["have_lo"] + (i * 104729 + 7) % (case["have_hi"] - case["have_lo"] + 1)
        padding = case["idle"] > 0 and i % case["idle"] == case["idle"] - 1
        new.append(n)
        lens.append(0 if padding else have + n)
    return new, lens


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    hq, hkv, d, page, prefix = case["hq"], case["hkv"], case["d"], case["page"], case["prefix"]
    dt = _dtype(case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)

    def pool(n):
        """A page pool, filled one slice at a time (the fp32 draw of a whole
        pool would double its footprint)."""
        p = torch.empty((n, hkv, page, d), device=dev, dtype=dt)
        for part in p.split(max(1, (1 << 26) // (hkv * page * d))):
            part.copy_(torch.randn(part.shape, generator=g, device=dev, dtype=torch.float32))
        return p

    new, lens = _lengths(case)
    row_ptr = [0]
    for n in new:
        row_ptr.append(row_ptr[-1] + n)
    total, rows = row_ptr[-1], row_ptr[-1] + case["spare"]
    attend = case["op"] == "attend"
    n_prefix = -(-prefix // page) if attend else 0
    per_seq = [-(-n // page) for n in lens]
    width = max(1, max(per_seq))
    n_pages = n_prefix + sum(per_seq) + 2
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    starts, at = [], n_prefix
    for n in per_seq:
        starts.append(at)
        at += n
    col = torch.arange(width, device=dev)
    count = torch.tensor(per_seq, device=dev)[:, None]
    first = torch.tensor(starts, device=dev)[:, None]
    table = torch.where(col < count, order[(first + col).clamp(max=n_pages - 1)], -1)
    st = dict(case=dict(case), total=total, max_new=max(new),
              k_pages=pool(n_pages), v_pages=pool(n_pages),
              page_table=table.to(torch.int32).contiguous(),
              row_ptr=torch.tensor(row_ptr, device=dev, dtype=torch.int32),
              seq_lens=torch.tensor(lens, device=dev, dtype=torch.int32))
    if attend:
        # queries and outputs of a model's attention layer; what the spare rows
        # hold stays, so it has the size of an average over many values
        st["q"] = randn(rows, hq, d)
        st["out"] = randn(rows, hq, d) * 2.0 ** -8
        st["prefix_pages"] = order[:n_prefix].contiguous()
    elif case["source"] == "cache":
        # rows [0, rows) of a contiguous head-major cache with room behind them
        st["k"], st["v"] = (randn(hkv, rows + 5, d)[:, :rows].transpose(0, 1) for _ in range(2))
    else:
        # the key and value columns of a fused projection's output
        qkv = randn(rows, hq + 2 * hkv, d)
        st["k"], st["v"] = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    if own:
        # what a serving program keeps beside its cache: angle tables, scratch
        from many_shot_icl_b200 import dbsa
        cfg = dbsa.DbsaConfig(hq, hkv, d, case["dtype"], case["theta"])
        n_pos = prefix + width * page
        st["cfg"] = cfg
        st["tables"] = torch.empty(dbsa.rope_tables_size(cfg, n_pos), dtype=torch.uint8, device=dev)
        dbsa.rope_tables(cfg, n_pos, st["tables"])
        if attend:
            st["workspace"] = torch.empty(
                dbsa.shared_prefix_workspace_size(cfg, case["seqs"], rows, prefix),
                dtype=torch.uint8, device=dev)
    return st


def _rotate(x, pos, theta):
    """Rotate-half RoPE of x [rows][heads][d] (any dtype) at pos [rows], in fp32
    with the angles taken in fp64."""
    d = x.shape[-1]
    w = theta ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    angle = pos.double()[:, None] * w
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    lo, hi = x[..., :d // 2].float(), x[..., d // 2:].float()
    return torch.cat((lo * c - hi * s, hi * c + lo * s), dim=-1)


def _rows(st):
    """Sequence and own-token index of each row that belongs to a sequence."""
    r = torch.arange(st["total"], device=st["row_ptr"].device, dtype=torch.int32)
    seq = torch.searchsorted(st["row_ptr"], r, right=True) - 1
    return seq, st["seq_lens"][seq] - st["row_ptr"][seq + 1] + r


def _append_plain(st):
    case = st["case"]
    n, page = st["total"], case["page"]
    seq, tok = _rows(st)
    to = st["page_table"][seq, tok // page].long()
    slot = (tok % page).long()
    st["k_pages"][to, :, slot] = _rotate(st["k"][:n], case["prefix"] + tok,
                                         case["theta"]).to(st["k_pages"].dtype)
    st["v_pages"][to, :, slot] = st["v"][:n]
    return st["k_pages"], st["v_pages"]


def _softmax_parts(scores, values):
    """(row maximum, sum of exponentials, exponentials times values)."""
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m.clamp(min=-3e38)).exp_()
    return m, p.sum(-1, keepdim=True), p @ values


def _attend_plain(st):
    case = st["case"]
    hq, hkv, d, page, prefix = case["hq"], case["hkv"], case["d"], case["page"], case["prefix"]
    g, n, n_seqs, max_new = hq // hkv, st["total"], case["seqs"], st["max_new"]
    seq, tok = _rows(st)
    u = torch.arange(n, device=seq.device) - st["row_ptr"][seq]
    q = _rotate(st["q"][:n], prefix + tok, case["theta"]) * (1.0 / math.sqrt(d))
    # every sequence's own keys, padded to the width of the page table
    width = st["page_table"].shape[1]
    own_pages = st["page_table"].clamp(min=0).long()
    k = st["k_pages"][own_pages].float().permute(0, 2, 1, 3, 4).reshape(n_seqs, hkv, width * page, d)
    v = st["v_pages"][own_pages].float().permute(0, 2, 1, 3, 4).reshape(n_seqs, hkv, width * page, d)
    qs = torch.zeros((n_seqs, max_new, hkv, g, d), device=q.device)
    qs[seq, u] = q.view(n, hkv, g, d)
    s = qs.permute(0, 2, 1, 3, 4).reshape(n_seqs, hkv, max_new * g, d) @ k.transpose(-1, -2)
    last = torch.full((n_seqs, max_new), -1, device=q.device, dtype=torch.int32)
    last[seq, u] = tok
    seen = torch.arange(width * page, device=q.device) <= last[:, :, None]
    s = s.view(n_seqs, hkv, max_new, g, -1).masked_fill_(~seen[:, None, :, None], -math.inf)
    m2, l2, o2 = _softmax_parts(s.view(n_seqs, hkv, max_new * g, -1), v)
    m2, l2, o2 = (x.view(n_seqs, hkv, max_new, g, -1)[seq, :, u] for x in (m2, l2, o2))
    if prefix > 0:
        pages = st["prefix_pages"].long()
        k = st["k_pages"][pages].float().transpose(0, 1).reshape(hkv, -1, d)[:, :prefix]
        v = st["v_pages"][pages].float().transpose(0, 1).reshape(hkv, -1, d)[:, :prefix]
        qp = q.view(n, hkv, g, d).transpose(0, 1).reshape(hkv, n * g, d)
        m1, l1, o1 = (x.view(hkv, n, g, -1).transpose(0, 1)
                      for x in _softmax_parts(qp @ k.transpose(-1, -2), v))
        m = torch.maximum(m1, m2)
        f1, f2 = (m1 - m).exp(), (m2 - m).exp()
        l2, o2 = l1 * f1 + l2 * f2, o1 * f1 + o2 * f2
    o = torch.where((tok >= 0)[:, None, None, None], o2 / l2, 0.0)
    st["out"][:n] = o.reshape(n, hq, d).to(st["out"].dtype)
    return st["out"]


def run(st):
    case = st["case"]
    if own:
        from many_shot_icl_b200 import dbsa
        if case["op"] == "append":
            dbsa.paged_append(st["cfg"], st["k"], st["v"], st["k_pages"], st["v_pages"],
                              st["page_table"], st["row_ptr"], st["seq_lens"], st["tables"],
                              pos0=case["prefix"])
            return st["k_pages"], st["v_pages"]
        dbsa.shared_prefix_attend(st["cfg"], st["q"], st["k_pages"], st["v_pages"],
                                  st["prefix_pages"], case["prefix"], st["page_table"],
                                  st["row_ptr"], st["seq_lens"], st["tables"], st["out"],
                                  st["workspace"])
        return st["out"]
    return _append_plain(st) if case["op"] == "append" else _attend_plain(st)


def work(case):
    new, lens = _lengths(case)
    live = [(n, ln) for n, ln in zip(new, lens) if ln > 0]
    elt = 4 if case["dtype"] == "f32" else 2
    kv_row = 2 * case["hkv"] * case["d"] * elt          # one token's key and value
    rows = sum(n for n, _ in live)
    if case["op"] == "append":
        # read and write every new key and value; 3 operations per rotated element
        return {"bytes": 2.0 * rows * kv_row, "flops": 3.0 * rows * case["hkv"] * case["d"]}
    keys = case["prefix"] + sum(ln for _, ln in live)
    pairs = sum(n * case["prefix"] + n * (ln - n) + n * (n + 1) // 2 for n, ln in live)
    return {"bytes": float(keys * kv_row + 2 * sum(new) * case["hq"] * case["d"] * elt),
            "flops": 4.0 * case["hq"] * case["d"] * pairs}


def _turn(x, pos, theta):
    """x [tokens][heads][d] in fp64, rotated as complex numbers."""
    d = x.shape[-1]
    freq = torch.tensor([theta ** (-2.0 * i / d) for i in range(d // 2)], dtype=torch.float64,
                        device=x.device)
    z = torch.complex(x[..., :d // 2], x[..., d // 2:])
    z = z * torch.polar(torch.ones_like(freq), freq * pos[:, None].double())[:, None]
    return torch.cat((z.real, z.imag), dim=-1)


def exact(case, seed):
    st = prepare(case, seed)
    new, lens = _lengths(case)
    page, prefix, hkv, d = case["page"], case["prefix"], case["hkv"], case["d"]
    g = case["hq"] // hkv
    dev = st["row_ptr"].device
    if case["op"] == "append":
        kp, vp = st.pop("k_pages").double(), st.pop("v_pages").double()
        row = 0
        for s, (n, ln) in enumerate(zip(new, lens)):
            t = torch.arange(ln - n, ln, device=dev)
            k, v = st["k"][row:row + n].double(), st["v"][row:row + n].double()
            k = _turn(k, prefix + t, case["theta"])
            for j in range((ln - n) // page, (ln - 1) // page + 1):
                a, b = max(j * page, ln - n), min((j + 1) * page, ln)
                p = int(st["page_table"][s, j]) if case["seqs"] > 1 else st["page_table"][s, j].long()
                kp[p, :, a - j * page:b - j * page] = k[a - ln + n:b - ln + n].transpose(0, 1)
                vp[p, :, a - j * page:b - j * page] = v[a - ln + n:b - ln + n].transpose(0, 1)
            row += n
        return kp, vp
    out = st["out"].double()
    tables = st["page_table"].tolist()
    for c in range(hkv):
        pk = st["k_pages"][st["prefix_pages"].long(), c].double().reshape(-1, d)[:prefix]
        pv = st["v_pages"][st["prefix_pages"].long(), c].double().reshape(-1, d)[:prefix]
        row = 0
        for s, (n, ln) in enumerate(zip(new, lens)):
            if ln == 0:
                out[row:row + n] = 0
            else:
                pages = tables[s][:-(-ln // page)]
                k = torch.cat([pk, st["k_pages"][pages, c].double().reshape(-1, d)[:ln]])
                v = torch.cat([pv, st["v_pages"][pages, c].double().reshape(-1, d)[:ln]])
                t = prefix + torch.arange(ln - n, ln, device=dev)
                q = _turn(st["q"][row:row + n, c * g:(c + 1) * g].double(), t, case["theta"])
                sc = torch.einsum("ngd,kd->ngk", q, k) / math.sqrt(d)
                hidden = torch.arange(prefix + ln, device=dev) > t[:, None]
                w = torch.softmax(sc.masked_fill(hidden[:, None], -math.inf), dim=-1)
                out[row:row + n, c * g:(c + 1) * g] = torch.einsum("ngk,kd->ngd", w, v)
            row += n
    return out
