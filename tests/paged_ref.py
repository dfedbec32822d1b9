"""Plain fp64 reference of the paged append and the shared-prefix attention,
and a batch builder, for their tests.  Loops over sequences and heads; shares
no code with the library."""
from __future__ import annotations

import math

import torch


def rotate(x, pos, theta):
    """x [tokens][heads][d] fp64 rotated (rotate-half) at pos [tokens]."""
    d = x.shape[-1]
    w = theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device=x.device) / d)
    a = pos.double()[:, None] * w
    c, s = a.cos()[:, None], a.sin()[:, None]
    lo, hi = x[..., :d // 2], x[..., d // 2:]
    return torch.cat((lo * c - hi * s, hi * c + lo * s), -1)


class Batch:
    """A pool of NaN pages, and sequences of given lengths whose rows of this
    call are the last n_new[s] of lens[s] tokens; every page that a length
    reaches gets a page id of a random permutation."""

    def __init__(self, cfg, page, prefix_len, n_new, lens, seed=0, spare_rows=0, width=None,
                 interleaved=False, device="cuda"):
        self.cfg, self.page, self.prefix_len = cfg, page, prefix_len
        self.n_new, self.lens = list(n_new), list(lens)
        g = torch.Generator().manual_seed(seed)
        self.gen = g
        hkv, d = cfg.n_kv_heads, cfg.head_dim
        self.dtype = torch.float32 if cfg.dtype == "f32" else torch.bfloat16
        per = [-(-n // page) for n in self.lens]
        n_prefix = -(-prefix_len // page)
        self.width = width or max(1, max(per))
        n_pages = n_prefix + sum(per) + 3
        order = torch.randperm(n_pages, generator=g).to(torch.int32)
        if interleaved:     # one allocation, K and V pages alternating
            both = torch.full((n_pages, 2, hkv, page, d), float("nan"), dtype=self.dtype,
                              device=device)
            self.k_pages, self.v_pages = both[:, 0], both[:, 1]
        else:
            self.k_pages = torch.full((n_pages, hkv, page, d), float("nan"), dtype=self.dtype,
                                      device=device)
            self.v_pages = torch.full_like(self.k_pages, float("nan"))
        table = torch.full((len(self.lens), self.width), -1, dtype=torch.int32)
        at = n_prefix
        for s, n in enumerate(per):
            table[s, :n] = order[at:at + n]
            at += n
        row_ptr = torch.zeros(len(self.lens) + 1, dtype=torch.int32)
        row_ptr[1:] = torch.cumsum(torch.tensor(self.n_new), 0)
        self.rows = int(row_ptr[-1]) + spare_rows
        self.prefix_pages = order[:n_prefix].to(device)
        self.page_table = table.to(device)
        self.row_ptr = row_ptr.to(device)
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device=device)
        self.device = device

    def randn(self, *shape, scale=1.0):
        x = torch.randn(shape, generator=self.gen) * scale
        return x.to(self.dtype).to(self.device)

    def fill(self, scale=1.0):
        """Random keys and values in every slot a token lives in; the other
        slots keep their NaN."""
        self._fill(self.prefix_pages.tolist(), self.prefix_len, scale)
        for s, n in enumerate(self.lens):
            self._fill(self.page_table[s].tolist(), n, scale)
        return self

    def _fill(self, pages, n, scale):
        hkv, d = self.cfg.n_kv_heads, self.cfg.head_dim
        for j in range(-(-n // self.page)):
            m = min(self.page, n - j * self.page)
            if 0 <= pages[j] < len(self.k_pages):
                self.k_pages[pages[j], :, :m] = self.randn(hkv, m, d, scale=scale)
                self.v_pages[pages[j], :, :m] = self.randn(hkv, m, d)

    def gather(self, pages, n, c):
        """(keys, values, present) of the first n tokens of a page list, fp64."""
        idx = torch.arange(n, device=self.device)
        p = torch.as_tensor(pages, device=self.device).long()[idx // self.page]
        ok = (p >= 0) & (p < len(self.k_pages))
        q = p.clamp(0, len(self.k_pages) - 1)
        return (self.k_pages[q, c, idx % self.page].double(),
                self.v_pages[q, c, idx % self.page].double(), ok)

    def attention(self, q):
        """(outputs, worst-case tolerances) for query rows q, fp64; rows of no
        sequence are NaN."""
        cfg = self.cfg
        hkv, d = cfg.n_kv_heads, cfg.head_dim
        g = cfg.n_q_heads // hkv
        scale = cfg.softmax_scale if cfg.softmax_scale > 0 else 1.0 / math.sqrt(d)
        # Rounding of the rotated query and of the probabilities, relative (half
        # a step), then the output's own.  fp32 sums of D or n terms add less
        # than (D + 8) 2^-24 of the absolute sum to a score, and n 2^-24 to a
        # mean of n values.
        half = torch.finfo(torch.bfloat16).eps / 2 if cfg.dtype != "f32" else 0.0
        f32 = 2.0 ** -24
        out = torch.full(q.shape, float("nan"), dtype=torch.float64, device=q.device)
        tol = torch.zeros_like(out)
        row = 0
        for s, (n, ln) in enumerate(zip(self.n_new, self.lens)):
            for c in range(hkv):
                kp, vp, okp = self.gather(self.prefix_pages, self.prefix_len, c)
                ko, vo, oko = self.gather(self.page_table[s], ln, c)
                k, v, ok = torch.cat([kp, ko]), torch.cat([vp, vo]), torch.cat([okp, oko])
                k, v = torch.where(ok[:, None], k, 0.0), torch.where(ok[:, None], v, 0.0)
                for i in range(n):
                    t = ln - n + i
                    cols = slice(c * g, (c + 1) * g)
                    if t < 0:
                        out[row + i, cols] = 0
                        continue
                    m = self.prefix_len + t + 1
                    see = ok[:m]
                    if not see.any():
                        out[row + i, cols] = 0
                        continue
                    pos = torch.full((1,), self.prefix_len + t, device=q.device)
                    qr = rotate(q[row + i, cols].double()[None], pos, cfg.rope_theta)[0]
                    sc = (qr @ k[:m].T) * scale
                    p = torch.softmax(sc.masked_fill(~see, -math.inf), -1)
                    o = p @ v[:m]
                    # scores move by at most e_j: p_j by a factor e^{+-2 max e}
                    # around its mean, the output by sum p_j (e^{e_j} - 1)
                    # |v_j - o| e^{max e}
                    e = (qr.abs() @ k[:m].abs().T) * scale * (half + (d + 8) * f32)
                    e = torch.where(see, e, 0.0)
                    dev = (v[:m][None] - o[:, None]).abs()
                    move = ((p * torch.expm1(e))[:, :, None] * dev).sum(1) * e.amax(-1).exp()[:, None]
                    spread = p @ v[:m].abs()
                    out[row + i, cols] = o
                    tol[row + i, cols] = (move + spread * (half + (m + 16) * f32)
                                          + o.abs() * (half + 2 * f32) + 1e-30)
            row += n
        return out, tol

    def tables(self):
        from many_shot_icl_b200 import dbsa
        n_pos = self.prefix_len + self.width * self.page
        t = torch.empty(dbsa.rope_tables_size(self.cfg, n_pos), dtype=torch.uint8,
                        device=self.device)
        dbsa.rope_tables(self.cfg, n_pos, t)
        return t

    def workspace(self):
        from many_shot_icl_b200 import dbsa
        n = dbsa.shared_prefix_workspace_size(self.cfg, len(self.lens), self.rows, self.prefix_len)
        return torch.full((n,), 0xFF, dtype=torch.uint8, device=self.device)   # NaN everywhere

    def attend(self, q, out=None, tables=None, workspace=None, stream=None):
        from many_shot_icl_b200 import dbsa
        if out is None:
            out = torch.full(q.shape, float("nan"), dtype=q.dtype, device=q.device)
        ws = self.workspace() if workspace is None else workspace
        dbsa.shared_prefix_attend(self.cfg, q, self.k_pages, self.v_pages, self.prefix_pages,
                                  self.prefix_len, self.page_table, self.row_ptr, self.seq_lens,
                                  self.tables() if tables is None else tables, out, ws,
                                  stream=stream)
        if workspace is None:
            assert dbsa.read_status(ws) == dbsa.OK
        return out

    def append(self, k, v, tables=None, stream=None):
        from many_shot_icl_b200 import dbsa
        dbsa.paged_append(self.cfg, k, v, self.k_pages, self.v_pages, self.page_table,
                          self.row_ptr, self.seq_lens, self.tables() if tables is None else tables,
                          pos0=self.prefix_len, stream=stream)


# Relative Frobenius bound: the worst-case roundings above, taken as independent
# and uniform (half / sqrt(3) rms each): rotated query (it moves scores by half /
# sqrt(3) of their own spread, which is below ~1 for N(0, 1) inputs),
# probabilities, output; root of the sum of squares 3.9e-3 for bf16, times 1.5.
# fp32: a score's error grows like sqrt(D) 2^-24, far below 1e-5.
REL_FRO = {"bf16": 6e-3, "f32": 1e-5}


def check(got, want, tol, dtype, what=""):
    """Every element inside its own worst case, and the whole inside REL_FRO;
    NaN exactly where the reference has it."""
    got = got.double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), what + ": rows written or missing"
    err = torch.where(nan, 0.0, (got - torch.where(nan, 0.0, want))).abs()
    over = err > tol
    assert not over.any(), "%s: %d elements beyond their bound, worst %.3e" % (
        what, int(over.sum()), float((err / tol.clamp(min=1e-30))[over].max()))
    norm = torch.where(nan, 0.0, want).norm()
    if norm > 0:
        rel = float(err.norm() / norm)
        assert rel <= REL_FRO[dtype], "%s: relative error %.2e" % (what, rel)
