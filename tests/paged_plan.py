"""How a shared-prefix attention call is cut into items and pieces, in plain
integers: a second writing of the split, for tests that need to know that the
shape they run reaches what they are about (several key tiles to a piece, more
items than CTAs).  Results never depend on it."""
from __future__ import annotations

N_CTAS = 2 * 148
OWN_WAVES, MAX_WAVES = 5, 8


class Plan:
    def __init__(self, cfg, prefix_len, n_new, lens):
        self.hkv, self.g = cfg.n_kv_heads, cfg.n_q_heads // cfg.n_kv_heads
        self.rows = rows = sum(n_new) * self.g
        f32 = cfg.dtype == "f32"
        self.tile_keys = 64
        self.prefix_tiles = -(-prefix_len // 64)
        self.tile_rows = 128
        if f32:
            self.tile_rows = 16
            while (self.tile_rows < 64 and
                   -(-rows // self.tile_rows) * (self.prefix_tiles + 1) * self.hkv > N_CTAS):
                self.tile_rows *= 2
        self.row_tiles = -(-rows // self.tile_rows)
        self.units = self.hkv * self.prefix_tiles
        self.groups = self._groups(cfg.head_dim) if prefix_len else 0
        self.own = []            # (first unit, tiles, rows) of each own-token entry
        at = 0
        for n, ln in zip(n_new, lens):
            for r0 in range(0, n * self.g, self.tile_rows):
                last = min(r0 + self.tile_rows, n * self.g) - 1
                seen = min(ln, ln - n + 1 + last // self.g)
                tiles = -(-seen // 64) if seen > 0 else 0
                self.own.append((at, tiles, last + 1 - r0))
                at += tiles * self.hkv
        self.own_units = at

    def _groups(self, d):
        best, best_time = 1, 0.0

        def consider(n):
            nonlocal best, best_time
            n = min(max(n, 1), self.units)
            waves = -(-n * self.row_tiles // N_CTAS)
            time = (waves * (self.units / n * 1.4 + 4.0)
                    + 0.17e-3 * (n + self.hkv) * self.rows * d / 128)
            if best_time == 0 or time < 0.99 * best_time:
                best, best_time = n, time

        cut = 64
        while cut > 1:
            consider(N_CTAS // self.row_tiles // cut)
            cut //= 2
        for w in range(1, min(self.row_tiles, MAX_WAVES) + 1):
            consider(w * N_CTAS // self.row_tiles)
        return best

    @property
    def prefix_items(self):
        return self.groups * self.row_tiles

    def prefix_pieces(self):
        """Key tiles (first, end) of each (range, KV head) piece."""
        out = []
        for j in range(self.groups):
            u, end = j * self.units // self.groups, (j + 1) * self.units // self.groups
            while u < end:
                kt0 = u % self.prefix_tiles
                n = min(self.prefix_tiles - kt0, end - u)
                out.append((kt0, kt0 + n))
                u += n
        return out

    @property
    def guided(self):
        return self.own_units >= 64 * N_CTAS

    def own_ranges(self):
        u = self.own_units
        if not self.guided:
            n = min(OWN_WAVES * N_CTAS, max(u // 4, min(u, N_CTAS)))
            return [(i * u // n, (i + 1) * u // n) for i in range(n)]
        cuts = [u * s // 16 for s in (0, 8, 12, 14, 15, 16)]
        return [(a + i * (b - a) // N_CTAS, a + (i + 1) * (b - a) // N_CTAS)
                for a, b in zip(cuts, cuts[1:]) for i in range(N_CTAS)]

    def own_pieces(self):
        """Key tiles and rows (first, end, rows) of each own-token piece."""
        out, e = [], 0
        flat = [(at + c * tiles, tiles, rows) for at, tiles, rows in self.own if tiles
                for c in range(self.hkv)]
        for u, end in self.own_ranges():
            while u < end:
                while flat[e][0] + flat[e][1] <= u:
                    e += 1
                kt0 = u - flat[e][0]
                n = min(flat[e][1] - kt0, end - u)
                out.append((kt0, kt0 + n, flat[e][2]))
                u += n
        return out
