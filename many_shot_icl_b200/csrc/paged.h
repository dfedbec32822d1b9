// Internal declarations of the paged cache and the shared-prefix attention:
// the batch as the kernels see it, the device-built plan, and how the work is
// cut into pieces.  Not part of the public ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "dbsa_internal.h"

namespace dbsa {

struct PagedPool {
  void *k, *v;
  int64_t page_stride;    // elements
  int32_t n_pages, page_size, page_shift;   // page_size = 1 << page_shift
  int32_t Hkv;
};

struct PagedBatch {
  const int32_t *row_ptr, *seq_lens, *page_table;
  int32_t n_seqs, n_rows, table_width, table_stride;
  int32_t cap;            // table_width * page_size
};

// The rows of one sequence in the batch and its own length with them; n = 0
// when its row_ptr entries are not rows of the batch.
struct SeqRows {
  int32_t row0, n, len;
};
__device__ __forceinline__ SeqRows seq_rows(const PagedBatch &b, int s) {
  SeqRows r;
  r.row0 = __ldg(b.row_ptr + s);
  const int32_t e = __ldg(b.row_ptr + s + 1);
  r.n = (r.row0 >= 0 && e <= b.n_rows && e > r.row0) ? e - r.row0 : 0;
  r.len = __ldg(b.seq_lens + s);
  if (r.len < 0 || r.len > b.cap) r.len = 0;
  return r;
}

// The sequence of a row and its own token there; sequence -1 for a row of none,
// a negative token for padding.
struct RowToken {
  int32_t seq, token;
  SeqRows rows;
};
// A decode step has one row per sequence in order, so row r is tried as
// sequence r (all three loads at once) before the search.
__device__ __forceinline__ RowToken row_token(const PagedBatch &b, int row) {
  RowToken t;
  t.seq = min(row, b.n_seqs - 1);
  t.rows = seq_rows(b, t.seq);
  if (row < t.rows.row0 || row >= t.rows.row0 + t.rows.n) {
    int lo = 0, hi = b.n_seqs;   // the first sequence that ends past the row
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(b.row_ptr + mid + 1) > row) hi = mid; else lo = mid + 1;
    }
    t.seq = lo < b.n_seqs ? lo : -1;
    if (lo < b.n_seqs) t.rows = seq_rows(b, lo);
    if (row < t.rows.row0 || row >= t.rows.row0 + t.rows.n) t.seq = -1;
  }
  t.token = t.rows.len - t.rows.n + (row - t.rows.row0);
  return t;
}

// ---- the plan of one attention call ----
//
// Query rows are packed per KV head: packed row r * g + hl is the batch's row
// r, local head hl.  The prefix is attended to by tiles of tile_rows packed
// rows, whichever sequences they belong to; own tokens by tiles that do not
// straddle a sequence.  Keys are counted in tiles of tile_keys.
//
// Prefix: the Hkv * prefix_tiles (KV head, key tile) units are cut into
// n_groups equal ranges, and each (range, row tile) is one item; the n_row_tiles
// items of a range are next to each other, so that they run at the same time
// and read its keys from memory once.
// Own tokens: the units of all (sequence, row tile, KV head) entries, in that
// order, are cut into ranges (OwnRanges), each an item.
// A CTA starts with the item of its own number; the others go to whichever CTA
// is free next (a ticket counter), since the SMs do not get equal shares of the
// memory's bandwidth.  What an item computes does not depend on who runs it.
//
// Every (item, KV head or entry) intersection is a piece: it leaves one partial
// (row maximum, sum of exponentials, weighted values) per row.
// Piece (head c, range j) of the prefix keeps packed row p at partial row
// (c + j) * rows + p: c + j is unique along the ranges, because from one piece
// to the next either the head or the range moves on.  The piece of own-token
// entry e in range i starts at own_base + first(e) + own_stride * i, where
// first(e) counts the rows of the entries before it: again unique, since a next
// piece adds either the rows of e or own_stride, which is no less.
struct PlanHead {
  int64_t units;           // own-token units, all entries
  int32_t n_entries;
  int32_t single;          // no sequence has more than one row tile: entry s is sequence s
  int32_t ticket;          // items taken beyond the first of each CTA
};
// One (sequence, row tile) of the own tokens, and the key-tile units (all heads)
// before it; one more record at the end holds their sum.  All that a piece needs,
// in one read.
struct alignas(16) Entry {
  int32_t seq, rt, row0, n;   // row0, n, len: of the sequence (SeqRows)
  int64_t units;
  int32_t len, pad;
};
struct AttendPlan {
  int32_t g, Hkv, D;
  int32_t tile_rows, tile_keys;
  int32_t rows;            // packed rows per KV head: n_rows * g
  int32_t n_row_tiles;     // ceil(rows / tile_rows)
  int32_t prefix_len, prefix_tiles;
  int32_t n_groups;        // ranges of the prefix
  int32_t n_ctas;
  int32_t own_ranges;      // at most
  int32_t own_stride;      // rows an own-token entry has at most
  int32_t max_entries;     // own-token (sequence, row tile) entries, at most
  int64_t own_base;        // first own-token partial row
  // device
  PlanHead *head;
  int4 *row_info;          // [n_rows]: row_token(): sequence, token, its first row, its rows
  int32_t *first_entry;    // [n_seqs + 1]
  Entry *entry;            // [max_entries + 1]
  void *q_rot;             // [Hkv][rows][D], cfg->dtype, rotated
  float *acc;              // [partial rows][D], not normalised
  float2 *ml;              // [partial rows]: (maximum in log2 units, sum)
};

// One piece: rows of a tile against key tiles [kt0, kt1) of one list of pages.
struct Piece {
  int32_t c;               // KV head
  int32_t row0, n_rows;    // packed rows
  int32_t kt0, kt1;
  int32_t n_keys;          // keys of the list that exist
  int32_t see0;            // row i sees keys below see0 + (off + i) / g, and n_keys
  int32_t off;
  int32_t shared;          // the prefix (1) or own tokens (0)
  const int32_t *pages;
  int64_t partial;         // partial row of the piece's first row
};

// The smallest j with floor((j + 1) * total / parts) > x, i.e. the part of
// [0, total) cut into `parts` ranges that holds x.  (In 32 bits where it can be:
// a 64-bit division costs ~100 instructions, and the merge kernel had ten.)
__device__ __forceinline__ int64_t part_of(int64_t x, int64_t parts, int64_t total) {
  const uint64_t y = (uint64_t)(x + 1) * (uint64_t)parts - 1;
  if (((uint64_t)total * (uint64_t)parts) >> 32 == 0) return (uint32_t)y / (uint32_t)total;
  return (int64_t)(y / (uint64_t)total);
}

// How the own-token units are cut into ranges.  No range may be empty, because
// the merge reads a partial of every range from a row's first to its last.
// Long: kOwnWaves ranges per CTA, long ones first (8/16 of the units in n_ctas
// ranges, then 4/16, 2/16, 1/16 and 1/16), so that there are few pieces and the
// CTAs still end together.  Short: equal ranges of four units at least, unless
// that leaves CTAs without work.
constexpr int kOwnWaves = 5;
struct OwnRanges {
  int64_t units, n;        // n ranges in all
  int32_t n_ctas;
  bool guided;

  __device__ __forceinline__ OwnRanges(const AttendPlan &p, int64_t units_)
      : units(units_), n_ctas(p.n_ctas) {
    guided = units >= 64 * (int64_t)n_ctas;
    n = guided ? (int64_t)kOwnWaves * n_ctas
               : min((int64_t)kOwnWaves * n_ctas, max(units / 4, min(units, (int64_t)n_ctas)));
  }
  // First unit of wave w: 16ths 0, 8, 12, 14, 15, 16.
  __device__ __forceinline__ int64_t wave(int w) const {
    return units * (16 - (w < 5 ? 16 >> w : 0)) / 16;
  }
  __device__ __forceinline__ int64_t begin(int64_t i) const {
    if (!guided) return i * units / n;
    const int w = (int)(i / n_ctas);
    if (w >= kOwnWaves) return units;
    const int64_t u = wave(w);
    return u + i % n_ctas * (wave(w + 1) - u) / n_ctas;
  }
  // The range that holds unit u.
  __device__ __forceinline__ int64_t of(int64_t u) const {
    if (!guided) return part_of(u, n, units);
    int w = 0;
    while (w + 1 < kOwnWaves && wave(w + 1) <= u) ++w;
    const int64_t u0 = wave(w);
    return (int64_t)w * n_ctas + part_of(u - u0, n_ctas, wave(w + 1) - u0);
  }
};

// Walks the pieces of one item in order.
struct PieceWalk {
  int64_t u, uend;         // units still to emit
  int32_t j, rt, e;        // range, row tile (prefix), entry (own tokens)
  bool own;

  // Items of the prefix are known from the call's arguments, without the plan
  // in device memory.
  static __device__ __forceinline__ bool is_shared(const AttendPlan &p, int64_t item) {
    return item < (int64_t)p.n_groups * p.n_row_tiles;
  }

  // Starts an item; false if there is none of that number.  Run by whole warps.
  __device__ bool start(const AttendPlan &p, int64_t item) {
    own = !is_shared(p, item);
    if (!own) {
      j = (int32_t)(item / p.n_row_tiles);
      rt = (int32_t)(item % p.n_row_tiles);
      const int64_t total = (int64_t)p.Hkv * p.prefix_tiles;
      u = j * total / p.n_groups;
      uend = (j + 1) * total / p.n_groups;
      return true;
    }
    item -= (int64_t)p.n_groups * p.n_row_tiles;
    const OwnRanges r(p, p.head->units);
    if (item >= r.n) return false;
    j = (int32_t)item;
    u = r.begin(item);
    uend = r.begin(item + 1);
    // the first entry that ends past u, 32 tries at a time
    int lo = 0, hi = p.head->n_entries;
    for (;;) {
      const int step = (hi - lo + 31) / 32;
      const int at = min(lo + ((int)(threadIdx.x & 31) + 1) * step, hi);
      const int first = __ffs(__ballot_sync(~0u, p.entry[at].units > u)) - 1;
      lo += first * step;
      if (step == 1) break;
      hi = min(lo + step, hi);
    }
    e = lo;
    return true;
  }

  // The next piece of the item; false if it has no more.
  __device__ bool next(const AttendPlan &p, const PagedBatch &b, const int32_t *prefix_pages,
                       Piece &o) {
    if (u >= uend) return false;
    if (!own) {
      o.c = (int32_t)(u / p.prefix_tiles);
      o.kt0 = (int32_t)(u % p.prefix_tiles);
      const int64_t n = min((int64_t)(p.prefix_tiles - o.kt0), uend - u);
      o.kt1 = o.kt0 + (int32_t)n;
      u += n;
      o.row0 = rt * p.tile_rows;
      o.n_rows = min(p.tile_rows, p.rows - o.row0);
      o.n_keys = p.prefix_len;
      o.see0 = p.prefix_len;
      o.off = 0;
      o.shared = 1;
      o.pages = prefix_pages;
      o.partial = (int64_t)(o.c + j) * p.rows + o.row0;
      return true;
    }
    Entry en = p.entry[e];
    int64_t last = p.entry[e + 1].units;
    while (last <= u) {
      en = p.entry[++e];
      last = p.entry[e + 1].units;
    }
    const int32_t tiles = (int32_t)(last - en.units) / p.Hkv;
    const int32_t rem = (int32_t)(u - en.units);
    o.c = rem / tiles;
    o.kt0 = rem % tiles;
    const int64_t n = min((int64_t)(tiles - o.kt0), uend - u);
    o.kt1 = o.kt0 + (int32_t)n;
    u += n;
    o.off = en.rt * p.tile_rows;
    o.row0 = en.row0 * p.g + o.off;
    o.n_rows = min(p.tile_rows, en.n * p.g - o.off);
    o.n_keys = en.len;
    o.see0 = en.len - en.n + 1;
    o.shared = 0;
    o.pages = b.page_table + (int64_t)en.seq * b.table_stride;
    o.partial = p.own_base + (int64_t)p.Hkv * o.row0 + (int64_t)o.c * o.n_rows +
                (int64_t)p.own_stride * j;
    return true;
  }
};

// Keys row i of a piece may see (it sees keys below the result).
__device__ __forceinline__ int32_t keys_seen(const Piece &p, int g, int i) {
  return p.shared ? p.n_keys : min(p.n_keys, p.see0 + (p.off + i) / g);
}

// Where rope_cs8() finds position p in tables laid out by rope_rows_at(): its rows
// of cosines are every second row of D / 2.
__device__ __forceinline__ int64_t rope_row_pos(int64_t p) {
  return (p >> kRopeShift << (kRopeShift + 1)) | (p & (kRopeLo - 1));
}

struct AttendArgs {
  PagedPool pool;
  PagedBatch batch;
  AttendPlan plan;
  const int32_t *prefix_pages;
  const void *q;
  int64_t q_row_stride;
  void *out;
  RopeTables rope;
  float scale_log2;
  int *status;
  uint64_t wait_limit_ns;
  int32_t withhold_tiles;
};

}  // namespace dbsa
