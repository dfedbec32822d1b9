// Paged cache: the append kernel, the attention call's preparation and merge
// kernels, and the C entry points.
//
// The cache holds keys already rotated at their positions (the Stage-1 cache
// holds them unrotated): a token's position in the shared prefix or behind it
// never changes, so its key is rotated once, when it is appended, and every
// later attention call streams it as it is.
#include <cuda_bf16.h>

#include <algorithm>

#include "dbsa_internal.h"
#include "paged.h"
#include "paged_attn.h"
#include "vec8.cuh"

namespace dbsa {
namespace {

// 8 consecutive elements from fp32 registers, rounded to nearest even once.
__device__ __forceinline__ void store8(bf16 *p, const float (&f)[8]) { store8_bf16(p, f); }
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// 8 consecutive elements, bit for bit.
template <typename T>
struct Raw8 {
  uint4 x[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) x[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void store(T *p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(p)[i] = x[i];
  }
};

// ------------------------------------------------------------------- append
// k'[i] = k[i] cos(pos w_i) - k[i + D/2] sin(pos w_i), k'[i + D/2] = k[i +
// D/2] cos + k[i] sin; v is copied.  Every element is read and written once:
// the kernel is bound by memory (long appends) or by the latency of its chain
// row -> sequence -> page -> store (decode steps).  Measured, 8 heads of 128,
// bf16, in short runs: 90 223 tokens from the head-major cache 118 us (6.3 TB/s
// read and written, 0.96 of the copy bandwidth; 123 us, 0.92, back to back at the
// power limit), 64 single tokens 2.6 us.  A block takes 256 / (D/16)
// rows of one KV head; a thread 8 rotation pairs of the row's key and the
// matching 16 elements of its value.
template <typename T>
struct AppendArgs {
  const T *k, *v;
  int64_t k_row, k_head, v_row, v_head;
  PagedPool pool;
  PagedBatch batch;
  int64_t pos0;
  RopeTables rope;
};

template <int D, typename T>
__global__ void __launch_bounds__(256) append_kernel(const AppendArgs<T> a) {
  pdl_enter();
  constexpr int H = D / 2, CP = H / 8;
  const int c = blockIdx.x % a.pool.Hkv;
  const int row = (blockIdx.x / a.pool.Hkv) * (256 / CP) + threadIdx.x / CP;
  const int i0 = (threadIdx.x % CP) * 8;
  if (row >= a.batch.n_rows) return;
  // key and value are requested before the slot they go to is known
  const T *ks = a.k + row * a.k_row + c * a.k_head, *vs = a.v + row * a.v_row + c * a.v_head;
  float lo[8], hi[8];
  Raw8<T> v_lo, v_hi;
  load8(ks + i0, lo);
  load8(ks + H + i0, hi);
  v_lo.load(vs + i0);
  v_hi.load(vs + H + i0);
  const RowToken t = row_token(a.batch, row);
  if (t.seq < 0 || t.token < 0) return;
  const int page = __ldg(a.batch.page_table + (int64_t)t.seq * a.batch.table_stride +
                         (t.token >> a.pool.page_shift));
  if (page < 0 || page >= a.pool.n_pages) return;
  float cs[8], sn[8];
  rope_cs8(a.rope, rope_row_pos(a.pos0 + t.token), i0, H, cs, sn);
  rotate8(lo, hi, cs, sn);
  const int64_t dst =
      page * a.pool.page_stride +
      ((int64_t)c * a.pool.page_size + (t.token & (a.pool.page_size - 1))) * D + i0;
  T *kd = static_cast<T *>(a.pool.k) + dst, *vd = static_cast<T *>(a.pool.v) + dst;
  store8(kd, lo);
  store8(kd + H, hi);
  v_lo.store(vd);
  v_hi.store(vd + H);
}

// ------------------------------------------------------------ attention: plan
// Exclusive prefix sum over the block's 256 threads; *total gets the sum.
__device__ int64_t block_scan(int64_t x, int64_t *total) {
  __shared__ int64_t warp_sum[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(~0u, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) before += warp_sum[w];
    all += warp_sum[w];
  }
  __syncthreads();
  *total = all;
  return before + inc - x;
}

// Units of one row tile of a sequence: the key tiles its last row sees, for
// every KV head.
__device__ __forceinline__ int64_t tile_units(const AttendPlan &p, const SeqRows &s, int rt) {
  const int64_t last = min((int64_t)(rt + 1) * p.tile_rows, (int64_t)s.n * p.g) - 1;
  const int64_t seen = min((int64_t)s.len, s.len - s.n + 1 + last / p.g);
  return seen > 0 ? (seen + p.tile_keys - 1) / p.tile_keys * p.Hkv : 0;
}

// The own-token entries and their units, by one block.
__device__ void build_plan(const AttendPlan &p, const PagedBatch &b) {
  const int tid = threadIdx.x;
  int64_t at = 0, units = 0, total;
  SeqRows s = {0, 0, 0};
  int more = 0;   // whether a sequence has several row tiles
  for (int s0 = 0; s0 < b.n_seqs; s0 += 256) {
    if (s0 + tid < b.n_seqs) {
      s = seq_rows(b, s0 + tid);
      more |= (int64_t)s.n * p.g > p.tile_rows;
    }
  }
  const int single = !__syncthreads_or(more);
  if (single) {   // entry = sequence (decode steps, short prompts): one pass
    for (int s0 = 0; s0 < b.n_seqs; s0 += 256) {
      const int e = s0 + tid;
      int64_t n = 0;
      if (e < b.n_seqs) {
        if (b.n_seqs > 256) s = seq_rows(b, e);
        if (s.n > 0) n = tile_units(p, s, 0);
      }
      const int64_t first = units + block_scan(n, &total);
      if (e < b.n_seqs) p.entry[e] = {e, 0, s.row0, s.n, first, s.len, 0};
      units += total;
    }
    at = b.n_seqs;
  } else {
    for (int s0 = 0; s0 < b.n_seqs; s0 += 256) {
      const int i = s0 + tid;
      int64_t n = 0;
      if (i < b.n_seqs) n = ((int64_t)seq_rows(b, i).n * p.g + p.tile_rows - 1) / p.tile_rows;
      const int64_t first = at + block_scan(n, &total);
      // more entries than max_entries need a decreasing row_ptr; none is written
      if (i < b.n_seqs) p.first_entry[i] = (int32_t)min(first, (int64_t)p.max_entries);
      at += total;
    }
    at = min(at, (int64_t)p.max_entries);
    if (tid == 0) p.first_entry[b.n_seqs] = (int32_t)at;
    __syncthreads();
    for (int e0 = 0; e0 < at; e0 += 256) {
      const int e = e0 + tid;
      int64_t n = 0;
      int32_t seq = 0, rt = 0;
      if (e < at) {
        int lo = 0, hi = b.n_seqs;   // the first sequence whose entries end past e
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (p.first_entry[mid + 1] > e) hi = mid; else lo = mid + 1;
        }
        seq = lo;
        rt = e - p.first_entry[lo];
        s = seq_rows(b, lo);
        n = tile_units(p, s, rt);
      }
      const int64_t first = units + block_scan(n, &total);
      if (e < at) p.entry[e] = {seq, rt, s.row0, s.n, first, s.len, 0};
      units += total;
    }
  }
  if (tid == 0) {
    p.entry[at].units = units;
    *p.head = {units, (int32_t)at, single, 0};
  }
}

// Queries rotated at their positions and packed per KV head (one rounding to
// the cache's type), the row table, the status word and (last block) the plan.
// Latency: two dependent reads and a store, ~2.5 us for a decode step; the
// attention kernel's prefix loads run meanwhile.
template <int D, typename T>
__global__ void __launch_bounds__(256) attend_prep_kernel(const AttendArgs a) {
  pdl_enter();
  constexpr int H = D / 2, CP = H / 8;
  const AttendPlan &p = a.plan;
  if (blockIdx.x == gridDim.x - 1) {
    if (threadIdx.x < kStatusBytes / 4) a.status[threadIdx.x] = 0;
    build_plan(p, a.batch);
    return;
  }
  const int c = blockIdx.x % p.Hkv;
  const int row = (blockIdx.x / p.Hkv) * (256 / CP) + threadIdx.x / CP;
  const int cp = threadIdx.x % CP, i0 = cp * 8;
  if (row >= a.batch.n_rows) return;
  const T *src = static_cast<const T *>(a.q) + row * a.q_row_stride + (int64_t)c * p.g * D + i0;
  T *dst = static_cast<T *>(p.q_rot) + ((int64_t)c * p.rows + (int64_t)row * p.g) * D + i0;
  // two heads at a time, the first two requested before the row's position
  float lo[2][8], hi[2][8], cs[8], sn[8];
  auto load = [&](int hl) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (hl + k < p.g) {
        load8(src + (int64_t)(hl + k) * D, lo[k]);
        load8(src + (int64_t)(hl + k) * D + H, hi[k]);
      }
  };
  load(0);
  const RowToken t = row_token(a.batch, row);
  if (c == 0 && cp == 0) p.row_info[row] = make_int4(t.seq, t.token, t.rows.row0, t.rows.n);
  const bool live = t.seq >= 0 && t.token >= 0;   // other rows: finite, never used
  rope_cs8(a.rope, rope_row_pos(live ? (int64_t)p.prefix_len + t.token : 0), i0, H, cs, sn);
  for (int hl = 0; hl < p.g; hl += 2) {
    if (hl > 0) load(hl);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (hl + k >= p.g) break;
      rotate8(lo[k], hi[k], cs, sn);
      if (!live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) lo[k][e] = hi[k][e] = 0.f;
      }
      store8(dst + (int64_t)(hl + k) * D, lo[k]);
      store8(dst + (int64_t)(hl + k) * D + H, hi[k]);
    }
  }
}

// ----------------------------------------------------------- attention: merge
// out = sum_i 2^(m_i - M) acc_i / sum_i 2^(m_i - M) l_i over the row's pieces,
// M = max m_i, in fp32.  Many pieces (W > 1): W warps per (row, head), which take
// the pieces in turn and meet in shared memory.  Few (W = 1): a warp per (row, KV
// head) does its g heads one after the other, the record of the row read once.
// Four warps a block, four pieces in flight per warp, lanes hold the columns.
// Bound by the latency of its chain of reads (L2): the row's record -> its entry
// -> the own partials; the prefix's partials are known from the arguments and are
// read meanwhile.  W follows the pieces that the prefix leaves a row (4 over 12, 2
// over 8); those of its own tokens are not counted, since the host does not know
// them, so that a row with a long history and little prefix has few warps.  With
// W = 4 throughout, 256 rows of 32 heads with 7 pieces each took 34 us; a warp per
// (row, head) took 50 us for 2 000 rows of 32 heads with 2 or 3.  But few rows (one
// warp per scheduler or less) leave the SMs idle while a warp does its heads in
// turn: 42 rows of 32 heads took 10.8 us with W = 1, 6.0 with 2.
constexpr int kMergeWarps = 4;
constexpr int kFewMergeRows = 4 * 148;

template <int D, typename T, int W>
__global__ void __launch_bounds__(32 * kMergeWarps) attend_merge_kernel(const AttendArgs a) {
  pdl_enter();
  constexpr int V = D / 32;   // columns per lane
  const AttendPlan &p = a.plan;
  const int heads = W == 1 ? p.Hkv : p.Hkv * p.g;   // units of work per row
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W, sub = (threadIdx.x >> 5) / W;
  const int rh = min((int)blockIdx.x * (kMergeWarps / W) + sub,
                     a.batch.n_rows * heads - 1);   // the last ones may be done twice
  const int row = rh / heads, c = W == 1 ? rh % heads : rh % heads / p.g;
  const int hl0 = W == 1 ? 0 : rh % heads % p.g, hl1 = W == 1 ? p.g : hl0 + 1;
  const int4 info = p.row_info[row];
  const PlanHead head = *p.head;

  float m, L, acc[V];   // of this warp's pieces of a head, acc and L relative to m
  // pieces first + i * step, i = i0, i0 + W, .. < n
  auto add = [&](int64_t first, int64_t step, int i0, int n) {
    for (int i = i0; i < n; i += 4 * W) {
      float2 ml[4];
      float x[4][V];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        ml[k] = make_float2(-INFINITY, 0.f);
        const int ii = i + k * W;
        if (ii < n) {
          const int64_t r = first + ii * step;
          ml[k] = p.ml[r];
          const float *src = p.acc + r * D + lane * V;
          if constexpr (V == 4) {
            const float4 y = *reinterpret_cast<const float4 *>(src);
            x[k][0] = y.x;
            x[k][1] = y.y;
            x[k][2] = y.z;
            x[k][3] = y.w;
          } else {
            const float2 y = *reinterpret_cast<const float2 *>(src);
            x[k][0] = y.x;
            x[k][1] = y.y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] = 0.f;
        }
      }
      const float mn = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), m);
      const float mu = mn == -INFINITY ? 0.f : mn, f = exp2f(m - mu);
      L *= f;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] *= f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float w = exp2f(ml[k].x - mu);
        L += w * ml[k].y;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += w * x[k][e];
      }
      m = mn;
    }
  };

  // pieces of the prefix: n1, of local head hl from f1 + hl
  int n1 = 0;
  int64_t f1 = 0;
  if (p.n_groups > 0) {
    const int64_t total = (int64_t)p.Hkv * p.prefix_tiles, u0 = (int64_t)c * p.prefix_tiles;
    const int64_t j0 = part_of(u0, p.n_groups, total);
    n1 = (int)(part_of(u0 + p.prefix_tiles - 1, p.n_groups, total) - j0) + 1;
    f1 = (c + j0) * p.rows + (int64_t)row * p.g;
  }
  // of the own tokens, in the row tile of local row `local`: n2 from f2
  const bool live = info.x >= 0 && info.y >= 0;
  int rt_of = -1, n2 = 0;
  int64_t f2 = 0;
  auto own = [&](int hl) {
    const int32_t local = (row - info.z) * p.g + hl, rt = local / p.tile_rows;
    if (rt != rt_of) {
      rt_of = rt;
      n2 = 0;
      const int64_t e = head.single ? info.x : (int64_t)p.first_entry[info.x] + rt;
      if (e < head.n_entries) {
        const int64_t u0 = p.entry[e].units;
        const int32_t tiles = (int32_t)(p.entry[e + 1].units - u0) / p.Hkv;
        if (tiles > 0) {
          const OwnRanges r(p, head.units);
          const int64_t i0 = r.of(u0 + (int64_t)c * tiles);
          n2 = (int)(r.of(u0 + (int64_t)(c + 1) * tiles - 1) - i0) + 1;
          const int32_t tile0 = rt * p.tile_rows, n_rows = min(p.tile_rows, info.w * p.g - tile0);
          f2 = p.own_base + (int64_t)p.Hkv * (info.z * p.g + tile0) + c * n_rows +
               p.own_stride * i0 - tile0;   // + local: the row
        }
      }
    }
    if (n2 > 0)   // the warps go on in turn after the prefix's pieces
      add(f2 + local, p.own_stride, (warp + W - n1 % W) % W, n2);
  };

  if constexpr (W == 1) {
    if (info.x < 0) return;   // a row of no sequence: left as it was
    T *out = static_cast<T *>(a.out) + ((int64_t)row * p.Hkv + c) * p.g * D + lane * V;
#pragma unroll 2
    for (int hl = hl0; hl < hl1; ++hl) {
      m = -INFINITY;
      L = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = 0.f;
      if (live) {
        add(f1 + hl, p.rows, 0, n1);
        own(hl);
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;   // 0: padding, or nothing seen
      T y[V];
#pragma unroll
      for (int e = 0; e < V; ++e) from_f32(acc[e] * inv, y[e]);
      if constexpr (sizeof(y) == 16)
        *reinterpret_cast<uint4 *>(out + hl * D) = *reinterpret_cast<uint4 *>(y);
      else if constexpr (sizeof(y) == 8)
        *reinterpret_cast<uint2 *>(out + hl * D) = *reinterpret_cast<uint2 *>(y);
      else
        *reinterpret_cast<uint32_t *>(out + hl * D) = *reinterpret_cast<uint32_t *>(y);
    }
  } else {
    __shared__ float shared[kMergeWarps][D + 2];
    float (*sh)[D + 2] = shared + sub * W;
    m = -INFINITY;
    L = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
    add(f1 + hl0, p.rows, warp, n1);
    if (live) own(hl0);
#pragma unroll
    for (int e = 0; e < V; ++e) sh[warp][lane * V + e] = acc[e];
    if (lane == 0) {
      sh[warp][D] = L;
      sh[warp][D + 1] = m;
    }
    __syncthreads();
    if (info.x < 0) return;
    float M = sh[0][D + 1];
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, sh[w][D + 1]);
    const float mu = M == -INFINITY ? 0.f : M;
    T *out = static_cast<T *>(a.out) + (int64_t)rh * D;
    for (int d = warp * 32 + lane; d < D; d += 32 * W) {
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float f = exp2f(sh[w][D + 1] - mu);
        num += f * sh[w][d];
        den += f * sh[w][D];
      }
      from_f32(live && den > 0.f ? num / den : 0.f, out[d]);
    }
  }
}

// ---------------------------------------------------------------- host side
size_t align_up(size_t x) { return (x + 255) / 256 * 256; }

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Positions [0, n) a table buffer of that many bytes covers.
int64_t table_positions(const dbsa_config *cfg, size_t bytes) {
  const int64_t n_hi =
      (int64_t)(bytes / (sizeof(float) * (size_t)cfg->head_dim)) - kRopeLo;
  return n_hi > 0 ? n_hi * kRopeLo : 0;
}

dbsa_status check_paged(const dbsa_config *cfg, const dbsa_paged_cache *cache,
                        const dbsa_paged_batch *b, int64_t pos0, const void *tables,
                        size_t tables_bytes, PagedPool *pool, PagedBatch *batch,
                        RopeTables *rope) {
  dbsa_status s = check_cfg(cfg);
  if (s != DBSA_OK) return s;
  if (!cache || !b) return fail(DBSA_ERR_INVALID_ARG, "cache or batch is NULL");
  if (!cache->k_pages || !cache->v_pages || !b->row_ptr || !b->seq_lens || !b->page_table ||
      !tables)
    return fail(DBSA_ERR_INVALID_ARG, "a tensor pointer is NULL");
  if (!aligned16(cache->k_pages) || !aligned16(cache->v_pages) || !aligned16(tables))
    return fail(DBSA_ERR_INVALID_ARG, "pages and tables must be 16-byte aligned");
  if (((reinterpret_cast<uintptr_t>(b->row_ptr) | reinterpret_cast<uintptr_t>(b->seq_lens) |
        reinterpret_cast<uintptr_t>(b->page_table)) & 3u) != 0)
    return fail(DBSA_ERR_INVALID_ARG, "row_ptr, seq_lens and page_table must be 4-byte aligned");
  const int ps = cache->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256)
    return fail(DBSA_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256 (got %d)", ps);
  if (cache->n_pages < 1) return fail(DBSA_ERR_INVALID_ARG, "n_pages must be >= 1");
  const int64_t page = (int64_t)cfg->n_kv_heads * ps * cfg->head_dim;
  if (cache->page_stride < page || cache->page_stride % 8 != 0)
    return fail(DBSA_ERR_INVALID_ARG,
                "page_stride must be a multiple of 8 and at least %lld (got %lld)",
                (long long)page, (long long)cache->page_stride);
  if (cache->page_stride > (int64_t(1) << 36))
    return fail(DBSA_ERR_INVALID_ARG, "page_stride too large");
  if (b->n_seqs < 1 || b->n_seqs > 65535)
    return fail(DBSA_ERR_INVALID_ARG, "n_seqs must be 1..65535 (got %d)", b->n_seqs);
  if (b->n_rows < 1 || b->n_rows > (1 << 30))
    return fail(DBSA_ERR_INVALID_ARG, "n_rows must be 1..2^30 (got %d)", b->n_rows);
  if (b->table_width < 1 || b->table_stride < b->table_width)
    return fail(DBSA_ERR_INVALID_ARG, "need 1 <= table_width <= table_stride");
  const int64_t own_cap = (int64_t)b->table_width * ps;
  // (key tiles of a sequence, times the heads, are counted in 32 bits)
  if (pos0 < 0 || pos0 > (1 << 30) || own_cap > (1 << 30) ||
      own_cap / 16 * cfg->n_kv_heads > INT32_MAX)
    return fail(DBSA_ERR_INVALID_ARG, "sequences too long");
  if (table_positions(cfg, tables_bytes) < pos0 + own_cap)
    return fail(DBSA_ERR_INVALID_ARG, "tables cover %lld positions, the batch can reach %lld",
                (long long)table_positions(cfg, tables_bytes), (long long)(pos0 + own_cap));
  pool->k = cache->k_pages;
  pool->v = cache->v_pages;
  pool->page_stride = cache->page_stride;
  pool->n_pages = cache->n_pages;
  pool->page_size = ps;
  pool->page_shift = ps == 16 ? 4 : ps == 32 ? 5 : ps == 64 ? 6 : ps == 128 ? 7 : 8;
  pool->Hkv = cfg->n_kv_heads;
  batch->row_ptr = b->row_ptr;
  batch->seq_lens = b->seq_lens;
  batch->page_table = b->page_table;
  batch->n_seqs = b->n_seqs;
  batch->n_rows = b->n_rows;
  batch->table_width = b->table_width;
  batch->table_stride = b->table_stride;
  batch->cap = (int32_t)own_cap;
  *rope = rope_rows_at(static_cast<const float *>(tables), cfg->head_dim);
  return DBSA_OK;
}

// How many ranges the prefix is cut into: the number for which waves of the CTAs
// x (key tiles of an item + a piece's own cost) + the partials' traffic is least,
// with the bf16 kernel's measured costs at D = 128: a key tile takes a CTA ~1.4 us
// (32 KB at its share of the memory, or 128 rows' arithmetic at the power limit),
// starting and ending a piece ~4 us, writing and merging the partials of a row
// ~0.17 ns x D / 128 of all CTAs' time.  fp32 calls are cut by the same costs,
// although a tile of 64 rows takes a CTA of their kernel ~20 us: they are not split
// as finely as they could be where they have few key tiles.  (More, shorter ranges
// would also even out the SMs' unequal speeds, but behind 90k tokens one row tile
// takes 69 us with one wave, 75 with two.)
constexpr int kMaxWaves = 8;
int prefix_groups(int rows, int n_row_tiles, int n_ctas, int Hkv, int D, int64_t units) {
  constexpr double kTile = 1.4, kPiece = 4.0, kRow = 0.17e-3;   // us
  int best = 1;
  double best_time = 0;
  auto consider = [&](int64_t groups) {
    groups = std::min<int64_t>(std::max<int64_t>(groups, 1), units);
    const double waves = (double)((groups * n_row_tiles + n_ctas - 1) / n_ctas);
    const double time = waves * ((double)units / (double)groups * kTile + kPiece) +
                        kRow * (double)(groups + Hkv) * rows * D / 128;
    if (best_time == 0 || time < 0.99 * best_time) {
      best = (int)groups;
      best_time = time;
    }
  };
  for (int cut = 64; cut > 1; cut /= 2) consider(n_ctas / n_row_tiles / cut);   // part of a wave
  for (int64_t w = 1; w <= std::min(n_row_tiles, kMaxWaves); ++w)
    consider(w * n_ctas / n_row_tiles);
  return best;
}

struct AttendLayout {
  AttendPlan p;
  size_t head, row_info, first_entry, entry, q_rot, acc, ml, total;
};
AttendLayout attend_layout(const dbsa_config *cfg, int32_t n_seqs, int32_t n_rows,
                           int64_t prefix_len) {
  const int rows = n_rows * (cfg->n_q_heads / cfg->n_kv_heads);
  const AttendShape shape = attend_shape(cfg, rows, prefix_len);
  AttendLayout l{};
  AttendPlan &p = l.p;
  p.g = cfg->n_q_heads / cfg->n_kv_heads;
  p.Hkv = cfg->n_kv_heads;
  p.D = cfg->head_dim;
  p.tile_rows = shape.tile_rows;
  p.tile_keys = shape.tile_keys;
  p.n_ctas = shape.n_ctas;
  p.rows = rows;
  p.n_row_tiles = (p.rows + p.tile_rows - 1) / p.tile_rows;
  p.prefix_len = (int32_t)prefix_len;
  p.prefix_tiles = (int32_t)((prefix_len + p.tile_keys - 1) / p.tile_keys);
  p.n_groups = prefix_len == 0 ? 0
                               : prefix_groups(p.rows, p.n_row_tiles, p.n_ctas, p.Hkv, p.D,
                                               (int64_t)p.Hkv * p.prefix_tiles);
  p.max_entries = n_seqs + p.rows / p.tile_rows;
  p.own_base = prefix_len == 0 ? 0 : (int64_t)(p.Hkv + p.n_groups) * p.rows;
  p.own_ranges = kOwnWaves * p.n_ctas;
  p.own_stride = std::min(p.tile_rows, p.rows);
  // Space is taken for at least what any smaller call needs, so that a workspace
  // made for the largest batch serves them all: prefix_groups() is not monotone,
  // nor is the choice of tile_rows.
  const int64_t units = (int64_t)p.Hkv * p.prefix_tiles, rows64 = rows;
  const int64_t prefix_rows =   // of n_groups * rows
      units == 0 ? 0
                 : std::max(rows64, std::min({units * rows64, p.n_ctas * rows64,
                                              (int64_t)kMaxWaves * p.n_ctas * shape.max_tile_rows}));
  const int64_t partial_rows =
      (int64_t)p.Hkv * rows * (units == 0 ? 1 : 2) + prefix_rows +
      (int64_t)std::min(shape.max_tile_rows, rows) * p.own_ranges;
  const size_t max_entries = (size_t)n_seqs + rows / shape.min_tile_rows;
  const size_t elt = cfg->dtype == DBSA_F32 ? 4 : 2;
  size_t off = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t o = align_up(off);
    off = o + bytes;
    return o;
  };
  l.head = take(sizeof(PlanHead));
  l.row_info = take((size_t)n_rows * sizeof(int4));
  l.first_entry = take(((size_t)n_seqs + 1) * sizeof(int32_t));
  l.entry = take((max_entries + 1) * sizeof(Entry));
  l.q_rot = take((size_t)p.Hkv * p.rows * p.D * elt);
  l.acc = take((size_t)partial_rows * p.D * sizeof(float));
  l.ml = take((size_t)partial_rows * sizeof(float2));
  l.total = align_up(off);
  return l;
}

// n_rows * g and the partial rows stay far inside 32 and 64 bits.
dbsa_status check_attend_size(const dbsa_config *cfg, int32_t n_seqs, int32_t n_rows,
                              int64_t prefix_len) {
  if (n_seqs < 1 || n_seqs > 65535)
    return fail(DBSA_ERR_INVALID_ARG, "n_seqs must be 1..65535 (got %d)", n_seqs);
  if (n_rows < 1 || (int64_t)n_rows * cfg->n_q_heads > (1 << 28))
    return fail(DBSA_ERR_INVALID_ARG, "n_rows must be 1..%d (got %d)",
                (1 << 28) / cfg->n_q_heads, n_rows);
  if (prefix_len < 0 || prefix_len > (1 << 30))
    return fail(DBSA_ERR_INVALID_ARG, "prefix_len must be 0..2^30");
  return DBSA_OK;
}

template <int D, typename T>
cudaError_t launch_attend_t(const AttendArgs &a, cudaStream_t st) {
  constexpr int RPB = 256 / (D / 16);
  const int64_t blocks = (int64_t)((a.batch.n_rows + RPB - 1) / RPB) * a.plan.Hkv + 1;
  cudaError_t e = pdl_launch(attend_prep_kernel<D, T>, dim3((unsigned)blocks), dim3(256), 0, st, a);
  if (e != cudaSuccess) return e;
  {
    ProfileScope prof(st);
    e = launch_attend_pieces(a, D, sizeof(T) == 4, st);
  }
  if (e != cudaSuccess) return e;
  // a row's pieces of the prefix: those of the ranges that its head meets
  const int pieces = a.plan.n_groups / a.plan.Hkv + 2;
  auto merge = [&](auto kernel, int w) {
    const int64_t rows = (int64_t)a.batch.n_rows * a.plan.Hkv * (w == 1 ? 1 : a.plan.g);
    const int per = kMergeWarps / w;
    return pdl_launch(kernel, dim3((unsigned)((rows + per - 1) / per)), dim3(32 * kMergeWarps), 0,
                      st, a);
  };
  if (pieces > 12) return merge(attend_merge_kernel<D, T, 4>, 4);
  if (pieces > 8 || (int64_t)a.batch.n_rows * a.plan.Hkv <= kFewMergeRows)
    return merge(attend_merge_kernel<D, T, 2>, 2);
  return merge(attend_merge_kernel<D, T, 1>, 1);
}

template <int D, typename T>
cudaError_t launch_append_t(const void *k, const void *v, const int64_t (&str)[4],
                            const PagedPool &pool, const PagedBatch &batch, int64_t pos0,
                            const RopeTables &rope, cudaStream_t st) {
  constexpr int RPB = 256 / (D / 16);
  AppendArgs<T> a;
  a.k = static_cast<const T *>(k);
  a.v = static_cast<const T *>(v);
  a.k_row = str[0];
  a.k_head = str[1];
  a.v_row = str[2];
  a.v_head = str[3];
  a.pool = pool;
  a.batch = batch;
  a.pos0 = pos0;
  a.rope = rope;
  const int64_t blocks = (int64_t)((batch.n_rows + RPB - 1) / RPB) * pool.Hkv;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return pdl_launch(append_kernel<D, T>, dim3((unsigned)blocks), dim3(256), 0, st, a);
}

}  // namespace
}  // namespace dbsa

using namespace dbsa;

extern "C" {

size_t dbsa_rope_tables_size(const dbsa_config *cfg, int64_t n_pos) {
  if (check_cfg(cfg) != DBSA_OK) return 0;
  if (n_pos < 1 || n_pos > (int64_t(1) << 31)) {
    fail(DBSA_ERR_INVALID_ARG, "n_pos must be 1..2^31");
    return 0;
  }
  return rope_table_bytes((int32_t)((n_pos + kRopeLo - 1) / kRopeLo), cfg->head_dim);
}

dbsa_status dbsa_rope_tables(const dbsa_config *cfg, int64_t n_pos, void *tables,
                             size_t tables_bytes, void *stream) {
  const size_t need = dbsa_rope_tables_size(cfg, n_pos);
  if (need == 0) return check_cfg(cfg) != DBSA_OK ? check_cfg(cfg) : DBSA_ERR_INVALID_ARG;
  if (!tables || !aligned16(tables))
    return fail(DBSA_ERR_INVALID_ARG, "tables is NULL or not 16-byte aligned");
  if (tables_bytes < need)
    return fail(DBSA_ERR_INVALID_ARG, "tables too small: %zu < %zu bytes", tables_bytes, need);
  // every position the bytes have room for: the calls take their size for the
  // positions that are covered
  const int32_t n_hi = (int32_t)(table_positions(cfg, tables_bytes) / kRopeLo);
  const cudaError_t e = launch_rope_rows(static_cast<float *>(tables), n_hi, cfg->head_dim,
                                         cfg->rope_theta, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "rope tables");
  count_launches(1);
  return DBSA_OK;
}

dbsa_status dbsa_paged_append(const dbsa_config *cfg, const void *k, int64_t k_row_stride,
                              int64_t k_head_stride, const void *v, int64_t v_row_stride,
                              int64_t v_head_stride, const dbsa_paged_cache *cache,
                              const dbsa_paged_batch *batch, int64_t pos0, const void *tables,
                              size_t tables_bytes, void *stream) {
  PagedPool pool;
  PagedBatch b;
  RopeTables rope;
  const dbsa_status s =
      check_paged(cfg, cache, batch, pos0, tables, tables_bytes, &pool, &b, &rope);
  if (s != DBSA_OK) return s;
  if (!k || !v) return fail(DBSA_ERR_INVALID_ARG, "a tensor pointer is NULL");
  if (!aligned16(k) || !aligned16(v))
    return fail(DBSA_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
  const int64_t str[4] = {k_row_stride, k_head_stride, v_row_stride, v_head_stride};
  for (int64_t x : str)
    if (x % 8 != 0) return fail(DBSA_ERR_INVALID_ARG, "strides must be multiples of 8");
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = cfg->dtype == DBSA_F32;
  cudaError_t e;
  if (cfg->head_dim == 128)
    e = f32 ? launch_append_t<128, float>(k, v, str, pool, b, pos0, rope, st)
            : launch_append_t<128, bf16>(k, v, str, pool, b, pos0, rope, st);
  else
    e = f32 ? launch_append_t<64, float>(k, v, str, pool, b, pos0, rope, st)
            : launch_append_t<64, bf16>(k, v, str, pool, b, pos0, rope, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged append");
  count_launches(1);
  return DBSA_OK;
}

size_t dbsa_shared_prefix_workspace_size(const dbsa_config *cfg, int32_t n_seqs, int32_t n_rows,
                                         int64_t prefix_len) {
  if (check_cfg(cfg) != DBSA_OK || check_attend_size(cfg, n_seqs, n_rows, prefix_len) != DBSA_OK)
    return 0;
  return attend_layout(cfg, n_seqs, n_rows, prefix_len).total;
}

dbsa_status dbsa_shared_prefix_attend(const dbsa_config *cfg, const void *q,
                                      int64_t q_row_stride, const dbsa_paged_cache *cache,
                                      const int32_t *prefix_pages, int64_t prefix_len,
                                      const dbsa_paged_batch *batch, const void *tables,
                                      size_t tables_bytes, void *out, void *workspace,
                                      size_t ws_bytes, void *stream) {
  const uint64_t wait_expiry = take_wait_expiry();
  AttendArgs a{};
  dbsa_status s = check_paged(cfg, cache, batch, prefix_len, tables, tables_bytes, &a.pool,
                              &a.batch, &a.rope);
  if (s != DBSA_OK) return s;
  if ((s = check_attend_size(cfg, batch->n_seqs, batch->n_rows, prefix_len)) != DBSA_OK) return s;
  if (!q || !out || (prefix_len > 0 && !prefix_pages))
    return fail(DBSA_ERR_INVALID_ARG, "a tensor pointer is NULL");
  if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(prefix_pages) & 3u) != 0)
    return fail(DBSA_ERR_INVALID_ARG, "q and out must be 16-byte aligned, prefix_pages 4-byte");
  if (q_row_stride % 8 != 0)
    return fail(DBSA_ERR_INVALID_ARG, "q_row_stride must be a multiple of 8");
  const AttendLayout l = attend_layout(cfg, batch->n_seqs, batch->n_rows, prefix_len);
  if ((s = check_ws(workspace, ws_bytes, l.total)) != DBSA_OK) return s;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.plan = l.p;
  a.plan.head = reinterpret_cast<PlanHead *>(ws + l.head);
  a.plan.row_info = reinterpret_cast<int4 *>(ws + l.row_info);
  a.plan.first_entry = reinterpret_cast<int32_t *>(ws + l.first_entry);
  a.plan.entry = reinterpret_cast<Entry *>(ws + l.entry);
  a.plan.q_rot = ws + l.q_rot;
  a.plan.acc = reinterpret_cast<float *>(ws + l.acc);
  a.plan.ml = reinterpret_cast<float2 *>(ws + l.ml);
  a.prefix_pages = prefix_pages;
  a.q = q;
  a.q_row_stride = q_row_stride;
  a.out = out;
  a.scale_log2 = scale_log2(cfg);
  a.status = reinterpret_cast<int *>(ws);
  a.wait_limit_ns = wait_expiry;
  a.withhold_tiles = wait_expiry != 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool f32 = cfg->dtype == DBSA_F32;
  cudaError_t e;
  if (cfg->head_dim == 128)
    e = f32 ? launch_attend_t<128, float>(a, st) : launch_attend_t<128, bf16>(a, st);
  else
    e = f32 ? launch_attend_t<64, float>(a, st) : launch_attend_t<64, bf16>(a, st);
  if (e != cudaSuccess) return cuda_fail(e, "shared-prefix attention");
  count_launches(3);
  return DBSA_OK;
}

}  // extern "C"
