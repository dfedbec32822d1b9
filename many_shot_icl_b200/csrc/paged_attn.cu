// Shared-prefix attention, the pieces: per (row tile, KV head, run of key
// tiles) one pass over the keys with the running maximum and sum of a softmax,
// leaving a partial per row.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "dbsa_internal.h"
#include "paged.h"
#include "paged_attn.h"
#include "sm100.cuh"
#include "vec8.cuh"

namespace dbsa {
namespace {

// ------------------------------------------------------ fp32 kernel
// fp32 caches are attended to in fp32 on the CUDA cores: tiles of 64 packed rows
// against 64 keys in shared memory, two CTAs of eight warps per SM.
//
// A warp owns R rows and one of KG groups of a tile's keys, and keeps its own
// running maximum, sums and outputs (lanes on columns); the groups are put
// together once, at the end of the piece.  Both follow the piece's rows: more
// than 32, R = 8, where each K and V read serves eight rows (with 4 the shared
// memory was the limit: prompts 589 us for 541); 17 to 32, R = 4; below, R = 4 and
// KG = 2, 4 or 8, so that a decode step, whose 4 rows would give one warp
// everything, keeps all eight busy.  For the scores a lane has two keys (KG = 1),
// one, or the D / 2 or D / 4 dimensions of one.
//
// K of the next tile is fetched (cp.async) once the scores are done, V once the
// outputs are, each while the other half of a tile is computed.  The other CTA
// of the SM fills the waits.  Bound: FMA and shared-memory reads (about even at
// R = 8) with many rows, memory with few.  Measured: 1 sequence of 32
// / 8 heads behind 90k tokens 140 us (0.81 of the copy bandwidth), 8 prompts of
// ~30 tokens behind 4k 541 us (0.4 of the FMA rate).
constexpr int kF32Rows = 64, kF32Keys = 64, kF32Warps = 8, kF32Threads = 32 * kF32Warps;

template <int D>
struct F32Smem {
  float q[kF32Rows][D];
  float k[kF32Keys][D + 4];   // rows 4 banks apart: float4 reads by 8 lanes do not collide
  float v[kF32Keys][D];
  union {
    float p[kF32Rows][kF32Keys];
    float ml[kF32Warps][4][2];   // at the end of a piece
    int32_t ticket;              // between pieces
  };
};
static_assert(sizeof(F32Smem<128>) <= 115712, "two CTAs per SM");

// 16 bytes to shared memory, zeros where there is no source.
__device__ __forceinline__ void copy16_async(void *dst, const void *src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)),
               "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// All groups but the last have landed (this thread's).
__device__ __forceinline__ void copy_wait_1() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Page of the row of the tile at k0 that lane i < 8 looks up for its warp (row
// warp + 8 i), -1 if there is none.
__device__ __forceinline__ int row_page(const Piece &pc, const PagedPool &pool, int k0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int key = k0 + warp + kF32Warps * lane;
  int page = -1;
  if (lane < kF32Keys / kF32Warps && key < pc.n_keys)
    page = __ldg(pc.pages + (key >> pool.page_shift));
  return page < pool.n_pages ? page : -1;
}

// One tile of keys or values: a warp copies a row at a time.
template <int D>
__device__ __forceinline__ void fetch_tile(float *dst, int stride, const void *pages,
                                           const Piece &pc, const PagedPool &pool, int k0,
                                           int page_of_lane) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kF32Keys / kF32Warps; ++i) {
    const int r = warp + kF32Warps * i;
    const int page = __shfl_sync(~0u, page_of_lane, i);
    const int64_t row = (int64_t)pc.c * pool.page_size + ((k0 + r) & (pool.page_size - 1));
    const float *src = static_cast<const float *>(pages) +
                       (page >= 0 ? page * pool.page_stride + row * D : 0) + lane * 4;
    if (lane * 4 < D) copy16_async(dst + r * stride + lane * 4, src, page >= 0);
  }
}

template <int D, int KG, int R>
__device__ __forceinline__ void f32_piece(const AttendArgs &a, const Piece &pc, F32Smem<D> &sm) {
  constexpr int V = D / 32, RG = kF32Warps / KG;
  constexpr int KPW = kF32Keys / KG;                // keys of a tile per warp
  constexpr int NK = KPW > 32 ? 2 : 1;              // keys per lane
  constexpr int PARTS = KPW < 32 ? 32 / KPW : 1;    // lanes per key
  const AttendPlan &p = a.plan;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rg = warp % RG, kg = warp / RG, row0 = rg * R;
  const int key_l = kg * KPW + lane % (KPW < 32 ? KPW : 32), part = lane / (KPW < 32 ? KPW : 32);

  int page = row_page(pc, a.pool, pc.kt0 * kF32Keys);
  fetch_tile<D>(&sm.k[0][0], D + 4, a.pool.k, pc, a.pool, pc.kt0 * kF32Keys, page);
  copy_commit();
  fetch_tile<D>(&sm.v[0][0], D, a.pool.v, pc, a.pool, pc.kt0 * kF32Keys, page);
  copy_commit();
  float m[R], l[R], o[R][V];
  int seen[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    seen[i] = row0 + i < pc.n_rows ? keys_seen(pc, p.g, row0 + i) : 0;
#pragma unroll
    for (int e = 0; e < V; ++e) o[i][e] = 0.f;
  }
  for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
    const int k0 = kt * kF32Keys, next = k0 + kF32Keys;
    const bool more = kt + 1 < pc.kt1;
    // which of this lane's keys are there
    bool live[NK];
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const int key = k0 + key_l + 32 * j;
      int pg = -1;
      if (key < pc.n_keys) pg = __ldg(pc.pages + (key >> a.pool.page_shift));
      live[j] = pg >= 0 && pg < a.pool.n_pages;
    }
    copy_wait_1();
    __syncthreads();   // K is in
    float s[R][NK] = {};
#pragma unroll 4
    for (int ch = 0; ch < D / 4 / PARTS; ++ch) {
      const int d = (part + PARTS * ch) * 4;
      float4 kk[NK];
#pragma unroll
      for (int j = 0; j < NK; ++j) kk[j] = *reinterpret_cast<const float4 *>(&sm.k[key_l + 32 * j][d]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float4 x = *reinterpret_cast<const float4 *>(&sm.q[row0 + i][d]);
#pragma unroll
        for (int j = 0; j < NK; ++j)
          s[i][j] += x.x * kk[j].x + x.y * kk[j].y + x.z * kk[j].z + x.w * kk[j].w;
      }
    }
    __syncthreads();   // K has been read
    if (more) {
      page = row_page(pc, a.pool, next);
      fetch_tile<D>(&sm.k[0][0], D + 4, a.pool.k, pc, a.pool, next, page);
    }
    copy_commit();
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
#pragma unroll
        for (int d = 16; d >= (PARTS > 1 ? KPW : 32); d >>= 1)
          s[i][j] += __shfl_xor_sync(~0u, s[i][j], d);
        s[i][j] = live[j] && k0 + key_l + 32 * j < seen[i] ? s[i][j] * a.scale_log2 : -INFINITY;
        mt = fmaxf(mt, s[i][j]);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(~0u, mt, d));
      const float mn = fmaxf(m[i], mt), mu = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - mu);
      m[i] = mn;
      l[i] *= f;   // summed over the lanes at the end
#pragma unroll
      for (int e = 0; e < V; ++e) o[i][e] *= f;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        const float w = exp2f(s[i][j] - mu);
        if (part == 0) {
          l[i] += w;
          sm.p[row0 + i][key_l + 32 * j] = w;
        }
      }
    }
    copy_wait_1();
    __syncthreads();   // V is in (and this warp's p)
#pragma unroll 2
    for (int k = 0; k < KPW; k += 4) {
      float4 pr[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        pr[i] = *reinterpret_cast<const float4 *>(&sm.p[row0 + i][kg * KPW + k]);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        float v[V];
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4 *>(&sm.v[kg * KPW + k + kk][lane * 4]);
          v[0] = x.x;
          v[1] = x.y;
          v[2] = x.z;
          v[3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2 *>(&sm.v[kg * KPW + k + kk][lane * 2]);
          v[0] = x.x;
          v[1] = x.y;
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float w = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
#pragma unroll
          for (int e = 0; e < V; ++e) o[i][e] += w * v[e];
        }
      }
    }
    __syncthreads();   // V has been read
    if (more) fetch_tile<D>(&sm.v[0][0], D, a.pool.v, pc, a.pool, next, page);
    copy_commit();
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) l[i] += __shfl_xor_sync(~0u, l[i], d);
  if constexpr (KG > 1) {
    static_assert(R == 4, "the exchange holds four rows a warp");
    // put the key groups together: group kg's outputs in the idle K tile
    float *part_o = &sm.k[0][0];
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int e = 0; e < V; ++e) part_o[(warp * R + i) * D + lane * V + e] = o[i][e];
      if (lane == 0) {
        sm.ml[warp][i][0] = m[i];
        sm.ml[warp][i][1] = l[i];
      }
    }
    __syncthreads();
    if (kg == 0) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float M = m[i];
#pragma unroll
        for (int g = 1; g < KG; ++g) M = fmaxf(M, sm.ml[rg + g * RG][i][0]);
        const float mu = M == -INFINITY ? 0.f : M;
        float f = exp2f(m[i] - mu);
        l[i] *= f;
#pragma unroll
        for (int e = 0; e < V; ++e) o[i][e] *= f;
#pragma unroll
        for (int g = 1; g < KG; ++g) {
          const int w = rg + g * RG;
          f = exp2f(sm.ml[w][i][0] - mu);
          l[i] += f * sm.ml[w][i][1];
#pragma unroll
          for (int e = 0; e < V; ++e) o[i][e] += f * part_o[(w * R + i) * D + lane * V + e];
        }
        m[i] = M;
      }
    }
  }
  if (kg == 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int r = row0 + i;
      if (r >= pc.n_rows) break;
      float *dst = p.acc + (pc.partial + r) * D + lane * V;
#pragma unroll
      for (int e = 0; e < V; ++e) dst[e] = o[i][e];
      if (lane == 0) p.ml[pc.partial + r] = make_float2(m[i], l[i]);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kF32Threads, 2) attend_f32_kernel(const __grid_constant__ AttendArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  F32Smem<D> &sm = *reinterpret_cast<F32Smem<D> *>(smem_raw);
  constexpr int CH = D / 4;
  const AttendPlan &p = a.plan;
  const int tid = threadIdx.x;
  PieceWalk walk;
  Piece pc;
  int64_t item = blockIdx.x;
  walk.u = walk.uend = 0;
  for (;;) {
    while (!walk.next(p, a.batch, a.prefix_pages, pc)) {
      if (!walk.start(p, item)) return;
      __syncthreads();   // the ticket before has been read
      if (tid == 0) sm.ticket = atomicAdd(&p.head->ticket, 1);
      __syncthreads();
      item = (int64_t)p.n_ctas + sm.ticket;
    }
    __syncthreads();   // the piece before is done with shared memory
    const float *qs = static_cast<const float *>(p.q_rot) + ((int64_t)pc.c * p.rows + pc.row0) * D;
    const int rows = pc.n_rows > 32 ? 64 : pc.n_rows > 16 ? 32 : 16;   // that are read
    for (int i = tid; i < rows * CH; i += kF32Threads) {
      const int r = i / CH, d = (i % CH) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < pc.n_rows) x = *reinterpret_cast<const float4 *>(qs + (int64_t)r * D + d);
      *reinterpret_cast<float4 *>(&sm.q[r][d]) = x;
    }
    // (the first barrier inside orders these writes before their use)
    if (pc.n_rows <= 4) f32_piece<D, 8, 4>(a, pc, sm);
    else if (pc.n_rows <= 8) f32_piece<D, 4, 4>(a, pc, sm);
    else if (pc.n_rows <= 16) f32_piece<D, 2, 4>(a, pc, sm);
    else if (pc.n_rows <= 32) f32_piece<D, 1, 4>(a, pc, sm);
    else f32_piece<D, 1, 8>(a, pc, sm);
  }
}

template <int D>
cudaError_t launch_f32(const AttendArgs &a, cudaStream_t st) {
  const cudaError_t e =
      cudaFuncSetAttribute(attend_f32_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)sizeof(F32Smem<D>));
  if (e != cudaSuccess) return e;
  return pdl_launch(attend_f32_kernel<D>, dim3(a.plan.n_ctas), dim3(kF32Threads),
                    sizeof(F32Smem<D>), st, a);
}

// ------------------------------------------------------ tensor-core kernel
// bf16 caches: tiles of 128 packed rows against 64 keys on tcgen05.
//
// Two CTAs per SM, 224 threads each, half of the SM's shared memory and tensor
// memory each, so that one CTA's waits are the other's work.  Per CTA:
//   warp 4     walks the pieces, publishes each in a ring of kPieceSlots, and
//              loads Q, K and V tiles by TMA, page by page (a box is at most one
//              page; lanes look the pages up and issue the boxes of a tile)
//   warp 5     owns the tensor memory; one thread issues S = Q K^T (both from
//              shared memory)
//   warp 6     one thread issues O += P V (P from tensor memory)
//   warps 0-3  softmax, one thread per row, and the partials' stores
// Tensor memory: two buffers of S (64 columns fp32; P, bf16, over the first 32
// of its S) and O (D columns): all 256 of the CTA's half at D = 128.  Q K^T of
// tile t + 1 runs while tile t is exponentiated, so the softmax warps find the
// next scores waiting and the chain from one tile to the next is the softmax
// alone.  An issuing thread spends ~125 cycles on each wait, met or not, and as
// much on each commit, so there are two of them and few barriers: S_FULL also
// says that the tile's K slot is free, PV_DONE that its V slot and its S buffer
// are.
// O is rescaled only when a row's maximum has grown by more than 2^8.
//
// Measured (one layer, 32 / 8 heads of 128, prefix of 90 223 tokens, short runs; back
// to back at the power limit a call for 64 sequences takes 17 % more): 1 sequence
// 56 us in this kernel, 370 MB, 6.5 TB/s between its ramps; 64 sequences 105 us,
// 0.85 PFLOP/s; 64 prompts of ~30 tokens 2.9 ms, 0.97 PFLOP/s at ~2 000 cycles
// per 128 x 128 scores, where the tensor core alone would take 1 024 with 128-key
// tiles and 1 536 with these (an instruction with A in shared memory takes 64
// cycles up to N = 128).  Bound by memory with few rows, by the card's power limit
// with many.
//
// Keys that do not exist (past the end of the list, or on a page that is not
// there) get probability 0, and their rows of V are zeroed in shared memory:
// 0 * NaN would poison the row.
constexpr int kTcRows = 128, kTcKeys = 64;
// Pieces of at most this many rows (a decode step's own tokens, a small batch
// behind the prefix) run 64-row instructions: rows 0..15 lie in the same lanes of
// the tensor memory, and half the tensor core's work, all of it on rows that do
// not exist, is saved.  What that buys is power: the calls run at its limit.
constexpr int kFewRows = 16;
constexpr int kTcSoftmaxWarps = 4, kTcProducerWarp = 4, kTcQkWarp = 5, kTcPvWarp = 6;
constexpr int kTcThreads = 224;
constexpr int kPieceSlots = 4;
constexpr int kAskAhead = 3;   // tiles
constexpr int kQBox = 32;   // query rows per TMA box: those of a softmax warp
constexpr uint64_t kWaitLimitNs = 4000000000ull;   // default: 4 s, far above any legitimate wait
constexpr uint64_t kDrainLimitNs = 200000000ull;   // 0.2 s for the exit drain
constexpr uint32_t kFull = 0xFFFFFFFFu;

template <int D>
struct Tc {
  static constexpr int NH = D / 64;                    // 64-column (128-byte) atoms of a row
  static constexpr uint32_t Q_BYTES = kTcRows * D * 2, KV_BYTES = kTcKeys * D * 2;
  // K and V tiles.  K slots go with the S buffers; V slots are one more, since
  // a tile's V is used a softmax later.
  static constexpr int NK = 2, NV = 3;
  enum Bar {
    Q_FULL /* [piece % 2] */, Q_EMPTY = Q_FULL + 2, DRAIN_QK = Q_EMPTY + 2, DRAIN_PV,
    S_FULL /* [K slot, S buffer] */,
    P_FULL = S_FULL + NK /* [S buffer] */, K_FULL = P_FULL + NK, V_FULL = K_FULL + NK,
    PV_DONE = V_FULL + NV /* [V slot] */, PIECE_FULL = PV_DONE + NV,
    PIECE_EMPTY = PIECE_FULL + kPieceSlots, COUNT = PIECE_EMPTY + kPieceSlots
  };
  static constexpr uint32_t TILES = Q_BYTES + (NK + NV) * KV_BYTES;
  // Two CTAs fit an SM (228 KB, 1 KB of it reserved per CTA), three do not: each
  // takes half of the tensor memory.
  static constexpr uint32_t NEED = TILES + 1024, SMEM = NEED > 80 * 1024 ? NEED : 80 * 1024;
  static_assert(SMEM <= 115712 && 3 * (SMEM + 1024) > 233472, "two CTAs per SM");
};

// Where the queries of a piece go: pieces of at most 64 rows take turns at the
// halves of the Q tile, so that one's can be loaded while the other's are in
// use (Q K^T then reads 64 rows past the piece's, whose results nobody uses).
constexpr int kQHalf = kTcRows / 2;
__device__ __forceinline__ int q_row0(uint32_t piece, int n_rows) {
  return n_rows <= kQHalf && (piece & 1) ? kQHalf : 0;
}

struct PieceRec {   // what the consumers need of a Piece
  int32_t n_rows, kt0, kt1, n_keys, see0, off, shared, pad;
  const int32_t *pages;
  int64_t partial;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ f32x2 f2_add(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(sm100::smem_u32(bar)), "r"(x), "r"(y), "r"(z),
      "r"(w)
      : "memory");
}
// Bounded wait on the way out: ignores the abort flag.
__device__ __forceinline__ void drain_wait(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = sm100::globaltimer_ns();
  while (!sm100::mbar_try_wait(bar, parity)) {
    if (sm100::globaltimer_ns() - t0 > kDrainLimitNs) return;
  }
}

// Page of keys 16 * lane .. of the tile at k0 (lanes 0..3), -1 if there is none.
__device__ __forceinline__ int group_page(const int32_t *pages, int k0, int n_keys,
                                          const PagedPool &pool, int lane) {
  const int key = k0 + 16 * lane;
  return lane < kTcKeys / 16 && key < n_keys ? __ldg(pages + (key >> pool.page_shift)) : -1;
}

template <int D>
__global__ void __launch_bounds__(kTcThreads, 2)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttendArgs a) {
  using namespace sm100;
  using C = Tc<D>;
  constexpr uint32_t QATOM = kTcRows * 128;       // one 64-column atom of the Q tile
  constexpr uint32_t ATOM = kTcKeys * 128;        // ... of a K or V tile
  // 128-row instructions, or 64-row ones
  constexpr uint32_t IDESC_QK = idesc_bf16_f32(kTcRows, kTcKeys, false);
  constexpr uint32_t IDESC_PV = idesc_bf16_f32(kTcRows, D, true);
  constexpr uint32_t IDESC_QK_64 = idesc_bf16_f32(64, kTcKeys, false);
  constexpr uint32_t IDESC_PV_64 = idesc_bf16_f32(64, D, true);
  constexpr uint32_t TMEM_COLS = 256, COL_S = 0, COL_O = 2 * kTcKeys;

  // Swizzled tiles sit on 1024-byte boundaries of shared memory: the dynamic
  // part starts on one, having nothing static before it (checked below).
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem, *sK = sQ + C::Q_BYTES, *sV = sK + C::NK * C::KV_BYTES;
  uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::TILES);
  PieceRec *ring = reinterpret_cast<PieceRec *>(bar + C::COUNT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(ring + kPieceSlots);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  static_assert(C::COUNT * 8 + kPieceSlots * sizeof(PieceRec) + 8 <= 1024, "barrier space");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttendPlan &p = a.plan;
  const uint64_t limit = a.wait_limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::COUNT; ++i) {
      uint32_t n = 1;
      if (i == C::P_FULL || i == C::P_FULL + 1) n = kTcSoftmaxWarps;
      if (i >= C::PIECE_EMPTY) n = kTcSoftmaxWarps + 2;   // softmax warps and the issuers
      mbar_init(&bar[i], n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kTcQkWarp) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  auto wait = [&](int b, uint32_t parity) -> bool {
    return mbar_wait(&bar[b], parity, abort_flag, a.status, limit, DBSA_ERR_TIMEOUT);
  };
  // one arrival for a whole warp, behind all its lanes' accesses
  auto arrive_warp = [&](int b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar[b]);
  };
  // waits run by a whole warp
  auto wait_warp = [&](int b, uint32_t parity) -> bool {
    return __all_sync(kFull, wait(b, parity));
  };

  if ((smem_u32(smem) & 1023u) != 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) atomicExch(a.status, DBSA_ERR_CUDA);
  } else if (warp == kTcProducerWarp) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_desc(&tmQ);
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    const int box = min(a.pool.page_size, kTcKeys);    // rows per TMA box
    const int n_boxes = kTcKeys / box * C::NH;         // of a K or V tile
    const int brow = lane / C::NH * box;               // this lane's box: first key, atom
    const int atom = lane % C::NH;
    const uint32_t box_bytes = (uint32_t)box * 128;
    const uint32_t dst = atom * ATOM + brow * 128;
    uint32_t n_pieces = 0, kn = 0, vn = 0;
    bool ok = true;
    PieceWalk walk;
    Piece pc = {};
    walk.u = walk.uend = 0;
    int64_t item = blockIdx.x;
    int32_t ticket = 0;    // lane 0
    bool asked = false;
    // The producer alone waits for the kernel before (which rotated the queries
    // and built the plan of the own tokens), and only when it needs them: the
    // first tiles of a prefix piece are loaded before that.  Their pages are
    // complete: the kernel before let this one start only after it had itself
    // waited for everything before it in the stream.
    bool entered = false, hold_q = false;
    auto enter = [&]() {
      if (!entered) asm volatile("griddepcontrol.wait;" ::: "memory");
      entered = true;
    };
    int rows_before = 0;   // rows of the piece before
    auto load_q = [&](uint32_t n) -> bool {
      enter();
      // the place's last user: two pieces back, or one if either needs it whole
      if (n >= 2 && !wait_warp(C::Q_EMPTY + (n & 1), (n / 2 - 1) & 1)) return false;
      if (n >= 1 && max(rows_before, pc.n_rows) > kQHalf &&
          !wait_warp(C::Q_EMPTY + ((n - 1) & 1), ((n - 1) / 2) & 1))
        return false;
      rows_before = pc.n_rows;
      // 32 rows a box, as many as hold rows of the piece: the rows behind them
      // keep what they held, for softmax warps that have no row of the piece
      const int boxes = (pc.n_rows + kQBox - 1) / kQBox;
      uint64_t *full = &bar[C::Q_FULL + (n & 1)];
      if (lane == 0) mbar_arrive_expect_tx(full, boxes * C::NH * kQBox * 128);
      __syncwarp();
      if (lane < boxes * C::NH) {
        const int b = lane / C::NH, h = lane % C::NH;
        tma_load_3d(sQ + h * QATOM + (q_row0(n, pc.n_rows) + b * kQBox) * 128, &tmQ, full, h * 64,
                    pc.row0 + b * kQBox, pc.c);
      }
      return true;
    };
    if (a.withhold_tiles) {
      enter();
      // test hook: nothing is published or loaded, so every wait of the
      // consumers runs out and raises the abort flag
      const uint64_t t0 = globaltimer_ns();
      while (!*abort_flag && globaltimer_ns() - t0 <= 2 * limit) __nanosleep(256);
      ok = false;
    }
    while (ok) {
      if (!walk.next(p, a.batch, a.prefix_pages, pc)) {
        if (n_pieces > 0 || !PieceWalk::is_shared(p, item)) enter();
        if (n_pieces > 0) {
          if (!asked && lane == 0) ticket = atomicAdd(&p.head->ticket, 1);
          asked = false;
          item = p.n_ctas + (int64_t)__shfl_sync(kFull, ticket, 0);
        }
        if (!walk.start(p, item) || !walk.next(p, a.batch, a.prefix_pages, pc)) break;
      }
      const uint32_t slot = n_pieces % kPieceSlots;
      if (n_pieces >= kPieceSlots &&
          !(ok = wait_warp(C::PIECE_EMPTY + slot, (n_pieces / kPieceSlots - 1) & 1)))
        break;
      if (lane == 0) {
        ring[slot] = {pc.n_rows, pc.kt0, pc.kt1, pc.n_keys, pc.see0,
                      pc.off,    pc.shared, 0,   pc.pages,  pc.partial};
        mbar_arrive(&bar[C::PIECE_FULL + slot]);
      }
      const uint32_t n = n_pieces++;
      hold_q = true;
      // in the order of their use: K of a tile, then V of the tile before
      int page = -1, next = -1, y = 0, next_y = 0;
      for (int kt = pc.kt0; kt <= pc.kt1; ++kt) {
        // The next ticket is asked for with the item's last tiles: not earlier, so
        // that slow SMs take fewer, and not after them, so that it is there in time.
        if (!asked && entered && walk.u == walk.uend && kt >= pc.kt1 - kAskAhead) {
          if (lane == 0) ticket = atomicAdd(&p.head->ticket, 1);
          asked = true;
        }
        // Q after the first K (whose slot is free before Q's place is), or, in
        // the first piece, once no K slot is left to fill
        if (hold_q && kt == pc.kt0 + (n == 0 ? C::NK : 1)) {
          if (!(ok = load_q(n))) break;
          hold_q = false;
        }
        if (kt < pc.kt1) {
          const int key = kt * kTcKeys + brow;
          next = -1;
          if (lane < n_boxes && key < pc.n_keys)
            next = __ldg(pc.pages + (key >> a.pool.page_shift));
          if (next >= a.pool.n_pages) next = -1;
          next_y = key & (a.pool.page_size - 1);
          const uint32_t ks = kn % C::NK;
          if (kn >= C::NK && !(ok = wait_warp(C::S_FULL + ks, (kn / C::NK - 1) & 1))) break;
          const uint32_t boxes = __popc(__ballot_sync(kFull, next >= 0));
          if (lane == 0) mbar_arrive_expect_tx(&bar[C::K_FULL + ks], boxes * box_bytes);
          __syncwarp();
          if (next >= 0)
            tma_load_4d(smem_u32(sK) + ks * C::KV_BYTES + dst, &tmK, &bar[C::K_FULL + ks],
                        atom * 64, next_y, pc.c, next);
          ++kn;
        }
        if (kt > pc.kt0) {
          const uint32_t vs = vn % C::NV;
          if (vn >= C::NV && !(ok = wait_warp(C::PV_DONE + vs, (vn / C::NV - 1) & 1))) break;
          const uint32_t boxes = __popc(__ballot_sync(kFull, page >= 0));
          if (lane == 0) mbar_arrive_expect_tx(&bar[C::V_FULL + vs], boxes * box_bytes);
          __syncwarp();
          if (page >= 0)
            tma_load_4d(smem_u32(sV) + vs * C::KV_BYTES + dst, &tmV, &bar[C::V_FULL + vs],
                        atom * 64, y, pc.c, page);
          ++vn;
        }
        page = next;
        y = next_y;
      }
      if (ok && hold_q && (ok = load_q(n))) hold_q = false;
    }
    // the end of the list
    if (ok) {
      const uint32_t slot = n_pieces % kPieceSlots;
      if (n_pieces < kPieceSlots ||
          (ok = wait_warp(C::PIECE_EMPTY + slot, (n_pieces / kPieceSlots - 1) & 1))) {
        if (lane == 0) {
          ring[slot].n_rows = 0;
          mbar_arrive(&bar[C::PIECE_FULL + slot]);
        }
      }
    }
    // every load must have landed before the CTA exits
    if (lane == 0) {
      // (the last piece's Q may not have been asked for)
      const uint32_t nq = hold_q ? n_pieces - 1 : n_pieces;
      for (uint32_t s = 0; s < 2; ++s)
        if (nq > s) drain_wait(&bar[C::Q_FULL + s], ((nq - 1 - s) / 2) & 1);
      for (uint32_t s = 0; s < C::NK; ++s)
        if (kn > s) drain_wait(&bar[C::K_FULL + s], ((kn - 1 - s) / C::NK) & 1);
      for (uint32_t s = 0; s < C::NV; ++s)
        if (vn > s) drain_wait(&bar[C::V_FULL + s], ((vn - 1 - s) / C::NV) & 1);
    }
  } else if (warp == kTcQkWarp || warp == kTcPvWarp) {
    // ------------------------------------------------------------ MMA issuers
    if (lane == 0) {
      const bool qk = warp == kTcQkWarp;
      const uint64_t dQ = sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024);
      const uint64_t dV = sdesc_sw128(smem_u32(sV), ATOM, 1024);
      uint32_t n_pieces = 0, tn = 0;
      // slot and phase of tile tn's V (P V) or of V two tiles before (Q K^T)
      uint32_t vs = 0, vph = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = n_pieces % kPieceSlots;
        if (!(ok = wait(C::PIECE_FULL + slot, (n_pieces / kPieceSlots) & 1))) break;
        const int n_rows = ring[slot].n_rows, kt0 = ring[slot].kt0, kt1 = ring[slot].kt1;
        const int n_keys = ring[slot].n_keys;
        if (n_rows == 0) break;
        mbar_arrive(&bar[C::PIECE_EMPTY + slot]);
        if (qk && !(ok = wait(C::Q_FULL + (n_pieces & 1), (n_pieces >> 1) & 1))) break;
        const uint64_t dq = dQ + q_row0(n_pieces, n_rows) * (128 >> 4);
        const int q_empty = C::Q_EMPTY + (n_pieces & 1);
        const uint32_t idesc = n_rows <= kFewRows ? (qk ? IDESC_QK_64 : IDESC_PV_64)
                                                  : (qk ? IDESC_QK : IDESC_PV);
        ++n_pieces;
        for (int kt = kt0; kt < kt1; ++kt, ++tn) {
          const uint32_t b = tn & 1, ph = (tn >> 1) & 1;
          if (qk) {
            if (!(ok = wait(C::K_FULL + b, ph))) break;
            if (tn >= 2) {   // P of the tile that had this S buffer has been used
              if (!(ok = wait(C::PV_DONE + vs, vph))) break;
              if (++vs == C::NV) {
                vs = 0;
                vph ^= 1;
              }
            }
            tc_fence_after();
            const uint64_t dk = dK + b * (C::KV_BYTES >> 4);
            const uint32_t d = tmem + COL_S + b * kTcKeys;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_bf16_ss(d, dq + (((kk >> 2) * QATOM + (kk & 3) * 32) >> 4),
                          dk + (((kk >> 2) * ATOM + (kk & 3) * 32) >> 4), idesc,
                          kk > 0 ? 1u : 0u);
            mma_commit(&bar[C::S_FULL + b]);
            if (kt == kt1 - 1) mma_commit(&bar[q_empty]);
          } else {
            if (!(ok = wait(C::V_FULL + vs, vph))) break;
            // P written, and O rescaled or (first tile) read out
            if (!(ok = wait(C::P_FULL + b, ph))) break;
            tc_fence_after();
            const uint64_t dv = dV + vs * (C::KV_BYTES >> 4);
            const uint32_t pcol = tmem + COL_S + b * kTcKeys;
            const uint32_t first = kt > kt0 ? 1u : 0u;
            const int valid = n_keys - kt * kTcKeys;
            if (valid > kTcKeys - 16) {
#pragma unroll
              for (int kk = 0; kk < kTcKeys / 16; ++kk)
                mma_bf16_ts(tmem + COL_O, pcol + kk * 8, dv + kk * 128, idesc,
                            kk > 0 ? 1u : first);
            } else {
              for (int kk = 0; kk * 16 < valid; ++kk)
                mma_bf16_ts(tmem + COL_O, pcol + kk * 8, dv + kk * 128, idesc,
                            kk > 0 ? 1u : first);
            }
            mma_commit(&bar[C::PV_DONE + vs]);
            if (++vs == C::NV) {
              vs = 0;
              vph ^= 1;
            }
          }
        }
      }
      // every instruction must be done before the tensor memory is given back
      mma_commit(&bar[qk ? C::DRAIN_QK : C::DRAIN_PV]);
      drain_wait(&bar[qk ? C::DRAIN_QK : C::DRAIN_PV], 0);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int row = warp * 32 + lane;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t t_o = tmem + lane_off + COL_O;
    const float sl2 = a.scale_log2;
    uint32_t n_pieces = 0, tn = 0;
    bool ok = true;
    while (ok) {
      const uint32_t slot = n_pieces % kPieceSlots;
      if (!(ok = wait_warp(C::PIECE_FULL + slot, (n_pieces / kPieceSlots) & 1))) break;
      const PieceRec pc = ring[slot];
      if (pc.n_rows == 0) break;
      arrive_warp(C::PIECE_EMPTY + slot);
      ++n_pieces;
      const bool idle = warp * 32 >= pc.n_rows;   // no row of this warp is one of the piece
      const int seen = pc.shared ? pc.n_keys : min(pc.n_keys, pc.see0 + (pc.off + row) / p.g);
      float m_ref = -INFINITY, l = 0.f;
      int page = group_page(pc.pages, pc.kt0 * kTcKeys, pc.n_keys, a.pool, lane);
      for (int kt = pc.kt0; kt < pc.kt1; ++kt, ++tn) {
        const int k0 = kt * kTcKeys, valid = min(kTcKeys, pc.n_keys - k0);
        // bit i: keys 16i .. 16i + 15 of the tile are on a page that is there
        const uint32_t groups = __ballot_sync(kFull, page >= 0 && page < a.pool.n_pages);
        page = group_page(pc.pages, k0 + kTcKeys, pc.n_keys, a.pool, lane);   // the next tile's
        const uint32_t t_s = tmem + lane_off + COL_S + (tn & 1) * kTcKeys;
        if (!(ok = wait_warp(C::S_FULL + (tn & 1), (tn >> 1) & 1))) break;
        tc_fence_after();
        if (valid % 16 != 0 || groups != (1u << ((valid + 15) / 16)) - 1) {
          // Rows of V that P V will read and no key stands for: zero them.  S of
          // tile t being complete says that P V of tile t - 2 is, so with three
          // slots this one's barrier is in this tile's phase or past it.
          const uint32_t vs = tn % C::NV;
          if (!(ok = wait_warp(C::V_FULL + vs, (tn / C::NV) & 1))) break;
          uint8_t *tile = sV + vs * C::KV_BYTES;
          const int rows = (valid + 15) / 16 * 16;
          for (int i = threadIdx.x; i < rows * C::NH * 8; i += kTcSoftmaxWarps * 32) {
            const int r = i / (C::NH * 8), x = i % (C::NH * 8);
            if (r >= valid || ((groups >> (r >> 4)) & 1u) == 0)
              *reinterpret_cast<uint4 *>(tile + (x >> 3) * ATOM + r * 128 + (x & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        if (!idle) {
          uint32_t s[2][32];
          tmem_ld32(t_s, s[0]);
          tmem_ld32(t_s + 32, s[1]);
          tmem_wait_ld(s[0]);
          tmem_wait_ld(s[1]);
          // keys this row sees of the tile
          const int lim = seen - k0;
          if (__any_sync(kFull, lim < kTcKeys) || groups != 0xFu) {
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c * 32 + e >= lim || ((groups >> (c * 2 + e / 16)) & 1u) == 0)
                  s[c][e] = __float_as_uint(-INFINITY);
          }
          float mt[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t *x = &s[c >> 1][(c & 1) * 16];
            mt[c] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
#pragma unroll
            for (int e = 2; e < 16; e += 2)
              mt[c] = max3(mt[c], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
          }
          // (lanes without a row hold anything: they must not move the others)
          const float mx =
              row < pc.n_rows ? max3(mt[0], mt[1], fmaxf(mt[2], mt[3])) * sl2 : -INFINITY;
          if (kt == pc.kt0) {
            m_ref = mx;
          } else if (__any_sync(kFull, mx > m_ref + 8.f)) {
            // O must hold the tiles before this one
            if (!(ok = wait_warp(C::PV_DONE + (tn - 1) % C::NV, ((tn - 1) / C::NV) & 1))) break;
            tc_fence_after();
            // (rows that need no new reference keep theirs: with another one their
            // probabilities would round differently, because of a neighbour)
            const float m_new = mx > m_ref + 8.f ? mx : m_ref;
            const float f = m_new == -INFINITY ? 1.f : ex2(m_ref - m_new);
            l *= f;
            m_ref = m_new;
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_ld16(t_o + c * 16, o);
              tmem_wait_ld16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st16(t_o + c * 16, o);
            }
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          const f32x2 sc2 = f2_pack(sl2, sl2), nmu2 = f2_pack(-mu, -mu);
          f32x2 sum2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t pw[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])), sc2,
                               nmu2),
                        x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              sum2[(e >> 1) & 1] = f2_add(sum2[(e >> 1) & 1], f2_pack(p0, p1));
              __nv_bfloat162 h = __floats2bfloat162_rn(p0, p1);
              pw[e >> 1] = *reinterpret_cast<uint32_t *>(&h);
            }
            tmem_st16(t_s + c * 16, pw);
          }
          tmem_wait_st();
          float s0, s1, s2, s3;
          f2_unpack(sum2[0], s0, s1);
          f2_unpack(sum2[1], s2, s3);
          l += (s0 + s1) + (s2 + s3);
        }
        tc_fence_before();
        arrive_warp(C::P_FULL + (tn & 1));
      }
      if (!ok) break;
      // P V of the last tile (that of the tile three before it, on the same
      // barrier, is done since the last S is)
      if (!(ok = wait_warp(C::PV_DONE + (tn - 1) % C::NV, ((tn - 1) / C::NV) & 1))) break;
      tc_fence_after();
      if (!idle) {
        float *dst = p.acc + (pc.partial + row) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(t_o + c * 32, o);
          tmem_wait_ld(o);
          if (row < pc.n_rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4 *>(dst + c * 32 + e) =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (row < pc.n_rows) p.ml[pc.partial + row] = make_float2(m_ref, l);
        tc_fence_before();   // O may be overwritten once P of the next piece is in
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kTcQkWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// bf16, boxes of 64 elements x `rows` rows, 128-byte swizzle.
bool encode_map(CUtensorMap *m, const void *ptr, int rank, const cuuint64_t *dims,
                const cuuint64_t *strides, int rows) {
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, one[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(ptr), dims, strides, box,
             one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_tc(const AttendArgs &a, cudaStream_t st) {
  using C = Tc<D>;
  const AttendPlan &p = a.plan;
  CUtensorMap mq, mk, mv;
  const cuuint64_t qd[3] = {D, (cuuint64_t)p.rows, (cuuint64_t)p.Hkv};
  const cuuint64_t qs[2] = {D * 2, (cuuint64_t)p.rows * D * 2};
  const cuuint64_t kd[4] = {D, (cuuint64_t)a.pool.page_size, (cuuint64_t)p.Hkv,
                            (cuuint64_t)a.pool.n_pages};
  const cuuint64_t ks[3] = {D * 2, (cuuint64_t)a.pool.page_size * D * 2,
                            (cuuint64_t)a.pool.page_stride * 2};
  const int box = a.pool.page_size < kTcKeys ? a.pool.page_size : kTcKeys;
  if (!encode_map(&mq, p.q_rot, 3, qd, qs, kQBox) || !encode_map(&mk, a.pool.k, 4, kd, ks, box) ||
      !encode_map(&mv, a.pool.v, 4, kd, ks, box))
    return cudaErrorInvalidValue;
  const cudaError_t e = cudaFuncSetAttribute(
      attend_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
  if (e != cudaSuccess) return e;
  AttendArgs b = a;
  if (b.wait_limit_ns == 0) b.wait_limit_ns = kWaitLimitNs;
  return pdl_launch(attend_tc_kernel<D>, dim3(p.n_ctas), dim3(kTcThreads), C::SMEM, st, mq, mk, mv,
                    b);
}

}  // namespace

AttendShape attend_shape(const dbsa_config *cfg, int rows, int64_t prefix_len) {
  constexpr int n_ctas = 2 * 148;
  if (cfg->dtype != DBSA_F32) return {kTcRows, kTcKeys, n_ctas, kTcRows, kTcRows};
  // fp32: a tile costs what its rows cost, so work that fits one wave of smaller
  // tiles takes those (25 rows x 32 heads behind 71 tokens: 29 us with 64-row
  // tiles).  One more key tile stands for the own tokens, whose lengths the host
  // does not know (their bound, table_width * page_size, is not used: rows of long
  // histories behind little prefix get small tiles all the same); tiles of less
  // than 16 rows would read long ones too often.
  constexpr int least = 16;
  int tile_rows = least;
  const int64_t keys = (prefix_len + kF32Keys - 1) / kF32Keys + 1;
  while (tile_rows < kF32Rows &&
         (rows + tile_rows - 1) / tile_rows * keys * cfg->n_kv_heads > n_ctas)
    tile_rows *= 2;
  return {tile_rows, kF32Keys, n_ctas, least, kF32Rows};
}

cudaError_t launch_attend_pieces(const AttendArgs &a, int head_dim, bool f32, cudaStream_t st) {
  if (f32) return head_dim == 128 ? launch_f32<128>(a, st) : launch_f32<64>(a, st);
  return head_dim == 128 ? launch_tc<128>(a, st) : launch_tc<64>(a, st);
}

}  // namespace dbsa
