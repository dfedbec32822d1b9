// Shared-prefix attention, the pieces: per (row tile, KV head, run of key
// tiles) one pass over the keys with the running maximum and sum of a softmax,
// leaving a partial per row.
#include <cuda_bf16.h>

#include <algorithm>

#include "dbsa_internal.h"
#include "paged.h"
#include "paged_attn.h"
#include "vec8.cuh"

namespace dbsa {
namespace {

// ------------------------------------------------------ CUDA-core kernel
// 32 packed rows against 64 keys at a time, everything in fp32 shared memory:
// scores with lanes on keys (warp w: rows 4w..4w+3, lane: keys lane, lane +
// 32), outputs with lanes on columns.
constexpr int kSimpleRows = 32, kSimpleKeys = 64, kSimpleThreads = 256;

template <int D>
struct SimpleSmem {
  float q[kSimpleRows][D];
  float k[kSimpleKeys][D + 4];   // rows 4 banks apart: float4 reads by 8 lanes do not collide
  float v[kSimpleKeys][D];
  float p[kSimpleRows][kSimpleKeys];
  int32_t live[kSimpleKeys];     // whether the key exists
};

template <typename T>
__device__ __forceinline__ void load8_f32(const T *src, float *dst) {
  float f[8];
  load8(src, f);
  reinterpret_cast<float4 *>(dst)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(dst)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

template <int D, typename T>
__global__ void __launch_bounds__(kSimpleThreads) attend_simple_kernel(const AttendArgs a) {
  pdl_enter();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimpleSmem<D> &sm = *reinterpret_cast<SimpleSmem<D> *>(smem_raw);
  constexpr int V = D / 32, CH = D / 8;
  const AttendPlan &p = a.plan;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  PieceWalk walk;
  walk.init(blockIdx.x);
  Piece pc;
  while (walk.next(p, a.batch, a.prefix_pages, pc)) {
    __syncthreads();   // the previous piece's reads of q are done
    const T *qs = static_cast<const T *>(p.q_rot) + ((int64_t)pc.c * p.rows + pc.row0) * D;
    for (int i = tid; i < kSimpleRows * CH; i += kSimpleThreads) {
      const int r = i / CH, d0 = (i % CH) * 8;
      if (r < pc.n_rows) {
        load8_f32(qs + (int64_t)r * D + d0, &sm.q[r][d0]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) sm.q[r][d0 + e] = 0.f;
      }
    }
    float m[4], l[4], o[4][V];
    int seen[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      seen[i] = warp * 4 + i < pc.n_rows ? keys_seen(pc, p.g, warp * 4 + i) : 0;
#pragma unroll
      for (int e = 0; e < V; ++e) o[i][e] = 0.f;
    }
    for (int kt = pc.kt0; kt < pc.kt1; ++kt) {
      const int k0 = kt * kSimpleKeys;
      __syncthreads();   // the previous tile's reads are done
      for (int i = tid; i < kSimpleKeys * CH; i += kSimpleThreads) {
        const int r = i / CH, d0 = (i % CH) * 8, key = k0 + r;
        int page = -1;
        if (key < pc.n_keys) page = __ldg(pc.pages + (key >> a.pool.page_shift));
        const bool live = page >= 0 && page < a.pool.n_pages;
        if (live) {
          const int64_t off =
              page * a.pool.page_stride +
              ((int64_t)pc.c * a.pool.page_size + (key & (a.pool.page_size - 1))) * D + d0;
          load8_f32(static_cast<const T *>(a.pool.k) + off, &sm.k[r][d0]);
          load8_f32(static_cast<const T *>(a.pool.v) + off, &sm.v[r][d0]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) sm.k[r][d0 + e] = sm.v[r][d0 + e] = 0.f;
        }
        if (d0 == 0) sm.live[r] = live;
      }
      __syncthreads();
      float s[4][2] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        const float4 k_0 = *reinterpret_cast<const float4 *>(&sm.k[lane][d]);
        const float4 k_1 = *reinterpret_cast<const float4 *>(&sm.k[lane + 32][d]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4 *>(&sm.q[warp * 4 + i][d]);
          s[i][0] += x.x * k_0.x + x.y * k_0.y + x.z * k_0.z + x.w * k_0.w;
          s[i][1] += x.x * k_1.x + x.y * k_1.y + x.z * k_1.z + x.w * k_1.w;
        }
      }
      const bool live0 = sm.live[lane] != 0, live1 = sm.live[lane + 32] != 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float s0 = live0 && k0 + lane < seen[i] ? s[i][0] * a.scale_log2 : -INFINITY;
        const float s1 = live1 && k0 + lane + 32 < seen[i] ? s[i][1] * a.scale_log2 : -INFINITY;
        float mt = fmaxf(s0, s1);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mt = fmaxf(mt, __shfl_xor_sync(~0u, mt, d));
        const float mn = fmaxf(m[i], mt), mu = mn == -INFINITY ? 0.f : mn;
        const float f = exp2f(m[i] - mu), p0 = exp2f(s0 - mu), p1 = exp2f(s1 - mu);
        m[i] = mn;
        l[i] = l[i] * f + p0 + p1;   // summed over the lanes at the end
#pragma unroll
        for (int e = 0; e < V; ++e) o[i][e] *= f;
        sm.p[warp * 4 + i][lane] = p0;
        sm.p[warp * 4 + i][lane + 32] = p1;
      }
      __syncwarp();
#pragma unroll 4
      for (int k = 0; k < kSimpleKeys; k += 4) {
        float4 pr[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pr[i] = *reinterpret_cast<const float4 *>(&sm.p[warp * 4 + i][k]);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float v[V];
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] = sm.v[k + kk][lane * V + e];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float w = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
#pragma unroll
            for (int e = 0; e < V; ++e) o[i][e] += w * v[e];
          }
        }
      }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float sum = l[i];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      const int r = warp * 4 + i;
      if (r < pc.n_rows) {
        float *dst = p.acc + (pc.partial + r) * D + lane * V;
#pragma unroll
        for (int e = 0; e < V; ++e) dst[e] = o[i][e];
        if (lane == 0) p.ml[pc.partial + r] = make_float2(m[i], sum);
      }
    }
  }
}

template <int D, typename T>
cudaError_t launch_simple(const AttendArgs &a, cudaStream_t st) {
  const cudaError_t e =
      cudaFuncSetAttribute(attend_simple_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)sizeof(SimpleSmem<D>));
  if (e != cudaSuccess) return e;
  return pdl_launch(attend_simple_kernel<D, T>, dim3(a.plan.n_ctas), dim3(kSimpleThreads),
                    sizeof(SimpleSmem<D>), st, a);
}

}  // namespace

AttendShape attend_shape(const dbsa_config *cfg) {
  (void)cfg;
  return {kSimpleRows, kSimpleKeys, 2 * 148};
}

cudaError_t launch_attend_pieces(const AttendArgs &a, int head_dim, bool f32, cudaStream_t st) {
  if (head_dim == 128)
    return f32 ? launch_simple<128, float>(a, st) : launch_simple<128, bf16>(a, st);
  return f32 ? launch_simple<64, float>(a, st) : launch_simple<64, bf16>(a, st);
}

}  // namespace dbsa
