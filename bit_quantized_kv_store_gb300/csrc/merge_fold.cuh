// merge_fold.cuh -- the fold of one (sequence, query head)'s split-T partials into 32
// of its output values by 256 threads, shared by the merge kernels.
#pragma once
#include "kernels.cuh"

namespace kvq {

// Shared memory of one fold.
struct FoldSmem {
  float m[32], z[32];  // per row: its maximum, then its z rescaled to the fold's
  float acc[32][33];
  int nan;
};

// kBatch: partitions a row-thread loads before using them (4; for a grid of few
// CTAs over many partitions 8, or 17 past 256 partitions, so that a 262K-key
// sequence's 513 take one round trip, still at two CTAs per SM: fewer round
// trips, more registers; for a grid of many waves 2, at six CTAs per SM: more
// CTAs resident, more round trips); the updates run in ascending partition
// order either way, so the bits are the same.
//
// Thread `tid` of the fold's 256 (whole warps; every thread of the CTA calls it,
// for the __syncthreads), the partials' rows m, z and accp = the partials'
// contexts at the first of the 32 values; np partials of Dv values.  Returns value
// `lane` of the 32 in the fold's first warp.
template <int kBatch>
__device__ __forceinline__ float merge_fold(const float* m, const float* z, const float* acc0, int Dv, int np, int tid,
                                            FoldSmem& sm) {
  const int lane = tid & 31;
  const int chunk = tid & 7, row = tid >> 3;
  const float* accp = acc0 + 4 * chunk;
  if (tid == 0) sm.nan = 0;

  // per-thread running partial over partitions row, row + 32, ...
  float Mt = -INFINITY, Zt = 0.f;
  float4 At = make_float4(0.f, 0.f, 0.f, 0.f);
  int nan_seen = 0;
  for (int i0 = row; i0 < np; i0 += kBatch * 32) {
    float mv[kBatch], zv[kBatch];
    float4 av[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {  // all loads of the batch first
      const int i = i0 + 32 * k;
      mv[k] = -INFINITY;
      zv[k] = 0.f;
      av[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < np) {
        mv[k] = m[i];
        if (chunk == 0) zv[k] = z[i];
        av[k] = *reinterpret_cast<const float4*>(accp + (int64_t)i * Dv);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + 32 * k >= np) break;
      nan_seen |= isnan(mv[k]) || isnan(zv[k]);  // (a bad page; keys whose every score is NaN, m = -inf)
      const float Mn = fmaxf(Mt, mv[k]);
      if (Mn == -INFINITY) continue;  // nothing attended so far
      const float wo = exp2f(Mt - Mn), wn = exp2f(mv[k] - Mn);
      Zt = fmaf(Zt, wo, zv[k] * wn);
      At.x = fmaf(At.x, wo, av[k].x * wn);
      At.y = fmaf(At.y, wo, av[k].y * wn);
      At.z = fmaf(At.z, wo, av[k].z * wn);
      At.w = fmaf(At.w, wo, av[k].w * wn);
      Mt = Mn;
    }
  }
  nan_seen = __any_sync(0xffffffffu, nan_seen);
  __syncthreads();  // sm.nan initialised
  if (nan_seen && lane == 0) sm.nan = 1;
  if (chunk == 0) {
    sm.m[row] = Mt;
    sm.z[row] = Zt;
  }
  __syncthreads();
  // M = max over the 32 rows; each row's partial rescaled to M
  float M = sm.m[0];
#pragma unroll
  for (int r = 1; r < 32; ++r) M = fmaxf(M, sm.m[r]);
  const bool empty = (M == -INFINITY);
  const float wr = (empty || Mt == -INFINITY) ? 0.f : exp2f(Mt - M);
  sm.acc[row][4 * chunk + 0] = At.x * wr;
  sm.acc[row][4 * chunk + 1] = At.y * wr;
  sm.acc[row][4 * chunk + 2] = At.z * wr;
  sm.acc[row][4 * chunk + 3] = At.w * wr;
  __syncthreads();  // every thread has read sm.m
  if (chunk == 0) sm.z[row] = Zt * wr;
  __syncthreads();
  float o = 0.f;
  if (tid < 32) {
    float Z = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) {  // ascending rows, a fixed order (unrolled: the loads go ahead of the adds)
      o += sm.acc[r][lane];
      Z += sm.z[r];
    }
    o = (empty || Z == 0.f) ? 0.f : o / Z;
    if (sm.nan) o = NAN;
  }
  return o;
}

}  // namespace kvq
