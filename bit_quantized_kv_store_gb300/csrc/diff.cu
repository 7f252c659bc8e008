// diff.cu -- differential attention's output heads: the first softmax map's output
// minus lambda times the second's, an optional norm over the head and a scale,
// (1) inside the merge of the split-T partials, (2) on heads already merged (the
// prefill's output).
//
//   y = o1 - lambda o2;  y * rsqrt(mean(y^2) + eps) * (w + offset);  * out_scale
//
// The two maps of an output head share their KV head, so one pass over the cache
// serves both (they are two query heads of its group), and what is left to do is
// here: the merge of "qwen27 CUDA: an opt-in 4-bit attention cache (262K on a
// 24 GB card)", section "What it is", with the subtraction before the rotation
// back (the rotation is linear, so it runs once instead of twice) and the norm on
// the result, without the merged heads going through memory.
//
// Bound: latency (one 32769-token sequence: 3.5 us after the decode's 12.4, the
// partials 1.6 MB in L2; a ragged batch of 32 up to 8000: 5.5 us after 61, 12.6 MB).
#include "merge_fold.cuh"
#include "rows.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

// ---------------------------------------------------------------- cluster helpers
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Store a float to `p`'s place in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ void st_cluster(float* p, uint32_t rank, float v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

__device__ __forceinline__ void put_out(void* out, int dtype, int64_t i, float v) {
  if (dtype == KVQ_DT_BF16) static_cast<__nv_bfloat16*>(out)[i] = __float2bfloat16_rn(v);
  else static_cast<float*>(out)[i] = v;
}

constexpr int kDiffGroups = 8;  // CTAs of an output head: 32 of its 256 values each

// The keys of sequence b, or -1 for a length out of range.
__device__ __forceinline__ int32_t keys_of(const MergeArgs& a, int b) {
  if (a.n_sel > 0) return a.n_sel;
  const int32_t T = a.seq_lens[b];
  return T < 0 || T > a.max_seq_len ? -1 : T;
}

// What needs the whole head, by one warp on its 256 differences: the TQ4 rows'
// transform, the norm, the scale.  Lane l ends with values 8 l .. 8 l + 7.
constexpr int kDiffE = 8;
__device__ __forceinline__ void finish_head(const MergeArgs& a, const DiffView& d, const void* signs, const float* all,
                                            int lane, float (&x)[kDiffE]) {
  constexpr int E = kDiffE;
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = all[E * lane + i];
  if (a.rotate_back == 2) tq4_transform<E>(x, lane_signs<E>(signs, lane), lane, true);
  if (d.norm.weight) {
    uint64_t p[1][E / 2], w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) p[0][i] = pk2(x[2 * i], x[2 * i + 1]);
    load_weight<E>(d.norm, lane, w);
    norm_rows<E, 32, 1>(p, w, d.norm.eps);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) upk2(p[0][i], x[2 * i], x[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] *= d.scale;
}

// A long sequence's few heads: one CTA of 512 threads per (32 output values, output
// head, sequence), two folds side by side, one for each map, then the difference
// in the first warp.  For what needs the whole head (`whole`) the 8 CTAs of the
// head are a cluster that put their values into each other's shared memory; each
// then works on all 256 and writes its own 32.
template <int kBatch>
__global__ void __launch_bounds__(512) merge_diff_kernel(const MergeArgs a, const DiffView d, const void* signs,
                                                         int whole) {
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * kDiffGroups;
  const int grp = blockIdx.x, ho = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, map = tid >> 8;
  const int64_t out0 = ((int64_t)b * (a.Hq >> 1) + ho) * D;
  const int32_t T = keys_of(a, b);
  if (T <= 0) {  // (the whole cluster: T is the sequence's)
    if (tid < 32) put_out(d.out, d.out_dtype, out0 + 32 * grp + lane, T < 0 ? NAN : 0.f);
    return;
  }
  const int np = static_cast<int>(((int64_t)T + a.part - 1) / a.part);
  if (whole) cluster_arrive();  // this CTA runs: its shared memory may be written
  __shared__ FoldSmem sm[2];
  __shared__ float second[32], all[D];
  const int64_t base = ((int64_t)b * a.Hq + 2 * ho + map) * a.P;
  const float o = merge_fold<kBatch>(a.ws_m + base, a.ws_z + base, a.ws_acc + base * D + 32 * grp, D, np, tid & 255,
                                     sm[map]);
  if (tid >= 256 && tid < 288) second[lane] = o;
  __syncthreads();
  float y = 0.f;
  if (tid < 32) {
    y = fmaf(-d.lambda[b * d.stride + ho], second[lane], o);
    if (a.rotate_back == 1) y = __fmul_rn(warp_fwht32(y, lane), kHadamardScale);
  }
  if (!whole) {
    if (tid < 32) put_out(d.out, d.out_dtype, out0 + 32 * grp + lane, y * d.scale);
    return;
  }
  cluster_wait();
  if (tid < 32) {
#pragma unroll
    for (int r = 0; r < kDiffGroups; ++r) st_cluster(&all[32 * grp + lane], r, y);
  }
  cluster_arrive();
  cluster_wait();
  if (tid >= 32) return;
  float x[kDiffE];
  finish_head(a, d, signs, all, lane, x);
  if (lane / (32 / kDiffGroups) == grp) {
#pragma unroll
    for (int i = 0; i < kDiffE; ++i) put_out(d.out, d.out_dtype, out0 + kDiffE * lane + i, x[i]);
  }
}

// Many heads, or few partitions: one CTA of T threads per (output head, sequence).
// The fold's arithmetic (merge_fold.cuh) in another arrangement, with the same bits: the running maximum of row r of 32 (partitions r, r + 32, ...)
// does not depend on the values, so one warp per map works out the rescaling
// weights of every partition once; the other dimension, 64 chunks of 4 values in
// T / 64 groups of 4 rows, is then plain multiply-adds over coalesced loads, the
// first of which are in flight meanwhile.  T: 512, or 256 for at most 16 partitions
// (rows 16 .. 31 are empty), which lets three CTAs share an SM instead of one.
// A batch of 32 sequences of up to 8000 keys, 16 partitions a head: 5.5 us; 12 us
// with 512 threads, 30 us with the cluster of 8 CTAs a head (thousands, each with
// its own barriers for 32 KB of partials).  One sequence's 12 heads of 65 partitions:
// 6.8 us here, 4.8 us there (the wait for the decode included).
constexpr int kRowMaxP = 1024;  // partitions whose weights fit in shared memory

template <int T>
struct RowMergeSmem {
  float acc[2][T / 16][256];
  float wr[2][32], z[2][32];
  float all[256], second[256];
  int nan[2], empty[2];
};

template <int kBatch, int T>
__global__ void __launch_bounds__(T) merge_diff_row_kernel(const MergeArgs a, const DiffView d, const void* signs) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  constexpr int RG = T / 64;  // groups of rows; each takes rows rg, rg + RG, .. of 4 RG
  RowMergeSmem<T>& sm = *reinterpret_cast<RowMergeSmem<T>*>(smem_raw);
  float2* wts = reinterpret_cast<float2*>(smem_raw + sizeof(RowMergeSmem<T>));  // [2][np] (old, new) weights
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * kDiffGroups;
  const int ho = blockIdx.x, b = blockIdx.y;
  const int tid = threadIdx.x, lane = tid & 31, warp = warp_index();
  const int64_t out0 = ((int64_t)b * (a.Hq >> 1) + ho) * D;
  const int32_t keys = keys_of(a, b);
  if (keys <= 0) {
    if (tid < D) put_out(d.out, d.out_dtype, out0 + tid, keys < 0 ? NAN : 0.f);
    return;
  }
  const int np = static_cast<int>(((int64_t)keys + a.part - 1) / a.part);
  const int64_t base = ((int64_t)b * a.Hq + 2 * ho) * a.P;  // map 1's partials follow map 0's
  const int chunk = tid & 63, rg = tid >> 6;
  const float* accp = a.ws_acc + base * D + 4 * chunk;
  auto load = [&](int i0, float4 (&v)[kBatch][2][4]) {  // partitions i0 + 32 k + rg + RG j of both maps
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + 32 * k + rg + RG * j;
          v[k][m][j] = i < np ? *reinterpret_cast<const float4*>(accp + ((int64_t)m * a.P + i) * D)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
        }
  };
  float4 v[kBatch][2][4];
  load(0, v);
  if (warp < 2) {  // map `warp`, row `lane`: the weights of its partitions
    const float* m = a.ws_m + base + (int64_t)warp * a.P;
    const float* z = a.ws_z + base + (int64_t)warp * a.P;
    float Mt = -INFINITY, Zt = 0.f;
    bool nan_seen = false;
    for (int i = lane; i < np; i += 32) {
      const float mi = m[i], zi = z[i];
      nan_seen |= isnan(mi) || isnan(zi);
      const float Mn = fmaxf(Mt, mi);
      float2 w = make_float2(1.f, 0.f);
      if (Mn != -INFINITY) {
        w = make_float2(exp2f(Mt - Mn), exp2f(mi - Mn));
        Zt = fmaf(Zt, w.x, zi * w.y);
        Mt = Mn;
      }
      wts[warp * np + i] = w;
    }
    float M = Mt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float wr = Mt == -INFINITY ? 0.f : exp2f(Mt - M);
    sm.wr[warp][lane] = wr;
    sm.z[warp][lane] = Zt * wr;
    const int any_nan = __any_sync(0xffffffffu, nan_seen);
    if (lane == 0) {
      sm.nan[warp] = any_nan;
      sm.empty[warp] = M == -INFINITY;
    }
  }
  __syncthreads();
  float4 A[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) A[m][j] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0;;) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + 32 * k + rg + RG * j;
          if (i >= np) continue;
          const float2 w = wts[m * np + i];
          const float4 u = v[k][m][j];
          A[m][j].x = fmaf(A[m][j].x, w.x, u.x * w.y);
          A[m][j].y = fmaf(A[m][j].y, w.x, u.y * w.y);
          A[m][j].z = fmaf(A[m][j].z, w.x, u.z * w.y);
          A[m][j].w = fmaf(A[m][j].w, w.x, u.w * w.y);
        }
    i0 += 32 * kBatch;
    if (i0 >= np) break;
    load(i0, v);
  }
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = rg + RG * j;
      if (r >= np) continue;
      const float wr = sm.wr[m][r];
      *reinterpret_cast<float4*>(&sm.acc[m][r][4 * chunk]) =
          make_float4(A[m][j].x * wr, A[m][j].y * wr, A[m][j].z * wr, A[m][j].w * wr);
    }
  __syncthreads();
  const int col = tid & 255, rows = min(np, 32);
  const auto folded = [&](int m) {  // value col of map m
    float o = 0.f, Z = 0.f;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) {  // ascending rows, as in the fold
      o += sm.acc[m][r][col];
      Z += sm.z[m][r];
    }
    o = (sm.empty[m] || Z == 0.f) ? 0.f : o / Z;
    return sm.nan[m] ? NAN : o;
  };
  float o0 = 0.f, o1 = 0.f;
  if constexpr (T == 512) {
    if (tid >= 256) sm.second[col] = folded(1);
    else o0 = folded(0);
    __syncthreads();
    if (tid < 256) o1 = sm.second[col];
  } else {
    o0 = folded(0);
    o1 = folded(1);
  }
  const bool whole = d.norm.weight != nullptr || a.rotate_back == 2;
  if (tid < 256) {
    float y = fmaf(-d.lambda[b * d.stride + ho], o1, o0);
    if (a.rotate_back == 1) y = __fmul_rn(warp_fwht32(y, lane), kHadamardScale);
    if (!whole) put_out(d.out, d.out_dtype, out0 + col, y * d.scale);
    else sm.all[col] = y;
  }
  if (!whole) return;
  __syncthreads();
  if (warp != 0) return;
  float x[kDiffE];
  finish_head(a, d, signs, sm.all, lane, x);
#pragma unroll
  for (int i = 0; i < kDiffE; ++i) put_out(d.out, d.out_dtype, out0 + kDiffE * lane + i, x[i]);
}

template <int kBatch, int T>
cudaError_t launch_row(const MergeArgs& a, const DiffView& d, const void* signs, int B, cudaStream_t s) {
  constexpr auto kern = merge_diff_row_kernel<kBatch, T>;
  constexpr int fixed = static_cast<int>(sizeof(RowMergeSmem<T>));
  cudaError_t e = set_max_smem_once<kern>(fixed + 2 * kRowMaxP * 8);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.Hq / 2, B), dim3(T), fixed + static_cast<size_t>(2) * a.P * 8, s, a, d, signs);
}

// The partials of a prompt chunk's ranges of keys, merged, subtracted and rotated
// back: one warp per (row, output head), lane l holding values 8 l .. 8 l + 7 of the
// head; ranges in ascending order.
__global__ void __launch_bounds__(256) prefill_diff_merge_kernel(const __grid_constant__ PrefillArgs a, FastDiv hd,
                                                                 int wide, const DiffView d) {
  pdl_wait();
  pdl_trigger();
  constexpr int E = 8, W = 256;
  const int lane = threadIdx.x & 31, heads = a.Hq / 2;
  const uint32_t i = blockIdx.x * (blockDim.x >> 5) + warp_index();  // row * output heads + head
  if (i >= static_cast<uint32_t>(a.n_q) * heads) return;
  const uint32_t row = fast_div(i, hd), h = i - row * hd.d;
  const RowsView in{a.ws_acc, 0, 0, KVQ_DT_F32, 1};
  const int64_t range = (int64_t)a.n_q * a.Hq;  // rows of a range
  uint64_t y1[1][E / 2];
  uint64_t(&y)[E / 2] = y1[0];
#pragma unroll
  for (int map = 0; map < 2; ++map) {
    const int64_t r0 = 2 * (int64_t)i + map;
    float M = -INFINITY;
    for (int s = 0; s < a.splits; ++s) M = fmaxf(M, a.ws_m[r0 + s * range]);
    uint64_t o[E / 2];
#pragma unroll
    for (int j = 0; j < E / 2; ++j) o[j] = pk2(0.f, 0.f);
    float Z = 0.f;
    for (int s = 0; s < a.splits; ++s) {
      const int64_t r = r0 + s * range;
      const float w = exp2f(a.ws_m[r] - M);  // NaN where the range's pages were bad
      Z = fmaf(a.ws_z[r], w, Z);
      RawRow<E, false> raw;
      load_raw<E, false>(in, r * W, lane, raw);
      uint64_t v[E / 2];
      unpack_row<E, false>(raw, v);
#pragma unroll
      for (int j = 0; j < E / 2; ++j) o[j] = fma2(v[j], pk2(w, w), o[j]);
    }
    const float inv = __fdiv_rn(1.f, Z);
    const float c = map == 0 ? inv : -d.lambda[row * d.stride + h] * inv;
#pragma unroll
    for (int j = 0; j < E / 2; ++j) y[j] = map == 0 ? mul2(o[j], pk2(c, c)) : fma2(o[j], pk2(c, c), y[j]);
  }
  if (a.rotate) rotate_row_had32<E>(y, lane);
  if (d.norm.weight) {
    uint64_t w[E / 2];
    load_weight<E>(d.norm, lane, w);
    norm_rows<E, 32, 1>(y1, w, d.norm.eps);
  }
#pragma unroll
  for (int j = 0; j < E / 2; ++j) y[j] = mul2(y[j], pk2(d.scale, d.scale));
  const RowsView out{d.out, 0, 0, d.out_dtype, wide};
  write_row<E>(out, (int64_t)i * W, lane, y);
}

// One warp per (row, output head); lane l holds elements E l .. E l + E - 1.  Bound:
// memory (4096 rows of 24 heads of 256, normed: 23.0 us to fp32, 6.6 TB/s, 97 % of the
// measured copy; 19.4 us to bf16).
template <int E>
__global__ void __launch_bounds__(256) diff_heads_kernel(const float* __restrict__ x, int64_t n, FastDiv hd, int wide,
                                                         const DiffView d) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = 32 * E;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp_index();  // row * output heads + head
  if (i >= n) return;
  const uint32_t row = fast_div(static_cast<uint32_t>(i), hd), h = static_cast<uint32_t>(i) - row * hd.d;
  const RowsView in{const_cast<float*>(x), 0, 0, KVQ_DT_F32, wide};
  RawRow<E, false> r1, r2;
  load_raw<E, false>(in, 2 * i * W, lane, r1);
  load_raw<E, false>(in, (2 * i + 1) * W, lane, r2);
  const float lam = d.lambda[row * d.stride + h];
  uint64_t p1[1][E / 2], q[E / 2];
  uint64_t(&p)[E / 2] = p1[0];
  unpack_row<E, false>(r1, p);
  unpack_row<E, false>(r2, q);
#pragma unroll
  for (int j = 0; j < E / 2; ++j) p[j] = fma2(pk2(-lam, -lam), q[j], p[j]);
  if (d.norm.weight) {
    load_weight<E>(d.norm, lane, q);
    norm_rows<E, 32, 1>(p1, q, d.norm.eps);
  }
#pragma unroll
  for (int j = 0; j < E / 2; ++j) p[j] = mul2(p[j], pk2(d.scale, d.scale));
  const RowsView out{d.out, 0, 0, d.out_dtype, wide};
  write_row<E>(out, i * W, lane, p);
}

}  // namespace

cudaError_t launch_merge_diff(const MergeArgs& a, const DiffView& d, const kvq_cache& c, int B, cudaStream_t s) {
  // A CTA for each head where that fills half the GPU, or where a head has few
  // partitions; 8 CTAs for each head of a long sequence.
  const int64_t heads = (int64_t)(a.Hq / 2) * B, n_sm = device_sm_count();
  cudaError_t e;
  if (a.P <= kRowMaxP && (a.P <= 32 || 2 * heads >= n_sm)) {
    e = a.P <= 16   ? launch_row<1, 256>(a, d, c.signs, B, s)
        : a.P <= 32 ? launch_row<1, 512>(a, d, c.signs, B, s)
                    : launch_row<2, 512>(a, d, c.signs, B, s);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
  }
  const int whole = (d.norm.weight != nullptr || a.rotate_back == 2) ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kDiffGroups, a.Hq / 2, B);
  cfg.blockDim = dim3(512);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kDiffGroups;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = whole ? 2 : 1;
  // (as the merge: more of a thread's partitions loaded at once where there are more)
  if (a.P > 128 && heads * kDiffGroups <= n_sm)
    e = a.P > 256 ? cudaLaunchKernelEx(&cfg, merge_diff_kernel<17>, a, d, c.signs, whole)
                  : cudaLaunchKernelEx(&cfg, merge_diff_kernel<8>, a, d, c.signs, whole);
  else
    e = cudaLaunchKernelEx(&cfg, merge_diff_kernel<4>, a, d, c.signs, whole);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_prefill_diff_merge(const PrefillArgs& a, const DiffView& d, cudaStream_t s) {
  const int64_t n = (int64_t)a.n_q * (a.Hq / 2);
  const int wide = (reinterpret_cast<uintptr_t>(d.out) & 31u) == 0 ? 1 : 0;
  cudaError_t e = launch_pdl(prefill_diff_merge_kernel, dim3(static_cast<unsigned>((n + 7) / 8)), dim3(256), 0, s, a,
                             make_fastdiv(static_cast<uint32_t>(a.Hq / 2)), wide, d);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_diff_heads(const float* x, int64_t rows, int Hq, int width, const DiffView& d, cudaStream_t s) {
  // launches of fewer than 2^31 output heads, so that the kernel divides in 32 bits
  const int64_t heads = Hq / 2, max_rows = ((int64_t(1) << 31) - 8) / heads;
  const size_t esz = d.out_dtype == KVQ_DT_BF16 ? 2 : 4;
  const FastDiv hd = make_fastdiv(static_cast<uint32_t>(heads));
  const int wide =
      (reinterpret_cast<uintptr_t>(x) & 31u) == 0 && (reinterpret_cast<uintptr_t>(d.out) & 31u) == 0 ? 1 : 0;
  for (int64_t r0 = 0; r0 < rows; r0 += max_rows) {
    const int64_t n = (rows - r0 < max_rows ? rows - r0 : max_rows) * heads;
    DiffView p = d;
    p.lambda += r0 * d.stride;
    p.out = static_cast<uint8_t*>(d.out) + r0 * heads * width * esz;
    const float* xr = x + r0 * Hq * width;
    const dim3 grid(static_cast<unsigned>((n + 7) / 8)), block(256);
    cudaError_t e;
    switch (width) {
      case 64: e = launch_pdl(diff_heads_kernel<2>, grid, block, 0, s, xr, n, hd, wide, p); break;
      case 128: e = launch_pdl(diff_heads_kernel<4>, grid, block, 0, s, xr, n, hd, wide, p); break;
      case 256: e = launch_pdl(diff_heads_kernel<8>, grid, block, 0, s, xr, n, hd, wide, p); break;
      case 512: e = launch_pdl(diff_heads_kernel<16>, grid, block, 0, s, xr, n, hd, wide, p); break;
      default: return cudaErrorInvalidValue;
    }
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace kvq
