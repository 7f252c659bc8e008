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

// One CTA of 512 threads per (32 output values, output head, sequence): two folds
// side by side, one for each map, then the difference in the first warp.  What
// needs the whole head -- the norm, and the TQ4 rows' transform -- is done after
// the 8 CTAs of the head, one cluster, have put their values into each other's
// shared memory (`whole`); each then works on all 256 and writes its own 32.
template <int kBatch>
__global__ void __launch_bounds__(512, kBatch > 4 ? 1 : kBatch == 2 ? 3 : 1)
    merge_diff_kernel(const MergeArgs a, const DiffView d, const void* signs, int whole) {
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * kDiffGroups;
  const int grp = blockIdx.x, ho = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, map = tid >> 8;
  const int64_t out0 = ((int64_t)b * (a.Hq >> 1) + ho) * D;
  int32_t T = a.n_sel;
  bool bad = false;
  if (a.n_sel == 0) {
    T = a.seq_lens[b];
    bad = T < 0 || T > a.max_seq_len;
  }
  const int np = bad ? 0 : static_cast<int>(((int64_t)T + a.part - 1) / a.part);
  if (np == 0) {  // (the whole cluster: T is the sequence's)
    if (tid < 32) put_out(d.out, d.out_dtype, out0 + 32 * grp + lane, bad ? NAN : 0.f);
    return;
  }
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
  constexpr int E = D / 32;
  float x[E];
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = all[E * lane + i];
  if (a.rotate_back == 2) tq4_transform<E>(x, lane_signs<E>(signs, lane), lane, true);
  if (d.norm.weight) {
    float w[E];
    load_weight<E>(d.norm, lane, w);
    norm_row<E>(x, w, d.norm.eps);
  }
  if (lane / (32 / kDiffGroups) == grp) {
#pragma unroll
    for (int i = 0; i < E; ++i) put_out(d.out, d.out_dtype, out0 + E * lane + i, x[i] * d.scale);
  }
}

// One warp per (row, output head); lane l holds elements E l .. E l + E - 1.
template <int E>
__global__ void __launch_bounds__(256) diff_heads_kernel(const float* __restrict__ x, int64_t n, FastDiv hd, int wide,
                                                         const DiffView d) {
  pdl_wait();
  pdl_trigger();
  constexpr int W = 32 * E;
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);  // row * output heads + head
  if (i >= n) return;
  const uint32_t row = fast_div(static_cast<uint32_t>(i), hd), h = static_cast<uint32_t>(i) - row * hd.d;
  const RowsView in{const_cast<float*>(x), 0, 0, KVQ_DT_F32, wide};
  float p[E], q[E];
  load_row<E>(in, 2 * i * W, lane, p);
  load_row<E>(in, (2 * i + 1) * W, lane, q);
  const float lam = d.lambda[row * d.stride + h];
#pragma unroll
  for (int j = 0; j < E; ++j) p[j] = fmaf(-lam, q[j], p[j]);
  if (d.norm.weight) {
    load_weight<E>(d.norm, lane, q);
    norm_row<E>(p, q, d.norm.eps);
  }
#pragma unroll
  for (int j = 0; j < E; ++j) p[j] *= d.scale;
  const RowsView out{d.out, 0, 0, d.out_dtype, wide};
  write_row<E>(out, i * W, lane, p);
}

}  // namespace

cudaError_t launch_merge_diff(const MergeArgs& a, const DiffView& d, const kvq_cache& c, int B, cudaStream_t s) {
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
  // the merge's rule on CTAs of twice the threads
  const int64_t ctas = (int64_t)kDiffGroups * (a.Hq / 2) * B, n_sm = device_sm_count();
  cudaError_t e;
  if (a.P > 128 && ctas <= n_sm)
    e = a.P > 256 ? cudaLaunchKernelEx(&cfg, merge_diff_kernel<17>, a, d, c.signs, whole)
                  : cudaLaunchKernelEx(&cfg, merge_diff_kernel<8>, a, d, c.signs, whole);
  else
    e = ctas > 4 * n_sm ? cudaLaunchKernelEx(&cfg, merge_diff_kernel<2>, a, d, c.signs, whole)
                        : cudaLaunchKernelEx(&cfg, merge_diff_kernel<4>, a, d, c.signs, whole);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_diff_heads(const float* x, int64_t rows, int Hq, int width, const DiffView& d, cudaStream_t s) {
  // launches of fewer than 2^31 output heads, so that the kernel divides in 32 bits
  const int64_t heads = Hq / 2, max_rows = ((int64_t(1) << 31) - 8) / heads;
  const size_t esz = d.out_dtype == KVQ_DT_BF16 ? 2 : 4;
  const FastDiv hd = make_fastdiv(static_cast<uint32_t>(heads));
  const int wide =
      (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (reinterpret_cast<uintptr_t>(d.out) & 15u) == 0 ? 1 : 0;
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
