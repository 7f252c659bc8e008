// latent.cu -- fp8 latent rows from a layer's projections in one launch: the latent
// part normed, the rope part position-rotated, both quantised and stored; and the
// absorbed queries' rope parts rotated beside their latent parts.
//
// Follows "KV cache quantization: fp8 (KV8) + 4-bit TurboQuant", KV8 base commit: the
// producer quantises the fresh normed and roped row (e4m3 bytes, a scale amax/448 for
// either part).  The arithmetic is that of the calls it stands for: the norm of a
// row of 512 and the rotation of one of 64 (rows.cuh, rope.cuh), the fp8 store's codes.
//
// One warp takes rows of one token one after another, the query heads and then the
// latent row, the next row's loads in flight: lane l holds latent elements 16 l ..
// 16 l + 15, and lanes 0 .. 3 the rope part's 64 as a row of their own.  The token's
// angles are worked out once per warp.
//
// Bound: memory (a query row is 1152 bytes in bf16 and 2304 out).  4096 tokens of 128
// heads: 307 us, 1.82 GB, 5.9 TB/s (88 % of the measured copy; 367 us without the
// next row's loads ahead, 328 us with ranges of heads for 1024 warps of an SM).  One
// token of 128 heads: 3.8 us, latency.
//
// This translation unit is compiled with -fmad=false.
#include "fp8_code.cuh"
#include "rope.cuh"

namespace kvq {

namespace {

constexpr int kLatent = 512, kRopePart = 64, kRopeLanes = kRopePart / kRopeE, kWarps = 8, kWarpsPerSm = 64;

// One part's codes and scale: LANES lanes of 16 values each.
template <int LANES>
__device__ __forceinline__ void fp8_part(const uint64_t (&x)[kRopeE / 2], uint8_t* codes, float* scale, int lane) {
  float v[kRopeE], amax = 0.f;
#pragma unroll
  for (int i = 0; i < kRopeE / 2; ++i) upk2(x[i], v[2 * i], v[2 * i + 1]);
#pragma unroll
  for (int i = 0; i < kRopeE; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float inv = __fdiv_rn(448.0f, amax);
  const bool zero = amax == 0.0f || isinf(inv);
  uint32_t w[kRopeE / 4];
#pragma unroll
  for (int q = 0; q < kRopeE / 4; ++q) {
    w[q] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[q] |= static_cast<uint32_t>(zero ? 0 : e4m3_encode(__fmul_rn(v[4 * q + i], inv))) << (8 * i);
  }
  if (lane < LANES) {
    *reinterpret_cast<uint4*>(codes + kRopeE * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    if (lane == 0) *scale = __fdiv_rn(amax, 448.0f);
  }
}

// BF: both inputs are bf16.
template <bool BF>
__global__ void __launch_bounds__(32 * kWarps) latent_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float4 angles_sh[kWarps][2 * kChunks];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = warp_index();
  const int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n_tok) return;
  // rows [h0, h1) of the token; row Hq is the latent row
  const int h0 = blockIdx.y * static_cast<int>(a.per), h1 = min(h0 + static_cast<int>(a.per), a.Hq + 1);
  const bool in = lane < kRopeLanes;
  RawRow<kRopeE, BF> raw, tail;  // the next row
#pragma unroll
  for (int i = 0; i < (BF ? kRopeE / 2 : kRopeE); ++i) tail.w[i] = 0;
  const auto load = [&](int h) {
    const RowsView& src = h == a.Hq ? a.k : a.q;
    const int64_t e0 = tok * src.ts + (h == a.Hq ? 0 : h * src.hs);
    load_raw<kRopeE, BF>(src, e0, lane, raw);
    if (in) load_raw<kRopeE, BF>(src, e0 + kLatent, lane, tail);
  };
  load(h0);
  RopeLane g;
  if (a.rope.rot != 0) {
    int32_t pos[4];
    load_pos(a.rope, tok, pos);
    make_angles(a.rope, pos, lane, a.status, angles_sh[warp]);
    g = rope_lane(a.rope, angles_sh[warp], in ? lane : 0, in ? lane : 0);
    if (!in) g.src[0] = g.src[1] = lane;
  }
  for (int h = h0; h < h1; ++h) {
    const bool latent = h == a.Hq;
    uint64_t x[1][kRopeE / 2], r[1][kRopeE / 2];
    unpack_row<kRopeE, BF>(raw, x[0]);
    unpack_row<kRopeE, BF>(tail, r[0]);
    if (h + 1 < h1) load(h + 1);
    if (a.rope.rot != 0) rope_rows<1>(a.rope, g, in ? lane : 0, r);
    if (!latent) {
      const int64_t o0 = tok * a.qo.ts + h * a.qo.hs;
      write_row<kRopeE>(a.qo, o0, lane, x[0]);
      if (in) write_row<kRopeE>(a.qo, o0 + kLatent, lane, r[0]);
      continue;
    }
    if (a.kn.weight) {
      uint64_t w[kRopeE / 2];
      load_weight<kRopeE>(a.kn, lane, w);
      norm_rows<kRopeE, 32, 1>(x, w, a.kn.eps);
    }
    const int32_t slot = a.slots[tok];
    if (slot < 0) return;
    if ((int64_t)slot >= (int64_t)a.c.num_pages * a.c.page_size) {
      if (lane == 0) set_status(a.status, KVQ_DEV_BAD_SLOT);
      return;
    }
    // (one head: the row's index is the slot)
    fp8_part<32>(x[0], static_cast<uint8_t*>(a.c.k) + (int64_t)slot * kLatent,
                 static_cast<float*>(a.c.k_scale) + slot, lane);
    fp8_part<kRopeLanes>(r[0], static_cast<uint8_t*>(a.c.v) + (int64_t)slot * kRopePart,
                         static_cast<float*>(a.c.v_scale) + slot, lane);
  }
}

}  // namespace

cudaError_t launch_latent(const NormRopeArgs& args, cudaStream_t s) {
  NormRopeArgs a = args;
  // the heads in as many ranges as fill the GPU a few times over
  const int64_t n_sm = device_sm_count() > 0 ? device_sm_count() : 1, rows = a.Hq + 1;
  int64_t per = (a.n_tok * rows + n_sm * kWarpsPerSm - 1) / (n_sm * kWarpsPerSm);
  a.per = per > rows ? rows : per;
  int wpc = kWarps;  // tokens per CTA
  while (wpc > 1 && a.n_tok < wpc) wpc >>= 1;
  const dim3 grid(static_cast<unsigned>((a.n_tok + wpc - 1) / wpc), static_cast<unsigned>((rows + a.per - 1) / a.per));
  const bool bf = a.k.dtype == KVQ_DT_BF16 && (a.Hq == 0 || a.q.dtype == KVQ_DT_BF16);
  cudaError_t e = bf ? launch_pdl(latent_kernel<true>, grid, dim3(32 * wpc), 0, s, a)
                     : launch_pdl(latent_kernel<false>, grid, dim3(32 * wpc), 0, s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace kvq
