// norm_rope.cu -- norms of queries and keys per head and rotary positions in one
// pass, alone or on the way into the cache: queries rotated into the cache's
// space, keys and values quantised and stored, in one launch.
//
// The stored rows follow the formats' definitions in kvq.h ("KV cache
// quantization: fp8 (KV8) + 4-bit TurboQuant", KV8 base commit: the producer
// quantises the fresh normed and roped row; "qwen27 CUDA: an opt-in 4-bit
// attention cache (262K on a 24 GB card)", section "What it is").
//
// The arithmetic per row, in fp32:
//   y = x * r * (w + offset), r = rsqrt(mean(x^2) + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin) for every rotary pair.
// The angle of a pair is 2 pi times the fraction of pos * turns, turns a 64-bit
// fixed-point fraction of a turn: the product wraps modulo one turn exactly, so
// a far position costs nothing in accuracy (an fp32 angle of 262144 radians is
// off by 0.016) and no fp64.  Its top 32 bits as a float in [-1, 1) go to
// sincospif: the rounding there is at most 2^-25 of half a turn, 1e-7 radians.
//
// A lane holds 16 consecutive elements of a row (32 bytes of bf16, one load), so a
// row of 256 lies over 16 lanes and a warp works on two heads of its token at once
// (D = 64, 128, 512: eight, four, one): against one row for a whole warp (183
// instructions a row of 256, 24.7 us for 4099 tokens of 24 heads) the reductions,
// the butterflies across lanes and the addressing are shared by more rows.  A warp
// takes `hpw` heads of one token, one batch after another with the next one's loads
// in flight; the angles (the same for every head) are computed once per warp,
// spread over its lanes, and read back from shared memory.  Bound: memory for a
// prompt chunk, the launch for a decode step.
//
// This translation unit is compiled with -fmad=false.
#include "rows.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

constexpr int kNoStore = -1;
constexpr int kMaxPairs = 128;
constexpr int kMaxWarps = 8;
constexpr int E = 16;  // elements of a lane

// cos and sin of the token's rotary pairs, once per warp, in shared memory: chunk c of
// 16 bytes holds (cos, cos, sin, sin) of pairs 2c and 2c + 1, as the packed
// products take them; a second copy has the sines negated, for the pairs' first
// elements.  Every 8 chunks are followed by one of padding, so that lanes that
// each read 8 consecutive chunks hit different banks.
constexpr int kChunks = kMaxPairs / 2 + kMaxPairs / 16;  // of a copy
__device__ __forceinline__ int chunk_place(int c) { return c + (c >> 3); }

__device__ __forceinline__ float2 angle(const RopeView& r, int pair, const int32_t (&pos)[4], int32_t* status) {
  const uint64_t w = r.table[pair];
  const int axis = static_cast<int>(w & 3u);
  int32_t p = pos[0];
#pragma unroll
  for (int a = 1; a < 4; ++a)
    if (axis == a) p = pos[a];
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(p)) * (w & ~uint64_t(3));
  float t = __fmul_rn(static_cast<float>(static_cast<int32_t>(phase >> 32)), 4.656612873077393e-10f);  // 2^-31
  if (axis >= r.axes) {
    set_status(status, KVQ_DEV_BAD_INDEX);
    t = NAN;
  }
  float2 cs;
  sincospif(t, &cs.y, &cs.x);
  return cs;
}

__device__ __forceinline__ void make_angles(const RopeView& r, int64_t tok, int lane, int32_t* status, float4* sh) {
  int32_t pos[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) pos[a] = a < r.axes ? r.pos[a * r.pos_stride + tok] : 0;
  for (int p = lane; p < (r.rot >> 1); p += 32) {
    const float2 cs = angle(r, p, pos, status);
    float* at = reinterpret_cast<float*>(&sh[chunk_place(p >> 1)]) + (p & 1);
    at[0] = cs.x;
    at[2] = cs.y;
    at += 4 * kChunks;
    at[0] = cs.x;
    at[2] = -cs.y;
  }
  __syncwarp();
}

// What the lane's rotation takes from where, worked out once per warp.  Half-split
// pairs (i, i + half), half a multiple of 8, go by blocks of 8 elements, two to a
// lane: a block's partner block lies half / 8 blocks away, in the same half of its
// lane or (half an odd multiple of 8) the other one.
struct RopeLane {
  const float4* cs[2];  // the blocks' first chunks (interleaved: cs[0] the lane's)
  int src[2];           // the lanes that hold the partner blocks
  bool in[2];           // whether a block is rotated at all
};

__device__ __forceinline__ RopeLane rope_lane(const RopeView& r, const float4* sh, int lane, int l) {
  RopeLane g;
  const int half = r.rot >> 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int e = E * l + 8 * k;
    g.in[k] = e < r.rot;
    const bool first = e < half;
    g.src[k] = lane - l + (!g.in[k] ? e : first ? e + half : e - half) / E;
    g.cs[k] = sh + (first ? kChunks : 0) + chunk_place(g.in[k] ? (first ? e : e - half) / 2 : 0);
  }
  if (r.interleaved) g.cs[0] = sh + chunk_place(g.in[0] ? E * l / 4 : 0);
  return g;
}

template <int SH, int U>
__device__ __forceinline__ void rope_half_split(const RopeLane& g, uint64_t (&x)[U][E / 2]) {
  uint64_t o[U][E / 2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float a, b;
      upk2(x[u][SH ? i ^ 4 : i], a, b);
      o[u][i] = pk2(__shfl_sync(0xffffffffu, a, g.src[i >> 2]), __shfl_sync(0xffffffffu, b, g.src[i >> 2]));
    }
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (g.in[k]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const ulonglong2 cs = reinterpret_cast<const ulonglong2*>(g.cs[k])[i];
#pragma unroll
        for (int u = 0; u < U; ++u)
          x[u][4 * k + i] = fma2(o[u][4 * k + i], cs.y, mul2(x[u][4 * k + i], cs.x));
      }
    }
}

// (a cos - b sin, b cos + a sin), each as one product and one fused add; l: the
// lane's place in its row.
template <int U>
__device__ __forceinline__ void rope_rows(const RopeView& r, const RopeLane& g, int l, uint64_t (&x)[U][E / 2]) {
  if (!r.interleaved) {
    if (r.rot & 16) rope_half_split<1, U>(g, x);
    else rope_half_split<0, U>(g, x);
    return;
  }
  if (!g.in[0]) return;
  const int e = E * l;
#pragma unroll
  for (int i = 0; i < E / 2; i += 2) {
    const float4 cs = g.cs[0][i / 2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float a, b;
      if (e + 2 * i < r.rot) {
        upk2(x[u][i], a, b);
        x[u][i] = pk2(__fmaf_rn(-b, cs.z, __fmul_rn(a, cs.x)), __fmaf_rn(a, cs.z, __fmul_rn(b, cs.x)));
      }
      if (e + 2 * i + 2 < r.rot) {
        upk2(x[u][i + 1], a, b);
        x[u][i + 1] = pk2(__fmaf_rn(-b, cs.w, __fmul_rn(a, cs.y)), __fmaf_rn(a, cs.w, __fmul_rn(b, cs.y)));
      }
    }
  }
}

// FMT: the cache's format, or kNoStore for rows that are only normed and rotated
// (then every head is a "query" and Hk is 0).  BF: every input is bf16.  LPR: lanes
// of a row.  U: batches of queries worked on side by side, so that one's shuffles
// are in flight during the other's arithmetic.
template <int LPR, int FMT, bool BF, int U>
__global__ void __launch_bounds__(32 * kMaxWarps, 2) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float4 angles_sh[kMaxWarps][2 * kChunks];
  pdl_wait();
  pdl_trigger();
  constexpr int D = E * LPR, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  const int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n_tok) return;
  // this warp's batches of RPW heads: first the queries', then K's, then V's
  const int qb = (a.Hq + RPW - 1) / RPW, kb = (a.Hk + RPW - 1) / RPW;
  const int b0 = blockIdx.y * a.hpw, b1 = min(b0 + a.hpw, qb + 2 * kb);

  // the next batch's rows, ahead of the work on a batch (and first of the angles)
  RawRow<E, BF> next[U];
  const uint8_t* at;  // the first one's address in this lane
  const auto row_of = [&](const RowsView& v, int h) { return element_at(v, tok * v.ts + h * v.hs + E * l); };
  const auto first_row = [&](int b) {  // of batch b, of whichever kind
    const bool is_q = b < qb, is_v = b >= qb + kb;
    const int h = (is_q ? b : is_v ? b - qb - kb : b - qb) * RPW + sub;
    const RowsView& v = is_q ? a.q : is_v ? a.v : a.k;
    at = row_of(v, h);
    if (h < (is_q ? a.Hq : a.Hk)) load_raw_at<E, BF>(at, v.dtype, v.wide, next[0]);
  };
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < (BF ? E / 2 : E); ++i) next[u].w[i] = 0;
  const int64_t step = (a.q.hs * RPW) << (a.q.dtype == KVQ_DT_BF16 ? 1 : 2);  // to the next batch of queries
  const int be = min(b1, qb);
  first_row(b0);
#pragma unroll
  for (int u = 1; u < U; ++u)
    if (b0 + u < be && (b0 + u) * RPW + sub < a.Hq) load_raw_at<E, BF>(at + u * step, a.q.dtype, a.q.wide, next[u]);
  int32_t slot = -1;
  if (FMT != kNoStore && b1 > qb) slot = a.slots[tok];
  RopeLane g;
  if (a.rope.rot != 0 && b0 < qb + kb) {
    make_angles(a.rope, tok, lane, a.status, angles_sh[warp]);
    g = rope_lane(a.rope, angles_sh[warp], lane, l);
  }

  uint64_t w[E / 2];
  uint32_t sw = 0;
  if constexpr (FMT == KVQ_FMT_TQ4) sw = lane_signs<E>(a.c.signs, l);
  if (b0 < qb) {
    if (a.qn.weight) load_weight<E>(a.qn, l, w);
    const int64_t out_step = (a.qo.hs * RPW) << (a.qo.dtype == KVQ_DT_BF16 ? 1 : 2);
    uint8_t* out = row_of(a.qo, b0 * RPW + sub);
    for (int b = b0; b < be; b += U) {
      uint64_t x[U][E / 2];
#pragma unroll
      for (int u = 0; u < U; ++u) unpack_row<E, BF>(next[u], x[u]);
      if (b + U < be) {
        at += U * step;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (b + U + u < be && (b + U + u) * RPW + sub < a.Hq)
            load_raw_at<E, BF>(at + u * step, a.q.dtype, a.q.wide, next[u]);
      } else if (FMT != kNoStore && b1 > qb) {
        first_row(qb);
      }
      if (a.qn.weight) norm_rows<E, LPR, U>(x, w, a.qn.eps);
      if (a.rope.rot != 0) rope_rows<U>(a.rope, g, l, x);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if constexpr (FMT == KVQ_FMT_Q4_HAD32) {
          if (a.rotate) rotate_row_had32<E>(x[u], lane);
        }
        if constexpr (FMT == KVQ_FMT_TQ4) {
          if (a.rotate) rotate_row_tq4<E, LPR>(x[u], sw, lane);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b + u < be && (b + u) * RPW + sub < a.Hq)
          write_row_at<E>(out + u * out_step, a.qo.dtype, a.qo.wide, x[u]);
      out += U * out_step;
    }
  }
  if constexpr (FMT != kNoStore) {
    if (b1 <= qb || slot < 0) return;
    if ((int64_t)slot >= (int64_t)a.c.num_pages * a.c.page_size) {
      if (lane == 0) set_status(a.status, KVQ_DEV_BAD_SLOT);
      return;
    }
    const uint32_t page = fast_div(static_cast<uint32_t>(slot), a.ps);
    const uint32_t off = static_cast<uint32_t>(slot) - page * a.ps.d;
    if (a.kn.weight && b0 < qb + kb) load_weight<E>(a.kn, l, w);
    for (int b = max(b0, qb); b < b1; ++b) {
      const bool is_v = b >= qb + kb;
      const int h = (is_v ? b - qb - kb : b - qb) * RPW + sub;
      const int64_t r = ((int64_t)page * a.Hk + h) * a.c.page_size + off;
      uint64_t x1[1][E / 2];
      uint64_t(&x)[E / 2] = x1[0];
      unpack_row<E, BF>(next[0], x);
      if (b + 1 < b1) first_row(b + 1);
      if (!is_v) {
        if (a.kn.weight) norm_rows<E, LPR, 1>(x1, w, a.kn.eps);
        if (a.rope.rot != 0) rope_rows<1>(a.rope, g, l, x1);
      }
      void* codes = is_v ? a.c.v : a.c.k;
      void* scales = is_v ? a.c.v_scale : a.c.k_scale;
      if constexpr (FMT == KVQ_FMT_BF16) {
        if (h < a.Hk)
          write_row_at<E>(static_cast<uint16_t*>(codes) + r * D + E * l, KVQ_DT_BF16, a.plane_wide, x);
      } else {
        __half s16;
        uint32_t word[2];
        if constexpr (FMT == KVQ_FMT_TQ4) {
          rotate_row_tq4<E, LPR>(x, sw, lane);
          float y[E];
#pragma unroll
          for (int i = 0; i < E / 2; ++i) upk2(x[i], y[2 * i], y[2 * i + 1]);
          tq4_row_codes<E, LPR>(y, word, s16);
          if (h < a.Hk && l == 0) static_cast<__half*>(scales)[r] = s16;
        } else {
          constexpr bool ROT = FMT == KVQ_FMT_Q4_HAD32;
          if constexpr (ROT) rotate_row_had32<E>(x, lane);
          q4_row_codes<E, ROT>(x, word, s16);
          if (h < a.Hk && l % (32 / E) == 0) static_cast<__half*>(scales)[r * (D / 32) + l / (32 / E)] = s16;
        }
        if (h < a.Hk) write_codes<E>(static_cast<uint8_t*>(codes) + r * (D / 2) + l * (E / 2), word);
      }
    }
  }
}

template <int LPR, int FMT>
cudaError_t launch_one(NormRopeArgs a, cudaStream_t s) {
  // Two waves of warps or more where there are rows for them (each warp computes
  // its token's angles once, so no more than that), the batches evenly over them.
  constexpr int RPW = 32 / LPR;
  const int total = (a.Hq + RPW - 1) / RPW + 2 * ((a.Hk + RPW - 1) / RPW);
  const int64_t target = static_cast<int64_t>(device_sm_count()) * 48;
  int64_t bpw = (a.n_tok * total + target - 1) / target;
  if (bpw > total) bpw = total;
  const int chunks = static_cast<int>((total + bpw - 1) / bpw);
  a.hpw = (total + chunks - 1) / chunks;
  int wpc = kMaxWarps;  // tokens per CTA
  while (wpc > 1 && a.n_tok < wpc) wpc >>= 1;
  const dim3 grid(static_cast<unsigned>((a.n_tok + wpc - 1) / wpc), (total + a.hpw - 1) / a.hpw);
  const bool bf = (a.Hq == 0 || a.q.dtype == KVQ_DT_BF16) &&
                  (a.Hk == 0 || (a.k.dtype == KVQ_DT_BF16 && a.v.dtype == KVQ_DT_BF16));
  const dim3 block(32 * wpc);
  cudaError_t e;
  if (a.hpw == 1)
    e = bf ? launch_pdl(norm_rope_kernel<LPR, FMT, true, 1>, grid, block, 0, s, a)
           : launch_pdl(norm_rope_kernel<LPR, FMT, false, 1>, grid, block, 0, s, a);
  else
    e = bf ? launch_pdl(norm_rope_kernel<LPR, FMT, true, 2>, grid, block, 0, s, a)
           : launch_pdl(norm_rope_kernel<LPR, FMT, false, 2>, grid, block, 0, s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int width, int fmt, cudaStream_t s) {
#define KVQ_BY_FORMAT(L)                                                          \
  switch (fmt) {                                                                  \
    case kNoStore: return launch_one<L, kNoStore>(a, s);                          \
    case KVQ_FMT_Q4_HAD32: return launch_one<L, KVQ_FMT_Q4_HAD32>(a, s);          \
    case KVQ_FMT_Q4_0: return launch_one<L, KVQ_FMT_Q4_0>(a, s);                  \
    case KVQ_FMT_TQ4: return launch_one<L, KVQ_FMT_TQ4>(a, s);                    \
    case KVQ_FMT_BF16: return launch_one<L, KVQ_FMT_BF16>(a, s);                  \
    default: return cudaErrorInvalidValue;                                        \
  }
  switch (width) {
    case 64: KVQ_BY_FORMAT(4)
    case 128: KVQ_BY_FORMAT(8)
    case 256: KVQ_BY_FORMAT(16)
    case 512:
      if (fmt == kNoStore) return launch_one<32, kNoStore>(a, s);
      if (fmt == KVQ_FMT_BF16) return launch_one<32, KVQ_FMT_BF16>(a, s);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
#undef KVQ_BY_FORMAT
}

}  // namespace kvq
