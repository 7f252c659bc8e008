// norm_rope.cu -- norms of queries and keys per head and rotary positions in one
// pass, alone or on the way into the cache: queries rotated into the cache's
// space, keys and values quantised and stored, in one launch.
//
// The stored rows follow the formats' definitions in kvq.h ("KV cache
// quantization: fp8 (KV8) + 4-bit TurboQuant", KV8 base commit: the producer
// quantises the fresh normed and roped row; "qwen27 CUDA: an opt-in 4-bit
// attention cache (262K on a 24 GB card)", section "What it is").
//
// The arithmetic per row of W = 32 E values, in fp32:
//   y = x * r * (w + offset), r = rsqrt(mean(x^2) + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin) for every rotary pair.
// The angle of a pair is 2 pi times the fraction of pos * turns, turns a 64-bit
// fixed-point fraction of a turn: the product wraps modulo one turn exactly, so
// a far position costs nothing in accuracy (an fp32 angle of 262144 radians is
// off by 0.016) and no fp64.  Its top 32 bits as a float in [-1, 1) go to
// sincospif: the rounding there is at most 2^-25 of half a turn, 1e-7 radians.
//
// One warp takes one token's rows, `hpw` heads one after another, lane l holding
// elements E l .. E l + E - 1, so the angles (the same for every head of the
// token) are computed once per warp, the norm is one warp reduction, and every
// transform of the store runs in registers and shuffles.  Bound: memory for a
// prompt chunk, the launch for a decode step.
//
// This translation unit is compiled with -fmad=false.
#include "rows.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

constexpr int kNoStore = -1;

// cos and sin of the rotary pairs that the lane's elements belong to.  Half-split
// pairs: one angle per element; interleaved: one per two elements (in cs[i / 2]).
template <int E>
struct Angles {
  float cs[E], sn[E];
  int partner;  // half-split: the lane that holds the pairs' other elements
  bool first;   // half-split: the lane holds the pairs' first elements
  bool in;      // half-split: the lane's elements are rotated (all or none)
};

__device__ __forceinline__ void angle(const RopeView& r, int pair, const int32_t (&pos)[4], int32_t* status,
                                      float& c, float& s) {
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
  sincospif(t, &s, &c);
}

template <int E>
__device__ __forceinline__ void make_angles(const RopeView& r, int64_t tok, int lane, int32_t* status, Angles<E>& g) {
  int32_t pos[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) pos[a] = a < r.axes ? r.pos[a * r.pos_stride + tok] : 0;
  const int e = E * lane, half = r.rot >> 1;
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      g.cs[i] = 1.0f;
      g.sn[i] = 0.0f;
      if (e + 2 * i < r.rot) angle(r, e / 2 + i, pos, status, g.cs[i], g.sn[i]);
    }
  } else {
    g.in = e < r.rot;
    g.first = e < half;
    g.partner = !g.in ? lane : g.first ? lane + half / E : lane - half / E;
    if (g.in) {
#pragma unroll
      for (int i = 0; i < E; ++i) angle(r, (g.first ? e : e - half) + i, pos, status, g.cs[i], g.sn[i]);
    }
  }
}

template <int E>
__device__ __forceinline__ void rope_row(const RopeView& r, const Angles<E>& g, int lane, float (&x)[E]) {
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      if (E * lane + 2 * i < r.rot) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = __fmaf_rn(-b, g.sn[i], __fmul_rn(a, g.cs[i]));
        x[2 * i + 1] = __fmaf_rn(a, g.sn[i], __fmul_rn(b, g.cs[i]));
      }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float o = __shfl_sync(0xffffffffu, x[i], g.partner);
      const float t = __fmaf_rn(g.first ? -o : o, g.sn[i], __fmul_rn(x[i], g.cs[i]));
      x[i] = g.in ? t : x[i];
    }
  }
}

// FMT: the cache's format, or kNoStore for rows that are only normed and rotated
// (then every head is a "query" and Hk is 0).
template <int E, int FMT>
__global__ void __launch_bounds__(256) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (tok >= a.n_tok) return;
  const int h0 = blockIdx.y * a.hpw, h1 = min(h0 + a.hpw, a.Hq + 2 * a.Hk);

  Angles<E> ang;
  if (a.rope.rot != 0 && h0 < a.Hq + a.Hk) make_angles<E>(a.rope, tok, lane, a.status, ang);

  float w[E];
  if (h0 < a.Hq) {
    if (a.qn.weight) load_weight<E>(a.qn, lane, w);
    for (int h = h0; h < min(h1, a.Hq); ++h) {
      float x[E];
      load_row<E>(a.q, tok * a.q.ts + h * a.q.hs, lane, x);
      if (a.qn.weight) norm_row<E>(x, w, a.qn.eps);
      if (a.rope.rot != 0) rope_row<E>(a.rope, ang, lane, x);
      if constexpr (FMT == KVQ_FMT_Q4_HAD32) {
        if (a.rotate) rotate_row_had32<E>(x, lane);
      }
      if constexpr (FMT == KVQ_FMT_TQ4) {
        if (a.rotate) tq4_transform<E>(x, lane_signs<E>(a.c.signs, lane), lane, false);
      }
      __syncwarp();  // in place: every lane has read its part of the row
      write_row<E>(a.qo, tok * a.qo.ts + h * a.qo.hs, lane, x);
    }
  }
  if constexpr (FMT != kNoStore) {
    if (h1 <= a.Hq) return;
    constexpr int D = 32 * E;
    const int32_t slot = a.slots[tok];
    if (slot < 0) return;
    if ((int64_t)slot >= (int64_t)a.c.num_pages * a.c.page_size) {
      if (lane == 0) set_status(a.status, KVQ_DEV_BAD_SLOT);
      return;
    }
    const uint32_t page = fast_div(static_cast<uint32_t>(slot), a.ps);
    const uint32_t off = static_cast<uint32_t>(slot) - page * a.ps.d;
    if (a.kn.weight && h0 < a.Hq + a.Hk) load_weight<E>(a.kn, lane, w);
    for (int h = max(h0, a.Hq); h < h1; ++h) {
      const bool is_v = h >= a.Hq + a.Hk;
      const int head = h - a.Hq - (is_v ? a.Hk : 0);
      const int64_t r = ((int64_t)page * a.Hk + head) * a.c.page_size + off;
      float x[E];
      const RowsView& src = is_v ? a.v : a.k;
      load_row<E>(src, tok * src.ts + head * src.hs, lane, x);
      if (!is_v) {
        if (a.kn.weight) norm_row<E>(x, w, a.kn.eps);
        if (a.rope.rot != 0) rope_row<E>(a.rope, ang, lane, x);
      }
      void* codes = is_v ? a.c.v : a.c.k;
      void* scales = is_v ? a.c.v_scale : a.c.k_scale;
      if constexpr (FMT == KVQ_FMT_BF16) {
        const RowsView row{codes, 0, 0, KVQ_DT_BF16, 1};
        write_row<E>(row, r * D, lane, x);
      } else if constexpr (FMT == KVQ_FMT_TQ4) {
        tq4_transform<E>(x, lane_signs<E>(a.c.signs, lane), lane, false);
        __half s16;
        const uint32_t word = tq4_row_codes<E>(x, s16);
        tq4_write_codes<E>(static_cast<uint8_t*>(codes) + r * (D / 2) + lane * (E / 2), word);
        if (lane == 0) static_cast<__half*>(scales)[r] = s16;
      } else {
        if constexpr (FMT == KVQ_FMT_Q4_HAD32) rotate_row_had32<E>(x, lane);
        __half s16;
        const uint32_t word = q4_row_codes<E>(x, s16);
        tq4_write_codes<E>(static_cast<uint8_t*>(codes) + r * (D / 2) + lane * (E / 2), word);
        if (lane % (32 / E) == 0) static_cast<__half*>(scales)[r * E + lane / (32 / E)] = s16;
      }
    }
  }
}

template <int E, int FMT>
cudaError_t launch_one(NormRopeArgs a, cudaStream_t s) {
  // Enough warps to fill the GPU, and no more: each computes its token's angles once.
  const int total = a.Hq + 2 * a.Hk;
  const int64_t target = static_cast<int64_t>(device_sm_count()) * 32;
  int64_t hpw = (a.n_tok * total + target - 1) / target;
  if (hpw > total) hpw = total;
  a.hpw = static_cast<int>(hpw < 1 ? 1 : hpw);
  int wpc = 8;  // tokens per CTA
  while (wpc > 1 && a.n_tok < wpc) wpc >>= 1;
  const dim3 grid(static_cast<unsigned>((a.n_tok + wpc - 1) / wpc), (total + a.hpw - 1) / a.hpw);
  cudaError_t e = launch_pdl(norm_rope_kernel<E, FMT>, grid, dim3(32 * wpc), 0, s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int width, int fmt, cudaStream_t s) {
#define KVQ_BY_FORMAT(E)                                                          \
  switch (fmt) {                                                                  \
    case kNoStore: return launch_one<E, kNoStore>(a, s);                          \
    case KVQ_FMT_Q4_HAD32: return launch_one<E, KVQ_FMT_Q4_HAD32>(a, s);          \
    case KVQ_FMT_Q4_0: return launch_one<E, KVQ_FMT_Q4_0>(a, s);                  \
    case KVQ_FMT_TQ4: return launch_one<E, KVQ_FMT_TQ4>(a, s);                    \
    case KVQ_FMT_BF16: return launch_one<E, KVQ_FMT_BF16>(a, s);                  \
    default: return cudaErrorInvalidValue;                                        \
  }
  switch (width) {
    case 64: KVQ_BY_FORMAT(2)
    case 128: KVQ_BY_FORMAT(4)
    case 256: KVQ_BY_FORMAT(8)
    case 512:
      if (fmt == kNoStore) return launch_one<16, kNoStore>(a, s);
      if (fmt == KVQ_FMT_BF16) return launch_one<16, KVQ_FMT_BF16>(a, s);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
#undef KVQ_BY_FORMAT
}

}  // namespace kvq
