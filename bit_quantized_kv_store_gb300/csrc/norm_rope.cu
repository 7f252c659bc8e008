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
// token) are computed once per warp, spread over its lanes and shared through
// shared memory, the norm is one warp reduction, and every transform of the store
// runs in registers and shuffles.  The next row's loads are in flight while a row
// is worked on.  Bound: memory for a prompt chunk, the launch for a decode step.
//
// This translation unit is compiled with -fmad=false.
#include "rows.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

constexpr int kNoStore = -1;
constexpr int kMaxPairs = 128;
constexpr int kMaxWarps = 8;

// cos and sin of the rotary pairs that the lane's elements belong to.  Half-split
// pairs: one angle per element (sn negative for the pairs' first elements);
// interleaved: pair i of the lane in cs[i], sn[i].
template <int E>
struct Angles {
  float cs[E], sn[E];
  int partner;  // half-split: the lane that holds the pairs' other elements
  bool in;      // half-split: the lane's elements are rotated (all or none)
};

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

// `sh`: the warp's kMaxPairs (cos, sin) in shared memory.
template <int E>
__device__ __forceinline__ void make_angles(const RopeView& r, int64_t tok, int lane, int32_t* status, float2* sh,
                                            Angles<E>& g) {
  int32_t pos[4];
#pragma unroll
  for (int a = 0; a < 4; ++a) pos[a] = a < r.axes ? r.pos[a * r.pos_stride + tok] : 0;
  const int e = E * lane, half = r.rot >> 1;
  for (int p = lane; p < half; p += 32) sh[p] = angle(r, p, pos, status);
  __syncwarp();
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const float2 cs = e + 2 * i < r.rot ? sh[e / 2 + i] : make_float2(1.0f, 0.0f);
      g.cs[i] = cs.x;
      g.sn[i] = cs.y;
    }
  } else {
    const bool first = e < half;
    g.in = e < r.rot;
    g.partner = !g.in ? lane : first ? lane + half / E : lane - half / E;
    if (g.in) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float2 cs = sh[(first ? e : e - half) + i];
        g.cs[i] = cs.x;
        g.sn[i] = first ? -cs.y : cs.y;
      }
    }
  }
}

// (a cos - b sin, b cos + a sin), each as one product and one fused add.
template <int E>
__device__ __forceinline__ void rope_row(const RopeView& r, const Angles<E>& g, int lane, uint64_t (&x)[E / 2]) {
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      if (E * lane + 2 * i < r.rot) {
        float a, b;
        upk2(x[i], a, b);
        x[i] = pk2(__fmaf_rn(-b, g.sn[i], __fmul_rn(a, g.cs[i])), __fmaf_rn(a, g.sn[i], __fmul_rn(b, g.cs[i])));
      }
  } else {
    float o[E];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float a, b;
      upk2(x[i], a, b);
      o[2 * i] = __shfl_sync(0xffffffffu, a, g.partner);
      o[2 * i + 1] = __shfl_sync(0xffffffffu, b, g.partner);
    }
    if (g.in) {
#pragma unroll
      for (int i = 0; i < E / 2; ++i)
        x[i] = fma2(pk2(o[2 * i], o[2 * i + 1]), pk2(g.sn[2 * i], g.sn[2 * i + 1]),
                    mul2(x[i], pk2(g.cs[2 * i], g.cs[2 * i + 1])));
    }
  }
}

// FMT: the cache's format, or kNoStore for rows that are only normed and rotated
// (then every head is a "query" and Hk is 0).  BF: every input is bf16.
template <int E, int FMT, bool BF>
__global__ void __launch_bounds__(32 * kMaxWarps) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  __shared__ float2 angles_sh[kMaxWarps][kMaxPairs];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  if (tok >= a.n_tok) return;
  const int h0 = blockIdx.y * a.hpw, h1 = min(h0 + a.hpw, a.Hq + 2 * a.Hk);
  const int q1 = min(h1, a.Hq), kv0 = max(h0, a.Hq);

  RawRow<E, BF> next;  // the next row, ahead of the angles' latency
  if (h0 < a.Hq) load_raw<E, BF>(a.q, tok * a.q.ts + h0 * a.q.hs, lane, next);
  int32_t slot = -1;
  if (FMT != kNoStore && h1 > a.Hq) slot = a.slots[tok];

  Angles<E> ang;
  if (a.rope.rot != 0 && h0 < a.Hq + a.Hk) make_angles<E>(a.rope, tok, lane, a.status, angles_sh[warp], ang);

  uint64_t w[E / 2];
  if (h0 < a.Hq) {
    if (a.qn.weight) load_weight<E>(a.qn, lane, w);
    for (int h = h0; h < q1; ++h) {
      uint64_t x[E / 2];
      unpack_row<E, BF>(next, x);
      if (h + 1 < q1) load_raw<E, BF>(a.q, tok * a.q.ts + (h + 1) * a.q.hs, lane, next);
      if (a.qn.weight) norm_row<E>(x, w, a.qn.eps);
      if (a.rope.rot != 0) rope_row<E>(a.rope, ang, lane, x);
      if constexpr (FMT == KVQ_FMT_Q4_HAD32) {
        if (a.rotate) rotate_row_had32<E>(x, lane);
      }
      if constexpr (FMT == KVQ_FMT_TQ4) {
        if (a.rotate) rotate_row_tq4<E>(x, lane_signs<E>(a.c.signs, lane), lane);
      }
      write_row<E>(a.qo, tok * a.qo.ts + h * a.qo.hs, lane, x);
    }
  }
  if constexpr (FMT != kNoStore) {
    if (h1 <= a.Hq || slot < 0) return;
    if ((int64_t)slot >= (int64_t)a.c.num_pages * a.c.page_size) {
      if (lane == 0) set_status(a.status, KVQ_DEV_BAD_SLOT);
      return;
    }
    constexpr int D = 32 * E;
    const uint32_t page = fast_div(static_cast<uint32_t>(slot), a.ps);
    const uint32_t off = static_cast<uint32_t>(slot) - page * a.ps.d;
    auto load_kv = [&](int h) {
      const bool is_v = h >= a.Hq + a.Hk;
      const RowsView& src = is_v ? a.v : a.k;
      load_raw<E, BF>(src, tok * src.ts + (h - a.Hq - (is_v ? a.Hk : 0)) * src.hs, lane, next);
    };
    load_kv(kv0);
    if (a.kn.weight && kv0 < a.Hq + a.Hk) load_weight<E>(a.kn, lane, w);
    for (int h = kv0; h < h1; ++h) {
      const bool is_v = h >= a.Hq + a.Hk;
      const int head = h - a.Hq - (is_v ? a.Hk : 0);
      const int64_t r = ((int64_t)page * a.Hk + head) * a.c.page_size + off;
      uint64_t x[E / 2];
      unpack_row<E, BF>(next, x);
      if (h + 1 < h1) load_kv(h + 1);
      if (!is_v) {
        if (a.kn.weight) norm_row<E>(x, w, a.kn.eps);
        if (a.rope.rot != 0) rope_row<E>(a.rope, ang, lane, x);
      }
      void* codes = is_v ? a.c.v : a.c.k;
      void* scales = is_v ? a.c.v_scale : a.c.k_scale;
      if constexpr (FMT == KVQ_FMT_BF16) {
        const RowsView row{codes, 0, 0, KVQ_DT_BF16, a.plane_wide};
        write_row<E>(row, r * D, lane, x);
      } else if constexpr (FMT == KVQ_FMT_TQ4) {
        rotate_row_tq4<E>(x, lane_signs<E>(a.c.signs, lane), lane);
        float y[E];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) upk2(x[i], y[2 * i], y[2 * i + 1]);
        __half s16;
        const uint32_t word = tq4_row_codes<E>(y, s16);
        tq4_write_codes<E>(static_cast<uint8_t*>(codes) + r * (D / 2) + lane * (E / 2), word);
        if (lane == 0) static_cast<__half*>(scales)[r] = s16;
      } else {
        constexpr bool ROT = FMT == KVQ_FMT_Q4_HAD32;
        if constexpr (ROT) rotate_row_had32<E>(x, lane);
        __half s16;
        const uint32_t word = q4_row_codes<E, ROT>(x, s16);
        tq4_write_codes<E>(static_cast<uint8_t*>(codes) + r * (D / 2) + lane * (E / 2), word);
        if (lane % (32 / E) == 0) static_cast<__half*>(scales)[r * E + lane / (32 / E)] = s16;
      }
    }
  }
}

template <int E, int FMT>
cudaError_t launch_one(NormRopeArgs a, cudaStream_t s) {
  // Three waves of warps or more where there are rows for them (each warp computes
  // its token's angles once, so no more than that), the heads evenly over them.
  const int total = a.Hq + 2 * a.Hk;
  const int64_t target = static_cast<int64_t>(device_sm_count()) * 96;
  int64_t hpw = (a.n_tok * total + target - 1) / target;
  if (hpw > total) hpw = total;
  const int chunks = static_cast<int>((total + hpw - 1) / hpw);
  a.hpw = (total + chunks - 1) / chunks;
  int wpc = kMaxWarps;  // tokens per CTA
  while (wpc > 1 && a.n_tok < wpc) wpc >>= 1;
  const dim3 grid(static_cast<unsigned>((a.n_tok + wpc - 1) / wpc), (total + a.hpw - 1) / a.hpw);
  const bool bf = (a.Hq == 0 || a.q.dtype == KVQ_DT_BF16) &&
                  (a.Hk == 0 || (a.k.dtype == KVQ_DT_BF16 && a.v.dtype == KVQ_DT_BF16));
  cudaError_t e = bf ? launch_pdl(norm_rope_kernel<E, FMT, true>, grid, dim3(32 * wpc), 0, s, a)
                     : launch_pdl(norm_rope_kernel<E, FMT, false>, grid, dim3(32 * wpc), 0, s, a);
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
