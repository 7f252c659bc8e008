// rows.cuh -- strided activation rows in a warp's registers: lane l holds elements
// E l .. E l + E - 1 of a row of 32 E values.  Loads and stores of bf16 and fp32
// rows, the per-row norm, and the 4-bit groups of a row in this layout (a group
// of 32 values spans 32 / E lanes).  Every floating-point operation that decides
// bits is an explicit IEEE-rounded intrinsic, so kernels of different
// translation units agree bit for bit.
#pragma once
#include "kernels.cuh"
#include "q4_code.cuh"

namespace kvq {

// The lane's E values of the row at element `e0` of the view (the row's start).
template <int E>
__device__ __forceinline__ void load_row(const RowsView& v, int64_t e0, int lane, float (&x)[E]) {
  const int64_t e = e0 + E * lane;
  if (v.dtype == KVQ_DT_BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(v.data) + e;
    if (v.wide) {
      uint32_t w[(E + 1) / 2];
      if constexpr (E >= 8) {
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
          const uint4 u = reinterpret_cast<const uint4*>(p)[i];
          w[4 * i] = u.x; w[4 * i + 1] = u.y; w[4 * i + 2] = u.z; w[4 * i + 3] = u.w;
        }
      } else if constexpr (E == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        w[0] = u.x; w[1] = u.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = __bfloat162float(p[i]);
    }
  } else {
    const float* p = static_cast<const float*>(v.data) + e;
    if (v.wide) {
      if constexpr (E >= 4) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const float4 u = reinterpret_cast<const float4*>(p)[i];
          x[4 * i] = u.x; x[4 * i + 1] = u.y; x[4 * i + 2] = u.z; x[4 * i + 3] = u.w;
        }
      } else {
        const float2 u = *reinterpret_cast<const float2*>(p);
        x[0] = u.x; x[1] = u.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) x[i] = p[i];
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The lane's E values into the row at element `e0`, rounded once (bf16) or as they are.
template <int E>
__device__ __forceinline__ void write_row(const RowsView& v, int64_t e0, int lane, const float (&x)[E]) {
  const int64_t e = e0 + E * lane;
  if (v.dtype == KVQ_DT_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(v.data) + e;
    if (v.wide) {
      uint32_t w[(E + 1) / 2];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      if constexpr (E >= 8) {
#pragma unroll
        for (int i = 0; i < E / 8; ++i)
          reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else if constexpr (E == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t*>(p) = w[0];
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
  } else {
    float* p = static_cast<float*>(v.data) + e;
    if (v.wide) {
      if constexpr (E >= 4) {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
          reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      } else {
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) p[i] = x[i];
    }
  }
}

// weight + offset of the lane's elements.
template <int E>
__device__ __forceinline__ void load_weight(const NormView& n, int lane, float (&w)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) w[i] = __fadd_rn(load_act(n.weight, n.dtype, E * lane + i), n.offset);
}

// x * r * w over the warp's row, r = 1 / sqrt(mean(x^2) + eps).  The squares are
// summed by a pairwise tree (in the lane, then across lanes) in fp32.
template <int E>
__device__ __forceinline__ void norm_row(float (&x)[E], const float (&w)[E], float eps) {
  float s[E];
#pragma unroll
  for (int i = 0; i < E; ++i) s[i] = __fmul_rn(x[i], x[i]);
#pragma unroll
  for (int h = 1; h < E; h <<= 1)
#pragma unroll
    for (int i = 0; i < E; i += 2 * h) s[i] = __fadd_rn(s[i], s[i + h]);
  float ss = s[0];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  const float r = rsqrtf(__fadd_rn(__fmul_rn(ss, 1.0f / (32 * E)), eps));
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], r), w[i]);
}

// blockdiag(H32) over the warp's row: the butterfly's stages h < E pair registers,
// the others pair lanes; the same operations on the same operands, in the same
// stage order, as warp_fwht32 (lane i's value x[i]).
template <int E>
__device__ __forceinline__ void rotate_row_had32(float (&x)[E], int lane) {
#pragma unroll
  for (int h = 1; h < E; h <<= 1)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (!(i & h)) {
        const float a = x[i], b = x[i + h];
        x[i] = __fadd_rn(a, b);
        x[i + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int o = 1; o < 32 / E; o <<= 1)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float p = __shfl_xor_sync(0xffffffffu, x[i], o);
      x[i] = (lane & o) ? __fsub_rn(p, x[i]) : __fadd_rn(x[i], p);
    }
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __fmul_rn(x[i], kHadamardScale);
}

// The 4-bit codes (element i of the lane in nibble i) of the lane's part of its
// group, and the group's fp16 scale: q4_group_code_warp's arithmetic in this layout.
template <int E>
__device__ __forceinline__ uint32_t q4_row_codes(const float (&y)[E], __half& s16) {
  float amax = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < E; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
  for (int o = 1; o < 32 / E; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  s16 = __float2half_rn(__fmul_rn(amax, 0.125f));
  if (__hisinf(s16)) s16 = __ushort_as_half(0x7BFFu);  // saturate to 65504
  const float s = __half2float(s16);
  uint32_t word = 0;
  const float r = rcp_approx(s);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    uint32_t code = 8;
    if (s != 0.0f && !q4_code_screened(y[i], r, code)) code = q4_code_exact(y[i], s);
    word = put_nibble(word, code, i);
  }
  return word;
}

}  // namespace kvq
