// tq4_code.cuh -- the TQ4 rows' signed row transform and the codes and scale of one
// transformed row across a warp (or an aligned part of one), shared by the kernels
// that store such rows.  Lane l of the row holds elements E l .. E l + E - 1, so
// the butterfly's first log2(E) stages run in registers and the others across
// lanes, and the pairwise tree of the sum of squares is the lanes' xor reduction.  Every
// floating-point operation is an explicit IEEE-rounded intrinsic.
#pragma once
#include "common.cuh"
#include "rows.cuh"

namespace kvq {

// Lloyd-Max magnitudes for 16 levels of N(0,1), rounded to fp16 (exact values).
__host__ __device__ constexpr float tq4_mag(int m) {
  return m == 0 ? 0.12841796875f : m == 1 ? 0.387939453125f : m == 2 ? 0.65673828125f : m == 3 ? 0.9423828125f
       : m == 4 ? 1.255859375f : m == 5 ? 1.6181640625f : m == 6 ? 2.068359375f : 2.732421875f;
}
// Midpoint between magnitudes m and m + 1 (exact: fp16 values summed in fp32).
__host__ __device__ constexpr float tq4_mid(int m) { return (tq4_mag(m) + tq4_mag(m + 1)) * 0.5f; }

template <int E>
__host__ __device__ constexpr float tq4_row_scale() {  // fp32(1 / sqrt(32 E))
  return E == 8 ? 0.0625f : E == 4 ? 0.0883883476483184405501f : 0.125f;
}

// In-place signed transform of the warp's row (forward: signs, butterfly, scale;
// inverse: butterfly, scale, signs).  `sw` holds this lane's E sign bits.
template <int E>
__device__ __forceinline__ void tq4_transform(float (&y)[E], uint32_t sw, int lane, bool inverse) {
  if (!inverse) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if ((sw >> i) & 1u) y[i] = -y[i];
  }
#pragma unroll
  for (int h = 1; h < E; h <<= 1)
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (!(i & h)) {
        const float a = y[i], b = y[i + h];
        y[i] = __fadd_rn(a, b);
        y[i + h] = __fsub_rn(a, b);
      }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float p = __shfl_xor_sync(0xffffffffu, y[i], o);
      y[i] = (lane & o) ? __fsub_rn(p, y[i]) : __fadd_rn(y[i], p);
    }
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = __fmul_rn(y[i], tq4_row_scale<E>());
  if (inverse) {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if ((sw >> i) & 1u) y[i] = -y[i];
  }
}

template <int E>
__device__ __forceinline__ uint32_t lane_signs(const void* signs, int lane) {
  const uint32_t w = static_cast<const uint32_t*>(signs)[(E * lane) >> 5];
  return w >> ((E * lane) & 31);
}

// tq4_transform (forward) on a row of LPR lanes in packed pairs: the same operations.
template <int E, int LPR>
__device__ __forceinline__ void rotate_row_tq4(uint64_t (&x)[E / 2], uint32_t sw, int lane) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    float a, b;
    upk2(x[i], a, b);
    x[i] = pk2((sw >> (2 * i)) & 1u ? -a : a, (sw >> (2 * i + 1)) & 1u ? -b : b);
  }
  lane_butterfly<E>(x);
  cross_butterfly<E, LPR>(x, lane);
  constexpr float c = tq4_row_scale<E * LPR / 32>();
  const uint64_t c2 = pk2(c, c);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], c2);
}

// The codes (element 8q + i of the lane in nibble i of word[q]) and the fp16 scale of
// the transformed row y of LPR lanes.
template <int E, int LPR>
__device__ __forceinline__ void tq4_row_codes(const float (&y)[E], uint32_t (&word)[(E + 7) / 8], __half& s16_out) {
  constexpr int D = LPR * E;
  // sum of squares by the pairwise tree: in-lane stages, then the xor reduction
  float q2[E];
#pragma unroll
  for (int i = 0; i < E; ++i) q2[i] = __fmul_rn(y[i], y[i]);
#pragma unroll
  for (int h = 1; h < E; h <<= 1)
#pragma unroll
    for (int i = 0; i < E; i += 2 * h) q2[i] = __fadd_rn(q2[i], q2[i + h]);
  float ss = q2[0];
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, o));
  __half s16 = __float2half_rn(__fsqrt_rn(__fmul_rn(ss, 1.0f / D)));
  if (__hisinf(s16)) s16 = __ushort_as_half(0x7BFFu);  // saturate to 65504
  const float s = __half2float(s16);

  // Element y has the code of the rounded quotient q = y / s: its magnitude is the number
  // of midpoints below |q|, bit 3 is q < 0.  Without the division: s (11 bits) times a
  // midpoint (at most 13) is exact, and the float above it divided by s lies more than
  // half a step above the midpoint (its step is more than 2^-24 of it, half the
  // midpoint's at most that), so |q| > mid exactly where |y| > s mid.  q is -0 where
  // |y| / s <= 2^-150; both sides times 2^126 s are normal numbers.
  float t[7];
#pragma unroll
  for (int j = 0; j < 7; ++j) t[j] = __fmul_rn(s, tq4_mid(j));
  const float tiny = __fmul_rn(s, -5.9604644775390625e-8f);  // -2^-24 s
#pragma unroll
  for (int q = 0; q < (E + 7) / 8; ++q) word[q] = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const float a = fabsf(y[i]);
    const bool hi = a > t[3];
    const bool mid = a > (hi ? t[5] : t[1]);
    const bool lo = a > (hi ? (mid ? t[6] : t[4]) : (mid ? t[2] : t[0]));
    const bool neg = __fmul_rn(y[i], 8.507059173023461586e37f) < tiny;
    uint32_t& w = word[i >> 3];
    if (hi) w |= 4u << (4 * (i & 7));
    if (mid) w |= 2u << (4 * (i & 7));
    if (lo) w |= 1u << (4 * (i & 7));
    if (neg) w |= 8u << (4 * (i & 7));
  }
  if (!(s > 0.0f)) {
#pragma unroll
    for (int q = 0; q < (E + 7) / 8; ++q) word[q] = 0;
  }
  s16_out = s16;
}

// Write the lane's E codes into its row of the codes plane.
template <int E>
__device__ __forceinline__ void write_codes(uint8_t* codes, const uint32_t (&word)[(E + 7) / 8]) {
  if constexpr (E == 16) {
    *reinterpret_cast<uint2*>(codes) = make_uint2(word[0], word[1]);
  } else if constexpr (E == 8) {
    *reinterpret_cast<uint32_t*>(codes) = word[0];
  } else if constexpr (E == 4) {
    *reinterpret_cast<uint16_t*>(codes) = static_cast<uint16_t>(word[0]);
  } else {
    *codes = static_cast<uint8_t>(word[0]);
  }
}

}  // namespace kvq
