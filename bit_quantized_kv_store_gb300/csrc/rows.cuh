// rows.cuh -- strided activation rows in a warp's registers: a row of E LPR values
// lies over LPR lanes (a warp, or an aligned part of one), its lane l holding
// elements E l .. E l + E - 1 as E / 2 packed fp32 pairs (element 2i in the low
// half of pair i).  Loads and stores of bf16 and fp32 rows, the per-row norm, the
// caches' row transforms and the 4-bit codes in this layout (a group of 32 values
// spans 32 / E lanes).  The transforms perform the operations
// of the store's butterflies on the same operands (two per packed instruction;
// across lanes p + x * (+-1), one rounding), so the stored bytes are the same.
#pragma once
#include "f32x2.cuh"
#include "kernels.cuh"
#include "q4_code.cuh"

namespace kvq {

// ---------------------------------------------------------------- loads and stores
// 32 bytes at once (address a multiple of 32).
__device__ __forceinline__ void ld256(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st256(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// N words (1, 2, 4, 8 or 16) at an address aligned to them (to 32 bytes past 8).
template <int N>
__device__ __forceinline__ void ld_words(const void* p, uint32_t* w) {
  if constexpr (N >= 8) {
#pragma unroll
    for (int i = 0; i < N; i += 8) ld256(static_cast<const uint32_t*>(p) + i, w + i);
  } else if constexpr (N == 4) {
    const uint4 u = *static_cast<const uint4*>(p);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = *static_cast<const uint2*>(p);
    w[0] = u.x; w[1] = u.y;
  } else {
    w[0] = *static_cast<const uint32_t*>(p);
  }
}
template <int N>
__device__ __forceinline__ void st_words(void* p, const uint32_t* w) {
  if constexpr (N >= 8) {
#pragma unroll
    for (int i = 0; i < N; i += 8) st256(static_cast<uint32_t*>(p) + i, w + i);
  } else if constexpr (N == 4) {
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if constexpr (N == 2) {
    *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    *static_cast<uint32_t*>(p) = w[0];
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The lane's part of a row as it lies in memory: E / 2 words of bf16 pairs (BF) or
// E fp32 words, kept like this while the row before it is worked on.  Without BF
// a bf16 row is converted as it is loaded.
template <int E, bool BF>
struct RawRow {
  uint32_t w[BF ? E / 2 : E];
};

// The lane's part of a row from its address there (`wide`, `dtype`: the row's view's).
template <int E, bool BF>
__device__ __forceinline__ void load_raw_at(const void* at, int dtype, int wide, RawRow<E, BF>& r) {
  if (BF || dtype == KVQ_DT_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(at);
    uint32_t w[E / 2];
    if (wide) {
      ld_words<E / 2>(p, w);
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) w[i] = p[2 * i] | static_cast<uint32_t>(p[2 * i + 1]) << 16;
    }
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      if constexpr (BF) {
        r.w[i] = w[i];
      } else {
        r.w[2 * i] = w[i] << 16;
        r.w[2 * i + 1] = w[i] & 0xFFFF0000u;
      }
    }
  } else if constexpr (!BF) {
    const uint32_t* p = static_cast<const uint32_t*>(at);
    if (wide) {
      ld_words<E>(p, r.w);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) r.w[i] = p[i];
    }
  }
}

// Address of element e of a view's data.
__device__ __forceinline__ uint8_t* element_at(const RowsView& v, int64_t e) {
  return static_cast<uint8_t*>(v.data) + (e << (v.dtype == KVQ_DT_BF16 ? 1 : 2));
}

// The lane's part of the row at element e0 of the view.
template <int E, bool BF>
__device__ __forceinline__ void load_raw(const RowsView& v, int64_t e0, int lane, RawRow<E, BF>& r) {
  load_raw_at<E, BF>(element_at(v, e0 + E * lane), v.dtype, v.wide, r);
}

template <int E, bool BF>
__device__ __forceinline__ void unpack_row(const RawRow<E, BF>& r, uint64_t (&x)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i)
    x[i] = BF ? pk2(__uint_as_float(r.w[i] << 16), __uint_as_float(r.w[i] & 0xFFFF0000u))
              : pk2(__uint_as_float(r.w[BF ? 0 : 2 * i]), __uint_as_float(r.w[BF ? 0 : 2 * i + 1]));
}

// The lane's part of a row to its address there, rounded once (bf16) or as it is.
template <int E>
__device__ __forceinline__ void write_row_at(void* at, int dtype, int wide, const uint64_t (&x)[E / 2]) {
  float f[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) upk2(x[i], f[2 * i], f[2 * i + 1]);
  if (dtype == KVQ_DT_BF16) {
    uint32_t w[E / 2];
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
    if (wide) {
      st_words<E / 2>(at, w);
    } else {
      uint16_t* p = static_cast<uint16_t*>(at);
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        p[2 * i] = static_cast<uint16_t>(w[i]);
        p[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
      }
    }
  } else if (wide) {
    uint32_t w[E];
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = __float_as_uint(f[i]);
    st_words<E>(at, w);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) static_cast<float*>(at)[i] = f[i];
  }
}

// The lane's part of the row at element e0 of the view.
template <int E>
__device__ __forceinline__ void write_row(const RowsView& v, int64_t e0, int lane, const uint64_t (&x)[E / 2]) {
  write_row_at<E>(element_at(v, e0 + E * lane), v.dtype, v.wide, x);
}

// ---------------------------------------------------------------- norm
// weight + offset of the lane's elements (n.wide: on a 32-byte boundary).
template <int E>
__device__ __forceinline__ void load_weight(const NormView& n, int lane, uint64_t (&w)[E / 2]) {
  const RowsView v{const_cast<void*>(n.weight), 0, 0, n.dtype, n.wide};
  RawRow<E, false> r;
  load_raw<E, false>(v, 0, lane, r);
  unpack_row<E, false>(r, w);
  const uint64_t o2 = pk2(n.offset, n.offset);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) w[i] = add2(w[i], o2);
}

// x * r * w over the row's LPR lanes, r = 1 / sqrt(mean(x^2) + eps), for U rows side
// by side.  The squares are summed in fp32: two chains of fused adds over the
// lane's pairs, then across lanes.
template <int E, int LPR, int U>
__device__ __forceinline__ void norm_rows(uint64_t (&x)[U][E / 2], const uint64_t (&w)[E / 2], float eps) {
  float ss[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint64_t s = mul2(x[u][0], x[u][0]);
    if constexpr (E >= 4) {
      uint64_t t = mul2(x[u][1], x[u][1]);
#pragma unroll
      for (int i = 2; i < E / 2; i += 2) {
        s = fma2(x[u][i], x[u][i], s);
        t = fma2(x[u][i + 1], x[u][i + 1], t);
      }
      s = add2(s, t);
    }
    float a, b;
    upk2(s, a, b);
    ss[u] = __fadd_rn(a, b);
  }
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) ss[u] = __fadd_rn(ss[u], __shfl_xor_sync(0xffffffffu, ss[u], o));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float r = rsqrtf(__fadd_rn(__fmul_rn(ss[u], 1.0f / (LPR * E)), eps));
    const uint64_t r2 = pk2(r, r);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) x[u][i] = mul2(mul2(x[u][i], r2), w[i]);
  }
}

// ---------------------------------------------------------------- row transforms
// Butterfly stages at element distances 1 .. E / 2, in the lane.
template <int E>
__device__ __forceinline__ void lane_butterfly(uint64_t (&x)[E / 2]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {  // distance 1: the halves of a pair
    float a, b;
    upk2(x[i], a, b);
    x[i] = pk2(__fadd_rn(a, b), __fsub_rn(a, b));
  }
#pragma unroll
  for (int h = 1; h < E / 2; h <<= 1)
#pragma unroll
    for (int i = 0; i < E / 2; ++i)
      if (!(i & h)) {
        const uint64_t a = x[i], b = x[i + h];
        x[i] = add2(a, b);
        x[i + h] = sub2(a, b);
      }
}

// Stages across lanes: partners o = 1 .. LANES / 2 lanes apart.
template <int E, int LANES>
__device__ __forceinline__ void cross_butterfly(uint64_t (&x)[E / 2], int lane) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    const float sgn = (lane & o) ? -1.0f : 1.0f;
    const uint64_t s2 = pk2(sgn, sgn);
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float a, b;
      upk2(x[i], a, b);
      const uint64_t p = pk2(__shfl_xor_sync(0xffffffffu, a, o), __shfl_xor_sync(0xffffffffu, b, o));
      x[i] = fma2(x[i], s2, p);
    }
  }
}

// blockdiag(H32) over the warp's row (warp_fwht32's stages and scale).
template <int E>
__device__ __forceinline__ void rotate_row_had32(uint64_t (&x)[E / 2], int lane) {
  lane_butterfly<E>(x);
  cross_butterfly<E, 32 / E>(x, lane);
  const uint64_t c2 = pk2(kHadamardScale, kHadamardScale);
#pragma unroll
  for (int i = 0; i < E / 2; ++i) x[i] = mul2(x[i], c2);
}

// The 4-bit codes (element 8q + i of the lane in nibble i of word[q]; E <= 8: all in
// word[0]) of the lane's part of its group, and the group's fp16 scale: q4_group_code_warp's arithmetic in this
// layout.  ROT: rotated values, whose groups hold no NaN beside finite values; all
// of a lane's codes then come from one packed estimate
//   t = min(fl(y * rcp(s) + 8), 15), u = fl(t + 1.5 * 2^23)
// (u's low mantissa bits hold rint_even(t)), taken when every t lies farther than
// the screen from a half-integer; t >= -1/2 for an fp16-normal, unsaturated scale.
template <int E, bool ROT>
__device__ __forceinline__ void q4_row_codes(const uint64_t (&x)[E / 2], uint32_t (&word)[(E + 7) / 8], __half& s16) {
  float y[E];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) upk2(x[i], y[2 * i], y[2 * i + 1]);
  float amax = fabsf(y[0]);
#pragma unroll
  for (int i = 1; i < E; ++i) amax = fmaxf(amax, fabsf(y[i]));
#pragma unroll
  for (int o = 1; o < 32 / E; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  s16 = __float2half_rn(__fmul_rn(amax, 0.125f));
  if (__hisinf(s16)) s16 = __ushort_as_half(0x7BFFu);  // saturate to 65504
  const float s = __half2float(s16);
#pragma unroll
  for (int q = 0; q < (E + 7) / 8; ++q) word[q] = 0x88888888u;  // scale 0: every code 8
  if (s == 0.0f) return;
  const float r = rcp_approx(s);
  if (ROT && s >= 6.103515625e-05f && s < 65504.0f) {  // (false for NaN)
    const uint64_t r2 = pk2(r, r), e2 = pk2(8.0f, 8.0f), m2 = pk2(12582912.0f, 12582912.0f);
    float dmax = 0.0f;
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      float ta, tb, da, db, ua, ub;
      upk2(fma2(x[i], r2, e2), ta, tb);
      const uint64_t t2 = pk2(fminf(ta, 15.0f), fminf(tb, 15.0f));
      const uint64_t u2 = add2(t2, m2);
      upk2(sub2(t2, sub2(u2, m2)), da, db);
      dmax = fmaxf(dmax, fmaxf(fabsf(da), fabsf(db)));
      upk2(u2, ua, ub);
      word[i >> 2] = put_nibble(word[i >> 2], __float_as_uint(ua), 2 * (i & 3));
      word[i >> 2] = put_nibble(word[i >> 2], __float_as_uint(ub), 2 * (i & 3) + 1);
    }
    if (dmax < kQ4Screen) return;
  }
  // value by value: the screened estimate, and the IEEE division for those it leaves
  // open, in a loop (rare, and sixteen divisions in a row would take registers from
  // the rest of the kernel)
  uint32_t open = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    uint32_t code;
    if (!q4_code_screened(y[i], r, code)) open |= 1u << i;
    word[i >> 3] = put_nibble(word[i >> 3], code, i & 7);
  }
  while (open) {
    const int i = __ffs(open) - 1;
    open &= open - 1;
    float v = y[0];
#pragma unroll
    for (int j = 1; j < E; ++j)
      if (j == i) v = y[j];
    const uint32_t code = q4_code_exact(v, s);
#pragma unroll
    for (int q = 0; q < (E + 7) / 8; ++q)
      if (i >> 3 == q) word[q] = put_nibble(word[q], code, i & 7);
  }
}

}  // namespace kvq
