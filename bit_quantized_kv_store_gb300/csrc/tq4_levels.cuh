// tq4_levels.cuh -- TQ4 codes as the levels they stand for, in registers, shared by the
// kernels that feed them to the tensor cores.
#pragma once
#include "common.cuh"

namespace kvq {

// A TQ4 code nibble is sign (bit 3) and magnitude index m (bits 0-2) of the
// level +-M_m of the 16-level Lloyd-Max codebook; the fp16 bits of M_0..M_7 are
// 0x301c 0x3635 0x3941 0x3b8a 0x3d06 0x3e79 0x4023 0x4177.  Byte tables of
// their low and high bytes, for prmt lookups indexed by m.
constexpr uint32_t kTqLo0 = 0x8a41351cu, kTqLo1 = 0x77237906u;  // low bytes of M_0..M_3, M_4..M_7
constexpr uint32_t kTqHi0 = 0x3b393630u, kTqHi1 = 0x41403e3du;  // high bytes

// The 8 codes of w (element i in nibble i: element 2b in the low nibble of
// byte b) -> 4 f16 pairs (elements 0,1 | 2,3 | 4,5 | 6,7), exactly the codebook
// levels.  The magnitudes select the levels' low and high bytes (prmt reads the
// low 16 bits of its selector: four 3-bit indices once the signs are masked);
// the signs are spread from bit 3 of each nibble to bit 7 of each high byte
// before the bytes are interleaved into pairs.
__device__ __forceinline__ uint4 tq4_levels8(uint32_t w) {
  const uint32_t mm = w & 0x77777777u;  // magnitudes of codes 0-3 (low half), 4-7 (high half)
  const uint32_t lo0 = prmt(kTqLo0, kTqLo1, mm), hi0s = prmt(kTqHi0, kTqHi1, mm);
  const uint32_t lo1 = prmt(kTqLo0, kTqLo1, mm >> 16), hi1s = prmt(kTqHi0, kTqHi1, mm >> 16);
  // x = w << 4 holds the signs of codes 0, 2, 4, 6 at bit 7 of its bytes 0-3;
  // w itself those of codes 1, 3, 5, 7
  const uint32_t x = w << 4;
  const uint32_t hi0 = hi0s ^ (prmt(x, w, 0x5140u) & 0x80808080u);  // codes 0, 1, 2, 3
  const uint32_t hi1 = hi1s ^ (prmt(x, w, 0x7362u) & 0x80808080u);  // codes 4, 5, 6, 7
  uint4 r;
  r.x = prmt(lo0, hi0, 0x5140u);  // (low, high) bytes of codes 0, 1
  r.y = prmt(lo0, hi0, 0x7362u);
  r.z = prmt(lo1, hi1, 0x5140u);
  r.w = prmt(lo1, hi1, 0x7362u);
  return r;
}

}  // namespace kvq
