// rope.cuh -- rotary positions of rows in a warp's registers (rows.cuh), 16 elements
// to a lane.
//
// The angle of a pair is 2 pi times the fraction of pos * turns, turns a 64-bit
// fixed-point fraction of a turn: the product wraps modulo one turn exactly, so
// a far position costs nothing in accuracy (an fp32 angle of 262144 radians is
// off by 0.016) and no fp64.  Its top 32 bits less the nearest quarter turn go to
// sincospif as a float of at most a quarter of half a turn: the rounding there is
// at most 2^-27 of half a turn, 2.4e-8 radians.
// Translation units that include this are compiled with -fmad=false, so that their
// rows agree bit for bit.
#pragma once
#include "rows.cuh"

namespace kvq {

constexpr int kMaxPairs = 128;
constexpr int kRopeE = 16;  // elements of a lane

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
  // the nearest quarter turn, and what is left of it in half turns, |t| <= 1/4
  const uint32_t h = static_cast<uint32_t>(phase >> 32) + 0x20000000u;
  const uint32_t quarter = h >> 30;
  float t = __fmul_rn(static_cast<float>(static_cast<int32_t>(h & 0x3FFFFFFFu) - 0x20000000), 4.656612873077393e-10f);
  if (axis >= r.axes) {
    set_status(status, KVQ_DEV_BAD_INDEX);
    t = NAN;
  }
  float s, c;
  sincospif(t, &s, &c);
  float2 cs = (quarter & 1) ? make_float2(s, c) : make_float2(c, s);
  if ((quarter + 1) & 2) cs.x = -cs.x;
  if (quarter & 2) cs.y = -cs.y;
  return cs;
}

// The token's positions on the rope's axes.
__device__ __forceinline__ void load_pos(const RopeView& r, int64_t tok, int32_t (&pos)[4]) {
#pragma unroll
  for (int a = 0; a < 4; ++a) pos[a] = a < r.axes ? r.pos[a * r.pos_stride + tok] : 0;
}

// LANES lanes work out one token's angles, `lane` this one's place among them; CH: the
// chunks of a copy.
template <int LANES = 32, int CH = kChunks>
__device__ __forceinline__ void make_angles(const RopeView& r, const int32_t (&pos)[4], int lane, int32_t* status,
                                            float4* sh) {
  __syncwarp();  // (the last token's have been read)
  for (int p = lane; p < (r.rot >> 1); p += LANES) {
    const float2 cs = angle(r, p, pos, status);
    float* at = reinterpret_cast<float*>(&sh[chunk_place(p >> 1)]) + (p & 1);
    at[0] = cs.x;
    at[2] = cs.y;
    at += 4 * CH;
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

template <int CH = kChunks>
__device__ __forceinline__ RopeLane rope_lane(const RopeView& r, const float4* sh, int lane, int l) {
  RopeLane g;
  const int half = r.rot >> 1;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int e = kRopeE * l + 8 * k;
    g.in[k] = e < r.rot;
    const bool first = e < half;
    g.src[k] = lane - l + (!g.in[k] ? e : first ? e + half : e - half) / kRopeE;
    g.cs[k] = sh + (first ? CH : 0) + chunk_place(g.in[k] ? (first ? e : e - half) / 2 : 0);
  }
  if (r.interleaved) g.cs[0] = sh + chunk_place(g.in[0] ? kRopeE * l / 4 : 0);
  return g;
}

template <int SH, int U>
__device__ __forceinline__ void rope_half_split(const RopeLane& g, uint64_t (&x)[U][kRopeE / 2]) {
  uint64_t o[U][kRopeE / 2];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < kRopeE / 2; ++i) {
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
__device__ __forceinline__ void rope_rows(const RopeView& r, const RopeLane& g, int l, uint64_t (&x)[U][kRopeE / 2]) {
  if (!r.interleaved) {
    if (r.rot & 16) rope_half_split<1, U>(g, x);
    else rope_half_split<0, U>(g, x);
    return;
  }
  if (!g.in[0]) return;
  const int e = kRopeE * l;
#pragma unroll
  for (int i = 0; i < kRopeE / 2; i += 2) {
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

}  // namespace kvq
