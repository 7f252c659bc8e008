// seqs.cuh -- the rows of several sequences over a paged cache, and the keys that they
// see: the last n rows of a sequence of T stored tokens sit at positions T - n .. T - 1,
// and the row at position p sees key j when j <= p and, with a window, j > p - window or
// j < sinks.  Shared by the attention kernels over ragged batches.
#pragma once
#include "rows.cuh"

namespace kvq {

struct SeqRows {
  int first;  // the sequence's first row in q and out
  int n;      // its rows
  int T;      // its stored tokens
  int state;  // kRowsOk, or why it is not computed
};
enum { kRowsOk = 0, kRowsSkip = 1 /* left as they are */, kRowsNan = 2 /* NaN */ };

// Behind every key and (negative) before every position; lengths and rows stay below it.
constexpr int kNoKey = 1 << 29;

// Sequence b's rows.
__device__ __forceinline__ SeqRows seq_rows(const SeqAttnArgs& a, int b) {
  SeqRows s;
  int last;
  if (a.cu_rows) {
    s.first = a.cu_rows[b];
    last = a.cu_rows[b + 1];
  } else {
    s.first = b;
    last = b + 1;
  }
  s.T = a.seq_lens[b];
  s.n = last - s.first;
  s.state = kRowsOk;
  if (s.first < 0 || last < s.first || last > a.n_rows || s.n > a.max_rows) {
    s.state = kRowsSkip;
    s.n = 0;
  } else if (s.T < 0 || s.T > a.max_seq_len || static_cast<int64_t>(s.T) > static_cast<int64_t>(a.max_pages) * a.c.page_size) {
    s.state = kRowsNan;
  }
  return s;
}

// Where a row's reference is a score (base 2) beyond this, its scores are taken in units that
// bring the reference down to it, so that their differences, and with them p and its place in
// fp16, are not off by as much as 32 bits are coarse there (32 at 2^28).  Two scores that differ
// by more than their operands' rounding, 2^-11 of them, are still 500 powers of two apart.
constexpr float kFarScore = 1048576.f;

__device__ __forceinline__ bool key_visible(int key, int p, int window, int sinks) {
  return key <= p && (window == 0 || key > p - window || key < sinks);
}

// The 16-key blocks that rows at positions p0 .. p1 (p1 >= 0) see some key of: blocks
// 0 .. head - 1 (the sinks', where a gap lies behind them), then from `body` on; block i
// of `count` is block_of(i).
struct KeyBlocks {
  int head, body, count;
  __device__ __forceinline__ int block_of(int i) const { return i < head ? i : i - head + body; }
};
__device__ __forceinline__ KeyBlocks key_blocks(int p0, int p1, int window, int sinks) {
  KeyBlocks k{0, 0, 0};
  const int end = (p1 >> 4) + 1;
  if (window > 0) {
    k.head = min((sinks + 15) >> 4, end);
    const int lo = max(p0, 0) - window + 1;
    k.body = max(max(lo, 0) >> 4, k.head);
  }
  k.count = k.head + max(0, end - k.body);
  return k;
}

// Whether every one of rows p0 .. p1 sees all keys k0 .. k0 + n - 1.
__device__ __forceinline__ bool all_visible(int k0, int n, int p0, int p1, int window, int sinks) {
  return k0 + n - 1 <= p0 && (window == 0 || k0 > p1 - window || k0 + n <= sinks);
}
// Whether some of rows p0 .. p1 sees key k (p0 <= p1).
__device__ __forceinline__ bool any_visible(int k, int p0, int p1, int window, int sinks) {
  return k <= p1 && (window == 0 || k > max(p0, k) - window || k < sinks);
}

// The D-point signed transform of a row whose element 32 G + lane is x[G].
template <int NG>
__device__ __forceinline__ void tq4_turn_lanes(float (&x)[NG], const uint32_t* signs, int lane, bool inverse) {
  if (!inverse) {
#pragma unroll
    for (int G = 0; G < NG; ++G)
      if ((signs[G] >> lane) & 1u) x[G] = -x[G];
  }
#pragma unroll
  for (int G = 0; G < NG; ++G) x[G] = warp_fwht32(x[G], lane);
#pragma unroll
  for (int h = 1; h < NG; h <<= 1)
#pragma unroll
    for (int G = 0; G < NG; ++G)
      if (!(G & h)) {
        const float u = x[G], v = x[G + h];
        x[G] = u + v;
        x[G + h] = u - v;
      }
  const float c = NG == 8 ? 0.0625f : NG == 4 ? 0.08838834764831845f : 0.125f;
#pragma unroll
  for (int G = 0; G < NG; ++G) x[G] *= c;
  if (inverse) {
#pragma unroll
    for (int G = 0; G < NG; ++G)
      if ((signs[G] >> lane) & 1u) x[G] = -x[G];
  }
}

// One output value, rounded into its type.
__device__ __forceinline__ void seq_store(const SeqAttnArgs& a, int row, int head, int e, float y) {
  const int64_t at = static_cast<int64_t>(row) * a.out.ts + static_cast<int64_t>(head) * a.out.hs + e;
  if (a.out.dtype == KVQ_DT_F32) static_cast<float*>(a.out.data)[at] = y;
  else static_cast<__nv_bfloat16*>(a.out.data)[at] = __float2bfloat16_rn(y);
}

// 8 values of every group of 32 of a row, the first of them element `at` of the view (< 0:
// zeros).
template <int NG>
__device__ __forceinline__ void seq_load_row(const RowsView& v, int64_t at, float (&x)[NG][8]) {
  if (at < 0) {
#pragma unroll
    for (int G = 0; G < NG; ++G)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[G][e] = 0.f;
  } else if (v.dtype == KVQ_DT_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(v.data) + at;
    uint32_t w[NG][4];
#pragma unroll
    for (int G = 0; G < NG; ++G) {
      if (v.wide) {
        ld_words<4>(p + 32 * G, w[G]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[G][i] = p[32 * G + 2 * i] | static_cast<uint32_t>(p[32 * G + 2 * i + 1]) << 16;
      }
    }
#pragma unroll
    for (int G = 0; G < NG; ++G)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[G][2 * i] = __uint_as_float(w[G][i] << 16);
        x[G][2 * i + 1] = __uint_as_float(w[G][i] & 0xFFFF0000u);
      }
  } else {
    const float* p = static_cast<const float*>(v.data) + at;
#pragma unroll
    for (int G = 0; G < NG; ++G) {
      if (v.wide) {
        ld_words<8>(p + 32 * G, reinterpret_cast<uint32_t*>(x[G]));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[G][e] = p[32 * G + e];
      }
    }
  }
}

// The rows' rotation (ALL: the D-point one with signs, else each group's; SCALE: to norm 1), for rows whose
// elements 32 G + 8 (lane >> 3) + e are x[G][e].
template <int NG, bool ALL, bool SCALE = true>
__device__ __forceinline__ void seq_turn(float (&x)[NG][8], const uint32_t* signs, int lane, bool inverse) {
  auto flip = [&] {
#pragma unroll
    for (int G = 0; G < NG; ++G) {
      const uint32_t s = signs[G] >> (8 * (lane >> 3));
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((s >> e) & 1u) x[G][e] = -x[G][e];
    }
  };
  if (ALL && !inverse) flip();
#pragma unroll
  for (int G = 0; G < NG; ++G) {
#pragma unroll
    for (int h = 1; h < 8; h <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(e & h)) {
          const float u = x[G][e], v = x[G][e + h];
          x[G][e] = u + v;
          x[G][e + h] = u - v;
        }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = __shfl_xor_sync(0xffffffffu, x[G][e], o);
        x[G][e] = lane & o ? y - x[G][e] : x[G][e] + y;
      }
  }
  if constexpr (ALL) {
#pragma unroll
    for (int h = 1; h < NG; h <<= 1)
#pragma unroll
      for (int G = 0; G < NG; ++G)
        if (!(G & h))
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float u = x[G][e], v = x[G + h][e];
            x[G][e] = u + v;
            x[G + h][e] = u - v;
          }
  }
  if constexpr (SCALE) {
    const float c = !ALL ? kHadamardScale : NG == 8 ? 0.0625f : NG == 4 ? 0.08838834764831845f : 0.125f;
#pragma unroll
    for (int G = 0; G < NG; ++G)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[G][e] *= c;
  }
  if (ALL && inverse) flip();
}

// 32 consecutive values of a row, from element `at` of the view on (< 0: zeros).
__device__ __forceinline__ void seq_load_32(const RowsView& v, int64_t at, float (&x)[4][8]) {
  if (at < 0) {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i >> 3][i & 7] = 0.f;
  } else if (v.dtype == KVQ_DT_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(v.data) + at;
    uint32_t w[16];
    if (v.wide) {
      ld_words<16>(p, w);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = p[2 * i] | static_cast<uint32_t>(p[2 * i + 1]) << 16;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i >> 2][2 * (i & 3)] = __uint_as_float(w[i] << 16);
      x[i >> 2][2 * (i & 3) + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float* p = static_cast<const float*>(v.data) + at;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (v.wide) {
        ld_words<8>(p + 8 * i, reinterpret_cast<uint32_t*>(x[i]));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = p[8 * i + e];
      }
    }
  }
}

// The 32-point butterfly of one thread's values, no scaling.
__device__ __forceinline__ void seq_turn_32(float (&x)[4][8]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(i & h)) {
        const int k = i + h;
        const float u = x[i >> 3][i & 7], v = x[k >> 3][k & 7];
        x[i >> 3][i & 7] = u + v;
        x[k >> 3][k & 7] = u - v;
      }
}

// 32 consecutive values to `at`, rounded into its type (`wide`: on a 32-byte boundary).
__device__ __forceinline__ void seq_store_32(void* at, int dtype, bool wide, const float (&x)[4][8]) {
  if (dtype == KVQ_DT_F32) {
    float* p = static_cast<float*>(at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (wide) {
        st_words<8>(p + 8 * i, reinterpret_cast<const uint32_t*>(x[i]));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[8 * i + e] = x[i][e];
      }
    }
  } else {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (wide) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = pack_bf16(x[2 * i + (e >> 2)][2 * (e & 3)], x[2 * i + (e >> 2)][2 * (e & 3) + 1]);
        st_words<8>(p + 16 * i, w);
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) p[16 * i + e] = __float2bfloat16_rn(x[2 * i + (e >> 3)][e & 7]);
      }
    }
  }
}

}  // namespace kvq
