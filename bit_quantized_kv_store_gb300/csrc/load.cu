// load.cu -- rows of the cache read back as the values they stand for: by slot, or
// ragged runs of positions by block table.
//
// The value of a code is the format's ("qwen27 CUDA: an opt-in 4-bit attention
// cache (262K on a 24 GB card)", section "What it is": Hadamard-rotated groups
// as 4-bit codes with an fp16 scale; "KV cache quantization: fp8 (KV8) + 4-bit
// TurboQuant": e4m3 rows with fp32 scales, and randomized-Hadamard rows with a
// 16-level codebook).  Rotating back takes the sums of the codes first and the
// scale after, so that the sums are exact:
//   Q4_HAD32: sums of 32 integers -8 .. 7 are at most 256 in magnitude, exact in
//     fp16, so the butterfly runs on packed fp16 pairs;
//   TQ4: the levels are multiples of 2^-13 below 4 and a sum of 256 of them is
//     below 2^10, 23 bits: exact in fp32.
// What is left is fl(sum * fl(scale / sqrt(n))) and the rounding into the output's
// type.
//
// One lane takes one group of 32 values: one 16-byte load of codes, the butterfly
// in registers (TQ4: its last stages across the row's lanes), and the 32 results
// as whole 32-byte sectors (256-bit stores), so no shared memory is needed to
// write full sectors.  Bound: memory (in bf16 the outputs are 3.6 times the
// codes' bytes).
#include <cuda_fp8.h>

#include "kernels.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

constexpr int kLoadBlock = 256;

// 32 bytes at once (address a multiple of 32).
__device__ __forceinline__ void st256(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// N (a multiple of 16) consecutive values into the view at element e (view.wide:
// the address is a multiple of 32 bytes).
template <int N>
__device__ __forceinline__ void put_values(const RowsView& v, int64_t e, const float (&x)[N]) {
  if (v.dtype == KVQ_DT_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(v.data) + e;
    if (v.wide) {
#pragma unroll
      for (int i = 0; i < N; i += 16) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = bf16_pair(x[i + 2 * j], x[i + 2 * j + 1]);
        st256(p + i, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
  } else {
    float* p = static_cast<float*>(v.data) + e;
    if (v.wide) {
#pragma unroll
      for (int i = 0; i < N; i += 8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[i + j]);
        st256(p + i, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = x[i];
    }
  }
}

enum Where { kSkip, kBad, kRow };

// The last sequence b with cu_lens[b] <= t (0 if there is none), by halving.
__device__ __forceinline__ int sequence_of(const LoadArgs& a, int64_t t) {
  int lo = 0, hi = a.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_lens[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Where output token t's row lies, or why it has none.
__device__ __forceinline__ Where locate(const LoadArgs& a, int64_t t, int32_t& page, uint32_t& off, int32_t& why) {
  if (a.slots) {
    const int32_t slot = a.slots[t];
    if (slot < 0) return kSkip;
    if ((int64_t)slot >= (int64_t)a.c.num_pages * a.c.page_size) {
      why = KVQ_DEV_BAD_SLOT;
      return kBad;
    }
    page = fast_div(static_cast<uint32_t>(slot), a.ps);
    off = static_cast<uint32_t>(slot) - page * a.ps.d;
    return kRow;
  }
  const int b = sequence_of(a, t);
  const int32_t start = a.cu_lens[b];
  if (t < start || t >= a.cu_lens[b + 1]) return kSkip;
  const int64_t p = t - start + (a.starts ? a.starts[b] : 0);
  if (p < 0 || p >= (int64_t)a.max_pages * a.c.page_size || p >= (int64_t(1) << 31)) {
    why = KVQ_DEV_BAD_LENGTH;
    return kBad;
  }
  const uint32_t col = fast_div(static_cast<uint32_t>(p), a.ps);
  off = static_cast<uint32_t>(p) - col * a.ps.d;
  page = a.block_tables[(int64_t)b * a.max_pages + col];
  if (page < 0 || page >= a.c.num_pages) {
    why = KVQ_DEV_BAD_PAGE;
    return kBad;
  }
  return kRow;
}

// The 32 codes of a group (16 bytes) as exact fp16 pairs (code - 8): register
// 4q + j holds elements 8q + j and 8q + j + 4.
__device__ __forceinline__ void q4_pairs(const uint4& u, __half2 (&p)[16]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    p[4 * q + 0] = u32_as_h2(nib_lo_pair(w[q]));
    p[4 * q + 1] = u32_as_h2(nib_hi_pair(w[q]));
    p[4 * q + 2] = u32_as_h2(nib_lo_pair(w[q] >> 8));
    p[4 * q + 3] = u32_as_h2(nib_hi_pair(w[q] >> 8));
  }
}

// The 32-point butterfly (unscaled) on those pairs; every sum is exact.
__device__ __forceinline__ void h2_butterfly(__half2 (&p)[16]) {
#pragma unroll
  for (int h = 1; h < 16; h <<= 1)  // element distances 1, 2, 8, 16
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & h)) {
        const __half2 s = __hadd2(p[i], p[i + h]), d = __hsub2(p[i], p[i + h]);
        p[i] = s;
        p[i + h] = d;
      }
  const __half2 pm = u32_as_h2(0xBC003C00u);  // (1, -1)
#pragma unroll
  for (int i = 0; i < 16; ++i)  // element distance 4: the halves of a register
    p[i] = __hfma2(p[i], pm, __lowhigh2highlow(p[i]));
}

// Byte `hi` (1) or 0 of the fp16 levels m .. m + 3, as a byte-permute table word.
__host__ __device__ constexpr uint32_t tq4_table(int m, int hi) {
  // the levels in fp16: 0.128.., 0.387.., 0.656.., 0.942.., 1.255.., 1.618.., 2.068.., 2.732..
  constexpr uint16_t lev[8] = {0x301C, 0x3635, 0x3941, 0x3B8A, 0x3D06, 0x3E79, 0x4023, 0x4177};
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>((lev[m + i] >> (8 * hi)) & 0xFF) << (8 * i);
  return w;
}

// The 8 levels (with sign) of a word of 8 TQ4 codes.
__device__ __forceinline__ void tq4_levels8(uint32_t w, float (&x)[8]) {
  const uint32_t m = w & 0x77777777u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // codes 4h .. 4h + 3
    const uint32_t sel = h ? m >> 16 : m;
    const uint32_t lo = prmt(tq4_table(0, 0), tq4_table(4, 0), sel), hi = prmt(tq4_table(0, 1), tq4_table(4, 1), sel);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = 4 * h + 2 * j;
      const uint32_t pair = prmt(lo, hi, j ? 0x7362u : 0x5140u);
      const float2 f = __half22float2(u32_as_h2(pair));
      x[c] = __uint_as_float(__float_as_uint(f.x) | ((w << (28 - 4 * c)) & 0x80000000u));
      x[c + 1] = __uint_as_float(__float_as_uint(f.y) | ((w << (24 - 4 * c)) & 0x80000000u));
    }
  }
}

// FMT: KVQ_FMT_Q4_HAD32, KVQ_FMT_Q4_0 or KVQ_FMT_TQ4; NG groups of 32 in a row.
// A thread takes one group of one row; groups, heads, K / V and tokens in this
// order.  rpt divides by a token's rows (its heads in the planes wanted, the
// first of which is K when kv0 == 0), so a launch keeps tokens * rows * NG < 2^31.
template <int FMT, int NG>
__global__ void __launch_bounds__(kLoadBlock) load_q4_kernel(const __grid_constant__ LoadArgs a, int kv0, FastDiv rpt) {
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * NG;
  const int Hk = a.c.num_kv_heads;
  const uint32_t idx = blockIdx.x * kLoadBlock + threadIdx.x;
  const int G = static_cast<int>(idx % NG);
  const uint32_t row = idx / NG;
  const uint32_t dt = fast_div(row, rpt);
  const uint32_t rt = row - dt * rpt.d;
  const uint32_t plane = fast_div(rt, a.hk);
  const int head = static_cast<int>(rt - plane * a.hk.d);
  const bool is_v = kv0 + static_cast<int>(plane) != 0;
  const int64_t t = a.t0 + dt;
  int32_t page = 0, why = 0;
  uint32_t off = 0;
  const Where at = t < a.n_tok ? locate(a, t, page, off, why) : kSkip;
  const int64_t r = ((int64_t)page * Hk + head) * a.c.page_size + off;
  const uint8_t* codes = static_cast<const uint8_t*>(is_v ? a.c.v : a.c.k);
  const __half* scales = static_cast<const __half*>(is_v ? a.c.v_scale : a.c.k_scale);
  float x[32];
  if constexpr (FMT == KVQ_FMT_TQ4) {
    float f = 0.f;
    uint4 u = make_uint4(0, 0, 0, 0);  // rows that are not read still take part in the exchanges
    if (at == kRow) {
      u = reinterpret_cast<const uint4*>(codes + r * (D / 2))[G];
      f = __half2float(scales[r]);
    }
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) tq4_levels8(w[q], *reinterpret_cast<float(*)[8]>(&x[8 * q]));
    if (a.rotate_back) {
#pragma unroll
      for (int h = 1; h < 32; h <<= 1)
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (!(i & h)) {
            const float p = x[i], q = x[i + h];
            x[i] = p + q;
            x[i + h] = p - q;
          }
#pragma unroll
      for (int o = 1; o < NG; o <<= 1) {  // the stages between the row's groups, its NG lanes
        const float sgn = (G & o) ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __fmaf_rn(x[i], sgn, __shfl_xor_sync(0xffffffffu, x[i], o));
      }
      f *= tq4_row_scale<NG>();
      const uint32_t sw = static_cast<const uint32_t*>(a.c.signs)[G];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        x[i] = __uint_as_float(__float_as_uint(x[i] * f) ^ ((sw << (31 - i)) & 0x80000000u));
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= f;
    }
  } else if (at == kRow) {
    const uint4 u = reinterpret_cast<const uint4*>(codes + r * (D / 2))[G];
    float f = __half2float(scales[r * NG + G]);
    __half2 p[16];
    q4_pairs(u, p);
    if (FMT == KVQ_FMT_Q4_HAD32 && a.rotate_back) {
      h2_butterfly(p);
      f *= kHadamardScale;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = __half22float2(p[4 * q + j]);
        x[8 * q + j] = v.x * f;
        x[8 * q + j + 4] = v.y * f;
      }
  }
  if (at == kSkip) return;
  if (at == kBad) {
    if (G == 0) set_status(a.status, why);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = NAN;
  }
  const RowsView& out = is_v ? a.v : a.k;
  put_values<32>(out, t * out.ts + head * out.hs + 32 * G, x);
}

// BF16 and fp8 latent rows: a thread takes 16 consecutive values of a row.  cpt
// divides by a token's 16-value chunks, cpr by a row's (fp8: the latent and rope
// parts are one row).
template <bool FP8>
__global__ void __launch_bounds__(kLoadBlock) load_wide_kernel(const __grid_constant__ LoadArgs a, int kv0, FastDiv cpt,
                                                               FastDiv cpr) {
  pdl_wait();
  pdl_trigger();
  const uint32_t idx = blockIdx.x * kLoadBlock + threadIdx.x;
  const uint32_t dt = fast_div(idx, cpt);
  const int64_t t = a.t0 + dt;
  if (t >= a.n_tok) return;
  const uint32_t ct = idx - dt * cpt.d;
  const uint32_t row = fast_div(ct, cpr);  // (fp8: 0)
  const int c = static_cast<int>(ct - row * cpr.d) * 16;
  int32_t page = 0, why = 0;
  uint32_t off = 0;
  const Where at = locate(a, t, page, off, why);
  if (at == kSkip) return;
  const int Hk = a.c.num_kv_heads, D = a.c.head_dim;
  float x[16];
  if (at == kBad) {
    if (c == 0) set_status(a.status, why);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = NAN;
  }
  if constexpr (FP8) {
    if (at == kRow) {
      const int64_t r = (int64_t)page * a.c.page_size + off;
      const bool rope = c >= D;
      const uint8_t* p = rope ? static_cast<const uint8_t*>(a.c.v) + r * a.c.rope_dim + (c - D)
                              : static_cast<const uint8_t*>(a.c.k) + r * D + c;
      const float sc = static_cast<const float*>(rope ? a.c.v_scale : a.c.k_scale)[r];
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const __half2_raw h =
            __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        x[2 * i] = f.x * sc;
        x[2 * i + 1] = f.y * sc;
      }
    }
    put_values<16>(a.k, t * a.k.ts + c, x);
  } else {
    const uint32_t plane = fast_div(row, a.hk);
    const int head = static_cast<int>(row - plane * a.hk.d);
    const bool is_v = kv0 + static_cast<int>(plane) != 0;
    const RowsView& out = is_v ? a.v : a.k;
    if (at == kRow) {
      const int64_t r = ((int64_t)page * Hk + head) * a.c.page_size + off;
      const uint4* p =
          reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(is_v ? a.c.v : a.c.k) + r * D + c);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint4 u = p[q];
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[8 * q + 2 * i] = __uint_as_float(w[i] << 16);
          x[8 * q + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    }
    put_values<16>(out, t * out.ts + head * out.hs + c, x);
  }
}

}  // namespace

cudaError_t launch_load(const LoadArgs& args, cudaStream_t s) {
  LoadArgs a = args;
  const int kv0 = a.k.data ? 0 : 1, kvs = (a.k.data ? 1 : 0) + (a.v.data ? 1 : 0);
  const int Hk = a.c.num_kv_heads, D = a.c.head_dim;
  const bool fp8 = a.c.format == KVQ_FMT_FP8_ROW, wide = fp8 || a.c.format == KVQ_FMT_BF16;
  const int NG = D / 32, cpr = (fp8 ? D + a.c.rope_dim : D) / 16;
  const int64_t rows = fp8 ? 1 : (int64_t)Hk * kvs;      // of a token
  const int64_t per_tok = rows * (wide ? cpr : NG);      // threads of a token
  if (per_tok >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
  const FastDiv fr = make_fastdiv(static_cast<uint32_t>(rows)), ft = make_fastdiv(static_cast<uint32_t>(per_tok)),
                fc = make_fastdiv(static_cast<uint32_t>(cpr));
  // launches of at most 2^30 threads, so that the kernels' indices stay 32-bit
  const int64_t max_tok = (int64_t(1) << 30) / per_tok, n_tok = a.n_tok;
  for (a.t0 = 0; a.t0 < n_tok; a.t0 += max_tok) {
    a.n_tok = n_tok - a.t0 < max_tok ? n_tok : a.t0 + max_tok;  // tokens [t0, n_tok) in this launch
    const dim3 grid(static_cast<unsigned>(((a.n_tok - a.t0) * per_tok + kLoadBlock - 1) / kLoadBlock)), block(kLoadBlock);
    cudaError_t e = cudaErrorInvalidValue;
#define KVQ_LOAD(F, N) e = launch_pdl(load_q4_kernel<F, N>, grid, block, 0, s, a, kv0, fr); break
    if (fp8) {
      e = launch_pdl(load_wide_kernel<true>, grid, block, 0, s, a, kv0, ft, fc);
    } else if (wide) {
      e = launch_pdl(load_wide_kernel<false>, grid, block, 0, s, a, kv0, ft, fc);
    } else if (a.c.format == KVQ_FMT_Q4_HAD32) {
      switch (NG) {
        case 1: KVQ_LOAD(KVQ_FMT_Q4_HAD32, 1);
        case 2: KVQ_LOAD(KVQ_FMT_Q4_HAD32, 2);
        case 4: KVQ_LOAD(KVQ_FMT_Q4_HAD32, 4);
        case 8: KVQ_LOAD(KVQ_FMT_Q4_HAD32, 8);
        default: break;
      }
    } else if (a.c.format == KVQ_FMT_Q4_0) {
      switch (NG) {
        case 1: KVQ_LOAD(KVQ_FMT_Q4_0, 1);
        case 2: KVQ_LOAD(KVQ_FMT_Q4_0, 2);
        case 4: KVQ_LOAD(KVQ_FMT_Q4_0, 4);
        case 8: KVQ_LOAD(KVQ_FMT_Q4_0, 8);
        default: break;
      }
    } else {
      switch (NG) {
        case 2: KVQ_LOAD(KVQ_FMT_TQ4, 2);
        case 4: KVQ_LOAD(KVQ_FMT_TQ4, 4);
        case 8: KVQ_LOAD(KVQ_FMT_TQ4, 8);
        default: break;
      }
    }
#undef KVQ_LOAD
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace kvq
