// load.cu -- rows of the cache read back as the values they stand for: by slot, or
// ragged runs of positions by block table.
//
// The value of a code is the format's ("qwen27 CUDA: an opt-in 4-bit attention
// cache (262K on a 24 GB card)", section "What it is": Hadamard-rotated groups
// as 4-bit codes with an fp16 scale; "KV cache quantization: fp8 (KV8) + 4-bit
// TurboQuant": e4m3 rows with fp32 scales, and randomized-Hadamard rows with a
// 16-level codebook).  Rotating back takes the sums of the codes first and the
// scale after, so that the sums are exact in fp32:
//   Q4_HAD32: 32 integers -8 .. 7;
//   TQ4: the levels are multiples of 2^-13 below 4, and a sum of 256 of them is
//     below 2^10: 23 bits.
// What is left is fl(sum * fl(scale / sqrt(n))) and the rounding into the output's
// type.
//
// The 32-point transform of a group is a product with a matrix of +-1, so it runs
// on the tensor cores (m16n8k16, fp16 operands that hold the codes exactly): as a
// butterfly in registers it took 230 instructions a group and the whole kernel was
// bound by issuing them (262144 tokens of 4 heads: 272 us, floor 203 us).  One
// warp tile is 8 groups of K and the same 8 of V (the 16 rows of the operand); the
// columns of the matrix are ordered so that a thread's results are 8 consecutive
// values, and the terms so that it loads 8 consecutive codes as one word.  The TQ4
// rows' stages between the groups of a row come first, as a product from the left
// with the groups' +-1 matrix; its sums enter the second product as two fp16 terms.
// (As stages across lanes on the results they were a third of the instructions.)
//
// Bound: memory (in bf16 the outputs are 3.6 times the codes' bytes).  262144 tokens
// of 4 heads to bf16: 218 us, 1.38 GB, 6.3 TB/s (93 % of the measured copy).  20011
// tokens of TQ4 rows to fp32: 34.1 us, 185 MB, 5.4 TB/s; 200011 to bf16: 265 us, 1.03 GB:
// the look-ups and the sums in two terms take 120 registers, and at 16 warps an SM half
// the issue slots wait (the FEW kernels spill 16 to 36 bytes a thread besides).  Rows
// without codes (load_wide_kernel): 65536 tokens of 4 bf16 heads 84 us, 6.4 TB/s;
// 262144 fp8 rows to bf16 81 us, 5.6 TB/s.  A lane writes 16 bytes next to its
// neighbours' or 32 by itself: stores of 16 bytes 32 apart reached 4.1 TB/s, these
// 7.5 TB/s, in a kernel that only writes.
#include <cuda_fp8.h>

#include "rows.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

constexpr int kLoadBlock = 256;

// N (8, or a multiple of 16) consecutive values to an address (`wide`: a multiple of
// their bytes, up to 32).
template <int N>
__device__ __forceinline__ void put_values(void* at, int dtype, int wide, const float (&x)[N]) {
  if (dtype == KVQ_DT_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(at);
    if (wide) {
      uint32_t w[N / 2];
#pragma unroll
      for (int i = 0; i < N / 2; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
      st_words<N / 2>(p, w);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) p[i] = __float2bfloat16_rn(x[i]);
    }
  } else {
    float* p = static_cast<float*>(at);
    if (wide) {
      uint32_t w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(x[i]);
      st_words<N>(p, w);
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

// Byte `hi` (1) or 0 of the fp16 levels m .. m + 3, as a byte-permute table word.
__host__ __device__ constexpr uint32_t tq4_table(int m, int hi) {
  // the levels in fp16: 0.128.., 0.387.., 0.656.., 0.942.., 1.255.., 1.618.., 2.068.., 2.732..
  constexpr uint16_t lev[8] = {0x301C, 0x3635, 0x3941, 0x3B8A, 0x3D06, 0x3E79, 0x4023, 0x4177};
  uint32_t w = 0;
  for (int i = 0; i < 4; ++i) w |= static_cast<uint32_t>((lev[m + i] >> (8 * hi)) & 0xFF) << (8 * i);
  return w;
}

// The 8 codes of a word as four exact fp16 pairs, and which codes a pair holds:
// pair 2s + u is (element 2s + u, element 2s + u + 4) for the 4-bit formats (code -
// 8), (element 4s + 2u, the next) for TQ4 (the levels, by byte permutes).
template <int FMT>
__device__ __forceinline__ void code_pairs(uint32_t w, uint32_t (&p)[4]) {
  if constexpr (FMT == KVQ_FMT_TQ4) {
    const uint32_t m = w & 0x77777777u;
#pragma unroll
    for (int s = 0; s < 2; ++s) {  // codes 4s .. 4s + 3
      const uint32_t sel = s ? m >> 16 : m;
      const uint32_t lo = prmt(tq4_table(0, 0), tq4_table(4, 0), sel);
      uint32_t hi = prmt(tq4_table(0, 1), tq4_table(4, 1), sel);
      // their signs into the levels' high bytes: every code byte twice, the first with
      // its low nibble's sign (bit 3) moved up, the second with its high nibble's (bit 7)
      const uint32_t y = prmt(w, 0u, s ? 0x3322u : 0x1100u);
      hi |= ((y & 0xFF00FF00u) | ((y << 4) & 0x00FF00FFu)) & 0x80808080u;
      p[2 * s] = prmt(lo, hi, 0x5140u);
      p[2 * s + 1] = prmt(lo, hi, 0x7362u);
    }
  } else {
    p[0] = nib_lo_pair(w);
    p[1] = nib_hi_pair(w);
    p[2] = nib_lo_pair(w >> 8);
    p[3] = nib_hi_pair(w >> 8);
  }
}

// The same pairs' codes in element order, as fp32.
template <int FMT>
__device__ __forceinline__ void code_values(uint32_t w, float (&x)[8]) {
  uint32_t p[4];
  code_pairs<FMT>(w, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(u32_as_h2(p[i]));
    x[FMT == KVQ_FMT_TQ4 ? 2 * i : i] = f.x;
    x[FMT == KVQ_FMT_TQ4 ? 2 * i + 1 : i + 4] = f.y;
  }
}

// The +-1 matrix's fragments of this lane (t = lane & 3, g = lane >> 2): step s of
// the two of 16 terms, half u, result columns 8 nt + g, which stand for output
// 8 (g >> 1) + 2 nt + (g & 1).  The sign of (element, output) is the parity of
// their common bits: bits 3 and 4 give the lane's base sign, the bits of the pair's
// place and of s, u, nt flip it.
template <int FMT>
struct SignMatrix {
  // the few distinct fragments, kept in registers: TQ4 [parity], 4-bit [u][nt >> 1][s & nt & 1]
  uint32_t m[FMT == KVQ_FMT_TQ4 ? 2 : 8];
  __device__ __forceinline__ explicit SignMatrix(int lane) {
    const int t = lane & 3, g = lane >> 2;
    const uint32_t b = (__popc(t & (g >> 1)) & 1) ? 0xBC00BC00u : 0x3C003C00u;  // -1, 1
    if constexpr (FMT == KVQ_FMT_TQ4) {  // pair place: element bit 0; u: bit 1; s: bit 2
      m[0] = b ^ ((g & 1) ? 0x80000000u : 0u);
      m[1] = m[0] ^ 0x80008000u;
    } else {  // u: element bit 0 (odd elements' entries are +-1/16); s: bit 1; pair place: bit 2
#pragma unroll
      for (int i = 0; i < 8; ++i)
        m[i] = b ^ ((i & 4) ? ((g & 1) ? 0x80008000u : 0u) ^ (0x3C003C00u ^ 0x2C002C00u) : 0u) ^
               ((i & 2) ? 0x80000000u : 0u) ^ ((i & 1) ? 0x80008000u : 0u);
    }
#pragma unroll
    for (uint32_t& r : m) asm volatile("" : "+r"(r));  // (not to be worked out again for every tile)
  }
  __device__ __forceinline__ uint32_t at(int s, int u, int nt) const {
    if constexpr (FMT == KVQ_FMT_TQ4) return m[((u & nt) ^ (s & (nt >> 1))) & 1];
    else return m[4 * u + (nt & 2) + (s & nt & 1)];
  }
};

// A sum of 8 TQ4 levels, a multiple of 2^-13 below 22, as two exact fp16 terms: the
// nearest multiple of 2^-6 (adding 1.5 * 2^17 rounds to one) and what is left.
__device__ __forceinline__ void split_sums(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const uint64_t x = pk2(x0, x1), m2 = pk2(196608.0f, 196608.0f), h = sub2(add2(x, m2), m2);
  float a, b;
  upk2(h, a, b);
  hi = pack_half2(a, b);
  upk2(sub2(x, h), a, b);
  lo = pack_half2(a, b);
}

// The codes of a word as mma operands.  4-bit formats: left biased, 1024 + c in the
// pairs of even elements and 1024 + 16 c in those of odd ones, whose matrix entries
// are +-1/16: the biases, 1024 and 64, cancel in every sum but outputs 0 and 1,
// whose accumulators start from minus theirs (kBias0, with the 8 of every code; kBias1).
constexpr float kBias0 = -(16.f * 1024.f + 16.f * 64.f + 32.f * 8.f), kBias1 = -(16.f * 1024.f - 16.f * 64.f);
template <int FMT>
__device__ __forceinline__ void code_operands(uint32_t w, uint32_t (&p)[4]) {
  if constexpr (FMT == KVQ_FMT_TQ4) {
    code_pairs<FMT>(w, p);
  } else {
    p[0] = nib_lo_pair_biased(w);
    p[1] = nib_hi_pair_biased(w);
    p[2] = nib_lo_pair_biased(w >> 8);
    p[3] = nib_hi_pair_biased(w >> 8);
  }
}

// FMT: KVQ_FMT_Q4_HAD32, KVQ_FMT_Q4_0 or KVQ_FMT_TQ4; NG groups of 32 in a row; ROT:
// rotate back.  A unit of work is 8 / NG tokens and hpu <= kHeads heads of them: lane
// 4g + t of its warp has the codes 8t .. 8t + 7 of group g of the 8 (group g % NG of
// token g / NG's row), in K and in V.  Every warp walks the units with the grid's
// stride, in three steps that overlap: where a unit's rows lie (a search and a
// block-table entry, two dependent loads) two units ahead, its codes and scales one
// ahead, the transform and the stores.  (One unit to a warp, each paying the chain
// of loads by itself: 262 us for 262144 tokens; with the outputs' types known to the
// compiler and three CTAs of an SM 220 us; the warps on equal ranges of units next to
// one another, far apart in memory, 245 us.)
// nb divides by a token's units; a launch has fewer than 2^31.  OUT: what is written,
// kBf16 or kF32 (K and V both, whole vectors), or kAny (as the views say).
// FEW: one or two heads, and a unit is all heads of kHeads / Hk token blocks; lane l
// finds the row of the unit's token l, and the tiles take them from there.
constexpr int kHeads = 4;
// CTAs of an SM: three (80 registers), two for the TQ4 rows, whose sums spill at 80
// (20011 tokens in fp32 61 us, against 34 us), and for FEW with its row addresses (two
// heads of 200011 tokens 111 us, against 95 us).
__host__ __device__ constexpr int load_ctas(int fmt, bool few) { return few || fmt == KVQ_FMT_TQ4 ? 2 : 3; }
enum Out { kAny, kBf16, kF32 };

template <int FMT, int NG, bool ROT, int OUT, bool FEW>
__global__ void __launch_bounds__(kLoadBlock, load_ctas(FMT, FEW)) load_q4_kernel(const __grid_constant__ LoadArgs a,
                                                                             FastDiv nb, int hpu, uint32_t units) {
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * NG;
  const int lane = threadIdx.x & 31, t4 = lane & 3, g = lane >> 2, G = g % NG;
  const int Hk = a.c.num_kv_heads;
  const bool with_k = OUT != kAny || a.k.data != nullptr, with_v = OUT != kAny || a.v.data != nullptr;
  const int k_dtype = OUT == kAny ? a.k.dtype : OUT == kBf16 ? KVQ_DT_BF16 : KVQ_DT_F32;
  const int v_dtype = OUT == kAny ? a.v.dtype : k_dtype;
  const int k_wide = OUT == kAny ? a.k.wide : 1, v_wide = OUT == kAny ? a.v.wide : 1;
  const SignMatrix<FMT> H(lane);
  uint64_t sign2[4];  // TQ4: the row signs of the lane's 8 outputs, +-1
  if constexpr (FMT == KVQ_FMT_TQ4 && ROT) {
    const uint32_t sw = static_cast<const uint32_t*>(a.c.signs)[G] >> (8 * t4);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sign2[j] = pk2((sw >> (2 * j)) & 1u ? -1.f : 1.f, (sw >> (2 * j + 1)) & 1u ? -1.f : 1.f);
  }
  constexpr float kBack = !ROT ? 1.0f : FMT == KVQ_FMT_TQ4 ? tq4_row_scale<NG>() : kHadamardScale;
  const float c0 = FMT != KVQ_FMT_TQ4 && t4 == 0 ? kBias0 : 0.f, c1 = FMT != KVQ_FMT_TQ4 && t4 == 0 ? kBias1 : 0.f;
  uint32_t hg = 0;  // TQ4: row g of the groups' +-1 matrix, terms 2 t4 and 2 t4 + 1, zero between tokens
  if constexpr (FMT == KVQ_FMT_TQ4 && ROT) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = 2 * t4 + e;
      if (g / NG == k / NG) hg |= ((__popc(G & (k % NG)) & 1) ? 0xBC00u : 0x3C00u) << (16 * e);
    }
  }
  // bytes between the heads of a token's rows
  const int64_t code_step = (int64_t)a.c.page_size * (D / 2);
  const int64_t scale_step = (int64_t)a.c.page_size * (FMT == KVQ_FMT_TQ4 ? 2 : 2 * NG);
  const int64_t ok_step = a.k.hs << (k_dtype == KVQ_DT_BF16 ? 1 : 2), ov_step = a.v.hs << (v_dtype == KVQ_DT_BF16 ? 1 : 2);

  struct Unit {
    int64_t t, row;  // the lane's token; its row in the planes at the unit's first head
    int h, why;
    Where at;
  };
  constexpr int TB = 8 / NG;  // tokens of a tile
  const int hs = FEW ? Hk >> 1 : 0;
  auto place = [&](uint32_t u, Unit& x) {
    int32_t page = 0, why = 0;
    uint32_t off = 0;
    if constexpr (FEW) {
      const int n = (kHeads >> hs) * TB;  // the unit's tokens, at most 32
      x.h = 0;
      x.t = a.t0 + (int64_t)u * n;
      x.at = lane < n && x.t + lane < a.n_tok ? locate(a, x.t + lane, page, off, why) : kSkip;
      if (x.at == kBad) set_status(a.status, why);
      x.row = x.at == kRow ? (int64_t)page * Hk * a.c.page_size + off : x.at == kBad ? -2 : -1;
    } else {
      const uint32_t tb = fast_div(u, nb);
      x.h = static_cast<int>(u - tb * nb.d) * hpu;
      x.t = a.t0 + (int64_t)tb * TB + g / NG;
      x.at = x.t < a.n_tok ? locate(a, x.t, page, off, why) : kSkip;
      x.why = why;
      x.row = ((int64_t)page * Hk + x.h) * a.c.page_size + off;
    }
  };
  // FEW: the lane's token of tile i within the unit, and the tile's head
  auto token = [&](int i) { return (i >> hs) * TB + g / NG; };
  auto head = [&](int i) { return i & ((1 << hs) - 1); };
  uint32_t word[kHeads][2];
  uint16_t scale[kHeads][2];
  auto fetch = [&](const Unit& x, uint32_t (&w)[kHeads][2], uint16_t (&sc)[kHeads][2]) {
    auto code_at = [&](int64_t row) { return row * (D / 2) + 16 * G + 4 * t4; };
    auto scale_at = [&](int64_t row) { return FMT == KVQ_FMT_TQ4 ? 2 * row : (row * NG + G) * 2; };
    const int64_t code0 = code_at(x.row), scale0 = scale_at(x.row);
    const uint8_t *ck = static_cast<const uint8_t*>(a.c.k), *cv = static_cast<const uint8_t*>(a.c.v);
    const uint8_t *sk = static_cast<const uint8_t*>(a.c.k_scale), *sv = static_cast<const uint8_t*>(a.c.v_scale);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      w[i][0] = w[i][1] = 0;
      sc[i][0] = sc[i][1] = 0x7E00;  // a position without a row stands for NaN
      bool have = x.at == kRow && i < hpu && x.h + i < Hk;
      int64_t ca = code0 + i * code_step, sa = scale0 + i * scale_step;
      if constexpr (FEW) {
        const int64_t row = __shfl_sync(0xffffffffu, x.row, token(i));
        have = row >= 0;
        ca = code_at(row) + head(i) * code_step;
        sa = scale_at(row) + head(i) * scale_step;
      }
      if (have) {
        if (with_k) {
          w[i][0] = *reinterpret_cast<const uint32_t*>(ck + ca);
          sc[i][0] = *reinterpret_cast<const uint16_t*>(sk + sa);
        }
        if (with_v) {
          w[i][1] = *reinterpret_cast<const uint32_t*>(cv + ca);
          sc[i][1] = *reinterpret_cast<const uint16_t*>(sv + sa);
        }
      }
    }
  };

  const uint32_t stride = gridDim.x * (kLoadBlock / 32);
  // Taken from lane 0 the warp's number makes the units' addresses uniform: rotated rows
  // to fp32 gain (30000 tokens of 4 heads 58.7 -> 51.3 us), rows to bf16 and unrotated
  // ones lose (262144 tokens 219 -> 222 us, 100011 of Q4_0 88 -> 99 us).
  uint32_t u = blockIdx.x * (kLoadBlock / 32) + (ROT && OUT != kBf16 ? warp_index() : threadIdx.x >> 5);
  if (u >= units) return;
  Unit cur, nxt = {};
  place(u, cur);
  fetch(cur, word, scale);
  bool more = units - u > stride;
  if (more) place(u + stride, nxt);
  for (;;) {
    // the next unit's rows, and where the one after it lies
    uint32_t nword[kHeads][2];
    uint16_t nscale[kHeads][2];
    Unit after = nxt;
    bool more2 = false;
    if (more) {
      fetch(nxt, nword, nscale);
      u += stride;
      more2 = units - u > stride;
      if (more2) place(u + stride, after);
    }
    if (!FEW && cur.at == kBad && cur.h == 0 && G == 0 && t4 == 0) set_status(a.status, cur.why);
    bool here = cur.at != kSkip;
    const int k_shift = k_dtype == KVQ_DT_BF16 ? 1 : 2, v_shift = v_dtype == KVQ_DT_BF16 ? 1 : 2;
    uint8_t* ok = static_cast<uint8_t*>(a.k.data) + ((cur.t * a.k.ts + cur.h * a.k.hs + 32 * G + 8 * t4) << k_shift);
    uint8_t* ov = static_cast<uint8_t*>(a.v.data) + ((cur.t * a.v.ts + cur.h * a.v.hs + 32 * G + 8 * t4) << v_shift);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      uint8_t *dk = ok, *dv = ov;
      if constexpr (FEW) {
        here = __shfl_sync(0xffffffffu, cur.row, token(i)) != -1;
        dk += (token(i) * a.k.ts + head(i) * a.k.hs) << k_shift;
        dv += (token(i) * a.v.ts + head(i) * a.v.hs) << v_shift;
      } else if (i >= hpu || cur.h + i >= Hk) {
        break;
      }
      float x[2][8];
      if constexpr (ROT) {
        uint32_t pk[4], pv[4];
        code_operands<FMT>(word[i][0], pk);
        code_operands<FMT>(word[i][1], pv);
        uint32_t lk[4], lv[4];  // TQ4: what the sums over the groups have below fp16
        if constexpr (FMT == KVQ_FMT_TQ4) {
          // the transform over the row's groups first: H of the groups times the pairs,
          // turned so that the groups are the terms; K and V are two blocks of one product
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float d[4];
            mma_f16_c(d, hg, 0u, 0u, hg, movmatrix_trans(pk[q]), movmatrix_trans(pv[q]), 0.f, 0.f, 0.f, 0.f);
            split_sums(d[0], d[1], pk[q], lk[q]);
            split_sums(d[2], d[3], pv[q], lv[q]);
          }
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
          float c[4];
          mma_f16_c(c, pk[0], pv[0], pk[1], pv[1], H.at(0, 0, nt), H.at(0, 1, nt), nt ? 0.f : c0, nt ? 0.f : c1,
                    nt ? 0.f : c0, nt ? 0.f : c1);
          mma_f16(c, pk[2], pv[2], pk[3], pv[3], H.at(1, 0, nt), H.at(1, 1, nt));
          if constexpr (FMT == KVQ_FMT_TQ4) {
            mma_f16(c, lk[0], lv[0], lk[1], lv[1], H.at(0, 0, nt), H.at(0, 1, nt));
            mma_f16(c, lk[2], lv[2], lk[3], lv[3], H.at(1, 0, nt), H.at(1, 1, nt));
          }
          x[0][2 * nt] = c[0];
          x[0][2 * nt + 1] = c[1];
          x[1][2 * nt] = c[2];
          x[1][2 * nt + 1] = c[3];
        }
      } else {
        code_values<FMT>(word[i][0], x[0]);
        code_values<FMT>(word[i][1], x[1]);
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const float f = __half2float(__ushort_as_half(scale[i][kv])) * kBack;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          uint64_t f2 = pk2(f, f);
          if constexpr (FMT == KVQ_FMT_TQ4 && ROT) f2 = mul2(f2, sign2[j / 2]);
          upk2(mul2(pk2(x[kv][j], x[kv][j + 1]), f2), x[kv][j], x[kv][j + 1]);
        }
      }
      if (here && with_k) put_values<8>(dk, k_dtype, k_wide, x[0]);
      if (here && with_v) put_values<8>(dv, v_dtype, v_wide, x[1]);
      if constexpr (!FEW) {
        ok += ok_step;
        ov += ov_step;
      }
    }
    if (!more) break;
    cur = nxt;
    nxt = after;
    more = more2;
#pragma unroll
    for (int i = 0; i < kHeads; ++i)
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        word[i][kv] = nword[i][kv];
        scale[i][kv] = nscale[i][kv];
      }
  }
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
    put_values<16>(element_at(a.k, t * a.k.ts + c), a.k.dtype, a.k.wide, x);
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
    put_values<16>(element_at(out, t * out.ts + head * out.hs + c), out.dtype, out.wide, x);
  }
}

}  // namespace

cudaError_t launch_load(const LoadArgs& args, cudaStream_t s) {
  LoadArgs a = args;
  const int kv0 = a.k.data ? 0 : 1, kvs = (a.k.data ? 1 : 0) + (a.v.data ? 1 : 0);
  const int Hk = a.c.num_kv_heads, D = a.c.head_dim;
  const bool fp8 = a.c.format == KVQ_FMT_FP8_ROW, wide = fp8 || a.c.format == KVQ_FMT_BF16;
  const int NG = D / 32, cpr = (fp8 ? D + a.c.rope_dim : D) / 16;
  const int64_t n_tok = a.n_tok;
  if (!wide) {
    // Units of 8 / NG tokens and hpu heads, walked by as many warps as are resident at
    // once.  hpu: the one whose rounds cost least, a round its heads' work and about
    // one head's for the unit itself, times the CTAs that share an SM (4096 tokens of 4
    // heads: one round and a bit of 4 heads would be two).
    const int64_t n_sm = device_sm_count() > 0 ? device_sm_count() : 1;
    const int64_t blocks8 = (n_tok * NG + 7) / 8;
    auto cost = [&](int64_t units, int tiles, int ctas) {
      const int64_t warps = n_sm * ctas * (kLoadBlock / 32);
      return (units + warps - 1) / warps * ctas * (tiles + 1);
    };
    int ctas_sm = load_ctas(a.c.format, false), hpu = 1;
    int64_t best = 0;
    for (int h = 1; h <= kHeads; h *= 2) {
      const int64_t c = cost(blocks8 * ((Hk + h - 1) / h), h, ctas_sm);
      if (h == 1 || c < best) best = c, hpu = h;
    }
    // One or two heads: a unit of several token blocks instead, by the same costs (one
    // head of 200011 tokens 50 us so, 96 us by single blocks; of 4001 tokens 3.5 and 4.4
    // us; 2048 tokens are one round of single blocks).
    const bool plain = kvs == 2 && a.k.wide && a.v.wide && a.k.dtype == a.v.dtype;
    const int64_t tpu = Hk <= 2 ? kHeads / Hk : 1;
    const bool few = plain && tpu > 1 && cost((blocks8 + tpu - 1) / tpu, kHeads, load_ctas(a.c.format, true)) < best;
    if (few) ctas_sm = load_ctas(a.c.format, true);
    const int64_t resident = n_sm * ctas_sm;
    // at most 2^30 units in a launch
    const int64_t per_tok = few ? 1 : (Hk + hpu - 1) / hpu, max_tok = (int64_t(1) << 30) / per_tok / 8 * 8;
    if (max_tok < 8) return cudaErrorInvalidValue;
    const FastDiv nb = make_fastdiv(static_cast<uint32_t>(per_tok));
    const int out = !plain ? kAny : a.k.dtype == KVQ_DT_BF16 ? kBf16 : kF32;
    const dim3 block(kLoadBlock);
    for (a.t0 = 0; a.t0 < n_tok; a.t0 += max_tok) {
      a.n_tok = n_tok - a.t0 < max_tok ? n_tok : a.t0 + max_tok;  // tokens [t0, n_tok) in this launch
      const int64_t blocks = ((a.n_tok - a.t0) * NG + 7) / 8;
      const int64_t units = few ? (blocks + tpu - 1) / tpu : blocks * per_tok;
      int64_t ctas = (units + kLoadBlock / 32 - 1) / (kLoadBlock / 32);
      if (ctas > resident) ctas = resident;
      const dim3 grid(static_cast<unsigned>(ctas));
      cudaError_t e = cudaErrorInvalidValue;
#define KVQ_LOAD_OUT(F, N, R, O, W) \
  launch_pdl(load_q4_kernel<F, N, R, O, W>, grid, block, 0, s, a, nb, hpu, static_cast<uint32_t>(units))
#define KVQ_LOAD(F, N, R)                                                                         \
  e = out == kBf16  ? few ? KVQ_LOAD_OUT(F, N, R, kBf16, true) : KVQ_LOAD_OUT(F, N, R, kBf16, false) \
      : out == kF32 ? few ? KVQ_LOAD_OUT(F, N, R, kF32, true) : KVQ_LOAD_OUT(F, N, R, kF32, false)   \
                    : KVQ_LOAD_OUT(F, N, R, kAny, false);                                         \
  break
#define KVQ_LOAD_NG(F, R)       \
  switch (NG) {                 \
    case 1: KVQ_LOAD(F, 1, R);  \
    case 2: KVQ_LOAD(F, 2, R);  \
    case 4: KVQ_LOAD(F, 4, R);  \
    case 8: KVQ_LOAD(F, 8, R);  \
    default: break;             \
  }
#define KVQ_LOAD_TQ(R)                      \
  switch (NG) {                             \
    case 2: KVQ_LOAD(KVQ_FMT_TQ4, 2, R);    \
    case 4: KVQ_LOAD(KVQ_FMT_TQ4, 4, R);    \
    case 8: KVQ_LOAD(KVQ_FMT_TQ4, 8, R);    \
    default: break;                         \
  }
    if (a.c.format == KVQ_FMT_TQ4) {
      if (a.rotate_back) {
        KVQ_LOAD_TQ(true)
      } else {
        KVQ_LOAD_TQ(false)
      }
    } else if (a.rotate_back) {  // Q4_HAD32
      KVQ_LOAD_NG(KVQ_FMT_Q4_HAD32, true)
    } else {  // the two 4-bit formats' codes have the same values
      KVQ_LOAD_NG(KVQ_FMT_Q4_0, false)
    }
#undef KVQ_LOAD_TQ
#undef KVQ_LOAD_NG
#undef KVQ_LOAD
#undef KVQ_LOAD_OUT
      if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
  }
  const int64_t per_tok = fp8 ? cpr : (int64_t)cpr * Hk * kvs;  // threads of a token
  if (per_tok >= (int64_t(1) << 30)) return cudaErrorInvalidValue;
  const FastDiv ft = make_fastdiv(static_cast<uint32_t>(per_tok)), fc = make_fastdiv(static_cast<uint32_t>(cpr));
  // launches of at most 2^30 threads, so that the kernel's indices stay 32-bit
  const int64_t max_tok = (int64_t(1) << 30) / per_tok;
  for (a.t0 = 0; a.t0 < n_tok; a.t0 += max_tok) {
    a.n_tok = n_tok - a.t0 < max_tok ? n_tok : a.t0 + max_tok;  // tokens [t0, n_tok) in this launch
    const dim3 grid(static_cast<unsigned>(((a.n_tok - a.t0) * per_tok + kLoadBlock - 1) / kLoadBlock)), block(kLoadBlock);
    cudaError_t e = fp8 ? launch_pdl(load_wide_kernel<true>, grid, block, 0, s, a, kv0, ft, fc)
                        : launch_pdl(load_wide_kernel<false>, grid, block, 0, s, a, kv0, ft, fc);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace kvq
