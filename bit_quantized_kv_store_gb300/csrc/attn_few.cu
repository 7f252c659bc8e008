// attn_few.cu -- attention of few rows a sequence (single new tokens, draft rows, short
// chunks) over the paged cache, with a sliding window and sinks, every row format.
//
// For a row at position p:  o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m) over the keys j
// that it sees (seqs.cuh), s_j = sm_scale log2(e) q . k_j, m a running reference.
//
// Bound by memory where a batch is large (each row of the cache is read once, 288 bytes
// a key and KV head of the 4-bit rows at 256 wide), by latency where it is not: a window
// of 4096 keys of one sequence is 4.7 MB, 0.7 us of the memory's time.  So the keys of a
// block of 8 columns (row x query head of one KV head) are dealt out to the warps of a
// cluster of CTAs, tile by tile, each warp with a ring of its own that cp.async fills;
// nothing synchronises between the first load and the last product.  The warps' partials
// are folded in shared memory, the CTAs' through distributed shared memory, in a fixed
// order, and the output is rotated back and rounded by the same launch.  Where one
// cluster would leave most of the GPU idle, several write partials and a second kernel
// folds them.
//
// 4-bit groups: a key's codes enter the tensor cores unsigned, without a conversion: c in
// bits 2 to 5 of a half is the subnormal c 2^-22, in bits 6 to 9 16 c 2^-22, and the query
// of such a dim carries the 1/16; the 8 that codes are biased by is in the accumulator's
// start (-8 sum q over the group).  So a group of scores is exact up to the query (fp16,
// 2^-11), and its scale multiplies the fp32 sum.  (The tensor cores
// line products of subnormals up as if their exponent were 2^-14 and cut a sum 23 bits
// below: 2^-15 of a code times the largest query element, a 2^-15 part of a score.  For
// values, whose small sums count, that is too much: they are converted, exactly, to c - 8.)
// On the way out the scale multiplies p instead of 32 values: p' = fp16(fp16(p) s), two
// roundings of 2^-11 at most.  p = 2^(11 + s_j - m), where m follows when s_j + log2 of the key's
// largest scale (if that is above 1) passes it by more than 4: p and p' use fp16 up to 2^15, and
// keep their bits down to 2^-25 of the largest p.  (TQ4 rows: p' = fp16(p s), and m counts small scales, too.)
// TQ4 rows: levels by byte lookups (tq4_levels.cuh), the row's scale on scores and p.
// bf16 rows: as they are; q and p in two bf16 halves (16 bits).
//
// Measured (one GB300, a graph of calls over inputs larger than L2): one token, window 1024 8.9
// us; 32 sequences, windows of 4096 keys 48.6 us (149 MB, 3.06 TB/s: about 560 instructions a
// block of 16 keys, 72 % of the issue slots while the keys last, and 15 us of start and fold); 16
// bf16 sequences, windows of 1024 19.7 us (67 MB, 3.4 TB/s).  About 1.3 us of each is metadata
// that is read behind the kernel in front, not beside it.  Loops are rolled because a call is
// short: unrolled, fetching the code took most of it (the first 11.7 us, so 7.6 then).
#include <algorithm>
#include <climits>

#include "f32x2.cuh"
#include "rows.cuh"
#include "seqs.cuh"
#include "tq4_levels.cuh"

namespace kvq {

constexpr uint32_t kCodeLo = 0x003C003Cu, kCodeHi = 0x03C003C0u;  // c 2^-22, 16 c 2^-22
enum { kFewQ4 = 0, kFewTq4 = 1, kFewBf16 = 2 };

template <int FMT, int D>
struct FewShape {
  static constexpr bool kBf = FMT == kFewBf16;
  static constexpr int kRow = kBf ? 2 * D : D / 2;           // bytes of a row of the k or v plane
  static constexpr int kChunks = kRow / 16;                  // 16-byte chunks of it
  static constexpr int kScaleRow = FMT == kFewQ4 ? D / 16 : FMT == kFewTq4 ? 2 : 0;  // bytes of its scales
  static constexpr int kBlocks = kBf || D == 256 ? 1 : 2;    // 16-key blocks of a tile
  static constexpr int kKeys = 16 * kBlocks;
  static constexpr int kPlane = kKeys * kRow;
  static constexpr int kScales = kKeys * kScaleRow;
  static constexpr int kStage = (2 * kPlane + 2 * kScales + 127) / 128 * 128;
  static constexpr int kStages = 2;
  static constexpr int kSteps = D / 16;                      // k-steps of the score product
};

template <int FMT, int D, int WARPS>
struct FewSmem {
  using S = FewShape<FMT, D>;
  static constexpr int kRing = S::kStage * S::kStages * WARPS;
  static constexpr int kFold = WARPS * 8 * D * 4;
  union {
    __align__(128) uint8_t ring[kRing > kFold ? kRing : kFold];
    float fold[WARPS][8][D];
  };
  // per lane, the score product's B operand: of a group's two steps; bf16 rows: of a step, (high b0, b1, low b0, b1)
  uint4 qf[S::kBf ? S::kSteps : S::kSteps / 2][32];
  float2 bias[D / 32][4];   // 4-bit groups: -8 sum of the group's queries (heads 2t, 2t + 1), as the codes' units
  float factor[8];          // per column: what its scores' units are worth
  float fm[WARPS][8], fz[WARPS][8], fw[WARPS][8];  // per warp and column: reference, sum, weight
  float m_own[8], z_own[8];
  float m[16][8], z[16][8];  // per CTA of the cluster and column
  __align__(16) float acc[8 * D];  // this CTA's pieces of the cluster's partials: [CTA][piece][values]
};

__device__ __forceinline__ void few_ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void few_ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 few_lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
// W words (1, 2 or 4) of shared memory.
template <int W>
__device__ __forceinline__ void few_lds(uint32_t a, uint32_t (&r)[W]) {
  if constexpr (W == 4) {
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
  } else if constexpr (W == 2) {
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a));
  } else {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(a));
  }
}
__device__ __forceinline__ uint32_t few_lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t few_lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
// The power of two that a key's p takes over from its scales, by the largest one's logarithm: 16
// where that is above 16, so that p, below 2^(15 - lsv), keeps four bits more and scales of 2^-10
// and up beside the large one lose none; 1 elsewhere, so that such a key beside it, or behind a
// sequence's end, or what is left of another in shared memory, does not change how others are
// rounded.
__device__ __forceinline__ float wide_unit(float lsv) { return lsv > 4.f ? 16.f : 1.f; }
__device__ __forceinline__ bool not_finite(uint32_t bf16) { return (bf16 & 0x7F80u) == 0x7F80u; }
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ float half_lo(uint32_t w) { return __low2float(u32_as_h2(w)); }
__device__ __forceinline__ float half_hi(uint32_t w) { return __high2float(u32_as_h2(w)); }
__device__ __forceinline__ float half_of(uint32_t h) { return __half2float(__ushort_as_half(static_cast<unsigned short>(h))); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Store to this CTA's shared address in CTA `rank` of the cluster.
__device__ __forceinline__ void cluster_st(float* p, uint32_t rank, float v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v) : "memory");
}

__device__ __forceinline__ void cluster_st4(float* p, uint32_t rank, const float4& v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}

// Byte offset of chunk c of row r in a plane's tile: rows of 16 kChunks bytes, the chunks
// turned so that eight rows' chunks of one number lie in eight different sixteenths of
// 128 bytes (what ldmatrix reads at once).
template <int CHUNKS>
__device__ __forceinline__ uint32_t few_off(int r, int c) {
  if constexpr (CHUNKS >= 8) return r * CHUNKS * 16 + ((c ^ (r & 7)) << 4);
  else return r * CHUNKS * 16 + ((c ^ ((r / (8 / CHUNKS)) & (CHUNKS - 1))) << 4);
}

__device__ __forceinline__ void split_bf16x2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x0, x1);
  const float2 f = __bfloat1622float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = pack_bf16(x0 - f.x, x1 - f.y);
}

template <int FMT, int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, FMT == kFewBf16 && D == 256 ? 1 : 4) attn_few_kernel(const __grid_constant__ SeqAttnArgs a) {
  using S = FewShape<FMT, D>;
  constexpr int NG = D / 32;
  extern __shared__ uint8_t smem_raw[];
  FewSmem<FMT, D, WARPS>& sm =
      *reinterpret_cast<FewSmem<FMT, D, WARPS>*>(smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const kvq_cache& c = a.c;
  const int b = blockIdx.z, kvh = blockIdx.y % c.num_kv_heads, cb = blockIdx.y / c.num_kv_heads;

  // what the sequence's rows see (lengths, rows and tables are often made by the kernel in front)
  pdl_wait();
  const SeqRows sr = seq_rows(a, b);
  const int cols = min(8, sr.n * a.group - 8 * cb);
  if (cols <= 0 || sr.state == kRowsSkip) {
    pdl_trigger();
    if (sr.state != kRowsOk && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
      set_status(a.status, KVQ_DEV_BAD_LENGTH);
    return;
  }
  const int base = sr.T - sr.n;  // position of the sequence's row 0
  const int i0 = 8 * cb / a.group, i1 = (8 * cb + cols - 1) / a.group;
  if (sr.state == kRowsNan) {
    pdl_trigger();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, KVQ_DEV_BAD_LENGTH);
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i < cols * D; i += WARPS * 32) {
        const int col = 8 * cb + i / D;
        seq_store(a, sr.first + col / a.group, kvh * a.group + col % a.group, i % D, NAN);
      }
    return;
  }
  const int p0 = base + i0, p1 = base + i1;
  KeyBlocks kb{0, 0, 0};
  if (p1 >= 0) kb = key_blocks(p0, p1, a.window, a.sinks);
  // its part of the blocks: a share, or (ragged sequences) so many of them
  const int all_tiles = (kb.count + S::kBlocks - 1) / S::kBlocks;
  int tile0, tile1, ranges;
  if (a.per > 0) {
    const int per = a.per / S::kBlocks;
    tile0 = min(all_tiles, per * static_cast<int>(blockIdx.x));
    tile1 = min(all_tiles, tile0 + per);
    ranges = max(1, (all_tiles + per - 1) / per);
    if (static_cast<int>(blockIdx.x) >= ranges) {
      pdl_trigger();
      return;
    }
  } else {
    tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * blockIdx.x / gridDim.x);
    tile1 = static_cast<int>(static_cast<int64_t>(all_tiles) * (blockIdx.x + 1) / gridDim.x);
    ranges = gridDim.x / cluster_size();
  }
  if (cluster_size() > 1) cluster_arrive();  // waited for before the first store to another CTA
  const int my_tiles = tile1 - tile0 > warp ? (tile1 - tile0 - warp + WARPS - 1) / WARPS : 0;

  // This warp's tiles are tile0 + warp + WARPS i.  Lane l holds the cache row of block l of
  // 32 at a time (32 / kBlocks tiles): -1 a page outside the pool, -2 behind the last block.
  constexpr int kBatch = 32 / S::kBlocks;
  const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_pages;
  auto find_rows = [&](int i) {
    const int tile = i + lane / S::kBlocks;
    const int blk = (tile0 + warp + WARPS * tile) * S::kBlocks + lane % S::kBlocks;
    if (tile >= my_tiles || blk >= kb.count) return -2;
    const int at = kb.block_of(blk), pg = static_cast<int>(fast_div(static_cast<uint32_t>(at), a.page_blocks));
    const int page = table[pg];
    if (page < 0 || page >= c.num_pages) return -1;
    return (page * c.num_kv_heads + kvh) * c.page_size + (at - pg * static_cast<int>(a.page_blocks.d)) * 16;
  };
  int rows_now = find_rows(0), rows_next = find_rows(kBatch);
  bool bad_page = rows_now == -1;

  uint8_t* const ring = sm.ring + warp * (S::kStage * S::kStages);
  auto issue = [&](int i) {  // the loads of tile i, into its stage of the ring
    uint8_t* st = ring + (i % S::kStages) * S::kStage;
#pragma unroll
    for (int sub = 0; sub < S::kBlocks; ++sub) {
      const int row0 = __shfl_sync(0xffffffffu, rows_now, (i % kBatch) * S::kBlocks + sub);
      if (row0 < 0) continue;
      const uint8_t* ks = static_cast<const uint8_t*>(c.k) + static_cast<int64_t>(row0) * S::kRow;
      const uint8_t* vs = static_cast<const uint8_t*>(c.v) + static_cast<int64_t>(row0) * S::kRow;
      uint8_t* dk = st + sub * 16 * S::kRow;
#pragma unroll
      for (int jj = 0; jj < (16 * S::kChunks + 31) / 32; ++jj) {
        const int j = lane + 32 * jj;
        const uint32_t off = few_off<S::kChunks>(j / S::kChunks, j % S::kChunks);
        cp_async_16(dk + off, ks + 16 * j);
        cp_async_16(dk + S::kPlane + off, vs + 16 * j);
      }
      if constexpr (S::kScaleRow > 0) {
        uint8_t* ds = st + 2 * S::kPlane + sub * 16 * S::kScaleRow;
        constexpr int kN = S::kScaleRow;  // 16-byte chunks of 16 rows' scales
        const int j = lane & 15;
        const void* plane = lane < 16 ? c.k_scale : c.v_scale;
        if (j < kN)
          cp_async_16(ds + (lane < 16 ? 0 : S::kScales) + 16 * j,
                      static_cast<const uint8_t*>(plane) + static_cast<int64_t>(row0) * S::kScaleRow + 16 * j);
      }
    }
  };
  auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
#pragma unroll 1
  for (int i = 0; i < S::kStages - 1; ++i) {
    if (i < my_tiles) issue(i);
    commit();
  }

  // ---------------- queries: into the cache's space, scaled to 2^10 .. 2^11, fp16 (bf16
  // rows: two bf16 halves).  Lane
  // (column l & 7, eighth l >> 3) holds 8 values of a group of 32; a warp has the groups
  // warp, warp + 4, ... (TQ4, whose rotation spans the row: it works out all and writes these).
  {
    const int n = lane & 7, eighth = lane >> 3, col = 8 * cb + n;
    constexpr bool kAll = FMT == kFewTq4;
    constexpr int kMine = kAll ? NG : (NG + WARPS - 1) / WARPS;
    const int64_t q_at = static_cast<int64_t>(sr.first + col / a.group) * a.q.ts +
                         static_cast<int64_t>(kvh * a.group + col % a.group) * a.q.hs + 8 * eighth;
    float x[kMine][8];
    if constexpr (kAll) {
      seq_load_row<NG>(a.q, n < cols ? q_at : -1, x);
      seq_turn<NG, true>(x, static_cast<const uint32_t*>(c.signs), lane, false);
    } else {
#pragma unroll
      for (int k = 0; k < kMine; ++k)
        seq_load_row<1>(a.q, n < cols && warp + WARPS * k < NG ? q_at + 32 * (warp + WARPS * k) : -1,
                        reinterpret_cast<float(&)[1][8]>(x[k]));
      if (c.format == KVQ_FMT_Q4_HAD32) seq_turn<kMine, false>(x, nullptr, lane, false);
    }
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < kMine; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[k][e] *= a.qscale;
        top = fmaxf(top, fabsf(x[k][e]));
      }
    if constexpr (FMT != kFewBf16) {
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      if constexpr (!kAll) {
        if (eighth == 0) sm.fm[warp][n] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, sm.fm[w][n]);
      }
    }
    float up = 1.f, unit = 1.f;
    if constexpr (FMT != kFewBf16) {
      // a power of two takes the largest element to [2^10, 2^11); NaN and infinities stay
      int ex = 0;
      if (top > 0.f && top < INFINITY) ex = 10 - (static_cast<int>(__float_as_uint(fmaxf(top, 1e-30f)) >> 23) - 127);
      up = __uint_as_float(static_cast<uint32_t>(min(ex, 110) + 127) << 23);
      unit = (FMT == kFewQ4 ? 4194304.f : 1.f) / up;
    }
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int G = kAll ? k : warp + WARPS * k;
      if (G % WARPS != warp || G >= NG) continue;
      uint32_t hi[4];
      if constexpr (FMT == kFewBf16) {
        // elements 8 eighth .. + 7 of the group: pairs t of the step 2G + eighth / 2, its B register eighth % 2
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) {
          uint32_t lo;
          split_bf16x2(x[k][2 * t4], x[k][2 * t4 + 1], hi[t4], lo);
          uint32_t* f = reinterpret_cast<uint32_t*>(&sm.qf[2 * G + (eighth >> 1)][n * 4 + t4]);
          f[eighth & 1] = hi[t4];
          f[2 + (eighth & 1)] = lo;
        }
      } else {
        // the order in which the codes come out of their words: 4-bit groups (0, 4) (1, 5) / 16
        // (2, 6) (3, 7) / 16, TQ4 in turn
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y0 = x[k][FMT == kFewQ4 ? i : 2 * i] * up, y1 = x[k][FMT == kFewQ4 ? i + 4 : 2 * i + 1] * up;
          const float part = FMT == kFewQ4 && (i & 1) ? 0.0625f : 1.f;
          hi[i] = pack_half2(y0 * part, y1 * part);
          if constexpr (FMT == kFewQ4) sum += (half_lo(hi[i]) + half_hi(hi[i])) * (i & 1 ? 16.f : 1.f);
        }
        sm.qf[G][n * 4 + eighth] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (FMT == kFewQ4) {
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          if (eighth == 0) reinterpret_cast<float*>(&sm.bias[G][n >> 1])[n & 1] = sum * -1.9073486328125e-06f;  // -8 2^-22
        }
      }
    }
    if (warp == 0 && lane < 8) sm.factor[n] = unit;
  }
  __syncthreads();

  // ---------------- the keys
  const uint32_t qf = smem_u32(&sm.qf[0][lane]);
  float f0 = sm.factor[2 * t], f1 = sm.factor[2 * t + 1];
  // positions of columns 2t, 2t + 1 and g (before any key where there is no such column)
  auto pos_of = [&](int n) { return n < cols ? base + (8 * cb + n) / a.group : -kNoKey; };
  const int pc0 = pos_of(2 * t), pc1 = pos_of(2 * t + 1), pcg = pos_of(g);

  float acc[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, z0 = 0.f, z1 = 0.f;

#pragma unroll 1
  for (int i = 0; i < my_tiles; ++i) {
    // ---- the loads of a tile ahead, then wait for this one's
    const int ahead = i + S::kStages - 1;
    if (ahead < my_tiles) {
      if (ahead % kBatch == 0) {
        rows_now = rows_next;
        rows_next = find_rows(ahead + kBatch);
        bad_page |= rows_now == -1;
      }
      issue(ahead);
    }
    commit();
    asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
    __syncwarp();

    const uint8_t* st = ring + (i % S::kStages) * S::kStage;
    const uint32_t kbase = smem_u32(st), vbase = kbase + S::kPlane, ksc = kbase + 2 * S::kPlane, vsc = ksc + S::kScales;
    const int blk0 = (tile0 + warp + WARPS * i) * S::kBlocks;
    int key0[S::kBlocks];
    bool edge = false;  // some key that some column does not see
#pragma unroll
    for (int sub = 0; sub < S::kBlocks; ++sub) {
      key0[sub] = blk0 + sub < kb.count ? kb.block_of(blk0 + sub) * 16 : kNoKey;
      edge |= !all_visible(key0[sub], 16, p0, p1, a.window, a.sinks);
    }

    // ---------------- scores of keys g, g + 8 of each block, columns 2t, 2t + 1
    float s[S::kBlocks][4];
#pragma unroll
    for (int sub = 0; sub < S::kBlocks; ++sub)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[sub][j] = 0.f;
    if constexpr (FMT == kFewBf16) {
      float sl[S::kBlocks][4] = {};
      const int kr = (lane & 7) + 8 * ((lane >> 3) & 1), kc = lane >> 4;
#pragma unroll 4
      for (int ks = 0; ks < S::kSteps; ++ks) {
        const uint4 q = few_lds128(qf + ks * 512);
#pragma unroll
        for (int sub = 0; sub < S::kBlocks; ++sub) {
          uint32_t ak[4];
          few_ldsm(kbase + sub * 16 * S::kRow + few_off<S::kChunks>(kr, 2 * ks + kc), ak);
          mma_bf16(s[sub], ak[0], ak[1], ak[2], ak[3], q.x, q.y);
          mma_bf16(sl[sub], ak[0], ak[1], ak[2], ak[3], q.z, q.w);
        }
      }
#pragma unroll
      for (int sub = 0; sub < S::kBlocks; ++sub)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[sub][j] += sl[sub][j];
    } else {
      // ldmatrix: matrices (keys 0-7, chunk 2u), (keys 8-15, 2u), (keys 0-7, 2u + 1), (keys 8-15, 2u + 1)
      const int lr = lane & 15, lc = lane >> 4;
      float sl[S::kBlocks][4] = {};
#pragma unroll 1
      for (int u = 0; u < D / 64; ++u) {
        uint32_t r[S::kBlocks][4];
        uint32_t sk[S::kBlocks][2];  // two groups' scales of keys g, g + 8
#pragma unroll
        for (int sub = 0; sub < S::kBlocks; ++sub) {
          if constexpr (FMT == kFewQ4) {
            sk[sub][0] = few_lds32(ksc + (sub * 16 + g) * S::kScaleRow + 4 * u);
            sk[sub][1] = few_lds32(ksc + (sub * 16 + g + 8) * S::kScaleRow + 4 * u);
          }
        }
#pragma unroll
        for (int sub = 0; sub < S::kBlocks; ++sub)
          few_ldsm(kbase + sub * 16 * S::kRow + few_off<S::kChunks>(lr, 2 * u + lc), r[sub]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int G = 2 * u + e;
          const uint4 qa = few_lds128(qf + G * 512);  // B of the group's two steps
          if constexpr (FMT == kFewQ4) {
            const float2 bi = sm.bias[G][t];
#pragma unroll
            for (int sub = 0; sub < S::kBlocks; ++sub) {
              const uint32_t ra = r[sub][2 * e], rb = r[sub][2 * e + 1];
              const uint32_t al = ra << 2, bl = rb << 2, ah = ra >> 6, bh = rb >> 6;
              const uint32_t a0 = al & kCodeLo, a1 = bl & kCodeLo, a2 = al & kCodeHi, a3 = bl & kCodeHi;
              const uint32_t c0 = ah & kCodeLo, c1 = bh & kCodeLo, c2 = ah & kCodeHi, c3 = bh & kCodeHi;
              float d[4];
              mma_f16_c(d, a0, a1, a2, a3, qa.x, qa.y, bi.x, bi.y, bi.x, bi.y);
              mma_f16(d, c0, c1, c2, c3, qa.z, qa.w);
              const float sg = e ? half_hi(sk[sub][0]) : half_lo(sk[sub][0]);
              const float sh = e ? half_hi(sk[sub][1]) : half_lo(sk[sub][1]);
              s[sub][0] = fmaf(sg, d[0], s[sub][0]);
              s[sub][1] = fmaf(sg, d[1], s[sub][1]);
              s[sub][2] = fmaf(sh, d[2], s[sub][2]);
              s[sub][3] = fmaf(sh, d[3], s[sub][3]);
            }
          } else {
#pragma unroll
            for (int sub = 0; sub < S::kBlocks; ++sub) {
              const uint4 A = tq4_levels8(r[sub][2 * e]), B = tq4_levels8(r[sub][2 * e + 1]);
              mma_f16(s[sub], A.x, B.x, A.y, B.y, qa.x, qa.y);
              mma_f16(sl[sub], A.z, B.z, A.w, B.w, qa.z, qa.w);
            }
          }
        }
      }
      if constexpr (FMT == kFewTq4) {
#pragma unroll
        for (int sub = 0; sub < S::kBlocks; ++sub) {
          const float sg = half_of(few_lds16(ksc + 2 * (sub * 16 + g))), sh = half_of(few_lds16(ksc + 2 * (sub * 16 + g + 8)));
          s[sub][0] = (s[sub][0] + sl[sub][0]) * sg;
          s[sub][1] = (s[sub][1] + sl[sub][1]) * sg;
          s[sub][2] = (s[sub][2] + sl[sub][2]) * sh;
          s[sub][3] = (s[sub][3] + sl[sub][3]) * sh;
        }
      }
#pragma unroll
      for (int sub = 0; sub < S::kBlocks; ++sub) {
        s[sub][0] *= f0;
        s[sub][1] *= f1;
        s[sub][2] *= f0;
        s[sub][3] *= f1;
      }
    }

    // ---------------- what is not seen; pages outside the pool
    const bool any_bad = __any_sync(0xffffffffu, bad_page);
    uint32_t strange[S::kBlocks] = {};  // bf16: rows of V that some column does not see and that hold infinities or NaN
    uint32_t keep[S::kBlocks][2];  // of column g: masks of the pairs of keys 2t, 2t + 1 and 2t + 8, 2t + 9
    if (edge || any_bad) {
#pragma unroll
      for (int sub = 0; sub < S::kBlocks; ++sub) {
        bool gone = false;
        if (any_bad) {
          const int blk = blk0 + sub;
          if (blk < kb.count) {
            const int page = table[kb.block_of(blk) * 16 / c.page_size];
            gone = page < 0 || page >= c.num_pages;
          }
          if (gone && lane == 0) set_status(a.status, KVQ_DEV_BAD_PAGE);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0[sub] + g + 8 * (j >> 1);
          if (!key_visible(key, j & 1 ? pc1 : pc0, a.window, a.sinks)) s[sub][j] = -INFINITY;
          else if (gone) s[sub][j] = NAN;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = key0[sub] + 2 * t + 8 * h;
          keep[sub][h] = (key_visible(key, pcg, a.window, a.sinks) ? 0x0000FFFFu : 0u) |
                         (key_visible(key + 1, pcg, a.window, a.sinks) ? 0xFFFF0000u : 0u);
        }
        if constexpr (FMT == kFewBf16) {
          // values that no column sees, and those of a bad page, become zeros: 0 x NaN is NaN
#pragma unroll 1
          for (int r = 0; r < 16; ++r) {
            uint4* at = reinterpret_cast<uint4*>(ring + (i % S::kStages) * S::kStage + S::kPlane + (sub * 16 + r) * S::kRow) + lane;
            if (gone || !any_visible(key0[sub] + r, p0, p1, a.window, a.sinks)) {
              if (lane < S::kChunks) *at = make_uint4(0, 0, 0, 0);
            } else if (p0 < p1) {
              bool odd = false;
              if (lane < S::kChunks) {
                const uint4 v = *at;
#pragma unroll
                for (int w = 0; w < 4; ++w) odd |= not_finite(word_of(v, w) & 0xFFFFu) || not_finite(word_of(v, w) >> 16);
              }
              if (__any_sync(0xffffffffu, odd)) strange[sub] |= 1u << r;
            }
          }
        }
      }
      __syncwarp();
    }

    // ---------------- the key's largest value scale, as the reference counts it
    float lsv = 0.f;  // of key `lane` of the tile
    bool wide = false;
    if constexpr (FMT == kFewQ4) {
      constexpr int kSW = D / 64;
      uint32_t w[kSW];
      few_lds<kSW>(vsc + (lane & (S::kKeys - 1)) * S::kScaleRow, w);
      __half2 h = u32_as_h2(w[0]);
#pragma unroll
      for (int k = 1; k < kSW; ++k) h = __hmax2(h, u32_as_h2(w[k]));
      const float top = fmaxf(__low2float(h), __high2float(h));
      lsv = fminf(fmaxf(__log2f(top), 0.f), 16.f);
      wide = lsv > 4.f;
    } else if constexpr (FMT == kFewTq4) {
      lsv = fminf(fmaxf(__log2f(half_of(few_lds16(vsc + 2 * (lane & (S::kKeys - 1))))), -60.f), 16.f);
    }

    // ---------------- online softmax (base 2)
    float top0, top1;
    float lg[S::kBlocks][2];
#pragma unroll
    for (int sub = 0; sub < S::kBlocks; ++sub) {
      lg[sub][0] = lg[sub][1] = 0.f;
      if constexpr (FMT != kFewBf16) {
        lg[sub][0] = __shfl_sync(0xffffffffu, lsv, sub * 16 + g);
        lg[sub][1] = __shfl_sync(0xffffffffu, lsv, sub * 16 + g + 8);
      }
    }
    auto find_top = [&] {
      top0 = top1 = -INFINITY;
#pragma unroll
      for (int sub = 0; sub < S::kBlocks; ++sub) {
        top0 = fmaxf(top0, fmaxf(s[sub][0] + lg[sub][0], s[sub][2] + lg[sub][1]));
        top1 = fmaxf(top1, fmaxf(s[sub][1] + lg[sub][0], s[sub][3] + lg[sub][1]));
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, o));
        top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, o));
      }
    };
    find_top();
    // the reference follows when it is passed by more than 4 (p' stays below 2^15)
    const bool up0 = top0 - m0 > 4.f, up1 = top1 - m1 > 4.f;
    if (__any_sync(0xffffffffu, up0 || up1)) {
      const float c0 = up0 ? fast_exp2(m0 - top0) : 1.f, c1 = up1 ? fast_exp2(m1 - top1) : 1.f;
      if constexpr (FMT != kFewBf16) {
        const float all0 = sm.factor[2 * t], all1 = sm.factor[2 * t + 1];
        const bool new0 = up0 && (fabsf(top0) > kFarScore || f0 != all0), new1 = up1 && (fabsf(top1) > kFarScore || f1 != all1);
        if (__any_sync(0xffffffffu, new0 || new1)) {  // a column's scores from here on in other units
          auto unit = [](float top, float f, float all) {
            const float far = fabsf(top * (all / f));
            return far > kFarScore ? all * (kFarScore / far) : all;
          };
          const float g0 = new0 ? unit(top0, f0, all0) : f0, g1 = new1 ? unit(top1, f1, all1) : f1;
          const float r0 = g0 / f0, r1 = g1 / f1;
          f0 = g0;
          f1 = g1;
#pragma unroll
          for (int sub = 0; sub < S::kBlocks; ++sub)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[sub][j] *= j & 1 ? r1 : r0;
          find_top();
        }
      }
      if (up0) m0 = top0;
      if (up1) m1 = top1;
      z0 *= c0;
      z1 *= c1;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        acc[k][0] *= c0;
        acc[k][1] *= c1;
        acc[k][2] *= c0;
        acc[k][3] *= c1;
      }
    }
    constexpr float kHead = FMT == kFewBf16 ? 0.f : 11.f;
    const float u0 = m0 == -INFINITY ? 0.f : m0 - kHead, u1 = m1 == -INFINITY ? 0.f : m1 - kHead;
    float p[S::kBlocks][4];
#pragma unroll
    for (int sub = 0; sub < S::kBlocks; ++sub) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[sub][j] = fast_exp2(s[sub][j] - (j & 1 ? u1 : u0));
      z0 += p[sub][0] + p[sub][2];
      z1 += p[sub][1] + p[sub][3];
    }

    // ---------------- context: value dims on M, keys on K, columns on N
    if constexpr (FMT == kFewBf16) {
      const int vr = (lane & 7) + 8 * (lane >> 4), vc = (lane >> 3) & 1;
#pragma unroll
      for (int sub = 0; sub < S::kBlocks; ++sub) {
        uint32_t h01, l01, h23, l23;
        split_bf16x2(p[sub][0], p[sub][1], h01, l01);
        split_bf16x2(p[sub][2], p[sub][3], h23, l23);
        const uint32_t bh0 = movmatrix_trans(h01), bl0 = movmatrix_trans(l01);
        const uint32_t bh1 = movmatrix_trans(h23), bl1 = movmatrix_trans(l23);
        // an infinity or NaN reaches the columns that see its key, one value at a time, and is
        // zero to the products, where it would reach every column (0 x NaN)
#pragma unroll 1
        for (uint32_t left = strange[sub]; left != 0; left &= left - 1) {
          const int r = __ffs(left) - 1;
          const float q0 = __shfl_sync(0xffffffffu, r < 8 ? p[sub][0] : p[sub][2], (r & 7) * 4 + t);
          const float q1 = __shfl_sync(0xffffffffu, r < 8 ? p[sub][1] : p[sub][3], (r & 7) * 4 + t);
          const bool on0 = key_visible(key0[sub] + r, pc0, a.window, a.sinks);
          const bool on1 = key_visible(key0[sub] + r, pc1, a.window, a.sinks);
          const uint32_t row = vbase + (sub * 16 + r) * S::kRow;
#pragma unroll
          for (int mb = 0; mb < D / 16; ++mb)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w = few_lds16(row + (few_off<S::kChunks>(sub * 16 + r, 2 * mb + h) - (sub * 16 + r) * S::kRow) + 2 * g);
              if (not_finite(w)) {
                if (on0) acc[mb][2 * h] = fmaf(q0, __uint_as_float(w << 16), acc[mb][2 * h]);
                if (on1) acc[mb][2 * h + 1] = fmaf(q1, __uint_as_float(w << 16), acc[mb][2 * h + 1]);
              }
            }
          __syncwarp();
          if (lane < S::kChunks) {
            uint32_t* at = reinterpret_cast<uint32_t*>(ring + (i % S::kStages) * S::kStage + S::kPlane + (sub * 16 + r) * S::kRow) + 4 * lane;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t x = at[w];
              at[w] = (not_finite(x & 0xFFFFu) ? 0u : x & 0xFFFFu) | (not_finite(x >> 16) ? 0u : x & 0xFFFF0000u);
            }
          }
          __syncwarp();
        }
#pragma unroll
        for (int mb = 0; mb < D / 16; ++mb) {
          uint32_t av[4];
          few_ldsm_t(vbase + sub * 16 * S::kRow + few_off<S::kChunks>(vr, 2 * mb + vc), av);
          mma_bf16(acc[mb], av[0], av[1], av[2], av[3], bh0, bh1);
          mma_bf16(acc[mb], av[0], av[1], av[2], av[3], bl0, bl1);
        }
      }
    } else {
      const int lr = lane & 15, lc = lane >> 4;
      const bool any_wide = FMT == kFewQ4 && __any_sync(0xffffffffu, wide);
#pragma unroll
      for (int sub = 0; sub < S::kBlocks; ++sub) {
        if constexpr (FMT == kFewTq4) {
          const float sg = half_of(few_lds16(vsc + 2 * (sub * 16 + g))), sh = half_of(few_lds16(vsc + 2 * (sub * 16 + g + 8)));
          p[sub][0] *= sg;
          p[sub][1] *= sg;
          p[sub][2] *= sh;
          p[sub][3] *= sh;
        } else if (any_wide) {  // (a key with a scale above 16: its p in units of the scale, here and below)
          const float eg = wide_unit(lg[sub][0]), eh = wide_unit(lg[sub][1]);
          p[sub][0] *= eg;
          p[sub][1] *= eg;
          p[sub][2] *= eh;
          p[sub][3] *= eh;
        }
        uint32_t b0 = movmatrix_trans(pack_half2(p[sub][0], p[sub][1]));
        uint32_t b1 = movmatrix_trans(pack_half2(p[sub][2], p[sub][3]));
        constexpr int kSW = FMT == kFewQ4 ? D / 64 : 1;
        uint32_t sv[4][kSW];  // scales of keys 2t, 2t + 1, 2t + 8, 2t + 9
        if constexpr (FMT == kFewQ4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = 2 * t + (k & 1) + 8 * (k >> 1);
            few_lds<kSW>(vsc + (sub * 16 + key) * S::kScaleRow, sv[k]);
            if (any_wide) {
              const float ek = wide_unit(__shfl_sync(0xffffffffu, lsv, sub * 16 + key));
              const __half2 e2 = __float2half2_rn(1.f / ek);  // (a power of two: exact)
#pragma unroll
              for (int w = 0; w < kSW; ++w) sv[k][w] = h2_as_u32(__hmul2(u32_as_h2(sv[k][w]), e2));
            }
          }
        } else if (edge || any_bad) {
          b0 &= keep[sub][0];  // (a scale that is not a number reaches no column that does not see it)
          b1 &= keep[sub][1];
        }
#pragma unroll
        for (int u = 0; u < D / 64; ++u) {
          uint32_t r[4];
          few_ldsm_t(vbase + sub * 16 * S::kRow + few_off<S::kChunks>(lr, 2 * u + lc), r);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int G = 2 * u + e;
            const uint32_t ra = r[2 * e], rb = r[2 * e + 1];  // keys 2t, 2t + 1 and 2t + 8, 2t + 9; dims 4g .. 4g + 3
            if constexpr (FMT == kFewQ4) {
              const uint32_t sel = e ? 0x7632u : 0x5410u;
              uint32_t w0 = h2_as_u32(__hmul2(u32_as_h2(b0), u32_as_h2(prmt(sv[0][u], sv[1][u], sel))));
              uint32_t w1 = h2_as_u32(__hmul2(u32_as_h2(b1), u32_as_h2(prmt(sv[2][u], sv[3][u], sel))));
              if (edge || any_bad) {
                w0 &= keep[sub][0];
                w1 &= keep[sub][1];
              }
              const uint32_t ah = ra >> 8, bh = rb >> 8;
              mma_f16(acc[2 * G], nib_lo_pair(ra), nib_hi_pair(ra), nib_lo_pair(rb), nib_hi_pair(rb), w0, w1);
              mma_f16(acc[2 * G + 1], nib_lo_pair(ah), nib_hi_pair(ah), nib_lo_pair(bh), nib_hi_pair(bh), w0, w1);
            } else {
              const uint4 A = tq4_levels8(ra), B = tq4_levels8(rb);  // (x, y): key 2t's dims 0 .. 3, (z, w): key 2t + 1's
              mma_f16(acc[2 * G], prmt(A.x, A.z, 0x5410u), prmt(A.x, A.z, 0x7632u), prmt(B.x, B.z, 0x5410u),
                      prmt(B.x, B.z, 0x7632u), b0, b1);
              mma_f16(acc[2 * G + 1], prmt(A.y, A.w, 0x5410u), prmt(A.y, A.w, 0x7632u), prmt(B.y, B.w, 0x5410u),
                      prmt(B.y, B.w, 0x7632u), b0, b1);
            }
          }
        }
      }
    }
    __syncwarp();
  }
  pdl_trigger();

  // ---------------- the warps' partials, folded
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    z0 += __shfl_xor_sync(0xffffffffu, z0, o);
    z1 += __shfl_xor_sync(0xffffffffu, z1, o);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();  // every ring is done with
  if (g == 0) {
    if constexpr (FMT != kFewBf16) {
      if (m0 != -INFINITY) m0 *= sm.factor[2 * t] / f0;
      if (m1 != -INFINITY) m1 *= sm.factor[2 * t + 1] / f1;
    }
    sm.fm[warp][2 * t] = m0;
    sm.fm[warp][2 * t + 1] = m1;
    sm.fz[warp][2 * t] = z0;
    sm.fz[warp][2 * t + 1] = z1;
  }
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    if constexpr (FMT == kFewBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sm.fold[warp][2 * t + (j & 1)][16 * k + g + 8 * (j >> 1)] = acc[k][j];
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int dim = 32 * (k >> 1) + 4 * g + 2 * (k & 1) + (j >> 1);
        sm.fold[warp][2 * t + (j & 1)][dim] = acc[k][j];
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < 8) {
    const int n = threadIdx.x;
    float M = -INFINITY, Z = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, sm.fm[w][n]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      // (a NaN sum goes on even where no score of its warp was a number)
      const float f = sm.fm[w][n] == -INFINITY ? (sm.fz[w][n] == sm.fz[w][n] ? 0.f : NAN) : fast_exp2(sm.fm[w][n] - M);
      Z = fmaf(sm.fz[w][n], f, Z);
      sm.fw[w][n] = f;
    }
    sm.m_own[n] = M;
    sm.z_own[n] = Z;
  }
  __syncthreads();
  // The CTA's partial goes piece by piece to the CTAs of the cluster that fold and store it: a
  // piece is a column's group of 32 values (TQ4: the whole column, which its rotation spans),
  // piece i is CTA i % cs's.  Stores to another CTA's shared memory wait for nothing.
  const uint32_t cs = cluster_size(), rank = cluster_rank();
  constexpr bool kWhole = FMT == kFewTq4;
  constexpr int kPiece = kWhole ? D : 32, kPieces = 8 * D / kPiece;
  if (cs > 1) cluster_wait();  // (every CTA has begun)
  const int per_cta = kPieces / static_cast<int>(cs);
#pragma unroll 2
  for (int i = 4 * threadIdx.x; i < 8 * D; i += 4 * WARPS * 32) {
    const int n = i / D, e = i % D, piece = i / kPiece;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = sm.fw[w][n];
      const float4 v = *reinterpret_cast<const float4*>(&sm.fold[w][n][e]);
      A.x = fmaf(v.x, f, A.x);
      A.y = fmaf(v.y, f, A.y);
      A.z = fmaf(v.z, f, A.z);
      A.w = fmaf(v.w, f, A.w);
    }
    const uint32_t owner = static_cast<uint32_t>(piece) % cs;
    cluster_st4(&sm.acc[(static_cast<int>(rank) * per_cta + piece / static_cast<int>(cs)) * kPiece + i % kPiece], owner, A);
  }
  // (the references and sums to everybody)
  for (int i = threadIdx.x; i < 8 * static_cast<int>(cs); i += WARPS * 32) {
    cluster_st(&sm.m[rank][i & 7], i >> 3, sm.m_own[i & 7]);
    cluster_st(&sm.z[rank][i & 7], i >> 3, sm.z_own[i & 7]);
  }
  if (cs > 1) cluster_sync_all();
  else __syncthreads();

  // ---------------- the cluster's partials of this CTA's pieces, folded in order
  const int range = blockIdx.x / cs;
  // (a piece of 32 by eight lanes, four values each; a column by a warp, D / 32 values each)
  constexpr int kLanes = kWhole ? 32 : 8, kV = kWhole ? NG : 4;
  const int sub = lane % kLanes;
#pragma unroll 1
  for (int local0 = warp * (32 / kLanes); local0 < per_cta; local0 += WARPS * (32 / kLanes)) {
    const int local = min(local0 + lane / kLanes, per_cta - 1);  // (the last one again, where there are fewer)
    const int piece = local * static_cast<int>(cs) + static_cast<int>(rank), n = piece * kPiece / D;
    float M = -INFINITY, Z = 0.f, x[kV] = {};
#pragma unroll 4
    for (int r = 0; r < static_cast<int>(cs); ++r) M = fmaxf(M, sm.m[r][n]);
#pragma unroll 4
    for (int r = 0; r < static_cast<int>(cs); ++r) {
      const float mr = sm.m[r][n], zr = sm.z[r][n];
      const float f = mr == -INFINITY ? (zr == zr ? 0.f : NAN) : fast_exp2(mr - M);
      Z = fmaf(zr, f, Z);
      const float* at = &sm.acc[(r * per_cta + local) * kPiece];
      if constexpr (kWhole) {
#pragma unroll
        for (int k = 0; k < kV; ++k) x[k] = fmaf(at[32 * k + sub], f, x[k]);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(at + 4 * sub);
        x[0] = fmaf(v.x, f, x[0]);
        x[1] = fmaf(v.y, f, x[1]);
        x[2] = fmaf(v.z, f, x[2]);
        x[3] = fmaf(v.w, f, x[3]);
      }
    }
    const int col = 8 * cb + n, row = sr.first + col / a.group, head = kvh * a.group + col % a.group;
    const int e0 = kWhole ? 0 : piece * 32 % D + 4 * sub;
    const bool live = n < cols;
    if (ranges > 1) {
      if (!live) continue;
      const int64_t part = (static_cast<int64_t>(range) * a.n_rows + row) * a.Hq + head;
      if (sub == 0 && e0 == 0) a.ws_m[part] = M, a.ws_z[part] = Z;
      if constexpr (kWhole) {
#pragma unroll
        for (int k = 0; k < kV; ++k) a.ws_acc[part * D + 32 * k + sub] = x[k];
      } else {
        *reinterpret_cast<float4*>(a.ws_acc + part * D + e0) = make_float4(x[0], x[1], x[2], x[3]);
      }
      continue;
    }
    const float inv = Z == 0.f ? 0.f : 1.f / Z;
#pragma unroll
    for (int k = 0; k < kV; ++k) x[k] *= inv;
    if constexpr (kWhole) {
      tq4_turn_lanes<kV>(x, static_cast<const uint32_t*>(c.signs), lane, true);
      if (live) {
#pragma unroll
        for (int k = 0; k < kV; ++k) seq_store(a, row, head, 32 * k + sub, x[k]);
      }
    } else {
      if (c.format == KVQ_FMT_Q4_HAD32) {
        const float s0 = x[0] + x[1], d0 = x[0] - x[1], s1 = x[2] + x[3], d1 = x[2] - x[3];
        x[0] = s0 + s1;
        x[1] = d0 + d1;
        x[2] = s0 - s1;
        x[3] = d0 - d1;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float y = __shfl_xor_sync(0xffffffffu, x[k], o);
            x[k] = lane & o ? y - x[k] : x[k] + y;
          }
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] *= kHadamardScale;
      }
      if (live) {
        const int64_t at = static_cast<int64_t>(row) * a.out.ts + static_cast<int64_t>(head) * a.out.hs + e0;
        if (a.out.wide && a.out.dtype == KVQ_DT_BF16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out.data) + at) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
        else if (a.out.wide)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out.data) + at) = make_float4(x[0], x[1], x[2], x[3]);
        else
#pragma unroll
          for (int k = 0; k < 4; ++k) seq_store(a, row, head, e0 + k, x[k]);
      }
    }
  }
}

// The ranges' partials of a row and head, folded in a fixed order, rotated back and rounded.
// Four warps take every fourth range: one warp's loads of all of them, four in flight, were
// 0.4 us a range.
template <int D>
__global__ void __launch_bounds__(128) attn_merge_kernel(const __grid_constant__ SeqAttnArgs a, int ranges) {
  constexpr int NG = D / 32;
  __shared__ float sm_x[4][D], sm_z[4];
  pdl_wait();
  pdl_trigger();
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const SeqRows sr = seq_rows(a, blockIdx.y);
  const int i = blockIdx.x;
  if (sr.state != kRowsOk || i >= sr.n * a.Hq) return;
  const int row = sr.first + i / a.Hq, head = i % a.Hq;
  if (a.per > 0) {  // as many as the column's block was cut into; one: stored already
    const int cb = (i / a.Hq * a.group + head % a.group) >> 3, base = sr.T - sr.n;
    const int p1 = base + (min(8 * cb + 8, sr.n * a.group) - 1) / a.group;
    ranges = p1 < 0 ? 1 : (key_blocks(base + 8 * cb / a.group, p1, a.window, a.sinks).count + a.per - 1) / a.per;
    if (ranges <= 1) return;
  }
  const int64_t stride = static_cast<int64_t>(a.n_rows) * a.Hq, part = static_cast<int64_t>(row) * a.Hq + head;
  float M = -INFINITY, Z = 0.f, x[NG] = {};
  for (int r = lane; r < ranges; r += 32) M = fmaxf(M, a.ws_m[part + r * stride]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll 4
  for (int r = warp; r < ranges; r += 4) {
    const float mr = a.ws_m[part + r * stride], zr = a.ws_z[part + r * stride];
    const float f = mr == -INFINITY ? (zr == zr ? 0.f : NAN) : fast_exp2(mr - M);
    Z = fmaf(zr, f, Z);
    const float* at = a.ws_acc + (part + r * stride) * D + lane;
#pragma unroll
    for (int k = 0; k < NG; ++k) x[k] = fmaf(at[32 * k], f, x[k]);
  }
#pragma unroll
  for (int k = 0; k < NG; ++k) sm_x[warp][32 * k + lane] = x[k];
  if (lane == 0) sm_z[warp] = Z;
  __syncthreads();
  if (warp != 0) return;
  Z = (sm_z[0] + sm_z[1]) + (sm_z[2] + sm_z[3]);
  const float inv = Z == 0.f ? 0.f : 1.f / Z;
#pragma unroll
  for (int k = 0; k < NG; ++k) {
    const int e = 32 * k + lane;
    x[k] = ((sm_x[0][e] + sm_x[1][e]) + (sm_x[2][e] + sm_x[3][e])) * inv;
  }
  if (a.c.format == KVQ_FMT_TQ4) {
    tq4_turn_lanes<NG>(x, static_cast<const uint32_t*>(a.c.signs), lane, true);
  } else if (a.c.format == KVQ_FMT_Q4_HAD32) {
#pragma unroll
    for (int k = 0; k < NG; ++k) x[k] = warp_fwht32(x[k], lane) * kHadamardScale;
  }
#pragma unroll
  for (int k = 0; k < NG; ++k) seq_store(a, row, head, 32 * k + lane, x[k]);
}

cudaError_t launch_attn_merge(const SeqAttnArgs& a, int ranges, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.max_rows) * a.Hq, a.num_seqs);
  switch (a.c.head_dim) {
    case 64: return launch_pdl(attn_merge_kernel<64>, grid, dim3(128), 0, s, a, ranges);
    case 128: return launch_pdl(attn_merge_kernel<128>, grid, dim3(128), 0, s, a, ranges);
    default: return launch_pdl(attn_merge_kernel<256>, grid, dim3(128), 0, s, a, ranges);
  }
}

// One wave of CTAs: four of the 4-bit rows' to an SM (registers), of the bf16 rows' as many as
// their rings leave room for.
static int few_fit(const kvq_cache& c) {
  return c.format != KVQ_FMT_BF16 || c.head_dim == 64 ? 4 : c.head_dim == 256 ? 1 : 3;
}

// The partials (of a row and head) that no plan passes: ranges x blocks of 8 columns is at most
// what runs at once, in the pieces of ragged sequences 12 times that
// (a piece has at least 0.339 all blocks / 2 fit n_sm blocks of 16 keys: 5.9 fit n_sm / blocks
// ranges and one more, and two where there are partials at all).
int64_t few_partials(const kvq_cache& c, bool ragged, int n_sm) {
  return static_cast<int64_t>(ragged ? 12 : 1) * 8 * few_fit(c) * n_sm;
}

FewPlan few_plan(const kvq_cache& c, int num_seqs, int Hq, int max_rows, int max_seq_len, int window, int sinks,
                 int n_sm) {
  const int group = Hq / c.num_kv_heads, D = c.head_dim;
  const int64_t blocks = static_cast<int64_t>(num_seqs) * c.num_kv_heads * ((static_cast<int64_t>(max_rows) * group + 7) / 8);
  int64_t keys = max_seq_len;
  if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + sinks + 64 + 8 / group);
  const int fit = few_fit(c);
  FewPlan p{1, 1, 0};
  if (window == 0 && num_seqs > 1) {
    // Sequences of any lengths: so many blocks of 16 keys a CTA, that sequences of half the
    // longest fill a wave (16 of 8000 tokens, 1 to 5 rows of 6 heads: equal shares 108 us,
    // so 64).  At least eight blocks for every warp, at most 32 ranges.
    const int64_t all = (keys + 15) / 16;
    int64_t per = (all * blocks / 2 + fit * static_cast<int64_t>(n_sm) - 1) / (fit * static_cast<int64_t>(n_sm));
    // Long pieces leave a long tail: where one has more than 96 blocks, three waves of shorter
    // ones (48 sequences up to 16000, 2 rows of 6 heads 191 -> 151 us, bf16 rows 357 -> 305).
    if (per > 96) per = std::max<int64_t>(96, per * 35 / 100);
    per = std::max<int64_t>(std::max<int64_t>(per, 32), (all + 31) / 32);
    p.per = static_cast<int>((per + 3) / 4 * 4);
    p.ranges = static_cast<int>(std::max<int64_t>(1, (all + p.per - 1) / p.per));
    if (p.ranges == 1) p.per = 0;
    return p;
  }
  // Clusters and ranges by what they are expected to cost: the blocks of a warp, which slow one
  // another down on an SM, more CTAs' beginnings, and a second launch for the fold of ranges.
  // All have to run at once: the clusters of a size that fit were counted (152 SMs, four CTAs to
  // an SM 148 of 4, 74 of 8, 33 of 16; one to an SM 36, 15 and 7), and a second wave costs what
  // the first does.  (The figures here are from before metadata was read behind the wait for the
  // kernel in front, 1.3 us a call.)  So of one sequence of 30000 tokens with 4 rows of 24 heads 46 us with three
  // clusters of 16 for each block of columns, 35 with eleven of 4; bf16 rows, one row, 45 and 27.
  // Clusters of 16 lie unevenly over the SMs and come as one range only (a window of 1024 keys of
  // one sequence; one of 4096 is nine clusters of 4).  TQ4 has 8 pieces that are folded, a CTA for each.
  const bool bf = c.format == KVQ_FMT_BF16;
  const int sub = !bf && D <= 128 ? 2 : 1;  // blocks of a warp's step
  const double unit = D / 256. * (bf ? 1.3 : c.format == KVQ_FMT_TQ4 ? 1.4 : 1.);
  const double step[4] = {1.2, 1.5, 1.9, 2.45};  // us a block, 1 to 4 CTAs on the SM
  const int64_t all = (keys + 15) / 16;
  double least = 0;
  for (int cs = c.format == KVQ_FMT_TQ4 ? 8 : 16; cs >= 1; cs /= 2) {
    const double share = cs == 16 ? 0.73 : cs == 8 ? (fit == 1 ? 0.78 : 0.88) : cs == 4 ? 0.94 : 1.;
    const int64_t room = static_cast<int64_t>(share * fit * n_sm / cs);
    for (int64_t r = 1; r <= (cs == 16 ? 1 : 64); ++r) {
      const int64_t per_step = 4 * sub * cs * r;
      if ((blocks * r > room && cs * r > 1) || (cs * r > 1 && per_step >= 2 * all)) break;
      const int64_t k = std::max<int64_t>(1, std::min<int64_t>(fit, (blocks * r * cs + n_sm - 1) / n_sm));
      const double waves = blocks > room ? static_cast<double>(blocks) / static_cast<double>(room) : 1.;
      const double cost = waves * (1.2 * static_cast<double>(k) + unit * step[k - 1] * static_cast<double>((all + per_step - 1) / per_step * sub)) +
                          (r > 1 ? 2.5 + 0.06 * static_cast<double>(r) : 0.);
      if (least == 0 || cost < least) {
        least = cost;
        p.cluster = cs;
        p.ranges = static_cast<int>(r);
      }
    }
  }
  return p;
}

template <int FMT, int D, int WARPS>
static cudaError_t launch_few(const SeqAttnArgs& a, const FewPlan& p, cudaStream_t s) {
  constexpr auto kern = attn_few_kernel<FMT, D, WARPS>;
  const size_t smem = sizeof(FewSmem<FMT, D, WARPS>) + 128;
  static_assert(sizeof(FewSmem<FMT, D, WARPS>) + 128 <= 232448, "shared memory");
  cudaError_t e = set_max_smem_once<kern, true>(static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t cbs = (static_cast<int64_t>(a.max_rows) * a.group + 7) / 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.cluster * p.ranges, static_cast<unsigned>(cbs * a.c.num_kv_heads), a.num_seqs);
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(p.cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || p.ranges == 1) return e;
  return launch_attn_merge(a, p.ranges, s);
}

template <int FMT>
static cudaError_t launch_few_dim(const SeqAttnArgs& a, const FewPlan& p, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch_few<FMT, 64, 4>(a, p, s);
    case 128: return launch_few<FMT, 128, 4>(a, p, s);
    default: return launch_few<FMT, 256, 4>(a, p, s);
  }
}

cudaError_t launch_attn_few(const SeqAttnArgs& a, const FewPlan& p, cudaStream_t s) {
  if (a.num_seqs == 0 || a.n_rows == 0 || a.max_rows == 0) return cudaSuccess;
  if (a.c.format == KVQ_FMT_BF16) return launch_few_dim<kFewBf16>(a, p, s);
  if (a.c.format == KVQ_FMT_TQ4) return launch_few_dim<kFewTq4>(a, p, s);
  return launch_few_dim<kFewQ4>(a, p, s);
}

}  // namespace kvq
