// attn_chunk.cu -- attention of many rows a sequence (prompt chunks) over the paged
// cache, ragged, with a sliding window and sinks, every row format, on pairs of SMs
// (tcgen05 with cta_group::2).
//
// For a row at position p:  o = sum_j 2^(s_j - m) v_j / sum_j 2^(s_j - m) over the keys j
// that it sees (seqs.cuh), s_j = sm_scale log2(e) q . k_j, m a running reference.
//
// Bound by the tensor cores: 4 x rows x keys x head_dim operations against a tile of keys
// that is read and decoded once for 256 rows.  A pair of CTAs takes 2 x floor(128 / group)
// positions of a sequence and the query heads of one KV head, 128 rows in each CTA's
// tensor memory, and walks the keys in tiles of 128.  B operands are shared by the pair:
// each CTA decodes 64 of a tile's keys and, of all 128, half of the value dims, so the
// decoding, the shared memory and its traffic are halved against one CTA alone (a product
// of 128 x 128 reads 128 bytes a cycle of shared memory, all there is; of 256 x 128 over
// the pair, 96).
// Roles, per CTA: warp 0 of the first CTA issues the products (scores of tile j + 1, then
// the context of tile j); warps 4 to 7 softmax, one row a thread; warps 8 to 11 decode
// keys, 12 to 15 values, from global memory through registers (the next tile's codes are
// loaded while this one's are converted) into operands without a swizzle: eight keys' 16
// bytes make a core matrix, so eight lanes write 128 contiguous bytes.  Keys are K-major;
// values lie with their dims contiguous (B with its columns contiguous), so neither is
// transposed.  Scores alternate between two buffers of tensor memory; p (fp16) goes over
// the scores it was made from and is the context product's A.
// Queries, keys and values are fp16 here (each within 2^-11; bf16 rows: bf16, as they
// are), a row's queries scaled by a power of two (to at most 2^15).  p is fp16: 2^(7 + s - m), at
// most 2^15, as the reference m follows when a row's scores pass it by more than 8 (by more than
// 6, for two bits more of p: 4096 rows at 16384 1498 -> 1677 us).  So a weight down to 2^-21 of
// the row's largest keeps its 11 bits, and one below is off by up to 2^-32 of the largest: where
// nearly all of the weight falls on a token whose value is near zero, as on a sequence's first,
// the output is made of such weights.  (bf16 rows: p is bf16, 2^(s - m) up to 2^8.)  Where a
// scale above 4096 turns up (8 s may not fit fp16), the pair goes over its keys once more
// with keys and values in units of 8 (a scale below 2^-11 is then rounded to 2^-22); nobody else
// pays for that, nor do slots that no row sees set it off.
//
// Measured (one GB300, 24 / 4 heads of 256, 4-bit rows): 4096 rows at 16384 1483 us (1251
// TFLOP/s), 2048 rows with a window of 4096 222 us.  The products alone, with everybody else
// only arriving, take 486 us of the 684 of 2048 rows at 16384; the softmax and the decoders add
// to them through shared memory and issue slots.  Every role's loop is rolled: four roles
// share a sub-partition's instruction fetch (unrolled 920 us).
#include <algorithm>

#include "f32x2.cuh"
#include "rows.cuh"
#include "seqs.cuh"
#include "tc05_pair.cuh"
#include "tq4_levels.cuh"

namespace kvq {

constexpr int kCkTile = 128;    // keys of a tile: 8 blocks of 16
constexpr int kCkThreads = 512;
constexpr int kCkRing = 5;       // units of raw codes that a decoding thread has in flight, and one
constexpr int kCkNotes = 512;  // keys that some rows of a pair see and others do not: up to 255 at either end
constexpr float kCkBigUnit = 0.125f;  // of keys and values in the second pass: 8 x 65504 fits fp16, and scales from 2^-11 on are exact
constexpr float kCkRaise = 8.f;  // a row's reference is raised when its scores passed it by more
constexpr float kCkHead = 7.f;   // p = 2^(this + s - m), at most 2^15 (fp16)
enum { kCkQ4 = 0, kCkTq4 = 1, kCkBf16 = 2 };

// tensor-memory columns (all 512 are allocated)
constexpr uint32_t kCkS = 0;    // 2 x 128: scores of even and odd tiles, then p
constexpr uint32_t kCkO = 256;  // head_dim: the output accumulator

template <int D>
struct __align__(1024) CkOperands {
  // core matrices of 8 rows x 16 bytes: element (row, d) of q, k at (row / 8) 16 D + (d / 8) 128 + (row % 8) 16,
  // element (key, n) of v at (n / 8) 2048 + (key / 8) 128 + (key % 8) 16, n its value dim in this CTA's half
  uint8_t q[128 * D * 2];
  uint8_t k[2][64 * D * 2];
  uint8_t v[2][128 * D];
};
template <int D>
struct CkSmem {
  union {
    CkOperands<D> op;
    float out[128][D + 1];  // at the end: this CTA's rows
  };
  uint4 raw[2][kCkRing][128];  // per plane, slot and decoding thread
  uint32_t raw_scale[2][kCkRing][128];
  // the CTA's 4 warps (q_ready: 16) arrive, and at the first CTA's the second's forwarder
  uint64_t k_ready[2], v_ready[2], p_ready[2], q_ready;
  uint64_t k_free[2], s_full[2], pv_done[2];    // each CTA's: the products arrive
  uint64_t drained;
  uint32_t row_top[128];                        // per row: its largest query element
  float factor[128];                            // per row: what its scores' units are worth
  float m[128], z[128];
  // values that are not numbers, of keys that not every row sees: four bits a key, one for each of
  // this CTA's groups (bf16 rows: one for this CTA's half of the dims)
  uint32_t noted[kCkNotes / 8];
  int any_noted;
  int over;  // a scale above 4096 was met, of a key that some row sees
  uint32_t tmem_base;
  int abort;
  int seq, block;
  SeqRows rows_of;  // the sequence's
};
constexpr size_t kCkMinSmem = 120 * 1024;  // one CTA to an SM: pairs that wait for tensor memory crosswise would wait forever

// Bounded wait, as the prefill's: gives up on the CTA's abort flag or after about 2 s.  PAIR:
// what the other CTA did before it arrived is visible, too.
template <bool PAIR = false, int D>
__device__ __forceinline__ bool ck_wait(CkSmem<D>& sm, uint64_t* bar, uint32_t parity, int32_t* status) {
  auto done = [&] { return PAIR ? pair_try_wait(bar, parity) : mbar_try_wait(bar, parity); };
  if (done()) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 0;; ++it) {
    if (done()) return true;
    if ((it & 31u) == 31u) {
      if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
      if (global_timer_ns() - t0 > 2000000000ull) {
        atomicExch(&sm.abort, 1);
        set_status(status, KVQ_DEV_TIMEOUT);
        return false;
      }
    }
  }
}
template <int D>
__device__ __forceinline__ bool ck_wait_warp(CkSmem<D>& sm, uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, ck_wait(sm, bar, parity, status));
}

__device__ __forceinline__ float ck_max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void ck_sts(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ bool ck_not_finite16(uint32_t bf16) { return (bf16 & 0x7F80u) == 0x7F80u; }

// Which tile of keys this is, for everybody who walks them.
struct CkWalk {
  KeyBlocks kb;
  int tile0, tiles;
  int p0, p1, window, sinks;
  __device__ __forceinline__ int key_of(int tile, int blk) const {  // the first key of block `blk` of 8
    const int i = (tile0 + tile) * 8 + blk;
    return i < kb.count ? kb.block_of(i) * 16 : kNoKey;
  }
  // Tiles [plain0, plain1) of the whole walk lie behind the sinks' blocks and every row sees
  // all of their keys; in the others (edges) some row may not.
  int plain0, plain1;
  __device__ __forceinline__ void find_plain() {
    const int shift = kb.head - kb.body;  // block i of the walk is block i - shift of the sequence
    plain0 = (kb.head + 7) >> 3;
    if (window > 0) plain0 = max(plain0, (((max(p1 - window + 1, 0) + 15) >> 4) + shift + 7) >> 3);
    plain1 = p0 < kCkTile - 1 ? 0 : ((((p0 - kCkTile + 1) >> 4) + shift) >> 3) + 1;
  }
  __device__ __forceinline__ bool edge(int tile) const { return tile0 + tile < plain0 || tile0 + tile >= plain1; }
  // The note of a key that some rows see and others do not: those behind the first row (1 ..
  // 255), and those that its window holds and the last row's does not (257 .. 511).
  enum { kEverybody = -1, kNobody = -2 };
  __device__ __forceinline__ int note_of(int key) const {
    if (!any_visible(key, p0, p1, window, sinks)) return kNobody;
    if (all_visible(key, 1, p0, p1, window, sinks)) return kEverybody;
    return key > p0 ? key - p0 : kCkNotes / 2 + key - (p0 - window);
  }
  __device__ __forceinline__ int key_of_note(int i) const { return i < kCkNotes / 2 ? p0 + i : p0 - window + i - kCkNotes / 2; }
};

// 8 codes of a word as fp16 operands, times (s, s): 4-bit groups in the order 0 4 1 5 2 6 3 7,
// TQ4 codes in their own.
template <int FMT>
__device__ __forceinline__ void ck_decode8(uint32_t w, __half2 s2, uint32_t (&o)[4]) {
  if constexpr (FMT == kCkQ4) {
    const uint32_t h = w >> 8;
    o[0] = h2_as_u32(__hmul2(u32_as_h2(nib_lo_pair(w)), s2));
    o[1] = h2_as_u32(__hmul2(u32_as_h2(nib_hi_pair(w)), s2));
    o[2] = h2_as_u32(__hmul2(u32_as_h2(nib_lo_pair(h)), s2));
    o[3] = h2_as_u32(__hmul2(u32_as_h2(nib_hi_pair(h)), s2));
  } else {
    const uint4 l = tq4_levels8(w);
    o[0] = h2_as_u32(__hmul2(u32_as_h2(l.x), s2));
    o[1] = h2_as_u32(__hmul2(u32_as_h2(l.y), s2));
    o[2] = h2_as_u32(__hmul2(u32_as_h2(l.z), s2));
    o[3] = h2_as_u32(__hmul2(u32_as_h2(l.w), s2));
  }
}
// Where element j of 8 lies among them, and the element that lies at position i.
template <int FMT>
__device__ __forceinline__ int ck_pos(int j) { return FMT == kCkQ4 ? (j & 3) * 2 + (j >> 2) : j; }
template <int FMT>
__device__ __forceinline__ int ck_elem(int i) { return FMT == kCkQ4 ? (i >> 1) + 4 * (i & 1) : i; }

// 0 x NaN: a value that is not a number, of a key that some rows do not see, is taken out of the
// operands and noted, for the rows that do see it.  (One that every row sees stays; one that
// nobody sees, in a slot behind the end or between sinks and window, is of no consequence.)
// Whether to take it out; `bit`: its group here.
template <int D>
__device__ __forceinline__ bool ck_note(CkSmem<D>& sm, const CkWalk& wk, int key, int bit) {
  const int note = wk.note_of(key);
  if (note >= 0) {
    atomicOr(&sm.noted[note >> 3], 1u << (4 * (note & 7) + bit));
    sm.any_noted = 1;
  }
  return note != CkWalk::kEverybody;
}

// ---------------------------------------------------------------- the decoders' part
// Four warps convert one plane's part of every tile: IS_K: 64 keys (those of this CTA),
// all dims; else 128 keys, this CTA's half of the dims.
// What a decoding thread fetches next. Pages are looked up for four tiles at once, one lane a
// block, and four tiles ahead: a tile's own look-up, waited for, held the first fetch of a pair
// back by a trip to memory (8 prompts 205 -> 197 us, five ragged chunks 447 -> 437).
struct CkFetch {
  int rows;  // lane l: the cache row of block l & 7 of tile l >> 3 of four
  int page;  // and that block's page of the next four, as the table has it
  int tile, unit, slot;
};

template <int FMT, int D, bool IS_K>
struct CkPart {
  static constexpr bool kBf = FMT == kCkBf16;
  static constexpr int kKeys = IS_K ? 64 : 128;
  static constexpr int kRowChunks = kBf ? D / 8 : D / 32;        // 16-byte chunks of a row
  static constexpr int kC = IS_K ? kRowChunks : kRowChunks / 2;  // of them here
  static constexpr int kUnits = kKeys * kC / 128;                // a thread's
  // 4-bit rows: a thread's units are key groups (of 8) kg0 + i kSpan, always the same chunk and
  // the same key of 16.  Their codes and scales come through a ring of its own in shared
  // memory, kCkRing - 1 units ahead (nobody else reads them, so only its own copies are
  // waited for).
  static constexpr int kSpan = kBf ? 0 : 16 / kC;
  const SeqAttnArgs& a;
  CkSmem<D>& sm;
  const CkWalk& wk;
  const int kvh, rank, tid;

  __device__ __forceinline__ int kg0() const { return tid / (8 * kC); }
  __device__ __forceinline__ int chunk() const { return (IS_K ? 0 : rank * kC) + (tid >> 3) % kC; }
  __device__ __forceinline__ int in16() const { return (kg0() & 1) * 8 + (tid & 7); }
  __device__ __forceinline__ uint32_t buf(int b) const { return smem_u32(IS_K ? sm.op.k[b] : sm.op.v[b]); }

  // Lane l: the first key of block l & 7 (of keys: of this CTA's four) of tile t0 + l / 8.
  __device__ __forceinline__ int lane_key(int t0) const {
    const int lane = tid & 31, tile = t0 + (lane >> 3);
    return tile < wk.tiles && (!IS_K || (lane & 7) < 4) ? wk.key_of(tile, IS_K ? rank * 4 + (lane & 3) : lane & 7) : kNoKey;
  }
  // Its page in the sequence's table: looked at only where the row is made of it, four tiles
  // later, so that the load is not waited for.
  __device__ __forceinline__ int find_page(int t0) const {
    const int key = lane_key(t0);
    if (key == kNoKey) return 0;
    return a.block_tables[static_cast<int64_t>(sm.seq) * a.max_pages + fast_div(static_cast<uint32_t>(key >> 4), a.page_blocks)];
  }
  // Its cache row: -1 a page outside the pool, -2 no such block.
  __device__ __forceinline__ int row_of(int t0, int page) const {
    const int key = lane_key(t0);
    if (key == kNoKey) return -2;
    if (page < 0 || page >= a.c.num_pages) {
      set_status(a.status, KVQ_DEV_BAD_PAGE);
      return -1;
    }
    const int blk = key >> 4, pg = static_cast<int>(fast_div(static_cast<uint32_t>(blk), a.page_blocks));
    return (page * a.c.num_kv_heads + kvh) * a.c.page_size + (blk - pg * static_cast<int>(a.page_blocks.d)) * 16;
  }
  __device__ __forceinline__ void next_tile(CkFetch& f) const {
    if ((++f.tile & 3) == 0) {
      f.rows = row_of(f.tile, f.page);
      f.page = find_page(f.tile + 4);
    }
  }
  // bf16 rows: unit i's key of the tile, and its place among the operands.
  __device__ __forceinline__ int unit_key(int i) const { return ((tid + 128 * i) / (8 * kC)) * 8 + (tid & 7); }
  __device__ __forceinline__ int unit_chunk(int i) const { return ((tid + 128 * i) >> 3) % kC; }
  __device__ __forceinline__ int place(int i) const {
    const int key = unit_key(i), n16 = unit_chunk(i);
    return IS_K ? (key >> 3) * 16 * D + n16 * 128 + (key & 7) * 16 : n16 * 2048 + (key >> 3) * 128 + (key & 7) * 16;
  }

  // The next unit (bf16 rows: tile, into the operands themselves; J: its number of both passes).
  __device__ __forceinline__ void fetch(CkFetch& f, int J) const {
    const kvq_cache& c = a.c;
    if constexpr (kBf) {
      const uint8_t* plane = static_cast<const uint8_t*>(IS_K ? c.k : c.v);
      const uint32_t at = buf(J & 1);
#pragma unroll 4
      for (int i = 0; i < kUnits; ++i) {
        const int key = unit_key(i);
        const int row0 = __shfl_sync(0xffffffffu, f.rows, (f.tile & 3) * 8 + (key >> 4));
        const uint32_t dst = at + place(i);
        if (row0 >= 0) {
          const uint8_t* src = plane + (static_cast<int64_t>(row0) + (key & 15)) * (2 * D) + ((IS_K ? 0 : rank * kC) + unit_chunk(i)) * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
        } else {  // no such key: zeros; a bad page's scores are NaN
          const uint32_t x = IS_K && row0 == -1 ? 0x7FFF7FFFu : 0u;
          ck_sts(dst, x, x, x, x);
        }
      }
      next_tile(f);
    } else {
      static_assert(kSpan % 2 == 0 && kUnits * kSpan * 8 == kKeys, "units");
      const int row0 = __shfl_sync(0xffffffffu, f.rows, (f.tile & 3) * 8 + (kg0() >> 1) + f.unit * (kSpan / 2));
      const uint32_t ring = smem_u32(&sm.raw[IS_K ? 0 : 1][0][tid]) + f.slot * 2048;
      const uint32_t ring_s = smem_u32(&sm.raw_scale[IS_K ? 0 : 1][0][tid]) + f.slot * 512;
      if (row0 >= 0) {
        const uint8_t* code_at = static_cast<const uint8_t*>(IS_K ? c.k : c.v) + in16() * (D / 2) + chunk() * 16;
        // (copies of 4 bytes: the scale beside another)
        const uint16_t* scale_at = static_cast<const uint16_t*>(IS_K ? c.k_scale : c.v_scale) + (scale_index() & ~1);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ring), "l"(code_at + static_cast<int64_t>(row0) * (D / 2))
                     : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ring_s),
                     "l"(scale_at + static_cast<int64_t>(row0) * (FMT == kCkQ4 ? D / 32 : 1))
                     : "memory");
      } else {  // no such key: zeros; a bad page's scores are NaN
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(ring_s), "r"(IS_K && row0 == -1 ? 0x7E007E00u : 0u) : "memory");
      }
      f.slot = f.slot == kCkRing - 1 ? 0 : f.slot + 1;
      if (++f.unit == kUnits) {
        f.unit = 0;
        next_tile(f);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ int scale_index() const { return FMT == kCkQ4 ? in16() * (D / 32) + chunk() : in16(); }

  // The first loads, of a pass whose first tile is number `first`.
  __device__ __forceinline__ CkFetch begin(int first) const {
    CkFetch f{0, find_page(0), 0, 0, 0};
    f.rows = row_of(0, f.page);
    f.page = find_page(4);
    if constexpr (kBf) {
      if (wk.tiles > 0) fetch(f, first);
    } else {
#pragma unroll 1
      for (int i = 0; i < kCkRing - 1; ++i) fetch(f, 0);
    }
    return f;
  }

  // All tiles.  big: the second pass, in units of 8; the buffers' and barriers' order goes on.
  __device__ __forceinline__ void run(CkFetch f, bool big) const {
    uint64_t* const ready = IS_K ? sm.k_ready : sm.v_ready;
    uint64_t* const freed = IS_K ? sm.k_free : sm.pv_done;
    const int lane = tid & 31;
    if constexpr (kBf) {
#pragma unroll 1
      for (int j = 0; j < wk.tiles; ++j) {
        if (j + 1 < wk.tiles) {
          if (j >= 1 && !ck_wait_warp(sm, &freed[(j + 1) & 1], ((j - 1) >> 1) & 1, a.status)) return;
          fetch(f, j + 1);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
        } else {
          asm volatile("cp.async.wait_group 0;" ::: "memory");
        }
        if constexpr (!IS_K) {
          if (wk.edge(j)) {
#pragma unroll 1
            for (int i = 0; i < kUnits; ++i) {
              const uint32_t at = buf(j & 1) + place(i);
              uint32_t w[4];
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at));
              bool found = false;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t x = (w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu;
                if (ck_not_finite16(x)) {
                  const int key = unit_key(i);
                  if (ck_note(sm, wk, wk.key_of(j, key >> 4) + (key & 15), 0)) {
                    found = true;
                    w[e >> 1] &= e & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                  }
                }
              }
              if (found) ck_sts(at, w[0], w[1], w[2], w[3]);
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[j & 1]);
      }
    } else {
      const int kg = kg0();
      const uint32_t pick = scale_index() & 1 ? 0x3232u : 0x1010u;
      const uint32_t dst0 = IS_K ? kg * 16 * D + (tid >> 3) % kC * 512 + (tid & 7) * 16
                                 : (tid >> 3) % kC * 8192 + kg * 128 + (tid & 7) * 16;
      constexpr uint32_t kStepUnit = IS_K ? kSpan * 16 * D : kSpan * 128, kStepWord = IS_K ? 128 : 2048;
      const uint32_t ring = smem_u32(&sm.raw[IS_K ? 0 : 1][0][tid]), ring_s = smem_u32(&sm.raw_scale[IS_K ? 0 : 1][0][tid]);
      const int first = big ? wk.tiles : 0;
      int slot = 0;
#pragma unroll 1
      for (int j = 0; j < wk.tiles; ++j) {
        const int J = first + j;
        const bool edge = !IS_K && wk.edge(j);
        if (J >= 2 && !ck_wait_warp(sm, &freed[J & 1], ((J >> 1) - 1) & 1, a.status)) return;
        uint32_t at = buf(J & 1) + dst0;
#pragma unroll 1
        for (int i = 0; i < kUnits; ++i) {
          fetch(f, 0);
          asm volatile("cp.async.wait_group %0;" ::"n"(kCkRing - 1) : "memory");
          uint32_t x[4], sw;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                       : "r"(ring + slot * 2048)
                       : "memory");
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(sw) : "r"(ring_s + slot * 512) : "memory");
          slot = slot == kCkRing - 1 ? 0 : slot + 1;
          uint32_t ss = prmt(sw, 0u, pick);
          if ((ss & 0x7FFFu) > 0x6C00u) {  // above 4096: a product may pass 65504; or not a number
            const int key = wk.key_of(j, (IS_K ? rank * 4 : 0) + ((kg + i * kSpan) >> 1)) + in16();
            if (!any_visible(key, wk.p0, wk.p1, wk.window, wk.sinks)) ss = 0;
            else if ((ss & 0x7C00u) != 0x7C00u) sm.over = 1;
            else if (edge && ck_note(sm, wk, key, (tid >> 3) % kC)) ss = 0;
          }
          __half2 s2 = u32_as_h2(ss);
          if (big) s2 = __hmul2(s2, __float2half2_rn(kCkBigUnit));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t o[4];
            ck_decode8<FMT>(x[k], s2, o);
            ck_sts(at + k * kStepWord, o[0], o[1], o[2], o[3]);
          }
          at += kStepUnit;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[J & 1]);
      }
    }
  }
};

// ---------------------------------------------------------------- the kernel

template <int FMT, int D>
__global__ void __launch_bounds__(kCkThreads, 1) attn_chunk_kernel(const __grid_constant__ SeqAttnArgs a) {
  constexpr int NG = D / 32;
  constexpr bool kBf = FMT == kCkBf16;
  extern __shared__ uint8_t smem_raw[];
  CkSmem<D>& sm = *reinterpret_cast<CkSmem<D>*>(smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = static_cast<int>(pair_rank());
  // One sequence: a KV head after another, so that whoever runs reads the same keys (4096 rows
  // at 16384 1409 us, the heads side by side 1428).  Several: every block's heads side by side,
  // so that no long block begins late (five ragged chunks: 10 us of 457 less than head after head).
  const int kv_heads = a.c.num_kv_heads, item = blockIdx.x >> 1, items = gridDim.x >> 1;
  const int kvh = a.num_seqs == 1 ? item / (items / kv_heads) : item % kv_heads, grp = a.group, qpb = 128 / grp;
  pdl_wait();

  // ---------------- which rows: blocks of 2 qpb positions, sequence by sequence, the last
  // (longest) of a sequence first
  if (warp == 0) {
    const int want = a.num_seqs == 1 ? item % (items / kv_heads) : item / kv_heads;
    const bool report = blockIdx.x == 0 && blockIdx.z == 0;
    int seq = -1, block = 0, before = 0;
    for (int b0 = 0; b0 < a.num_seqs && (seq < 0 || report); b0 += 32) {
      int mine = 0;
      SeqRows r{};
      if (b0 + lane < a.num_seqs) {
        r = seq_rows(a, b0 + lane);
        if (report && r.state != kRowsOk) set_status(a.status, KVQ_DEV_BAD_LENGTH);
        mine = (r.n + 2 * qpb - 1) / (2 * qpb);
      }
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, before + upto > want);
      if (seq < 0 && over != 0) {
        const int l = __ffs(over) - 1;
        const int last = before + __shfl_sync(0xffffffffu, upto, l) - 1;
        seq = b0 + l;
        block = last - want;
        if (lane == l) sm.rows_of = r;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) sm.seq = seq, sm.block = block;
  }
  if (threadIdx.x < 128) sm.row_top[threadIdx.x] = 0;
  if (threadIdx.x >= 128 && threadIdx.x < 128 + kCkNotes / 8) sm.noted[threadIdx.x - 128] = 0;
  if (threadIdx.x == 32) {
    for (int h = 0; h < 2; ++h) {
      mbar_init(&sm.k_ready[h], rank == 0 ? 5 : 4);
      mbar_init(&sm.v_ready[h], rank == 0 ? 5 : 4);
      mbar_init(&sm.p_ready[h], rank == 0 ? 5 : 4);
      mbar_init(&sm.k_free[h], 1);
      mbar_init(&sm.s_full[h], 1);
      mbar_init(&sm.pv_done[h], 1);
    }
    mbar_init(&sm.drained, 1);
    mbar_init(&sm.q_ready, rank == 0 ? 17 : 16);
    sm.abort = 0;
    sm.any_noted = 0;
    sm.over = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int seq = sm.seq;
  if (seq < 0) {  // more blocks than there are (the grid is sized by a bound)
    pdl_trigger();
    return;
  }
  const SeqRows sr = sm.rows_of;
  const int base = sr.T - sr.n;
  const int ib = sm.block * 2 * qpb, i0 = ib + rank * qpb;  // the pair's, this CTA's first row
  const int my_rows = max(0, min(qpb, sr.n - i0)) * grp;
  if (sr.state == kRowsNan) {
    pdl_trigger();
    if (blockIdx.z == 0)
      for (int i = threadIdx.x; i < my_rows * D; i += kCkThreads) {
        const int r = i / D;
        seq_store(a, sr.first + i0 + r / grp, kvh * grp + r % grp, i % D, NAN);
      }
    return;
  }
  CkWalk wk;
  wk.p0 = base + ib;
  wk.p1 = base + min(sr.n, ib + 2 * qpb) - 1;
  wk.window = a.window;
  wk.sinks = a.sinks;
  wk.kb = KeyBlocks{0, 0, 0};
  if (wk.p1 >= 0) wk.kb = key_blocks(wk.p0, wk.p1, a.window, a.sinks);
  const int all_tiles = (wk.kb.count + 7) / 8;
  wk.tile0 = static_cast<int>(static_cast<int64_t>(all_tiles) * blockIdx.z / gridDim.z);
  wk.tiles = static_cast<int>(static_cast<int64_t>(all_tiles) * (blockIdx.z + 1) / gridDim.z) - wk.tile0;
  wk.find_plain();
  const int nt = wk.tiles;

  if (warp == 1) pair_tmem_alloc(&sm.tmem_base, 512);

  tc_fence_before();
  __syncwarp();
  pair_arrive_all();  // both CTAs' barriers and tensor memory (waited for behind the queries)

  // ---------------- the decoders' first loads, ahead of the queries
  CkFetch fetch{};
  if (warp >= 12) fetch = CkPart<FMT, D, false>{a, sm, wk, kvh, rank, static_cast<int>(threadIdx.x & 127)}.begin(0);
  else if (warp >= 8) fetch = CkPart<FMT, D, true>{a, sm, wk, kvh, rank, static_cast<int>(threadIdx.x & 127)}.begin(0);

  // ---------------- queries: into the cache's space, scaled, fp16 (bf16 rows: bf16).  A thread
  // has a row's group of 32 (two of them at 256 wide), which it rotates in registers; eight
  // lanes write a core matrix.  The scale is a row's power of two that takes a bound of its
  // values to 2^14 .. 2^15: rotated ones are at most sqrt(32) times the row's largest.
  // (TQ4, whose rotation spans the row: eight rows a warp, four lanes a row.)
  {
    // the power of two that takes a bound `top` to 2^14 .. 2^15; NaN and infinities stay
    auto scale_for = [](float top) {
      int ex = 0;
      if (top > 0.f && top < INFINITY) ex = 14 - (static_cast<int>(__float_as_uint(fmaxf(top, 1e-30f)) >> 23) - 127);
      return __uint_as_float(static_cast<uint32_t>(max(min(ex, 110), -110) + 127) << 23);
    };
    // (the factor of a row's scores is not negative: the maximum is taken before it)
    const float sign = a.qscale < 0.f ? -1.f : 1.f;
    auto q_at = [&](int r) {
      return static_cast<int64_t>(sr.first + i0 + r / grp) * a.q.ts + static_cast<int64_t>(kvh * grp + r % grp) * a.q.hs;
    };
    auto pack = [&](const float* x, float by, uint32_t at) {  // eight values of a row
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float lo = x[ck_elem<FMT>(2 * i)] * by, hi = x[ck_elem<FMT>(2 * i + 1)] * by;
        w[i] = kBf ? pack_bf16(lo, hi) : pack_half2(lo, hi);
      }
      ck_sts(at, w[0], w[1], w[2], w[3]);
    };
    if constexpr (FMT == kCkTq4) {
      const int r = 8 * warp + (lane & 7);
      float x[NG][8];
      seq_load_row<NG>(a.q, r < my_rows ? q_at(r) + 8 * (lane >> 3) : -1, x);
      seq_turn<NG, true>(x, static_cast<const uint32_t*>(a.c.signs), lane, false);
      float top = 0.f;
#pragma unroll
      for (int G = 0; G < NG; ++G)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[G][e]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      const float up = scale_for(top);
      const uint32_t dst = smem_u32(sm.op.q) + warp * 16 * D + (lane & 7) * 16 + (lane >> 3) * 128;
#pragma unroll
      for (int G = 0; G < NG; ++G) pack(x[G], up * sign, dst + 512 * G);
      if (lane < 8) sm.factor[r] = fmaxf(fabsf(a.qscale) / up, 1e-37f);
    } else {
      const int r = 32 * (warp & 3) + lane;
      const bool rot = a.c.format == KVQ_FMT_Q4_HAD32;
      constexpr int kMine = NG >= 4 ? NG / 4 : 1;
      float x[kMine][4][8];
      float top = 0.f;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int G = (warp >> 2) + 4 * k;
        const bool on = r < my_rows && G < NG;
        seq_load_32(a.q, on ? q_at(r) + 32 * G : -1, x[k]);
#pragma unroll
        for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(x[k][i >> 3][i & 7]));
      }
      float up = 1.f;
      if constexpr (!kBf) {
        atomicMax(&sm.row_top[r], __float_as_uint(top));  // (not negative: ordered as its bits)
        __syncthreads();
        top = __uint_as_float(sm.row_top[r]);
        up = scale_for(rot ? top * 5.65685424949238f : top);
      }
      const uint32_t dst = smem_u32(sm.op.q) + (r >> 3) * 16 * D + (r & 7) * 16;
#pragma unroll
      for (int k = 0; k < kMine; ++k) {
        const int G = (warp >> 2) + 4 * k;
        if (G >= NG) continue;
        if (rot) seq_turn_32(x[k]);
        const float by = up * sign * (rot ? kHadamardScale : 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) pack(x[k][i], by, dst + (4 * G + i) * 128);
      }
      if (warp < 4) sm.factor[r] = fmaxf(fabsf(a.qscale) / up, 1e-37f);
    }
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.q_ready);
  }

  pair_wait_all();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;
  const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;

  bool big = false;  // the second pass
  int first = 0;
#pragma unroll 1
  for (;;) {
    if (warp < 4) {
      // ---------------- products
      if (warp == 0 && rank == 0 && lane == 0) {
        constexpr uint32_t id_qk = pair_idesc(kBf, false, 256, kCkTile), id_pv = pair_idesc(kBf, true, 256, D);
        const uint64_t dq = umma_desc(smem_u32(sm.op.q), 128, 16 * D);
        const uint64_t dk[2] = {umma_desc(smem_u32(sm.op.k[0]), 128, 16 * D), umma_desc(smem_u32(sm.op.k[1]), 128, 16 * D)};
        const uint64_t dv[2] = {umma_desc(smem_u32(sm.op.v[0]), 128, 2048), umma_desc(smem_u32(sm.op.v[1]), 128, 2048)};
        const bool ok = ck_wait<true>(sm, &sm.q_ready, 0, a.status);
        for (int j = 0; j <= nt && ok; ++j) {
          if (j < nt) {
            const int J = first + j, b = J & 1;
            if (!ck_wait<true>(sm, &sm.k_ready[b], (J >> 1) & 1, a.status)) break;
            tc_fence_after();
            const uint32_t s = tbase + kCkS + 128 * b;
#pragma unroll
            for (int st = 0; st < D / 16; ++st) pair_umma_ss(s, dq + 16 * st, dk[b] + 16 * st, id_qk, st > 0 ? 1u : 0u);
            pair_commit(&sm.k_free[b]);
            pair_commit(&sm.s_full[b]);
          }
          if (j >= 1) {
            const int jp = j - 1, J = first + jp, b = J & 1;
            if (!ck_wait<true>(sm, &sm.v_ready[b], (J >> 1) & 1, a.status)) break;
            if (!ck_wait<true>(sm, &sm.p_ready[b], (J >> 1) & 1, a.status)) break;
            tc_fence_after();
            const uint32_t p = tbase + kCkS + 128 * b;
#pragma unroll
            for (int st = 0; st < kCkTile / 16; ++st)
              pair_umma_ts(tbase + kCkO, p + 8 * st, dv[b] + 16 * st, id_pv, jp > 0 || st > 0 ? 1u : 0u);
            pair_commit(&sm.pv_done[b]);
          }
        }
        // every product issued has finished before the operands and the tensor memory go
        // (bounded, and independent of the abort flag)
        pair_commit(&sm.drained);
        const uint64_t t0 = global_timer_ns();
        while (!pair_try_wait(&sm.drained, big ? 1 : 0)) {
          if (global_timer_ns() - t0 > 2000000000ull) {
            atomicExch(&sm.abort, 1);
            set_status(a.status, KVQ_DEV_TIMEOUT);
            break;
          }
        }
      } else if (warp > 0 && rank == 1 && lane == 0) {
        // ---------------- the second CTA's operands, announced to the first by a thread with
        // nothing else in flight (a release to the cluster waits for all that its thread has)
        uint64_t* const mine = warp == 1 ? sm.k_ready : warp == 2 ? sm.v_ready : sm.p_ready;
        if (warp == 1 && !big && ck_wait(sm, &sm.q_ready, 0, a.status)) pair_arrive(pair_addr(&sm.q_ready, 0));
        for (int j = 0; j < nt; ++j) {
          const int J = first + j;
          if (!ck_wait(sm, &mine[J & 1], (J >> 1) & 1, a.status)) break;
          pair_arrive(pair_addr(&mine[J & 1], 0));
        }
      }
    } else if (warp < 8) {
      // ---------------- softmax, one row a thread
      const int r = 32 * (warp & 3) + lane;
      const int p = r < my_rows ? base + i0 + r / grp : -kNoKey;
      ck_wait_warp(sm, &sm.q_ready, 0, a.status);  // (the factors)
      const float f_all = sm.factor[r] * (big ? 1.f / kCkBigUnit : 1.f);
      float f = f_all;
      float m_run = -INFINITY, z = 0.f;
      for (int j = 0; j < nt; ++j) {
        const int J = first + j, b = J & 1;
        if (!ck_wait_warp(sm, &sm.s_full[b], (J >> 1) & 1, a.status)) break;
        tc_fence_after();
        const uint32_t s_at = tbase + lane_off + kCkS + 128 * b;
        const bool edge = wk.edge(j);
        uint32_t seen[4] = {~0u, ~0u, ~0u, ~0u};  // of the tile's keys
        if (edge) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int key = wk.key_of(j, k);
            auto below = [](int n) { return n <= 0 ? 0u : n >= 16 ? 0xFFFFu : (1u << n) - 1u; };
            uint32_t bits = below(p - key + 1);
            if (a.window > 0) bits &= ~below(p - a.window - key + 1) | below(a.sinks - key);
            seen[k >> 1] = (seen[k >> 1] & (k & 1 ? 0x0000FFFFu : 0xFFFF0000u)) | bits << (16 * (k & 1));
          }
        }
        auto load = [&](int cc, uint32_t (&v)[32]) {  // 32 of the tile's scores
          tmem_ld32(s_at + 32 * cc, v);
          tmem_wait_ld();
          if (edge) {
            const uint32_t on = cc == 0 ? seen[0] : cc == 1 ? seen[1] : cc == 2 ? seen[2] : seen[3];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((on >> i) & 1u)) v[i] = 0xFF800000u;
          }
        };
        float t4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t v[32];
          load(cc, v);
#pragma unroll
          for (int i = 0; i < 32; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) t4[k] = ck_max3(t4[k], __uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
        }
        float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
        if (top != -INFINITY) top *= f;
        // the reference is raised only when a row's scores passed it by more (base 2)
        const bool raise = top - m_run > kCkRaise;
        float corr = 1.f;
        if (raise) {
          corr = m_run == -INFINITY ? 1.f : fast_exp2(m_run - top);  // (z and the context are zero until then)
          z *= corr;
          m_run = top;
          if (fabsf(top) > kFarScore || f != f_all) {  // the row's scores from here on in other units
            m_run = top * (f_all / f);
            f = f_all;
            if (fabsf(m_run) > kFarScore) {
              f *= kFarScore / fabsf(m_run);
              m_run = copysignf(kFarScore, m_run);
            }
          }
        }
        const float mu = m_run == -INFINITY ? 0.f : m_run - (kBf ? 0.f : kCkHead);
        if (j > 0 && __any_sync(0xffffffffu, raise && corr != 1.f)) {
          if (!ck_wait_warp(sm, &sm.pv_done[(J - 1) & 1], ((J - 1) >> 1) & 1, a.status)) break;
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t o[16];
            tmem_ld16(tbase + lane_off + kCkO + 16 * cc, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            tmem_st16(tbase + lane_off + kCkO + 16 * cc, o);
          }
          tmem_wait_st();
        }
        const uint64_t f2 = pk2(f, f), mu2 = pk2(-mu, -mu);
        uint64_t z2[2] = {0, 0};
        // p of 32 keys goes to 16 columns whose scores have been read
#pragma unroll 2
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t v[32], pk[16];
          load(cc, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float e0, e1;
            upk2(fma2(pk2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, mu2), e0, e1);
            e0 = fast_exp2(e0);
            e1 = fast_exp2(e1);
            z2[i & 1] = add2(z2[i & 1], pk2(e0, e1));
            pk[i] = kBf ? pack_bf16(e0, e1) : pack_half2(e0, e1);
          }
          tmem_st16(s_at + 16 * cc, pk);
        }
        {
          float e0, e1;
          upk2(add2(z2[0], z2[1]), e0, e1);
          z += e0 + e1;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready[b]);
      }
      sm.m[r] = m_run == -INFINITY ? m_run : m_run * (f_all / f);
      sm.z[r] = z;
      const int last = first + nt - 1;
      if (nt > 0) ck_wait_warp(sm, &sm.pv_done[last & 1], (last >> 1) & 1, a.status);
    } else {
      if (warp < 12) {
        const CkPart<FMT, D, true> part{a, sm, wk, kvh, rank, static_cast<int>(threadIdx.x & 127)};
        if (big) fetch = part.begin(first);
        part.run(fetch, big);
      } else {
        const CkPart<FMT, D, false> part{a, sm, wk, kvh, rank, static_cast<int>(threadIdx.x & 127)};
        if (big) fetch = part.begin(first);
        part.run(fetch, big);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");  // (those behind the last tile's, or behind a wait that gave up)
    }
    // Both CTAs are done: every product has finished (the softmax warps waited for the last).
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    pair_sync();
    tc_fence_after();
    if constexpr (!kBf) {
      if (big) break;
      big = (pair_ld_u32(pair_addr(&sm.over, 0)) | pair_ld_u32(pair_addr(&sm.over, 1))) != 0;
      if (!big) break;
      first = nt;
      if (threadIdx.x < kCkNotes / 8) sm.noted[threadIdx.x] = 0;
      if (threadIdx.x == 0) sm.any_noted = 0;
      pair_sync();
    } else {
      break;
    }
  }

  // ---------------- the rows: out of tensor memory, over the operands, rotated back, stored
  const int ranges = gridDim.z;
  const uint32_t noted = pair_ld_u32(pair_addr(&sm.any_noted, 0)) | pair_ld_u32(pair_addr(&sm.any_noted, 1));
  // A thread takes a row's groups of 32 out of tensor memory, rotates them back and stores
  // them.  Over the operands and eight rows a warp where a rotation spans the row (TQ4) or
  // some value is not a number.
  const bool staged = (FMT == kCkTq4 && ranges == 1) || noted != 0;
  {
    const int r = 32 * (warp & 3) + lane, row = sr.first + i0 + r / grp, head = kvh * grp + r % grp;
    const bool live = r < my_rows, rot = a.c.format == KVQ_FMT_Q4_HAD32 && ranges == 1;
    const float zr = sm.z[r];
    const float unit = big ? 1.f / kCkBigUnit : 1.f;
    const bool failed = (pair_ld_u32(pair_addr(&sm.abort, 0)) | pair_ld_u32(pair_addr(&sm.abort, 1))) != 0;
    const float inv = failed ? NAN : ranges > 1 ? unit : zr == 0.f ? 0.f : unit / zr;
    const int64_t part = (static_cast<int64_t>(blockIdx.z) * a.n_rows + row) * a.Hq + head;
    if (ranges > 1 && live && warp < 4) a.ws_m[part] = sm.m[r], a.ws_z[part] = zr;
#pragma unroll 1
    for (int G = warp >> 2; G < NG; G += 4) {
      uint32_t o[32];
      __syncwarp();
      if (nt > 0) {
        tmem_ld32(tbase + lane_off + kCkO + 32 * G, o);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = 0;
      }
      float x[4][8];
      const float by = inv * (rot ? kHadamardScale : 1.f);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i >> 3][ck_elem<FMT>(i & 7)] = __uint_as_float(o[i]) * by;
      if (staged) {
#pragma unroll
        for (int i = 0; i < 32; ++i) sm.out[r][32 * G + i] = x[i >> 3][i & 7];
        continue;
      }
      if (rot) seq_turn_32(x);
      if (!live) continue;
      if (ranges > 1) seq_store_32(a.ws_acc + part * D + 32 * G, KVQ_DT_F32, true, x);
      else
        seq_store_32(element_at(a.out, static_cast<int64_t>(row) * a.out.ts + static_cast<int64_t>(head) * a.out.hs + 32 * G),
                     a.out.dtype, a.out.wide, x);
    }
  }
  tc_fence_before();
  if (staged) {
    __syncthreads();
    // values that are not numbers, into the rows that see their keys
    for (int other = 0; other < 2; ++other) {
      if (pair_ld_u32(pair_addr(&sm.any_noted, other)) == 0) continue;
      for (int r = threadIdx.x; r < my_rows; r += kCkThreads) {
        const int p = base + i0 + r / grp;
        for (int i8 = 0; i8 < kCkNotes / 8; ++i8)
          for (uint32_t left = pair_ld_u32(pair_addr(&sm.noted[i8], other)); left != 0;) {
            const int sub = (__ffs(left) - 1) >> 2, i = 8 * i8 + sub;
            const uint32_t which = (left >> (4 * sub)) & 15u;
            left &= ~(15u << (4 * sub));
            if (!key_visible(wk.key_of_note(i), p, a.window, a.sinks)) continue;
            if constexpr (kBf) {
              // the value's elements, from the cache again (its page is a good one: it was read)
              const int key = wk.key_of_note(i), pg = static_cast<int>(fast_div(static_cast<uint32_t>(key >> 4), a.page_blocks));
              const int page = a.block_tables[static_cast<int64_t>(seq) * a.max_pages + pg];
              const int64_t at = (static_cast<int64_t>(page) * kv_heads + kvh) * a.c.page_size + (key - pg * a.c.page_size);
              const uint16_t* v = static_cast<const uint16_t*>(a.c.v) + at * D + other * (D / 2);
              for (int e = 0; e < D / 2; ++e) {
                const uint32_t x = v[e];
                if (ck_not_finite16(x)) sm.out[r][other * (D / 2) + e] += __uint_as_float(x << 16);
              }
            } else {
              for (int k = 0; k < (NG + 1) / 2; ++k)
                if ((which >> k) & 1u)
                  for (int e = 0; e < 32; ++e) sm.out[r][(other * (NG / 2) + k) * 32 + e] = NAN;
            }
          }
      }
    }
    __syncthreads();
    {
      const int r = 8 * warp + (lane & 7);  // (rows behind the last are zeros, or of no consequence)
      const int row = sr.first + i0 + r / grp, head = kvh * grp + r % grp;
      const bool live = r < my_rows;
      const int64_t out_at = static_cast<int64_t>(row) * a.out.ts + static_cast<int64_t>(head) * a.out.hs + 8 * (lane >> 3);
      const int64_t part = (static_cast<int64_t>(blockIdx.z) * a.n_rows + row) * a.Hq + head;
      auto get = [&](int G, float(&x)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = sm.out[r][32 * G + 8 * (lane >> 3) + e];
      };
      auto put = [&](int G, const float(&x)[8]) {
        if (!live) return;
        if (ranges > 1) {
          st_words<8>(a.ws_acc + part * D + 32 * G + 8 * (lane >> 3), reinterpret_cast<const uint32_t*>(x));
        } else if (a.out.dtype == KVQ_DT_F32) {
          float* p = static_cast<float*>(a.out.data) + out_at + 32 * G;
          if (a.out.wide) {
            st_words<8>(p, reinterpret_cast<const uint32_t*>(x));
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = x[e];
          }
        } else {
          __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.out.data) + out_at + 32 * G;
          if (a.out.wide) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
            st_words<4>(p, w);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = __float2bfloat16_rn(x[e]);
          }
        }
      };
      if (8 * warp < my_rows) {
        if (FMT == kCkTq4 && ranges == 1) {
          float x[NG][8];
#pragma unroll
          for (int G = 0; G < NG; ++G) get(G, x[G]);
          seq_turn<NG, true>(x, static_cast<const uint32_t*>(a.c.signs), lane, true);
#pragma unroll
          for (int G = 0; G < NG; ++G) put(G, x[G]);
        } else {
          const bool rot = ranges == 1 && a.c.format == KVQ_FMT_Q4_HAD32;
#pragma unroll 2
          for (int G = 0; G < NG; ++G) {
            float x[1][8];
            get(G, x[0]);
            if (rot) seq_turn<1, false, false>(x, nullptr, lane, true);
            put(G, x[0]);
          }
        }
      }
    }
  }
  pair_sync();  // (its notes are read until here, and its tensor memory)
  if (warp == 1) pair_tmem_dealloc(tbase, 512);
}

// The pairs of CTAs of a call, by a bound: sequences' blocks are whole.
int64_t chunk_blocks(int n_rows, int num_seqs, int max_rows, int group) {
  const int64_t per = 2 * (128 / group);
  return std::min<int64_t>((max_rows + per - 1) / per * num_seqs, n_rows / per + num_seqs);
}

// The partials (of a row and head) that no call passes: ranges x pairs is at most what runs at
// once, and a pair has up to 256 rows.
int64_t chunk_partials(int n_sm) { return static_cast<int64_t>(std::max(1, n_sm / 2)) * 256; }

int chunk_ranges(const kvq_cache& c, int n_rows, int num_seqs, int Hq, int max_rows, int max_seq_len, int window, int sinks,
                 int n_sm) {
  const int group = Hq / c.num_kv_heads;
  const int64_t items = chunk_blocks(n_rows, num_seqs, max_rows, group) * c.num_kv_heads;
  int64_t keys = max_seq_len;
  if (window > 0) keys = std::min<int64_t>(keys, static_cast<int64_t>(window) + sinks + std::min(max_rows, 256 / group) + 32);
  const int64_t tiles = (keys + kCkTile - 1) / kCkTile;
  const int64_t pairs = std::max(1, n_sm / 2);
  if (items <= 0 || 2 * items > pairs) return 1;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(pairs / items, tiles / 4), 32)));
}

template <int FMT, int D>
static cudaError_t launch_chunk(const SeqAttnArgs& a, int ranges, cudaStream_t s) {
  constexpr auto kern = attn_chunk_kernel<FMT, D>;
  constexpr size_t smem = std::max(sizeof(CkSmem<D>) + 1024, kCkMinSmem);
  static_assert(smem <= 232448, "shared memory");
  cudaError_t e = set_max_smem_once<kern>(static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * chunk_blocks(a.n_rows, a.num_seqs, a.max_rows, a.group) * a.c.num_kv_heads),
                     1, ranges);
  cfg.blockDim = dim3(kCkThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || ranges == 1) return e;
  return launch_attn_merge(a, ranges, s);
}

template <int FMT>
static cudaError_t launch_chunk_dim(const SeqAttnArgs& a, int ranges, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch_chunk<FMT, 64>(a, ranges, s);
    case 128: return launch_chunk<FMT, 128>(a, ranges, s);
    default: return launch_chunk<FMT, 256>(a, ranges, s);
  }
}

cudaError_t launch_attn_chunk(const SeqAttnArgs& a, int ranges, cudaStream_t s) {
  if (a.num_seqs == 0 || a.n_rows == 0 || a.max_rows == 0) return cudaSuccess;
  if (a.c.format == KVQ_FMT_BF16) return launch_chunk_dim<kCkBf16>(a, ranges, s);
  if (a.c.format == KVQ_FMT_TQ4) return launch_chunk_dim<kCkTq4>(a, ranges, s);
  return launch_chunk_dim<kCkQ4>(a, ranges, s);
}

}  // namespace kvq
