// norm_rope.cu -- norms of queries and keys per head and rotary positions in one
// pass, alone or on the way into the cache: queries rotated into the cache's
// space, keys and values quantised and stored, in one launch.
//
// The stored rows follow the formats' definitions in kvq.h ("KV cache
// quantization: fp8 (KV8) + 4-bit TurboQuant", KV8 base commit: the producer
// quantises the fresh normed and roped row; "qwen27 CUDA: an opt-in 4-bit
// attention cache (262K on a 24 GB card)", section "What it is").
//
// The arithmetic per row, in fp32:
//   y = x * r * (w + offset), r = rsqrt(mean(x^2) + eps)
//   (a, b) -> (a cos - b sin, b cos + a sin) for every rotary pair.
// The angles and their use are in rope.cuh.
//
// A lane holds 16 consecutive elements of a row (32 bytes of bf16, one load), so a
// row of 256 lies over 16 lanes and a warp works on two heads of its token at once
// (D = 64, 128, 512: eight, four, one); with a row over the whole warp, 8 elements
// to a lane, a row took 183 instructions (now 92) and 4099 tokens of 24 heads
// 24.7 us, since the reductions, the butterflies across lanes and the addressing
// were shared by fewer rows.  The angles (the same for every head) are worked out
// once per token and warp, spread over its lanes, and read back from shared memory.
//
// Bound (times of calls in a graph).  4099 x 24 heads of 256, bf16 to bf16 with norm
// and three axes: 19.1 us, 101 MB, 5.3 TB/s (78 % of the measured copy; the same kernel
// without norm and rotation takes as long, so what is left is filling and draining the
// memory pipe).  4096 tokens of 24 + 4 + 4 heads to rotated fp32 queries and 4-bit rows:
// 34.2 us, 172 MB, 5.0 TB/s (Q4_0 rows 32.2, bf16 rows 33.0 us, floors 25.5 and 27.3);
// 31 us without the norm, the rotations and the codes' arithmetic.  The rest is latency at
// 16 warps an SM: 20.2 M instructions leave half the issue slots empty, waiting for
// shared memory and the shuffles.  TQ4 rows 49.5 us: four of their eight butterfly
// stages go across lanes, 64 shuffles a row, and the kernels of one type spill 52 to 68
// bytes a thread.  One token: the launch.
// Measured and not kept (the 4096-token chunk with its read-back, then 41.7 us): K and V
// rows two batches side by side like the queries' 47.3 us, one batch at 80 registers
// and 24 warps an SM 49.7 us, five CTAs of four warps at 96 registers 51.4 us.
//
// This translation unit is compiled with -fmad=false.
#include "rope.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

constexpr int kNoStore = -1;
constexpr int E = kRopeE;  // elements of a lane
constexpr int kMaxWarps = 4, kMinCtas = 4;  // of a CTA, and CTAs of an SM (128 registers)
// What a kernel is made for: whole vectors of one input and one output type, or
// (kAny) whatever the views say.
enum Mode { kAny, kBf16ToBf16, kBf16ToF32, kF32ToF32 };

// FMT: the cache's format, or kNoStore for rows that are only normed and rotated
// (then every head is a "query" and Hk is 0).  LPR: lanes of a row.  Bf16 queries go
// by two batches side by side (U), so that one's shuffles are in flight during the
// other's arithmetic.  All tokens' batches in one line are cut into equal ranges, one
// for each warp (a.per batches): no warp waits for another's last token, and a warp
// works out the angles of the few tokens that its range touches.  The next token's
// positions, slot and first rows are loaded during a token's last batches.
// FEW (rows that are only normed and rotated, few heads): a batch is one head of RPW
// tokens next to one another instead, each with its own angles ("token" then stands
// for such a group).
template <int LPR, int FMT, int MODE, bool FEW>
__global__ void __launch_bounds__(32 * kMaxWarps, kMinCtas) norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kTokenChunks = FEW ? E * LPR / 4 + E * LPR / 32 : kChunks;  // of a copy of a token's angles
  __shared__ float4 angles_sh[kMaxWarps][(FEW ? 32 / LPR : 1) * 2 * kTokenChunks];
  pdl_wait();
  pdl_trigger();
  constexpr int D = E * LPR, RPW = 32 / LPR;
  constexpr bool BF = MODE == kBf16ToBf16 || MODE == kBf16ToF32;
  constexpr int U = BF && !FEW ? 2 : 1;
  const int lane = threadIdx.x & 31, warp = warp_index(), l = lane % LPR, sub = lane / LPR;
  // a token's batches of RPW heads: first the queries', then K's, then V's
  const int qb = FEW ? a.Hq : (a.Hq + RPW - 1) / RPW, kb = (a.Hk + RPW - 1) / RPW, total = qb + 2 * kb;
  const int64_t all = (FEW ? (a.n_tok + RPW - 1) / RPW : a.n_tok) * total;
  int64_t left = ((int64_t)blockIdx.x * (blockDim.x >> 5) + warp) * a.per;  // this warp's first batch
  if (left >= all) return;
  int64_t tok = left / total;
  int b0 = static_cast<int>(left - tok * total);
  left = all - left < a.per ? all - left : a.per;  // its batches

  const auto in_type = [&](const RowsView& v) { return MODE == kAny ? v.dtype : BF ? KVQ_DT_BF16 : KVQ_DT_F32; };
  const auto wide = [&](const RowsView& v) { return MODE == kAny ? v.wide : 1; };
  const int out_type = MODE == kAny ? a.qo.dtype : MODE == kBf16ToBf16 ? KVQ_DT_BF16 : KVQ_DT_F32;
  const auto query = [&](int b) { return FEW ? b : b * RPW + sub; };  // the lane's head of a batch
  const auto token = [&](int64_t t) { return FEW ? t * RPW + sub : t; };
  const auto live = [&](int64_t t, int b) { return FEW ? token(t) < a.n_tok : query(b) < a.Hq; };
  // address of the lane's part of head h's row, and bytes from a batch of queries to the next
  const auto row_of = [&](const RowsView& v, int type, int64_t t, int h) {
    return static_cast<uint8_t*>(v.data) + ((t * v.ts + h * v.hs + E * l) << (type == KVQ_DT_BF16 ? 1 : 2));
  };
  const int64_t step = (a.q.hs * (FEW ? 1 : RPW)) << (in_type(a.q) == KVQ_DT_BF16 ? 1 : 2);
  const int64_t out_step = (a.qo.hs * (FEW ? 1 : RPW)) << (out_type == KVQ_DT_BF16 ? 1 : 2);

  RawRow<E, BF> next[U];  // the rows after those being worked on
  const uint8_t* at;      // the first one's address in this lane
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < (BF ? E / 2 : E); ++i) next[u].w[i] = 0;
  const auto load_kv = [&](int64_t t, int b) {
    const bool is_v = b >= qb + kb;
    const int h = (is_v ? b - qb - kb : b - qb) * RPW + sub;
    const RowsView& v = is_v ? a.v : a.k;
    if (h < a.Hk) load_raw_at<E, BF>(row_of(v, in_type(v), t, h), in_type(v), wide(v), next[0]);
  };
  const auto load_q = [&](int64_t t, int b, int end) {  // U batches of queries from b on, before `end`, at `at`
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (b + u < end && live(t, b + u))
        load_raw_at<E, BF>(at + u * step, in_type(a.q), wide(a.q), next[u]);
  };
  int32_t pos[4] = {}, slot = -1;
  const auto first_rows = [&](int64_t t, int b, int end) {  // of token t's batches [b, end), with its positions and slot
    if (b < qb) {
      at = row_of(a.q, in_type(a.q), token(t), query(b));
      load_q(t, b, min(end, qb));
    } else if (FMT != kNoStore) {
      load_kv(t, b);
    }
    if (a.rope.rot != 0 && b < qb + kb && (!FEW || live(t, b))) load_pos(a.rope, token(t), pos);
    if (FMT != kNoStore && end > qb) slot = a.slots[t];
  };
  const auto end_of = [&](int b, int64_t n) { return static_cast<int>(n < total - b ? b + n : total); };
  int b1 = end_of(b0, left);
  first_rows(tok, b0, b1);

  RopeLane g;
  float4* const angles = angles_sh[warp] + (FEW ? sub * 2 * kTokenChunks : 0);
  if (a.rope.rot != 0) g = rope_lane<kTokenChunks>(a.rope, angles, lane, l);
  uint32_t sw = 0;
  if constexpr (FMT == KVQ_FMT_TQ4) sw = lane_signs<E>(a.c.signs, l);
  uint64_t w[E / 2];
  int weights = 0;  // whose they are: 1 the queries', 2 the keys'

  for (;;) {
    const int be = min(b1, qb);
    const bool stores = FMT != kNoStore && b1 > qb;
    const int64_t rest = left - (b1 - b0);  // batches of the tokens after this one
    const int nb1 = end_of(0, rest);
    if (a.rope.rot != 0 && b0 < qb + kb) make_angles<FEW ? LPR : 32, kTokenChunks>(a.rope, pos, FEW ? l : lane, a.status, angles);
    const int32_t this_slot = slot;
    if (b0 < qb) {
      if (a.qn.weight && weights != 1) load_weight<E>(a.qn, l, w), weights = 1;
      uint8_t* out = row_of(a.qo, out_type, token(tok), query(b0));
      for (int b = b0; b < be; b += U) {
        uint64_t x[U][E / 2];
#pragma unroll
        for (int u = 0; u < U; ++u) unpack_row<E, BF>(next[u], x[u]);
        if (b + U < be) {
          at += U * step;
          load_q(tok, b + U, be);
        } else if (stores) {
          load_kv(tok, qb);
        } else if (rest > 0) {
          first_rows(tok + 1, 0, nb1);
        }
        if (a.qn.weight) norm_rows<E, LPR, U>(x, w, a.qn.eps);
        if (a.rope.rot != 0) {
          if constexpr (FMT == kNoStore) {
            rope_rows<U>(a.rope, g, l, x);
          } else {  // one after the other: the partners of both would spill
#pragma unroll
            for (int u = 0; u < U; ++u) rope_rows<1>(a.rope, g, l, *reinterpret_cast<uint64_t(*)[1][E / 2]>(&x[u]));
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if constexpr (FMT == KVQ_FMT_Q4_HAD32) {
            if (a.rotate) rotate_row_had32<E>(x[u], lane);
          }
          if constexpr (FMT == KVQ_FMT_TQ4) {
            if (a.rotate) rotate_row_tq4<E, LPR>(x[u], sw, lane);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (b + u < be && live(tok, b + u)) write_row_at<E>(out + u * out_step, out_type, wide(a.qo), x[u]);
        out += U * out_step;
      }
    }
    if constexpr (FMT != kNoStore) {
      if (stores) {
        const bool in_pool = (int64_t)this_slot < (int64_t)a.c.num_pages * a.c.page_size, keep = this_slot >= 0 && in_pool;
        if (!in_pool && lane == 0) set_status(a.status, KVQ_DEV_BAD_SLOT);
        const uint32_t page = keep ? fast_div(static_cast<uint32_t>(this_slot), a.ps) : 0;
        const uint32_t off = static_cast<uint32_t>(this_slot) - page * a.ps.d;
        if (a.kn.weight && b0 < qb + kb && weights != 2) load_weight<E>(a.kn, l, w), weights = 2;
        for (int b = max(b0, qb); b < b1; ++b) {
          const bool is_v = b >= qb + kb;
          const int h = (is_v ? b - qb - kb : b - qb) * RPW + sub;
          const int64_t r = ((int64_t)page * a.Hk + h) * a.c.page_size + off;
          uint64_t x1[1][E / 2];
          uint64_t(&x)[E / 2] = x1[0];
          unpack_row<E, BF>(next[0], x);
          if (b + 1 < b1) load_kv(tok, b + 1);
          else if (rest > 0) first_rows(tok + 1, 0, nb1);
          if (!keep) continue;
          if (!is_v) {
            if (a.kn.weight) norm_rows<E, LPR, 1>(x1, w, a.kn.eps);
            if (a.rope.rot != 0) rope_rows<1>(a.rope, g, l, x1);
          }
          void* codes = is_v ? a.c.v : a.c.k;
          void* scales = is_v ? a.c.v_scale : a.c.k_scale;
          if constexpr (FMT == KVQ_FMT_BF16) {
            if (h < a.Hk)
              write_row_at<E>(static_cast<uint16_t*>(codes) + r * D + E * l, KVQ_DT_BF16, a.plane_wide, x);
          } else {
            __half s16;
            uint32_t word[2];
            if constexpr (FMT == KVQ_FMT_TQ4) {
              rotate_row_tq4<E, LPR>(x, sw, lane);
              float y[E];
#pragma unroll
              for (int i = 0; i < E / 2; ++i) upk2(x[i], y[2 * i], y[2 * i + 1]);
              tq4_row_codes<E, LPR>(y, word, s16);
              if (h < a.Hk && l == 0) static_cast<__half*>(scales)[r] = s16;
            } else {
              constexpr bool ROT = FMT == KVQ_FMT_Q4_HAD32;
              if constexpr (ROT) rotate_row_had32<E>(x, lane);
              q4_row_codes<E, ROT>(x, word, s16);
              if (h < a.Hk && l % (32 / E) == 0) static_cast<__half*>(scales)[r * (D / 32) + l / (32 / E)] = s16;
            }
            if (h < a.Hk) write_codes<E>(static_cast<uint8_t*>(codes) + r * (D / 2) + l * (E / 2), word);
          }
        }
      }
    }
    if (rest <= 0) break;
    ++tok;
    left = rest;
    b0 = 0;
    b1 = nb1;
  }
}

template <int LPR, int FMT, bool FEW>
cudaError_t launch_ranges(NormRopeArgs a, cudaStream_t s) {
  // One range of batches for each resident warp, one batch where there are fewer; and
  // CTAs of fewer warps where that leaves SMs without one.  (Rounded up to an even
  // number, for the pairs of query batches: 1001 fp32 tokens of 32 + 8 + 8 heads of 128
  // with their read-back 16.3 us instead of 15.0, 4096 tokens 41.5 instead of 40.9.)
  constexpr int RPW = 32 / LPR;
  const int64_t total = FEW ? a.Hq : (a.Hq + RPW - 1) / RPW + 2 * ((a.Hk + RPW - 1) / RPW);
  const int64_t n_sm = device_sm_count() > 0 ? device_sm_count() : 1;
  const int64_t resident = n_sm * kMinCtas * kMaxWarps, all_batches = (FEW ? (a.n_tok + RPW - 1) / RPW : a.n_tok) * total;
  const int64_t per = (all_batches + resident - 1) / resident;
  a.per = per;
  const int64_t warps = (all_batches + per - 1) / per;
  int wpc = kMaxWarps;
  while (wpc > 1 && warps < n_sm * wpc) wpc >>= 1;
  const dim3 grid(static_cast<unsigned>((warps + wpc - 1) / wpc)), block(32 * wpc);
  const bool kv = a.Hk > 0, q = a.Hq > 0;
  const bool whole = (!q || (a.q.wide && a.qo.wide)) && (!kv || (a.k.wide && a.v.wide));
  const auto all = [&](int t) { return (!q || a.q.dtype == t) && (!kv || (a.k.dtype == t && a.v.dtype == t)); };
  const bool out_f32 = !q || a.qo.dtype == KVQ_DT_F32;
  cudaError_t e;
  // One batch a warp: the kernel of any type, which takes it alone.  Two batches side by
  // side have nothing to overlap then and cost TQ4 rows their spills (100 tokens of 24 + 4
  // heads 4.5 us so, 5.4 us by type; bf16 rows 3.65 and 3.8 us; one token of 4-bit rows
  // 3.1 to 3.3 and 3.0 to 3.1 us).
  if (!whole || per == 1)
    e = launch_pdl(norm_rope_kernel<LPR, FMT, kAny, FEW>, grid, block, 0, s, a);
  else if (all(KVQ_DT_BF16))
    e = out_f32 ? launch_pdl(norm_rope_kernel<LPR, FMT, kBf16ToF32, FEW>, grid, block, 0, s, a)
                : launch_pdl(norm_rope_kernel<LPR, FMT, kBf16ToBf16, FEW>, grid, block, 0, s, a);
  else if (all(KVQ_DT_F32) && out_f32)
    e = launch_pdl(norm_rope_kernel<LPR, FMT, kF32ToF32, FEW>, grid, block, 0, s, a);
  else
    e = launch_pdl(norm_rope_kernel<LPR, FMT, kAny, FEW>, grid, block, 0, s, a);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

template <int LPR, int FMT>
cudaError_t launch_one(const NormRopeArgs& a, cudaStream_t s) {
  // Few heads: half a batch of one token's heads or more would be empty, and there are
  // more such batches than resident warps (one head of 128, 10336 tokens: 8.5 us so,
  // 13.2 us by tokens; one of 64, 16384 tokens: 5.3 and 12.8 us; below that many tokens
  // the angles are better spread over a whole warp).
  constexpr int RPW = 32 / LPR;
  if constexpr (FMT == kNoStore && RPW > 1)
    if (2 * a.Hq <= RPW && a.n_tok > (int64_t)device_sm_count() * kMinCtas * kMaxWarps)
      return launch_ranges<LPR, FMT, true>(a, s);
  return launch_ranges<LPR, FMT, false>(a, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, int width, int fmt, cudaStream_t s) {
#define KVQ_BY_FORMAT(L)                                                          \
  switch (fmt) {                                                                  \
    case kNoStore: return launch_one<L, kNoStore>(a, s);                          \
    case KVQ_FMT_Q4_HAD32: return launch_one<L, KVQ_FMT_Q4_HAD32>(a, s);          \
    case KVQ_FMT_Q4_0: return launch_one<L, KVQ_FMT_Q4_0>(a, s);                  \
    case KVQ_FMT_TQ4: return launch_one<L, KVQ_FMT_TQ4>(a, s);                    \
    case KVQ_FMT_BF16: return launch_one<L, KVQ_FMT_BF16>(a, s);                  \
    default: return cudaErrorInvalidValue;                                        \
  }
  switch (width) {
    case 64: KVQ_BY_FORMAT(4)
    case 128: KVQ_BY_FORMAT(8)
    case 256: KVQ_BY_FORMAT(16)
    case 512:
      if (fmt == kNoStore) return launch_one<32, kNoStore>(a, s);
      if (fmt == KVQ_FMT_BF16) return launch_one<32, KVQ_FMT_BF16>(a, s);
      return cudaErrorInvalidValue;
    default: return cudaErrorInvalidValue;
  }
#undef KVQ_BY_FORMAT
}

}  // namespace kvq
