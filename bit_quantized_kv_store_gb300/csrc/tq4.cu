// tq4.cu -- the TQ4 rows: store (randomized Hadamard over the row, Lloyd-Max
// codebook at radius / sqrt(n)) and the signed row rotation of queries and
// outputs.
//
// Follows "KV cache quantization: fp8 (KV8) + 4-bit TurboQuant", PR body, "Why
// rotated-int4": a randomized-Hadamard rotation makes the coordinates of a row
// close to Gaussian and keeps its radius, so a fixed 16-level Lloyd-Max
// codebook for N(0,1), scaled by radius / sqrt(n), quantizes every coordinate
// with one scale per row.
//
// One warp per row; lane l holds elements E l .. E l + E - 1 (E = D / 32), so
// the butterfly's first log2(E) stages run in registers and the other five
// across lanes, and the pairwise tree of the sum of squares is the warp's
// xor reduction.  This TU is compiled with -fmad=false: the squares and sums
// round exactly as written.
#include "kernels.cuh"
#include "tq4_code.cuh"

namespace kvq {

namespace {

template <int E>
__global__ void __launch_bounds__(256) store_tq4_kernel(kvq_cache c, const void* __restrict__ k,
                                                        const void* __restrict__ v, int dtype, int64_t n_tok,
                                                        const int32_t* __restrict__ slots, int32_t* status) {
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * E;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp_index();
  const int Hk = c.num_kv_heads;
  if (row >= n_tok * Hk * 2) return;
  const int kv = static_cast<int>(row & 1);
  const int64_t tok = (row >> 1) / Hk;
  const int head = static_cast<int>((row >> 1) % Hk);
  const int32_t slot = slots[tok];
  if (slot < 0) return;
  if ((int64_t)slot >= (int64_t)c.num_pages * c.page_size) {
    if (lane == 0) set_status(status, KVQ_DEV_BAD_SLOT);
    return;
  }
  const int64_t r = ((int64_t)(slot / c.page_size) * Hk + head) * c.page_size + slot % c.page_size;
  const void* src = kv ? v : k;
  const int64_t base = (tok * Hk + head) * D + E * lane;

  float y[E];
#pragma unroll
  for (int i = 0; i < E; ++i) y[i] = load_act(src, dtype, base + i);
  tq4_transform<E>(y, lane_signs<E>(c.signs, lane), lane, false);

  __half s16;
  uint32_t word[1];
  tq4_row_codes<E, 32>(y, word, s16);
  uint8_t* codes = static_cast<uint8_t*>(kv ? c.v : c.k) + r * (D / 2) + lane * (E / 2);
  write_codes<E>(codes, word);
  if (lane == 0) static_cast<__half*>(kv ? c.v_scale : c.k_scale)[r] = s16;
}

template <int E>
__global__ void __launch_bounds__(256) tq4_rotate_kernel(const void* __restrict__ signs, const void* x, int dtype,
                                                         float* y, int64_t rows, int inverse) {
  pdl_wait();
  pdl_trigger();
  constexpr int D = 32 * E;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp_index();
  if (row >= rows) return;
  float v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = load_act(x, dtype, row * D + E * lane + i);
  __syncwarp();  // every lane has read its inputs before any lane writes (y may alias x)
  tq4_transform<E>(v, lane_signs<E>(signs, lane), lane, inverse != 0);
#pragma unroll
  for (int i = 0; i < E; ++i) y[row * D + E * lane + i] = v[i];
}

}  // namespace

cudaError_t launch_store_tq4(const kvq_cache& c, const void* k, const void* v, int dtype, int64_t n_tok,
                             const int32_t* slots, int32_t* status, cudaStream_t s) {
  if (n_tok == 0) return cudaSuccess;
  const int64_t rows = n_tok * c.num_kv_heads * 2;
  const dim3 blocks(static_cast<unsigned>((rows + 7) / 8));
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = launch_pdl(store_tq4_kernel<2>, blocks, dim3(256), 0, s, c, k, v, dtype, n_tok, slots, status); break;
    case 128: e = launch_pdl(store_tq4_kernel<4>, blocks, dim3(256), 0, s, c, k, v, dtype, n_tok, slots, status); break;
    case 256: e = launch_pdl(store_tq4_kernel<8>, blocks, dim3(256), 0, s, c, k, v, dtype, n_tok, slots, status); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_tq4_rotate(const kvq_cache& c, const void* x, int dtype, float* y, int64_t rows, int inverse,
                              cudaStream_t s) {
  if (rows == 0) return cudaSuccess;
  const dim3 blocks(static_cast<unsigned>((rows + 7) / 8));
  cudaError_t e;
  switch (c.head_dim) {
    case 64: e = launch_pdl(tq4_rotate_kernel<2>, blocks, dim3(256), 0, s, c.signs, x, dtype, y, rows, inverse); break;
    case 128: e = launch_pdl(tq4_rotate_kernel<4>, blocks, dim3(256), 0, s, c.signs, x, dtype, y, rows, inverse); break;
    case 256: e = launch_pdl(tq4_rotate_kernel<8>, blocks, dim3(256), 0, s, c.signs, x, dtype, y, rows, inverse); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace kvq
