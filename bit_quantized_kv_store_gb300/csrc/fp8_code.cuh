// fp8_code.cuh -- the e4m3 code of a value of a latent row.
#pragma once
#include <cuda_fp8.h>

#include <cstdint>

namespace kvq {

__device__ __forceinline__ uint8_t e4m3_encode(float x) {
  if (isnan(x)) return 0;  // NaN is stored as the inert code 0
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3));
}

}  // namespace kvq
