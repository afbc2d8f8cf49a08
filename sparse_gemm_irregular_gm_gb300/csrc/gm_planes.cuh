// gm_planes.cuh -- an fp32 value as three bf16 ones, x = x0 + x1 + x2 with x0 the nearest bf16 of x and so
// on, which keeps all 24 bits: operands of the tensor-core products.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace gm {

constexpr uint32_t kRoundsPast = 0x7f7f8000u;  // bits of |x| from which the nearest bf16 is none that is finite
__device__ __forceinline__ uint32_t take_plane(float& x, bool third, bool ordinary) {  // leaves in x what is left of it
  __nv_bfloat16 a = __float2bfloat16_rn(x);
  float left = x - __bfloat162float(a);
  if (!ordinary && !third) {
    if (fabsf(x) == INFINITY) a = __ushort_as_bfloat16(0), left = x;
    else if (x != x) left = 0.f;  // NaN stands in the first plane
    else if ((__float_as_uint(x) & INT32_MAX) >= kRoundsPast) a = __float2bfloat16_rz(x), left = x - __bfloat162float(a);
  }
  x = left;
  return __bfloat16_as_ushort(a);
}

}  // namespace gm
