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

// A matrix laid out as an operand: 16 bits, or three planes of f32, rows padded with zeros to ld, a multiple of 8; a
// thread writes 8 elements of each plane at once. VEC: the rows of src start on 16-byte boundaries. `first` of `stride` threads.
template <bool F32, bool VEC>
__device__ __forceinline__ void lay_out(const void* __restrict__ src, int64_t rows, int dim, int64_t src_ld,
                                        uint16_t* __restrict__ dst, int ld, int64_t first, int64_t stride) {
  const unsigned per_row = static_cast<unsigned>(ld) / 8;
  const int64_t n = rows * ld, pieces = rows * per_row;
  for (int64_t i = first; i < pieces; i += stride) {
    int64_t r;
    int c;
    if (pieces < (int64_t(1) << 32)) {
      const unsigned q = static_cast<unsigned>(i) / per_row;
      r = q, c = static_cast<int>((static_cast<unsigned>(i) - q * per_row) * 8);
    } else {
      r = i / per_row, c = static_cast<int>(i - r * per_row) * 8;
    }
    const int left = dim - c;  // at least 1
    if constexpr (!F32) {
      const uint16_t* p = static_cast<const uint16_t*>(src) + r * src_ld + c;
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = (2 * j < left ? p[2 * j] : 0u) | (2 * j + 1 < left ? static_cast<uint32_t>(p[2 * j + 1]) << 16 : 0u);
      *reinterpret_cast<uint4*>(dst + i * 8) = make_uint4(x[0], x[1], x[2], x[3]);
    } else {
      const float* p = static_cast<const float*>(src) + r * src_ld + c;
      float x[8];
      if (VEC && left >= 8) {
        const float4 u = reinterpret_cast<const float4*>(p)[0], v = reinterpret_cast<const float4*>(p)[1];
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = j < left ? p[j] : 0.f;
      }
      uint32_t largest = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) largest = max(largest, __float_as_uint(x[j]) & INT32_MAX);
      const bool ordinary = largest < kRoundsPast;
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t a = take_plane(x[j], q == 2, ordinary), b = take_plane(x[j + 1], q == 2, ordinary);
          y[j / 2] = a | (b << 16);
        }
        *reinterpret_cast<uint4*>(dst + q * n + i * 8) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  }
}

}  // namespace gm
