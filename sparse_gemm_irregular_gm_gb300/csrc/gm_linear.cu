// gm_linear.cu -- a product with bias, activation and residual (include/gm_layers.h): host driver, and the
// kernels around the tensor-core products of gm_loss_prod.cu.
//
// Forward: one product whose end adds the bias, writes z if the backward call will want it, applies the activation and
// adds the residual. Few tiles along a long row are split along it; the parts are joined by a second kernel with the same
// end. Backward: dz = grad * act'(z) is laid out as an operand, its columns summed on the way (db), then dX = dz W
// and dW = dz^T X are products of the kind that the losses' gradients are.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gm_act.cuh"
#include "gm_device.cuh"
#include "gm_host.h"
#include "gm_layers.h"
#include "gm_loss.h"
#include "gm_planes.cuh"
#include "gm_umma.cuh"

namespace gm {

namespace {

__device__ __forceinline__ float element(const void* p, int64_t i, int type) {
  return type == GM_LOSS_F32    ? static_cast<const float*>(p)[i]
         : type == GM_LOSS_BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i])
                                : __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void set_element(void* p, int64_t i, int type, float x) {
  if (type == GM_LOSS_F32) static_cast<float*>(p)[i] = x;
  else if (type == GM_LOSS_BF16) static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(x);
  else static_cast<__half*>(p)[i] = __float2half_rn(x);
}
__device__ __forceinline__ float activated(float z, int act, bool fine) {
  if (act == GM_ACT_RELU) return z < 0.f ? 0.f : z;
  if (act == GM_ACT_GELU) return z * (fine ? normal_below<true>(z) : normal_below<false>(z));
  if (act == GM_ACT_GELU_TANH) return z * (fine ? logistic<true>(gelu_tanh_arg(z)) : logistic<false>(gelu_tanh_arg(z)));
  if (act == GM_ACT_SILU) return z * (fine ? logistic<true>(z) : logistic<false>(z));
  return z;
}

// Four elements from i on, `have` of them; wide: they lie together on a boundary of their own.
__device__ __forceinline__ void get_four(const void* p, int64_t i, int type, bool wide, int have, float (&v)[4]) {
  if (wide && type == GM_LOSS_F32) {
    const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else if (wide) {
    const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t w[2] = {x.x, x.y};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 y = type == GM_LOSS_BF16 ? make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u))
                                            : __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      v[2 * j] = y.x, v[2 * j + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = j < have ? element(p, i + j, type) : 0.f;
  }
}
__device__ __forceinline__ void set_four(void* p, int64_t i, int type, bool wide, int have, const float (&v)[4]) {
  if (wide && type == GM_LOSS_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  } else if (wide) {
    uint32_t w[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (type == GM_LOSS_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __floats2half2_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < have) set_element(p, i + j, type, v[j]);
  }
}

// y and z from the parts of X W^T, a thread four columns: 512 x 4096 in two parts, 25 MB, 6 us; an element a thread, found by a
// division of 64 bits, took 14. Parts are made of so few tiles that 32 bits count the fours.
__global__ void __launch_bounds__(256) k_linear_join(const float* __restrict__ acc, int splits, int64_t rows, int64_t outs,
                                                     int64_t acc_ld, const LinearEnd e, void* y, int64_t y_ld, int type, bool wide,
                                                     const uint8_t* __restrict__ lost) {
  chain_wait();
  const bool gone = __any_sync(kFull, lost_word(lost) != 0);  // parts that were never written: NaN, not what lies there
  const uint32_t a_row = static_cast<uint32_t>(acc_ld / 4), n = static_cast<uint32_t>(rows) * a_row, stride = gridDim.x * blockDim.x;
  for (uint32_t i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t r = i / a_row, c = int64_t(i - static_cast<uint32_t>(r) * a_row) * 4;
    const int have = static_cast<int>(outs - c);
    if (have <= 0) continue;
    const float* p = acc + r * acc_ld + c;
    float v[4] = {0.f, 0.f, 0.f, 0.f}, t[4];
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
      const float4 x = *reinterpret_cast<const float4*>(p + s * rows * acc_ld);  // columns from outs on are not written: not used
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
    if (gone) v[0] = v[1] = v[2] = v[3] = NAN;
    if (e.bias) {
      get_four(e.bias, c, type, wide, have, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += t[j];
    }
    if (e.keep) set_four(e.z, r * e.z_ld + c, type, wide, have, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = activated(v[j], e.act, type == GM_LOSS_F32);
    if (e.residual) {
      get_four(e.residual, r * e.residual_ld + c, type, wide, have, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += t[j];
    }
    set_four(y, r * y_ld + c, type, wide, have, v);
  }
}

// X and W laid out as operands where they cannot be read in place: in one launch, or by blocks of the next kernel's.
struct Lay {
  const void* src;  // null: nothing to lay out
  int64_t rows, src_ld;
  uint16_t* dst;
  int dim, ld;
  bool wide;        // rows of src start on 16-byte boundaries
  unsigned blocks;
};
struct Lays {
  Lay m[2];
  unsigned blocks() const { return m[0].blocks + m[1].blocks; }
};
constexpr int kLayThreads = 256;

template <bool F32>
__device__ __forceinline__ void lay_out_all(const Lays& l, unsigned block) {
  const Lay& m = l.m[block < l.m[0].blocks ? 0 : 1];
  if (block >= l.m[0].blocks) block -= l.m[0].blocks;
  const int64_t first = static_cast<int64_t>(block) * kLayThreads + threadIdx.x, stride = static_cast<int64_t>(m.blocks) * kLayThreads;
  if (F32 && m.wide) lay_out<F32, true>(m.src, m.rows, m.dim, m.src_ld, m.dst, m.ld, first, stride);
  else lay_out<F32, false>(m.src, m.rows, m.dim, m.src_ld, m.dst, m.ld, first, stride);
}
template <bool F32>
__global__ void __launch_bounds__(kLayThreads) k_operands(const Lays l) {
  chain_wait();
  lay_out_all<F32>(l, blockIdx.x);
}

// f16 has too short a range for small gradients times small slopes (gradients of 1e-4 at z near -4 came to a row of dW a third off), so
// such a dz is scaled, as G is (Scales): by the power of two that brings the largest finite |grad|, hence about the largest |dz|, into
// [2^13, 2^14). What lies under 2^-14 then loses at most half of 2^-24: 2^-38 of the largest. One pass more over grad, which
// k_dz then finds in L2 where it fits: backward of 8192 x 1024 x 4096 f16 gelu 139 us, 120 without a scale (as bf16 is).
// dz = grad * act'(z), as an operand of the two products: 16 bits, with few rows a second plane of what rounding took; three
// bf16 planes of f32. Sums of its columns over the block's rows, in fp32, go to sums[part]. A warp takes 256 columns of
// a row, a thread 8 of them. The blocks after these lay out X and W. Bound by memory and by gelu's slope together: 8192 x 4096 bf16,
// 201 MB, 41 us, 4.9 TB/s or 72 % of what a copy reaches (5 longer with all rows of a turn asked for before any is worked on).
struct DzArgs {
  const void *grad, *z;  // z null: dz is grad
  int64_t grad_ld, z_ld, rows, outs, rows_a_block;
  int act, type;
  bool wide;             // rows start on 16-byte boundaries
  uint16_t* dz;          // null: not wanted
  int64_t ld, plane;
  int planes;
  float* sums;           // null: not wanted
  unsigned slabs, blocks;
  const uint32_t* largest;  // of k_largest, by which dz is scaled; null: it is not
  int n_largest;
  uint32_t* weights;        // [2]: what Scales takes the scale off again by
};
constexpr int kDzWarps = kLayThreads / 32, kDzColumns = 256;

// Eight elements as they are in memory; `have` of them, the others 0.
template <bool F32>
struct Raw8 {
  uint32_t w[F32 ? 8 : 4];
  __device__ __forceinline__ void read(const void* p, int have, bool wide) {
    constexpr int kQuads = F32 ? 2 : 1;
#pragma unroll
    for (int q = 0; q < 4 * kQuads; ++q) w[q] = 0;
    if (wide && have >= 8) {
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const uint4 x = static_cast<const uint4*>(p)[q];
        w[4 * q] = x.x, w[4 * q + 1] = x.y, w[4 * q + 2] = x.z, w[4 * q + 3] = x.w;
      }
    } else if (have > 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= have) continue;
        if constexpr (F32) w[i] = static_cast<const uint32_t*>(p)[i];
        else w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << (i & 1 ? 16 : 0);
      }
    }
  }
  __device__ __forceinline__ void get(bool bf16, float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (F32) {
        v[2 * i] = __uint_as_float(w[2 * i]), v[2 * i + 1] = __uint_as_float(w[2 * i + 1]);
      } else if (bf16) {
        v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        v[2 * i] = y.x, v[2 * i + 1] = y.y;
      }
    }
  }
};

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The largest |grad| of those of a block that are finite: its bits, one word a block.
__global__ void __launch_bounds__(kLayThreads) k_largest(const uint16_t* __restrict__ grad, int64_t ld, int64_t rows, int64_t outs, bool wide,
                                                         uint32_t* __restrict__ out) {
  constexpr int kAhead = 4;
  __shared__ uint32_t sh[kLayThreads / 32];
  chain_wait();
  const unsigned per_row = static_cast<unsigned>((outs + 7) / 8);
  const int64_t pieces = rows * per_row, stride = static_cast<int64_t>(gridDim.x) * kLayThreads;
  uint32_t most = 0;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kLayThreads + threadIdx.x; i0 < pieces; i0 += kAhead * stride) {
    Raw8<false> x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int64_t i = i0 + j * stride;
      const int64_t r = pieces < (int64_t(1) << 32) ? static_cast<unsigned>(i) / per_row : i / per_row, c = (i - r * per_row) * 8;
      x[j].read(grad + r * ld + c, i < pieces ? static_cast<int>(min(int64_t(8), outs - c)) : 0, wide);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
#pragma unroll
      for (const uint32_t w : x[j].w) {
        const uint32_t v = w & 0x7fff7fffu;
        most = __vmaxu2(most, v & ~__vcmpgeu2(v, 0x7c007c00u));
      }
  }
  most = __reduce_max_sync(kFull, max(most & 0xffffu, most >> 16));
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (const uint32_t w : sh) most = max(most, w);
  out[blockIdx.x] = most;
}

template <bool F32>
__device__ __forceinline__ void times_slope(float (&g)[8], const float (&z)[8], int act) {
#pragma unroll
  for (int i = 0; i < 8; ++i) g[i] *= slope<F32>(z[i], act);
}

template <bool F32>
__global__ void __launch_bounds__(32 * kDzWarps, 3) k_dz(const DzArgs a, const Lays lays) {
  __shared__ float sh[kDzWarps][kDzColumns];
  chain_wait();
  if (blockIdx.x >= a.blocks) {
    lay_out_all<F32>(lays, blockIdx.x - a.blocks);
    return;
  }
  constexpr int kBytes = F32 ? 4 : 2;
  constexpr int kAhead = F32 ? 1 : 2;  // rows of a warp at a time; as many more are under way meanwhile
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned slab = blockIdx.x % a.slabs, part = blockIdx.x / a.slabs;
  const int64_t col = static_cast<int64_t>(slab) * kDzColumns + lane * 8;
  const int have = static_cast<int>(max(int64_t(0), min(int64_t(8), a.outs - col)));
  const bool bf16 = a.type != GM_LOSS_F16, write = a.dz && col < a.ld;  // ld is a multiple of 8
  const int64_t first = part * a.rows_a_block, end = min(a.rows, first + a.rows_a_block);
  const char* grad = static_cast<const char*>(a.grad) + ((first + warp) * a.grad_ld + col) * kBytes;
  const char* z_at = static_cast<const char*>(a.z) + ((first + warp) * a.z_ld + col) * kBytes;
  uint16_t* out = a.dz + (first + warp) * a.ld + col;
  const int64_t grad_step = a.grad_ld * kBytes * kDzWarps, z_step = a.z_ld * kBytes * kDzWarps, out_step = a.ld * kDzWarps;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.f;
  Raw8<F32> g_next[kAhead], z_next[kAhead];
  auto ask = [&](int64_t r) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int in = r + k * kDzWarps < end ? have : 0;  // what is not there is 0, and so is its dz
      g_next[k].read(grad, in, a.wide);
      if (a.z) z_next[k].read(z_at, in, a.wide);
      grad += grad_step, z_at += z_step;
    }
  };
  ask(first + warp);
  float by = 1.f;
  if (!F32 && a.largest) {
    __shared__ uint32_t sh_most[kDzWarps];
    uint32_t most = 0;
    for (int i = threadIdx.x; i < a.n_largest; i += 32 * kDzWarps) most = max(most, a.largest[i]);
    most = __reduce_max_sync(kFull, most);
    if (lane == 0) sh_most[warp] = most;
    __syncthreads();
    for (const uint32_t w : sh_most) most = max(most, w);
    const float weight = __half2float(__ushort_as_half(static_cast<unsigned short>(most)));
    by = scale_for(weight);
    if (blockIdx.x == 0 && threadIdx.x < 2) a.weights[threadIdx.x] = __float_as_uint(weight);
  }
  for (int64_t r0 = first + warp; r0 < end; r0 += kDzWarps * kAhead) {
    Raw8<F32> g_raw[kAhead], z_raw[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      g_raw[k] = g_next[k];
      if (a.z) z_raw[k] = z_next[k];
    }
    ask(r0 + kDzWarps * kAhead);
#pragma unroll
    for (int k = 0; k < kAhead; ++k, out += out_step) {
      float g[8];
      g_raw[k].get(bf16, g);
      if (a.z) {
        float z[8];
        z_raw[k].get(bf16, z);
        if (a.act == GM_ACT_GELU) times_slope<F32>(g, z, GM_ACT_GELU);
        else if (a.act == GM_ACT_SILU) times_slope<F32>(g, z, GM_ACT_SILU);
        else if (a.act == GM_ACT_GELU_TANH) times_slope<F32>(g, z, GM_ACT_GELU_TANH);
        else times_slope<F32>(g, z, GM_ACT_RELU);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += g[i];
      if (!write || r0 + k * kDzWarps >= end) continue;
      if (!F32 && a.largest) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= by;
      }
      if (!F32 && a.planes == 1) {
        *reinterpret_cast<uint4*>(out) =
            make_uint4(pack2(g[0], g[1], bf16), pack2(g[2], g[3], bf16), pack2(g[4], g[5], bf16), pack2(g[6], g[7], bf16));
        continue;
      }
#pragma unroll 1
      for (int p = 0; p < a.planes; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          uint32_t h[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float& u = g[i + j];
            if constexpr (F32) {
              h[j] = take_plane(u, p == 2, (__float_as_uint(u) & INT32_MAX) < kRoundsPast);
            } else if (bf16) {
              const __nv_bfloat16 y = __float2bfloat16_rn(u);
              h[j] = __bfloat16_as_ushort(y), u = (h[j] & 0x7f80u) == 0x7f80u ? 0.f : u - __bfloat162float(y);  // of inf: nothing
            } else {
              const __half y = __float2half_rn(u);
              h[j] = __half_as_ushort(y), u = (h[j] & 0x7c00u) == 0x7c00u ? 0.f : u - __half2float(y);
            }
          }
          w[i / 2] = h[0] | (h[1] << 16);
        }
        *reinterpret_cast<uint4*>(out + p * a.plane) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  if (!a.sums) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) sh[warp][lane * 8 + i] = acc[i];
  __syncthreads();
  const int64_t c = static_cast<int64_t>(slab) * kDzColumns + threadIdx.x;
  float x = 0.f;
#pragma unroll
  for (int w = 0; w < kDzWarps; ++w) x += sh[w][threadIdx.x];
  if (c < a.outs) a.sums[part * a.outs + c] = x;
}

// ---- few rows ------------------------------------------------------------------------------------
// One row of X, or up to 4 of f32 (whose tensor-core form reads and writes W four times more): a warp reads OUTS rows of W together, 16
// bytes a lane (VEC; else single elements), eight such loads under way, and multiplies in fp32. Bound by the bytes of W
// and, with 2^24 of them, by the launch: 1 x 4096 x 4096 bf16 11 us from memory, 3 TB/s (21 on the tensor cores); 1024 x 32768
// f32, 134 MB: one row 34, two 40, four 56 (five, on the tensor cores, 124). Two rows of 16 bits are faster on the tensor cores
// (1024 x 32768: 36 us here, 26 there).
constexpr int kFewWarps = 8;
template <bool F32, bool VEC, int ROWS, int OUTS>
__global__ void __launch_bounds__(32 * kFewWarps, ROWS == 1 ? 3 : 2) k_linear_few(const gm_linear p, const LinearEnd e, void* y, int64_t y_ld) {
  chain_wait();
  constexpr int kBytes = F32 ? 4 : 2, kTurns = (F32 ? 4 : 8) / OUTS;
  const int lane = threadIdx.x & 31, dim = static_cast<int>(p.dim);
  const bool bf16 = p.type != GM_LOSS_F16;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kFewWarps * OUTS;
  auto part = [&](const void* m, int64_t row, int64_t ld, int at, Raw8<F32>& v) {
    const char* q = static_cast<const char*>(m) + row * ld * kBytes;
    if constexpr (VEC) {
      const int c = at + lane * 8;
      v.read(q + static_cast<int64_t>(c) * kBytes, min(8, dim - c), true);  // dim is a multiple of 8
    } else {
#pragma unroll
      for (int i = 0; i < (F32 ? 8 : 4); ++i) v.w[i] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = at + lane + 32 * i;
        if (c >= dim) continue;
        if constexpr (F32) v.w[i] = reinterpret_cast<const uint32_t*>(q)[c];
        else v.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(q)[c]) << (i & 1 ? 16 : 0);
      }
    }
  };
  for (int64_t o0 = (static_cast<int64_t>(blockIdx.x) * kFewWarps + (threadIdx.x >> 5)) * OUTS; o0 < p.n_outs; o0 += step) {
    float acc[ROWS][OUTS] = {};
    for (int at = 0; at < dim; at += 256 * kTurns) {
      Raw8<F32> w[kTurns][OUTS], x_raw[kTurns];
#pragma unroll
      for (int t = 0; t < kTurns; ++t)
#pragma unroll
        for (int k = 0; k < OUTS; ++k) part(p.w, min(o0 + k, p.n_outs - 1), p.w_ld, at + t * 256, w[t][k]);
      if constexpr (ROWS == 1) {
#pragma unroll
        for (int t = 0; t < kTurns; ++t) part(p.x, 0, p.x_ld, at + t * 256, x_raw[t]);
      }
#pragma unroll
      for (int t = 0; t < kTurns; ++t) {
        float v[OUTS][8];
#pragma unroll
        for (int k = 0; k < OUTS; ++k) w[t][k].get(bf16, v[k]);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
          float x[8];
          if constexpr (ROWS > 1) part(p.x, min(int64_t(r), p.n_rows - 1), p.x_ld, at + t * 256, x_raw[t]);
          x_raw[t].get(bf16, x);
#pragma unroll
          for (int k = 0; k < OUTS; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[r][k] = fmaf(x[i], v[k][i], acc[r][k]);
        }
      }
    }
    float mine = 0.f;  // lane r * OUTS + k has the sum of that row and out
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
#pragma unroll
      for (int k = 0; k < OUTS; ++k) {
        const float sum = warp_reduce_sum(acc[r][k]);
        if (lane == r * OUTS + k) mine = sum;
      }
    const int64_t row = lane / OUTS, out = o0 + lane % OUTS;
    if (row >= ROWS || row >= p.n_rows || out >= p.n_outs) continue;
    if (e.bias) mine += element(e.bias, out, p.type);
    if (e.keep) set_element(e.z, row * e.z_ld + out, p.type, mine);
    mine = activated(mine, e.act, F32);
    if (e.residual) mine += element(e.residual, row * e.residual_ld + out, p.type);
    set_element(y, row * y_ld + out, p.type, mine);
  }
}

// ---- host ----------------------------------------------------------------------------------------
struct LinearCall {
  gm_linear p = {};
  gm_layer_config cfg = {};
  cudaStream_t s = nullptr;
  int sms = 0;
  int* status = nullptr;
  int planes() const { return p.type == GM_LOSS_F32 ? 3 : 1; }
};

// Few rows go to a kernel that reads W once as it lies, instead of the tensor cores.
bool few(const LinearCall& c) { return c.p.n_rows <= (c.p.type == GM_LOSS_F32 ? 4 : 1); }

gm_status check_matrix(const void* p, int64_t ld, int64_t cols, int64_t rows, int32_t type, bool needed) {
  if (!p) return needed && rows > 0 ? GM_ERR_INVALID_ARG : GM_OK;
  if (!aligned(p, elem_bytes(type)) || ld < cols) return GM_ERR_INVALID_ARG;
  return ld > kMostLd ? GM_ERR_INDEX_OVERFLOW : GM_OK;
}

gm_status check_linear(LinearCall& c, const gm_linear* p, const gm_layer_config* cfg, void* stream) {
  if (!p || p->n_rows < 0 || p->dim < 1 || p->n_outs < 1) return GM_ERR_INVALID_ARG;
  if (p->n_rows > kMostIndex || p->dim > (int64_t(1) << 24) || p->n_outs > (int64_t(1) << 24)) return GM_ERR_INDEX_OVERFLOW;
  if (p->type != GM_LOSS_F32 && p->type != GM_LOSS_BF16 && p->type != GM_LOSS_F16) return GM_ERR_INVALID_ARG;
  if (p->activation < GM_ACT_NONE || p->activation > GM_ACT_SILU) return GM_ERR_INVALID_ARG;
  gm_status rc = check_matrix(p->x, p->x_ld, p->dim, p->n_rows, p->type, true);
  if (rc == GM_OK) rc = check_matrix(p->w, p->w_ld, p->dim, p->n_outs, p->type, true);
  if (rc != GM_OK) return rc;
  c.p = *p;
  if (cfg) c.cfg = *cfg;
  if (c.cfg.workspace && (!aligned(c.cfg.workspace, 256) || c.cfg.workspace_bytes < 0)) return GM_ERR_INVALID_ARG;
  c.s = static_cast<cudaStream_t>(stream);
  return GM_OK;
}

gm_status begin(LinearCall& c) {
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  c.sms = sm_count(kMostBlocks);
  c.status = loss_status_word();
  if (c.sms > 0 && c.status) return GM_OK;
  cudaGetLastError();
  return GM_ERR_CUDA;
}
gm_status finish(bool launched) { return cudaGetLastError() != cudaSuccess || !launched ? GM_ERR_CUDA : GM_OK; }

// How a source is laid out, and the operand that it is then.
Lay lay_of(const Source& m, const Arena& a, int sms) {
  Lay l = {};
  if (!m.packed) return l;
  l.src = m.p;
  l.rows = m.rows;
  l.src_ld = m.src_ld;
  l.dst = a.at<uint16_t>(m.off);
  l.dim = static_cast<int>(m.dim);
  l.ld = static_cast<int>(m.ld);
  l.wide = aligned(m.p, 16) && (m.rows <= 1 || m.src_ld * elem_bytes(m.type) % 16 == 0);
  l.blocks = grid_for(m.rows * m.ld / 8, kLayThreads, int64_t(sms) * 16);
  return l;
}

// Tiles of a product: blocks a tile, its columns, and how many parts its sum is cut into.
struct Tiling {
  int cg = 1, bn = 64;
  int64_t splits = 1;
};
// The least of rounds of tiles times what a stage of one takes (SM clocks, measured: 16 bits, and three planes of f32, whose
// pairs hold two stages only), times stages, with a start and an end a round; parts cost a launch and their way through memory.
// us, forward with gelu, by tiles of 2 x 256 (pairs), 256, 128 and 64 columns: 8192 x 1024 x 4096 bf16: 54, 60, 69, 107;
// 512 x 4096 x 4096: 33, 31, 23, 33; 24 x 1024 x 32768: 27, 21, 25, 33; 4096 x 1024 x 1024 f32: 99, -, 71, 85.
// In 1, 2, 4, 8 parts: 24 x 16384 x 1024 by 128: 59, 35, 23, 17; 512 x 4096 x 4096: 23, 29, 32, 38.
Tiling tile_for(int64_t m, int64_t n, int64_t k_blocks, int planes, int sms, bool pairs = true) {
  Tiling best;
  double least = 1e300;
  struct Kind { int cg, bn; double stage, stage32; };
  const Kind kinds[] = {{2, 256, 600, 10400}, {1, 256, 700, 0}, {1, 128, 456, 3400}, {1, 64, 375, 2060}};
  for (const Kind& k : kinds) {
    if ((planes == 3 && k.cg == 1 && k.bn == 256) || (k.cg == 2 && !pairs)) continue;
    const int64_t slots = sms / k.cg, tiles = div_up(m, 128 * k.cg) * div_up(n, k.bn);
    const double stage = planes == 3 ? k.stage32 : k.stage;
    for (int64_t want = 1; want <= 16; want *= 2) {
      if (want > 1 && (tiles * want > slots || k_blocks / want < 8)) break;
      const int64_t per = div_up(k_blocks, want), parts = div_up(k_blocks, per);
      const double cost = div_up(tiles * parts, slots) * (per * stage + 2500.0 + 12.0 * k.bn) +
                          (parts > 1 ? 6000.0 + static_cast<double>(m) * n * parts * 0.0025 : 0.0);
      if (cost < least) least = cost, best = Tiling{k.cg, k.bn, parts};
    }
  }
  return best;
}

struct LinearForward {
  Arena a;
  Source x, w;
  Tiling t;
  size_t o_lost = 0, o_acc = 0;
  int64_t acc_ld = 0;
  explicit LinearForward(const LinearCall& c)
      : x(c.p.x, c.p.n_rows, c.p.dim, c.p.x_ld, c.p.type), w(c.p.w, c.p.n_outs, c.p.dim, c.p.w_ld, c.p.type) {
    if (few(c)) return;
    o_lost = a.add(kMostBlocks);
    x.plan(a);
    w.plan(a);
    t = tile_for(c.p.n_rows, c.p.n_outs, div_up(c.p.dim, 64), c.planes(), c.sms);
    if (t.splits > 1) {
      acc_ld = up(c.p.n_outs, 32);
      o_acc = a.add(t.splits * c.p.n_rows * acc_ld * 4);
    }
  }
};

// Rows of 32 elements from p on, read 16 bytes at a time.
bool wide_rows(const void* p, int64_t ld, int64_t rows, int64_t es) { return aligned(p, 16) && (rows <= 1 || ld * es % 16 == 0); }
// By TMA where its rows start and end on 16-byte boundaries; boxes of 32 rows of 32 elements.
bool linear_result(CUtensorMap* m, bool* by_tma, void* out, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  *by_tma = wide_rows(out, ld, rows, es) && cols * es % 16 == 0;
  if (!*by_tma) return true;
  if (rows <= 1) ld = up(cols, 16 / es);
  return encode(m, Operand{out, rows, cols, ld, rows * ld, 1, static_cast<int>(es)}, 32, static_cast<int>(32 * es));
}

template <bool F32, bool VEC, int ROWS>
cudaError_t launch_few_rows(const LinearCall& c, const LinearEnd& e, void* y, int64_t y_ld) {
  // short rows of W several at a time, so that the loads under way are as many
  const gm_linear& p = c.p;
  const int outs = p.dim > 1024 / (F32 ? 2 : 1) ? 1 : p.dim > 512 / (F32 ? 2 : 1) ? 2 : 4;
  const unsigned grid = grid_for(p.n_outs, kFewWarps * outs, int64_t(c.sms) * 16);
  auto* k = outs == 1 ? k_linear_few<F32, VEC, ROWS, 1> : outs == 2 ? k_linear_few<F32, VEC, ROWS, 2> : k_linear_few<F32, VEC, ROWS, 4>;
  return launch_chained(k, grid, 32 * kFewWarps, 0, c.s, 1, p, e, y, y_ld);
}
template <bool VEC>
cudaError_t launch_few(const LinearCall& c, const LinearEnd& e, void* y, int64_t y_ld) {
  if (c.p.type != GM_LOSS_F32) return launch_few_rows<false, VEC, 1>(c, e, y, y_ld);
  return c.p.n_rows == 1 ? launch_few_rows<true, VEC, 1>(c, e, y, y_ld)
         : c.p.n_rows == 2 ? launch_few_rows<true, VEC, 2>(c, e, y, y_ld) : launch_few_rows<true, VEC, 4>(c, e, y, y_ld);
}

gm_status forward(LinearCall& c, LinearEnd e, void* y, int64_t y_ld) {
  gm_status rc = begin(c);
  if (rc != GM_OK) return rc;
  if (few(c)) {
    const int64_t es = elem_bytes(c.p.type);
    const bool vec = wide_rows(c.p.x, c.p.x_ld, c.p.n_rows, es) && wide_rows(c.p.w, c.p.w_ld, c.p.n_outs, es) && c.p.dim % 8 == 0;
    return finish((vec ? launch_few<true>(c, e, y, y_ld) : launch_few<false>(c, e, y, y_ld)) == cudaSuccess);
  }
  const int64_t m = c.p.n_rows, n = c.p.n_outs, es = elem_bytes(c.p.type);
  LinearForward p(c);
  rc = p.a.open(c.cfg.workspace, c.cfg.workspace_bytes, c.s);
  if (rc != GM_OK) return rc;
  const Lays lays{{lay_of(p.x, p.a, c.sms), lay_of(p.w, p.a, c.sms)}};
  if (lays.blocks() &&
      launch_chained(c.p.type == GM_LOSS_F32 ? k_operands<true> : k_operands<false>, lays.blocks(), kLayThreads, 0, c.s, 1, lays) != cudaSuccess)
    return finish(false);
  const Operand ox = p.x.operand(p.a), ow = p.w.operand(p.a);
  ProdMaps maps;
  if (!encode(&maps.a, ox, prod_box_rows_a()) || !encode(&maps.b, ow, prod_box_rows_b(p.t.cg, p.t.bn))) return GM_ERR_CUDA;
  maps.o = maps.z = maps.a;
  ProdArgs g = {};
  g.planes = c.planes();
  g.g_planes = 1;
  g.bf16 = c.p.type != GM_LOSS_F16;
  g.m = m;
  g.n = n;
  g.m_tiles = static_cast<int>(div_up(m, 128 * p.t.cg));
  g.n_tiles = static_cast<int>(div_up(n, p.t.bn));
  g.k_blocks = static_cast<int>(div_up(c.p.dim, 64));
  g.k_per_split = static_cast<int>(div_up(g.k_blocks, p.t.splits));
  g.splits = static_cast<int>(div_up(g.k_blocks, g.k_per_split));
  g.chunk = kChunk;
  g.group = group_of_tiles(g.m_tiles, 128 * p.t.cg, c.p.dim, g.planes);
  g.status = c.status;
  g.lost = p.a.at<uint8_t>(p.o_lost);
  g.lost_first = true;
  g.out = y;
  g.out_ld = y_ld;
  g.out_type = c.p.type;
  e.bias_wide = aligned(e.bias, 16);
  e.residual_wide = wide_rows(e.residual, e.residual_ld, m, es);
  bool set;
  float* acc = nullptr;
  if (g.splits > 1) {
    g.acc = true;
    acc = p.a.at<float>(p.o_acc);
    set = encode(&maps.o, Operand{acc, m, n, p.acc_ld, m * p.acc_ld, g.splits, 4}, 32);
  } else {
    set = linear_result(&maps.o, &g.by_tma, y, m, n, y_ld, es);
    if (set && e.keep) set = linear_result(&maps.z, &e.z_by_tma, e.z, m, n, e.z_ld, es);
  }
  if (!set) return GM_ERR_CUDA;
  g.lin = e;
  bool ok = launch_prod(Prod::kLinear, p.t.cg, p.t.bn, maps, g, c.sms, c.s) == cudaSuccess;
  if (ok && acc) {
    auto four = [&](const void* q, int64_t ld) { return !q || (aligned(q, 4 * es) && (m <= 1 || ld % 4 == 0)); };
    const bool wide = n % 4 == 0 && four(y, y_ld) && four(e.keep ? e.z : nullptr, e.z_ld) && four(e.residual, e.residual_ld) && four(e.bias, 0);
    ok = launch_chained(k_linear_join, grid_for(m * (p.acc_ld / 4), 256), 256, 0, c.s, 1, static_cast<const float*>(acc), g.splits, m, n,
                        p.acc_ld, e, y, y_ld, static_cast<int>(c.p.type), wide, static_cast<const uint8_t*>(g.lost)) == cudaSuccess;
  }
  return finish(ok);
}

struct LinearGrads {
  const void* grad;
  int64_t grad_ld;
  const void* z;
  int64_t z_ld;
  void* dx;
  int64_t dx_ld;
  void* dw;
  int64_t dw_ld;
  void* db;
};

constexpr int kLargestAnSm = 8;  // blocks of k_largest

// One of the two products that read dz, and the sum of its parts.
struct SumPlan {
  int cg, bn;
  int64_t splits, acc_ld, k_blocks;
  size_t o_acc = 0;
  SumPlan(Arena& a, int64_t rows, int64_t cols, int64_t k, int planes, int sms, bool pairs) {
    k_blocks = div_up(k, 64);
    const Tiling t = tile_for(rows, cols, k_blocks, planes, sms, pairs);
    cg = t.cg, bn = t.bn, splits = t.splits;
    acc_ld = up(cols, 32);
    if (splits > 1) o_acc = a.add(splits * rows * acc_ld * 4);
  }
};

struct LinearBackward {
  Arena a;
  Source x, w;
  int planes, dz_planes;
  int64_t dz_ld, parts, rows_a_part;  // parts: of db's sum
  SumPlan dx, dw;
  bool scaled;                        // dz is (relu's is grad itself, or 0)
  size_t o_lost, o_dz, o_sums, o_largest = 0, o_weights = 0;
  explicit LinearBackward(const LinearCall& c)
      : x(c.p.x, c.p.n_rows, c.p.dim, c.p.x_ld, c.p.type),
        w(c.p.w, c.p.n_outs, c.p.dim, c.p.w_ld, c.p.type),
        planes(c.planes()),
        // Rounding dz costs digits (8192 x 1024 x 4096 bf16 gelu: gradients 2.4e-3 from 64 bits, 1.7e-3 without); a second plane doubles
        // the products' time, 90 us of 188 there, but none where they wait for W and dW
        dz_planes(planes == 3 ? 3 : c.p.activation != GM_ACT_NONE && c.p.n_rows <= 128 ? 2 : 1),
        dx(a, c.p.n_rows, c.p.dim, c.p.n_outs, planes, c.sms, dz_planes != 2),  // no pairs of blocks for two planes of dz
        dw(a, c.p.n_outs, c.p.dim, c.p.n_rows, planes, c.sms, dz_planes != 2) {
    const int64_t m = c.p.n_rows, n = c.p.n_outs;
    x.plan(a);
    w.plan(a);
    o_lost = a.add(2 * kMostBlocks);
    dz_ld = up(n, 8);
    o_dz = a.add(dz_planes * m * dz_ld * 2);
    const int64_t slabs = div_up(n, kDzColumns);
    parts = std::max<int64_t>(1, std::min(3 * c.sms / slabs, div_up(m, 4 * kDzWarps)));  // one round of blocks
    rows_a_part = div_up(m, parts);
    parts = div_up(m, rows_a_part);
    o_sums = a.add(parts * n * 4);
    const int act = c.p.activation;
    scaled = c.p.type == GM_LOSS_F16 && (act == GM_ACT_GELU || act == GM_ACT_GELU_TANH || act == GM_ACT_SILU);
    if (scaled) {
      o_largest = a.add(c.sms * kLargestAnSm * 4);
      o_weights = a.add(8);
    }
  }
};

gm_status backward(LinearCall& c, const LinearGrads& q) {
  gm_status rc = begin(c);
  if (rc != GM_OK) return rc;
  const int64_t m = c.p.n_rows, n = c.p.n_outs, dim = c.p.dim, es = elem_bytes(c.p.type);
  const int32_t type = c.p.type;
  if (m == 0) {
    bool ok = true;
    if (q.dw) ok = cudaMemset2DAsync(q.dw, q.dw_ld * es, 0, dim * es, n, c.s) == cudaSuccess;
    if (ok && q.db) ok = cudaMemsetAsync(q.db, 0, n * es, c.s) == cudaSuccess;
    return finish(ok);
  }
  LinearBackward p(c);
  rc = p.a.open(c.cfg.workspace, c.cfg.workspace_bytes, c.s);
  if (rc != GM_OK) return rc;
  const bool act = c.p.activation != GM_ACT_NONE;
  const bool in_place = !act && type != GM_LOSS_F32 && wide_rows(q.grad, q.grad_ld, m, 2);  // grad is dz, and an operand
  const bool products = q.dx || q.dw;
  Operand odz{q.grad, m, n, m <= 1 ? up(n, 8) : q.grad_ld, m * q.grad_ld, 1};
  Lays lays = {};
  if (q.dx) lays.m[0] = lay_of(p.w, p.a, c.sms);
  if (q.dw) lays.m[1] = lay_of(p.x, p.a, c.sms);
  uint32_t* weights = nullptr;
  const bool dz_or_db = (products && !in_place) || q.db;
  if (dz_or_db || lays.blocks()) {
    DzArgs d = {};
    d.grad = q.grad;
    d.grad_ld = q.grad_ld;
    d.z = act ? q.z : nullptr;
    d.z_ld = q.z_ld;
    d.rows = m;
    d.outs = n;
    d.rows_a_block = p.rows_a_part;
    d.act = c.p.activation;
    d.type = type;
    d.wide = wide_rows(q.grad, q.grad_ld, m, es) && (!act || wide_rows(q.z, q.z_ld, m, es));
    if (products && !in_place) {
      d.dz = p.a.at<uint16_t>(p.o_dz);
      d.ld = p.dz_ld;
      d.plane = m * p.dz_ld;
      d.planes = p.dz_planes;
      odz = Operand{d.dz, m, n, d.ld, d.plane, d.planes};
    }
    if (d.dz && p.scaled) {
      uint32_t* largest = p.a.at<uint32_t>(p.o_largest);
      const unsigned grid = grid_for(m * div_up(n, 8), 4 * kLayThreads, int64_t(c.sms) * kLargestAnSm);
      if (launch_chained(k_largest, grid, kLayThreads, 0, c.s, 1, static_cast<const uint16_t*>(q.grad), q.grad_ld, m, n, wide_rows(q.grad, q.grad_ld, m, es),
                         largest) != cudaSuccess)
        return finish(false);
      d.largest = largest;
      d.n_largest = static_cast<int>(grid);
      d.weights = weights = p.a.at<uint32_t>(p.o_weights);
    }
    if (q.db) d.sums = p.a.at<float>(p.o_sums);
    d.slabs = static_cast<unsigned>(div_up(n, kDzColumns));
    d.blocks = dz_or_db ? d.slabs * static_cast<unsigned>(p.parts) : 0;
    if (launch_chained(type == GM_LOSS_F32 ? k_dz<true> : k_dz<false>, d.blocks + lays.blocks(), 32 * kDzWarps, 0, c.s, 1, d, lays) != cudaSuccess)
      return finish(false);
    if (q.db) sum_splits(d.sums, p.parts, 1, n, n, q.db, n, type, nullptr, c.s);
  }
  bool ok = true;
  auto product = [&](Prod kind, const SumPlan& t, const Operand& b, int64_t rows, void* out, int64_t out_ld, uint8_t* lost) {
    ProdMaps maps;
    if (!encode(&maps.a, odz, kind == Prod::kDh ? prod_box_rows_a() : 64) || !encode(&maps.b, b, 64)) return false;
    maps.z = maps.a;
    ProdArgs g = {};
    g.planes = p.planes;
    g.g_planes = odz.planes;
    g.bf16 = type != GM_LOSS_F16;
    g.m = rows;
    g.n = dim;
    g.m_tiles = static_cast<int>(div_up(rows, 128 * t.cg));
    g.n_tiles = static_cast<int>(div_up(dim, t.bn));
    g.k_blocks = static_cast<int>(t.k_blocks);
    g.k_per_split = static_cast<int>(div_up(t.k_blocks, t.splits));
    g.splits = static_cast<int>(t.splits);
    g.chunk = kChunk;
    g.parts = true;
    g.group = 1;
    g.status = c.status;
    g.lost = lost;
    g.lost_first = true;
    g.weights = weights;  // two alike: one scale for all rows
    float* acc = nullptr;
    bool set;
    if (t.splits > 1) {
      acc = p.a.at<float>(t.o_acc);
      g.acc = g.by_tma = true;
      set = encode(&maps.o, Operand{acc, rows, dim, t.acc_ld, rows * t.acc_ld, g.splits, 4}, 32);
    } else {
      set = set_result(&maps.o, g, out, rows, dim, out_ld, type);
      if (t.bn == 64 && es == 2) g.by_tma = false;  // half a tile is less than a box
    }
    if (!set || launch_prod(kind, t.cg, t.bn, maps, g, c.sms, c.s) != cudaSuccess) return false;
    if (acc) sum_splits(acc, t.splits, rows, dim, t.acc_ld, out, out_ld, type, lost, c.s);
    return true;
  };
  uint8_t* lost = p.a.at<uint8_t>(p.o_lost);
  if (q.dx) ok = product(Prod::kDh, p.dx, p.w.operand(p.a), m, q.dx, q.dx_ld, lost);
  if (ok && q.dw) ok = product(Prod::kDw, p.dw, p.x.operand(p.a), n, q.dw, q.dw_ld, lost + kMostBlocks);
  return finish(ok);
}

}  // namespace

}  // namespace gm

extern "C" gm_status gm_linear_forward(const gm_linear* p, const gm_layer_config* cfg, void* stream, const void* bias,
                                       const void* residual, int64_t residual_ld, void* y, int64_t y_ld, void* z,
                                       int64_t z_ld) {
  using namespace gm;
  NvtxRange range("gm_linear_forward");
  LinearCall c;
  gm_status rc = check_linear(c, p, cfg, stream);
  if (rc != GM_OK) return rc;
  if (!aligned(bias, elem_bytes(p->type))) return GM_ERR_INVALID_ARG;
  rc = check_matrix(residual, residual_ld, p->n_outs, p->n_rows, p->type, false);
  if (rc == GM_OK) rc = check_matrix(y, y_ld, p->n_outs, p->n_rows, p->type, true);
  if (rc == GM_OK) rc = check_matrix(z, z_ld, p->n_outs, p->n_rows, p->type, false);
  if (rc != GM_OK) return rc;
  if (y && y == residual && y_ld != residual_ld && p->n_rows > 1) return GM_ERR_INVALID_ARG;
  if (p->n_rows == 0) return GM_OK;
  LinearEnd e = {};
  e.bias = bias;
  e.residual = residual;
  e.residual_ld = residual_ld;
  e.act = p->activation;
  e.keep = z != nullptr;
  e.z = z;
  e.z_ld = z_ld;
  return forward(c, e, y, y_ld);
}

extern "C" gm_status gm_linear_backward(const gm_linear* p, const gm_layer_config* cfg, void* stream, const void* grad,
                                        int64_t grad_ld, const void* z, int64_t z_ld, void* dx, int64_t dx_ld, void* dw,
                                        int64_t dw_ld, void* dbias) {
  using namespace gm;
  NvtxRange range("gm_linear_backward");
  LinearCall c;
  gm_status rc = check_linear(c, p, cfg, stream);
  if (rc == GM_OK) rc = check_matrix(grad, grad_ld, p->n_outs, p->n_rows, p->type, true);
  if (rc == GM_OK) rc = check_matrix(z, z_ld, p->n_outs, p->n_rows, p->type, p->activation != GM_ACT_NONE);
  if (rc == GM_OK) rc = check_matrix(dx, dx_ld, p->dim, p->n_rows, p->type, false);
  if (rc == GM_OK) rc = check_matrix(dw, dw_ld, p->dim, p->n_outs, p->type, false);
  if (rc != GM_OK) return rc;
  if (!aligned(dbias, elem_bytes(p->type)) || (p->n_rows > 0 && !dx && !dw && !dbias)) return GM_ERR_INVALID_ARG;
  return backward(c, LinearGrads{grad, grad_ld, z, z_ld, dx, dx_ld, dw, dw_ld, dbias});
}

extern "C" gm_status gm_linear_workspace(const gm_linear* p, int32_t backward, int64_t* bytes) {
  using namespace gm;
  if (!bytes || (backward != 0 && backward != 1)) return GM_ERR_INVALID_ARG;
  LinearCall c;
  const gm_status rc = check_linear(c, p, nullptr, nullptr);
  if (rc != GM_OK) return rc;
  *bytes = 0;
  if (c.p.n_rows == 0) return GM_OK;
  c.sms = sm_count(kMostBlocks);
  if (c.sms <= 0) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  *bytes = static_cast<int64_t>(backward ? LinearBackward(c).a.used : LinearForward(c).a.used);
  return GM_OK;
}
