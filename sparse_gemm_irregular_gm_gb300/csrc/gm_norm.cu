// gm_norm.cu -- the norms around a residual with its gate and scale (include/gm_layers.h), forward and
// backward.
//
// Every element is read and written once: a group of threads holds a row in registers, the row's
// means are the group's sums. Bound by memory. The backward pass also sums over rows (gradients of
// weights, of a gate that is a vector): a thread keeps its columns from row to row, adds them up in
// registers, and the blocks' sums are joined by a second kernel in a fixed order, so no value is
// added atomically. Rows longer than a block holds (kHeldDim) are walked several times instead.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gm_device.cuh"
#include "gm_host.h"
#include "gm_layers.h"
#include "gm_loss.h"
#include "gm_umma.cuh"

namespace gm {

namespace {

constexpr int kPer = 8;           // elements of a row a thread holds together: 16 bytes of a 16-bit type
constexpr int kHeldDim = 4096;    // of a row held by at most 512 threads
constexpr int kSums = 5;          // over rows, at most: before, after, gate, before_bias, after_bias
enum { kSumBefore, kSumAfter, kSumGate, kSumBeforeBias, kSumAfterBias };

// Elements as they are in memory: 8 of them in 4 words (f32: 8).
template <int TYPE>
constexpr int kWords = TYPE == GM_LOSS_F32 ? 8 : 4;
template <int TYPE>
struct Raw {
  uint32_t w[kWords<TYPE>];
};

__device__ __forceinline__ float lower16(uint32_t x, bool bf16) {
  return bf16 ? __uint_as_float(x << 16) : __half2float(__ushort_as_half(static_cast<unsigned short>(x)));
}
template <int TYPE>
__device__ __forceinline__ void unpack(const Raw<TYPE>& r, float (&v)[kPer]) {
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if constexpr (TYPE == GM_LOSS_F32) v[i] = __uint_as_float(r.w[i]);
    else v[i] = lower16(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2] & 0xffffu, TYPE == GM_LOSS_BF16);
  }
}
template <int TYPE>
__device__ __forceinline__ uint32_t round16(float x) {
  if constexpr (TYPE == GM_LOSS_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  else return __half_as_ushort(__float2half_rn(x));
}
template <int TYPE>
__device__ __forceinline__ Raw<TYPE> pack(const float (&v)[kPer]) {
  Raw<TYPE> r;
  if constexpr (TYPE == GM_LOSS_F32) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.w[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; i += 2) r.w[i / 2] = round16<TYPE>(v[i]) | (round16<TYPE>(v[i + 1]) << 16);
  }
  return r;
}

// Columns of a thread: VEC (rows and vectors start and end on 16 bytes): 8 consecutive ones; else one
// of every `group`, so that a warp's loads of single elements lie together.
template <bool VEC>
__device__ __forceinline__ int64_t column(int64_t t, int group, int i) {
  return VEC ? t * kPer + i : t + static_cast<int64_t>(i) * group;
}
// t: the thread's place in its group, plus kPer * group (VEC: group) for the next turn of a long row.
template <int TYPE, bool VEC>
__device__ __forceinline__ Raw<TYPE> load(const void* row, int64_t t, int group, int64_t dim) {
  Raw<TYPE> r;
#pragma unroll
  for (int i = 0; i < kWords<TYPE>; ++i) r.w[i] = 0;
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < kWords<TYPE> / 4; ++h)
      if (t * kPer + h * 4 < dim) {
        const uint4 x = reinterpret_cast<const uint4*>(row)[t * (kWords<TYPE> / 4) + h];
        r.w[4 * h] = x.x, r.w[4 * h + 1] = x.y, r.w[4 * h + 2] = x.z, r.w[4 * h + 3] = x.w;
      }
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t c = column<false>(t, group, i);
      if (c >= dim) continue;
      if constexpr (TYPE == GM_LOSS_F32) r.w[i] = static_cast<const uint32_t*>(row)[c];
      else r.w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(row)[c]) << (i & 1 ? 16 : 0);
    }
  }
  return r;
}
template <int TYPE, bool VEC>
__device__ __forceinline__ void store(void* row, int64_t t, int group, int64_t dim, const float (&v)[kPer]) {
  const Raw<TYPE> r = pack<TYPE>(v);
  if constexpr (VEC) {
#pragma unroll
    for (int h = 0; h < kWords<TYPE> / 4; ++h)
      if (t * kPer + h * 4 < dim)
        reinterpret_cast<uint4*>(row)[t * (kWords<TYPE> / 4) + h] =
            make_uint4(r.w[4 * h], r.w[4 * h + 1], r.w[4 * h + 2], r.w[4 * h + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int64_t c = column<false>(t, group, i);
      if (c >= dim) continue;
      if constexpr (TYPE == GM_LOSS_F32) static_cast<uint32_t*>(row)[c] = r.w[i];
      else static_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2]);
    }
  }
}
template <int TYPE>
__device__ __forceinline__ const void* row_at(const void* p, int64_t row, int64_t ld) {
  return static_cast<const char*>(p) + row * ld * (TYPE == GM_LOSS_F32 ? 4 : 2);
}
template <int TYPE>
__device__ __forceinline__ void* row_at(void* p, int64_t row, int64_t ld) {
  return static_cast<char*>(p) + row * ld * (TYPE == GM_LOSS_F32 ? 4 : 2);
}

// Threads that work on a row: 32 to 512 (long rows: 1024). Two sums over them, known to each. A group of one
// warp needs no barrier; the others meet at one of their own, and the sums' places alternate, so that one
// barrier a sum is enough.
struct Group {
  int size, id, t;
  float2* sh;  // [2][32] of this group
  int turn = 0;
  __device__ __forceinline__ Group(int size, float2* all) : size(size), id(threadIdx.x / size), t(threadIdx.x % size) {
    sh = all + id * 64;
  }
  __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      a += __shfl_xor_sync(kFull, a, d);
      b += __shfl_xor_sync(kFull, b, d);
    }
    if (size > 32) {
      float2* at = sh + 32 * turn;
      turn ^= 1;
      if ((t & 31) == 0) at[t >> 5] = make_float2(a, b);
      asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
      const int warps = size >> 5, lane = t & 31;
      const float2 x = lane < warps ? at[lane] : make_float2(0.f, 0.f);
      a = x.x, b = x.y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        a += __shfl_xor_sync(kFull, a, d);
        b += __shfl_xor_sync(kFull, b, d);
      }
    }
    return make_float2(a, b);
  }
};

struct NormArgs {
  gm_norm n;
  float inv_dim;
  void *x_out, *y;
  int64_t x_out_ld, y_ld;
  float4* stats;
};

// What a thread does with its eight columns of a row; shared by the kernels that hold a row and those that
// walk it.
template <int TYPE, bool VEC>
struct Columns {
  const gm_norm& n;
  int64_t t;
  int group;
  __device__ __forceinline__ void get(const void* p, float (&v)[kPer]) const {
    unpack<TYPE>(load<TYPE, VEC>(p, t, group, n.dim), v);
  }
  __device__ __forceinline__ void row(const void* p, int64_t row, int64_t ld, float (&v)[kPer]) const {
    get(row_at<TYPE>(p, row, ld), v);
  }
  __device__ __forceinline__ bool inside(int i) const { return column<VEC>(t, group, i) < n.dim; }
  // scale * gate
  __device__ __forceinline__ void factor(int64_t row_, float (&v)[kPer]) const {
    if (n.gate_kind == GM_GATE_NONE) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) v[i] = n.scale;
      return;
    }
    row(n.gate, n.gate_kind == GM_GATE_MATRIX ? row_ : 0, n.gate_ld, v);
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] *= n.scale;
  }
  // n(f) * after + after_bias
  __device__ __forceinline__ void project(const float (&unit)[kPer], float (&p)[kPer]) const {
    if (!n.after) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) p[i] = unit[i];
      return;
    }
    weigh(n.after, n.after_bias, unit, p);
  }
  __device__ __forceinline__ void weigh(const void* weight, const void* bias, const float (&unit)[kPer],
                                        float (&p)[kPer]) const {
    float w[kPer];
    get(weight, w);
    if (bias) {
      float b[kPer];
      get(bias, b);
#pragma unroll
      for (int i = 0; i < kPer; ++i) p[i] = fmaf(unit[i], w[i], b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) p[i] = unit[i] * w[i];
    }
  }
  // x' from x and f, given f's statistics
  __device__ __forceinline__ void update(int64_t row_, float2 of_f, const float (&f)[kPer], float (&x)[kPer]) const {
    float u[kPer], g[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) u[i] = n.after ? (f[i] - of_f.x) * of_f.y : f[i];
    project(u, u);
    factor(row_, g);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = fmaf(g[i], u[i], x[i]);
  }
};

// Mean and 1 / size of a row; SUM(g) gives the row's sum of g(i, value) over its elements.
template <class SUM>
__device__ __forceinline__ float2 statistics(const gm_norm& n, float inv_dim, SUM&& sum) {
  float mean = 0.f;
  if (n.norm == GM_NORM_LAYER) mean = sum([](float v) { return v; }) * inv_dim;
  const float square = sum([mean](float v) { return (v - mean) * (v - mean); }) * inv_dim;
  return make_float2(mean, 1.f / sqrtf(square + n.eps));
}

// ---- forward -------------------------------------------------------------------------------------
// A row in registers: NV turns of 8 columns a thread.
template <int TYPE, bool VEC, int NV>
__global__ void __launch_bounds__(512) k_norm_forward(const NormArgs a, int group) {
  __shared__ float2 sh[512 / 32 * 64];
  chain_wait();
  Group g(group, sh);
  const int groups = blockDim.x / group;
  const gm_norm& n = a.n;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id; row < n.n_rows;
       row += static_cast<int64_t>(gridDim.x) * groups) {
    float x[NV][kPer];
    float2 of_f = make_float2(0.f, 1.f), of_x = make_float2(0.f, 1.f);
    auto cols = [&](int v) { return Columns<TYPE, VEC>{n, g.t + int64_t(v) * (VEC ? group : group * kPer), group}; };
    auto row_sum = [&](const float (&v)[NV][kPer]) {
      return [&](auto&& f) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < kPer; ++i) s += cols(k).inside(i) ? f(v[k][i]) : 0.f;
        return g.sum(s, 0.f).x;
      };
    };
#pragma unroll
    for (int k = 0; k < NV; ++k) cols(k).row(n.x, row, n.x_ld, x[k]);
    if (n.f) {
      float f[NV][kPer];
#pragma unroll
      for (int k = 0; k < NV; ++k) cols(k).row(n.f, row, n.f_ld, f[k]);
      if (n.after) of_f = statistics(n, a.inv_dim, row_sum(f));
#pragma unroll
      for (int k = 0; k < NV; ++k) cols(k).update(row, of_f, f[k], x[k]);
    }
    if (a.x_out) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        store<TYPE, VEC>(row_at<TYPE>(a.x_out, row, a.x_out_ld), cols(k).t, group, n.dim, x[k]);
    }
    if (a.y) {
      of_x = statistics(n, a.inv_dim, row_sum(x));
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[k][i] = (x[k][i] - of_x.x) * of_x.y;
        cols(k).weigh(n.before, n.before_bias, x[k], x[k]);
        store<TYPE, VEC>(row_at<TYPE>(a.y, row, a.y_ld), cols(k).t, group, n.dim, x[k]);
      }
    }
    if (a.stats && g.t == 0) a.stats[row] = make_float4(of_f.x, of_f.y, of_x.x, of_x.y);
  }
}

// Rows longer than that: a block walks its row once for each sum and once to write it. What it reads again
// comes from L2. x is read for the last time before x_out is written, which may be the same memory.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(1024) k_norm_forward_long(const NormArgs a) {
  __shared__ float2 sh[64];
  chain_wait();
  const int group = blockDim.x;
  Group g(group, sh);
  const gm_norm& n = a.n;
  for (int64_t row = blockIdx.x; row < n.n_rows; row += gridDim.x) {
    float2 of_f = make_float2(0.f, 1.f), of_x = make_float2(0.f, 1.f);
    auto walk = [&](auto&& body) {
      for (int64_t at = 0; at < n.dim; at += group * kPer) {
        const Columns<TYPE, VEC> c{n, g.t + (VEC ? at / kPer : at), group};
        body(c);
      }
    };
    auto updated = [&](const Columns<TYPE, VEC>& c, float (&x)[kPer]) {
      c.row(n.x, row, n.x_ld, x);
      if (!n.f) return;
      float f[kPer];
      c.row(n.f, row, n.f_ld, f);
      c.update(row, of_f, f, x);
    };
    auto total = [&](auto&& values) {
      return [&](auto&& f) {
        float s = 0.f;
        walk([&](const Columns<TYPE, VEC>& c) {
          float v[kPer];
          values(c, v);
#pragma unroll
          for (int i = 0; i < kPer; ++i) s += c.inside(i) ? f(v[i]) : 0.f;
        });
        return g.sum(s, 0.f).x;
      };
    };
    if (n.after)
      of_f = statistics(n, a.inv_dim, total([&](const Columns<TYPE, VEC>& c, float (&v)[kPer]) { c.row(n.f, row, n.f_ld, v); }));
    if (a.y) of_x = statistics(n, a.inv_dim, total(updated));
    walk([&](const Columns<TYPE, VEC>& c) {
      float x[kPer];
      updated(c, x);
      if (a.x_out) store<TYPE, VEC>(row_at<TYPE>(a.x_out, row, a.x_out_ld), c.t, group, n.dim, x);
      if (a.y) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = (x[i] - of_x.x) * of_x.y;
        c.weigh(n.before, n.before_bias, x, x);
        store<TYPE, VEC>(row_at<TYPE>(a.y, row, a.y_ld), c.t, group, n.dim, x);
      }
    });
    if (a.stats && g.t == 0) a.stats[row] = make_float4(of_f.x, of_f.y, of_x.x, of_x.y);
  }
}

// ---- backward ------------------------------------------------------------------------------------
struct BackArgs {
  gm_norm n;
  gm_norm_grads o;
  float inv_dim;
  const float4* stats;
  const void *gx, *gy;
  int64_t gx_ld, gy_ld;
  bool need_x;      // whether anything but before and before_bias is wanted
  float* sums;      // [block][kSums][dim]
  float4* means;    // long rows: [row] the four means of the formulas
};

// A thread's columns of one row on the way back.
template <int TYPE, bool VEC>
struct Back {
  float gy[kPer], unit[kPer], unit_f[kPer], p[kPer], factor[kPer], dx[kPer], dp[kPer];
  // gy, n(x'), n(f), p, scale * gate
  __device__ __forceinline__ void start(const BackArgs& a, const Columns<TYPE, VEC>& c, int64_t row, float4 st,
                                        const Raw<TYPE>& x_raw, const Raw<TYPE>& f_raw, const Raw<TYPE>& gy_raw) {
    const gm_norm& n = a.n;
    float x[kPer];
    unpack<TYPE>(x_raw, x);
    unpack<TYPE>(gy_raw, gy);
    if (n.f) {
      unpack<TYPE>(f_raw, unit_f);
      if (n.after) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) unit_f[i] = (unit_f[i] - st.x) * st.y;
      }
      c.project(unit_f, p);
      c.factor(row, factor);
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = fmaf(factor[i], p[i], x[i]);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) unit[i] = (x[i] - st.z) * st.w;
  }
  // sums of d n(x') and of d, d = gy * before
  __device__ __forceinline__ float2 sums_x(const BackArgs& a, const Columns<TYPE, VEC>& c, float (&d)[kPer]) const {
    c.get(a.n.before, d);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      d[i] *= gy[i];
      s.x += c.inside(i) ? d[i] * unit[i] : 0.f;
      s.y += d[i];
    }
    return s;
  }
  __device__ __forceinline__ void to_x(const BackArgs& a, const Raw<TYPE>& gx_raw, const float (&d)[kPer], float2 mean,
                                       float4 st) {
    unpack<TYPE>(gx_raw, dx);
    if (!a.gy) return;
    if (a.n.norm != GM_NORM_LAYER) mean.y = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dx[i] = fmaf(d[i] - fmaf(unit[i], mean.x, mean.y), st.w, dx[i]);
  }
  // dp, and sums of e n(f) and of e, e = dp * after
  __device__ __forceinline__ float2 sums_f(const BackArgs& a, const Columns<TYPE, VEC>& c, float (&e)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) dp[i] = factor[i] * dx[i];
    float2 s = make_float2(0.f, 0.f);
    if (!a.n.after) return s;
    c.get(a.n.after, e);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      e[i] *= dp[i];
      s.x += c.inside(i) ? e[i] * unit_f[i] : 0.f;
      s.y += c.inside(i) ? e[i] : 0.f;
    }
    return s;
  }
  __device__ __forceinline__ void to_f(const BackArgs& a, const float (&e)[kPer], float2 mean, float4 st, float (&df)[kPer]) const {
    if (a.n.norm != GM_NORM_LAYER) mean.y = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      df[i] = a.n.after ? (e[i] - fmaf(unit_f[i], mean.x, mean.y)) * st.y : dp[i];
  }
  // by the gate's elements
  __device__ __forceinline__ void to_gate(const BackArgs& a, float (&dg)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) dg[i] = a.n.scale * dx[i] * p[i];
  }
  template <int N>
  __device__ __forceinline__ void add(const BackArgs& a, float (&acc)[N][kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[kSumBefore][i] = fmaf(gy[i], unit[i], acc[kSumBefore][i]);
    if constexpr (N > kSumBeforeBias) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[kSumBeforeBias][i] += gy[i];
    }
    if (!a.need_x || !a.n.f) return;
    if (a.n.after) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[kSumAfter][i] = fmaf(dp[i], unit_f[i], acc[kSumAfter][i]);
      if constexpr (N > kSumAfterBias) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[kSumAfterBias][i] += dp[i];
      }
    }
    if (a.n.gate_kind == GM_GATE_VECTOR) {
      float dg[kPer];
      to_gate(a, dg);
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[kSumGate][i] += dg[i];
    }
  }
};

// A row's four tensors as they are in memory.
template <int TYPE>
struct RowIn {
  Raw<TYPE> x, f, gx, gy;
  float4 st;
};
template <int TYPE, bool VEC>
__device__ __forceinline__ RowIn<TYPE> read_row(const BackArgs& a, int64_t t, int group, int64_t row) {
  RowIn<TYPE> r = {};
  const gm_norm& n = a.n;
  r.st = a.stats[row];
  r.x = load<TYPE, VEC>(row_at<TYPE>(n.x, row, n.x_ld), t, group, n.dim);
  if (n.f) r.f = load<TYPE, VEC>(row_at<TYPE>(n.f, row, n.f_ld), t, group, n.dim);
  if (a.gx) r.gx = load<TYPE, VEC>(row_at<TYPE>(a.gx, row, a.gx_ld), t, group, n.dim);
  if (a.gy) r.gy = load<TYPE, VEC>(row_at<TYPE>(a.gy, row, a.gy_ld), t, group, n.dim);
  return r;
}

// Rows held by a group; the next row is under way while one is worked on. SUMS: 3 (no biases) or 5.
template <int TYPE, bool VEC, int SUMS>
__global__ void __launch_bounds__(512) k_norm_backward(const BackArgs a, int group) {
  __shared__ float2 sh[512 / 32 * 64];
  chain_wait();
  Group g(group, sh);
  const int groups = blockDim.x / group;
  const gm_norm& n = a.n;
  const Columns<TYPE, VEC> c{n, g.t, group};
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  float acc[SUMS][kPer];
#pragma unroll
  for (int s = 0; s < SUMS; ++s)
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[s][i] = 0.f;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id;
  RowIn<TYPE> next;
  if (row < n.n_rows) next = read_row<TYPE, VEC>(a, g.t, group, row);
  for (; row < n.n_rows; row += step) {
    const RowIn<TYPE> in = next;
    if (row + step < n.n_rows) next = read_row<TYPE, VEC>(a, g.t, group, row + step);
    Back<TYPE, VEC> b;
    b.start(a, c, row, in.st, in.x, in.f, in.gy);
    if (a.need_x) {
      float d[kPer];
      float2 mean = make_float2(0.f, 0.f);
      if (a.gy) {
        mean = b.sums_x(a, c, d);
        mean = g.sum(mean.x, mean.y);
        mean.x *= a.inv_dim, mean.y *= a.inv_dim;
      }
      b.to_x(a, in.gx, d, mean, in.st);
      if (a.o.x) store<TYPE, VEC>(row_at<TYPE>(a.o.x, row, a.o.x_ld), g.t, group, n.dim, b.dx);
      if (n.f) {
        mean = b.sums_f(a, c, d);
        if (n.after && a.o.f) {
          mean = g.sum(mean.x, mean.y);
          mean.x *= a.inv_dim, mean.y *= a.inv_dim;
        }
        if (a.o.f) {
          float df[kPer];
          b.to_f(a, d, mean, in.st, df);
          store<TYPE, VEC>(row_at<TYPE>(a.o.f, row, a.o.f_ld), g.t, group, n.dim, df);
        }
        if (a.o.gate && n.gate_kind == GM_GATE_MATRIX) {
          b.to_gate(a, d);
          store<TYPE, VEC>(row_at<TYPE>(a.o.gate, row, a.o.gate_ld), g.t, group, n.dim, d);
        }
      }
    }
    if (a.sums) b.add(a, acc);
  }
  if (!a.sums) return;
  // the block's groups one after another, in shared memory
  extern __shared__ float block_sums[];  // [SUMS][dim] where a block has several groups
  float* out = a.sums + static_cast<int64_t>(blockIdx.x) * kSums * n.dim;
  float* to = groups > 1 ? block_sums : out;
  for (int k = 0; k < groups; ++k) {
    if (g.id == k) {
#pragma unroll
      for (int s = 0; s < SUMS; ++s)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (c.inside(i)) {
            float* at = to + s * n.dim + column<VEC>(g.t, group, i);
            *at = k > 0 ? *at + acc[s][i] : acc[s][i];
          }
    }
    if (groups > 1) __syncthreads();
  }
  if (groups > 1)
    for (int64_t i = threadIdx.x; i < SUMS * n.dim; i += blockDim.x) out[i] = block_sums[i];
}

// Rows longer than that: a block walks its row three times and leaves the row's means, by which
// k_norm_columns sums over rows.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(512) k_norm_backward_long(const BackArgs a) {
  __shared__ float2 sh[64];
  chain_wait();
  const int group = blockDim.x;
  Group g(group, sh);
  const gm_norm& n = a.n;
  for (int64_t row = blockIdx.x; row < n.n_rows; row += gridDim.x) {
    float2 mean_x = make_float2(0.f, 0.f), mean_f = make_float2(0.f, 0.f);
    auto walk = [&](auto&& body) {
      for (int64_t at = 0; at < n.dim; at += group * kPer) {
        const Columns<TYPE, VEC> c{n, g.t + (VEC ? at / kPer : at), group};
        const RowIn<TYPE> in = read_row<TYPE, VEC>(a, c.t, group, row);
        Back<TYPE, VEC> b;
        b.start(a, c, row, in.st, in.x, in.f, in.gy);
        body(c, b, in);
      }
    };
    auto mean_of = [&](float2 s) {
      s = g.sum(s.x, s.y);
      return make_float2(s.x * a.inv_dim, s.y * a.inv_dim);
    };
    float2 s = make_float2(0.f, 0.f);
    if (a.gy) {
      walk([&](const Columns<TYPE, VEC>& c, Back<TYPE, VEC>& b, const RowIn<TYPE>&) {
        float d[kPer];
        const float2 x = b.sums_x(a, c, d);
        s.x += x.x, s.y += x.y;
      });
      mean_x = mean_of(s);
    }
    auto to_x = [&](const Columns<TYPE, VEC>& c, Back<TYPE, VEC>& b, const RowIn<TYPE>& in) {
      float d[kPer];
      if (a.gy) b.sums_x(a, c, d);
      b.to_x(a, in.gx, d, mean_x, in.st);
    };
    if (n.after && a.o.f) {
      s = make_float2(0.f, 0.f);
      walk([&](const Columns<TYPE, VEC>& c, Back<TYPE, VEC>& b, const RowIn<TYPE>& in) {
        float e[kPer];
        to_x(c, b, in);
        const float2 x = b.sums_f(a, c, e);
        s.x += x.x, s.y += x.y;
      });
      mean_f = mean_of(s);
    }
    walk([&](const Columns<TYPE, VEC>& c, Back<TYPE, VEC>& b, const RowIn<TYPE>& in) {
      to_x(c, b, in);
      if (a.o.x) store<TYPE, VEC>(row_at<TYPE>(a.o.x, row, a.o.x_ld), c.t, group, n.dim, b.dx);
      if (!n.f) return;
      float e[kPer], df[kPer];
      b.sums_f(a, c, e);
      if (a.o.f) {
        b.to_f(a, e, mean_f, in.st, df);
        store<TYPE, VEC>(row_at<TYPE>(a.o.f, row, a.o.f_ld), c.t, group, n.dim, df);
      }
      if (a.o.gate && n.gate_kind == GM_GATE_MATRIX) {
        b.to_gate(a, df);
        store<TYPE, VEC>(row_at<TYPE>(a.o.gate, row, a.o.gate_ld), c.t, group, n.dim, df);
      }
    });
    if (g.t == 0) a.means[row] = make_float4(mean_x.x, mean_x.y, mean_f.x, mean_f.y);
  }
}

// Sums over rows of long rows: a block takes 32 * kPer columns of a range of rows, its 8 warps every eighth.
constexpr int kColumnWarps = 8, kColumns = 32 * kPer;
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(32 * kColumnWarps) k_norm_columns(const BackArgs a, int64_t rows_a_block) {
  __shared__ float sh[kSums][kColumns];
  chain_wait();
  const gm_norm& n = a.n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * kColumns;
  const Columns<TYPE, VEC> c{n, (VEC ? col0 / kPer : col0) + lane, 32};
  float acc[kSums][kPer];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[s][i] = 0.f;
  const int64_t first = blockIdx.y * rows_a_block, end = min(n.n_rows, first + rows_a_block);
  for (int64_t row = first + warp; row < end; row += kColumnWarps) {
    const RowIn<TYPE> in = read_row<TYPE, VEC>(a, c.t, 32, row);
    Back<TYPE, VEC> b;
    b.start(a, c, row, in.st, in.x, in.f, in.gy);
    if (a.need_x) {
      const float4 m = a.means[row];
      float d[kPer];
      if (a.gy) b.sums_x(a, c, d);
      b.to_x(a, in.gx, d, make_float2(m.x, m.y), in.st);
      if (n.f) b.sums_f(a, c, d);
    }
    b.add(a, acc);
  }
  for (int k = 0; k < kColumnWarps; ++k) {
    if (warp == k) {
#pragma unroll
      for (int s = 0; s < kSums; ++s)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          float* at = &sh[s][column<VEC>(lane, 32, i)];
          *at = k > 0 ? *at + acc[s][i] : acc[s][i];
        }
    }
    __syncthreads();
  }
  float* out = a.sums + static_cast<int64_t>(blockIdx.y) * kSums * n.dim;
  for (int i = threadIdx.x; i < kSums * kColumns; i += blockDim.x) {
    const int64_t col = col0 + i % kColumns;
    if (col < n.dim) out[i / kColumns * n.dim + col] = sh[i / kColumns][i % kColumns];
  }
}

// The blocks' sums joined: 32 columns a block, its 8 warps every eighth part. blockIdx.y: which sum.
struct JoinTo {
  void* out[kSums];
};
template <int TYPE>
__global__ void __launch_bounds__(256) k_norm_join(const float* __restrict__ sums, int parts, int64_t dim, const JoinTo to) {
  __shared__ float sh[8][32];
  chain_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.y;
  void* out = to.out[s];
  if (!out) return;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float x = 0.f;
  if (col < dim) {
    const float* p = sums + s * dim + col;
#pragma unroll 8
    for (int k = warp; k < parts; k += 8) x += p[static_cast<int64_t>(k) * kSums * dim];
  }
  sh[warp][lane] = x;
  __syncthreads();
  if (warp != 0 || col >= dim) return;
#pragma unroll
  for (int k = 1; k < 8; ++k) x += sh[k][lane];
  if constexpr (TYPE == GM_LOSS_F32) static_cast<float*>(out)[col] = x;
  else static_cast<uint16_t*>(out)[col] = static_cast<uint16_t>(round16<TYPE>(x));
}

// ---- host ----------------------------------------------------------------------------------------
gm_status check_norm(const gm_norm* n, bool forward) {
  if (!n || n->n_rows < 0 || n->dim < 1) return GM_ERR_INVALID_ARG;
  if (n->n_rows > kMostIndex || n->dim > (int64_t(1) << 24)) return GM_ERR_INDEX_OVERFLOW;
  if (n->type != GM_LOSS_F32 && n->type != GM_LOSS_BF16 && n->type != GM_LOSS_F16) return GM_ERR_INVALID_ARG;
  if (n->norm != GM_NORM_RMS && n->norm != GM_NORM_LAYER) return GM_ERR_INVALID_ARG;
  if (n->gate_kind < GM_GATE_NONE || n->gate_kind > GM_GATE_MATRIX) return GM_ERR_INVALID_ARG;
  if (!std::isfinite(n->scale) || !std::isfinite(n->eps) || n->eps < 0.f) return GM_ERR_INVALID_ARG;
  const bool rows = n->n_rows > 0;
  if (n->after_bias && !n->after) return GM_ERR_INVALID_ARG;
  if (n->before_bias && !n->before) return GM_ERR_INVALID_ARG;
  if ((n->after || n->gate_kind != GM_GATE_NONE) && rows && !n->f) return GM_ERR_INVALID_ARG;
  if ((n->gate_kind == GM_GATE_VECTOR || (n->gate_kind == GM_GATE_MATRIX && rows)) && !n->gate) return GM_ERR_INVALID_ARG;
  if (rows && !n->x) return GM_ERR_INVALID_ARG;
  const int64_t es = elem_bytes(n->type);
  for (const void* p : {n->x, n->f, n->after, n->after_bias, n->gate, n->before, n->before_bias})
    if (!aligned(p, es)) return GM_ERR_INVALID_ARG;
  if (n->x_ld < n->dim || (n->f && n->f_ld < n->dim) || (n->gate_kind == GM_GATE_MATRIX && n->gate_ld < n->dim))
    return GM_ERR_INVALID_ARG;
  if (n->x_ld > kMostLd || n->f_ld > kMostLd || n->gate_ld > kMostLd) return GM_ERR_INDEX_OVERFLOW;
  return GM_OK;
}

gm_status check_rows(const gm_norm& n, const void* p, int64_t ld) {
  if (!p) return GM_OK;
  if (!aligned(p, elem_bytes(n.type)) || ld < n.dim) return GM_ERR_INVALID_ARG;
  return ld > kMostLd ? GM_ERR_INDEX_OVERFLOW : GM_OK;
}

// Whether all rows (ld 0: one vector) start and end on 16-byte boundaries.
struct Sixteen {
  bool ok = true;
  int64_t es, dim, rows;
  explicit Sixteen(const gm_norm& n) : es(elem_bytes(n.type)), dim(n.dim), rows(n.n_rows) {
    ok = dim * es % 16 == 0;
    (*this)(n.x, n.x_ld)(n.f, n.f_ld)(n.after, 0)(n.after_bias, 0)(n.before, 0)(n.before_bias, 0);
    (*this)(n.gate, n.gate_kind == GM_GATE_MATRIX ? n.gate_ld : 0);
  }
  Sixteen& operator()(const void* p, int64_t ld) {
    if (p) ok = ok && aligned(p, 16) && (rows <= 1 || ld * es % 16 == 0);
    return *this;
  }
};

// Threads of a row held in registers, `turns` times 8 columns each.
int group_of(int64_t dim, int turns) { return static_cast<int>(up(div_up(dim, kPer * turns), 32)); }

template <class F>
cudaError_t by_type(int32_t type, bool vec, F&& f) {
  using std::integral_constant;
#define GM_BY(T)                                                                                   \
  return vec ? f(integral_constant<int, T>(), integral_constant<bool, true>()) : f(integral_constant<int, T>(), integral_constant<bool, false>())
  switch (type) {
    case GM_LOSS_F32: GM_BY(GM_LOSS_F32);
    case GM_LOSS_BF16: GM_BY(GM_LOSS_BF16);
    default: GM_BY(GM_LOSS_F16);
  }
#undef GM_BY
}

gm_status done(cudaError_t e) { return cudaGetLastError() != cudaSuccess || e != cudaSuccess ? GM_ERR_CUDA : GM_OK; }

gm_status norm_forward(const gm_norm& n, cudaStream_t s, void* x_out, int64_t x_out_ld, void* y, int64_t y_ld, float* stats) {
  const bool vec = Sixteen(n)(x_out, x_out_ld)(y, y_ld).ok;
  const NormArgs a{n, 1.f / static_cast<float>(n.dim), x_out, y, x_out_ld, y_ld, reinterpret_cast<float4*>(stats)};
  return done(by_type(n.type, vec, [&](auto t, auto v) {
    constexpr int T = decltype(t)::value;
    constexpr bool V = decltype(v)::value;
    if (n.dim > kHeldDim)
      return launch_chained(k_norm_forward_long<T, V>, grid_for(n.n_rows, 1), n.dim > 2 * kHeldDim ? 1024 : 512, 0, s, 1, a);
    // 4 turns for many long rows, so that several rows are under way on an SM; one thread a column group for few
    const int turns = n.dim > 1024 && n.n_rows >= 512 ? 2 : 1;
    const int group = group_of(n.dim, turns), block = std::max(group, 128) / group * group;
    const unsigned grid = grid_for(n.n_rows, block / group, int64_t(1) << 30);
    return turns == 2 ? launch_chained(k_norm_forward<T, V, 2>, grid, block, 0, s, 1, a, group)
                      : launch_chained(k_norm_forward<T, V, 1>, grid, block, 0, s, 1, a, group);
  }));
}

// How a backward call is cut, and where its workspace lies.
struct NormPlan {
  Arena a;
  bool long_rows;
  int group = 0, block = 0;
  int64_t parts, rows_a_part = 0;  // of the sums over rows
  size_t o_sums, o_means = 0;
  NormPlan(const gm_norm& n, int sms) {
    long_rows = n.dim > kHeldDim;
    if (long_rows) {
      const int64_t slabs = div_up(n.dim, kColumns);
      parts = std::max<int64_t>(1, std::min<int64_t>(div_up(4 * sms, slabs), div_up(n.n_rows, 4 * kColumnWarps)));
      rows_a_part = div_up(n.n_rows, parts);
      parts = div_up(n.n_rows, rows_a_part);
      o_means = a.add(n.n_rows * 16);
    } else {
      group = group_of(n.dim, 1);
      block = std::max(group, 256) / group * group;
      parts = std::min<int64_t>(div_up(n.n_rows, block / group), sms * std::max(1, 512 / block));
    }
    o_sums = a.add(parts * kSums * n.dim * 4);
  }
};

gm_status norm_backward(const gm_norm& n, const gm_layer_config& cfg, cudaStream_t s, const float* stats, const void* gx,
                        int64_t gx_ld, const void* gy, int64_t gy_ld, const gm_norm_grads& o) {
  const int sms = sm_count(kMostBlocks);
  if (sms <= 0) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  const int64_t es = elem_bytes(n.type);
  if (n.n_rows == 0) {
    for (void* p : {o.after, o.after_bias, o.before, o.before_bias, n.gate_kind == GM_GATE_VECTOR ? o.gate : nullptr})
      if (p && cudaMemsetAsync(p, 0, n.dim * es, s) != cudaSuccess) {
        cudaGetLastError();
        return GM_ERR_CUDA;
      }
    return GM_OK;
  }
  NormPlan p(n, sms);
  const gm_status rc = p.a.open(cfg.workspace, cfg.workspace_bytes, s);
  if (rc != GM_OK) return rc;
  JoinTo to = {};
  to.out[kSumBefore] = o.before;
  to.out[kSumAfter] = o.after;
  to.out[kSumGate] = n.gate_kind == GM_GATE_VECTOR ? o.gate : nullptr;
  to.out[kSumBeforeBias] = o.before_bias;
  to.out[kSumAfterBias] = o.after_bias;
  bool sums = false;
  for (void* q : to.out) sums = sums || q;
  const bool biases = o.before_bias || o.after_bias;
  BackArgs a{n, o, 1.f / static_cast<float>(n.dim), reinterpret_cast<const float4*>(stats), gx, gy, gx_ld, gy_ld};
  a.need_x = o.x || o.f || o.gate || o.after || o.after_bias;
  a.sums = sums ? p.a.at<float>(p.o_sums) : nullptr;
  a.means = p.long_rows ? p.a.at<float4>(p.o_means) : nullptr;
  Sixteen all(n);
  all(gx, gx_ld)(gy, gy_ld)(o.x, o.x_ld)(o.f, o.f_ld)(o.gate, n.gate_kind == GM_GATE_MATRIX ? o.gate_ld : 0);
  return done(by_type(n.type, all.ok, [&](auto t, auto v) {
    constexpr int T = decltype(t)::value;
    constexpr bool V = decltype(v)::value;
    cudaError_t e = cudaSuccess;
    if (p.long_rows) {
      if (a.need_x) e = launch_chained(k_norm_backward_long<T, V>, grid_for(n.n_rows, 1), 512, 0, s, 1, a);
      if (e == cudaSuccess && sums) {
        const dim3 grid(static_cast<unsigned>(div_up(n.dim, kColumns)), static_cast<unsigned>(p.parts));
        e = launch_chained(k_norm_columns<T, V>, grid, 32 * kColumnWarps, 0, s, 1, a, p.rows_a_part);
      }
    } else {
      const int groups = p.block / p.group;
      const size_t smem = sums && groups > 1 ? (biases ? 5 : 3) * n.dim * 4 : 0;
      e = biases ? launch_chained(k_norm_backward<T, V, 5>, static_cast<unsigned>(p.parts), p.block, smem, s, 1, a, p.group)
                 : launch_chained(k_norm_backward<T, V, 3>, static_cast<unsigned>(p.parts), p.block, smem, s, 1, a, p.group);
    }
    if (e == cudaSuccess && sums) {
      const dim3 grid(static_cast<unsigned>(div_up(n.dim, 32)), biases ? 5 : 3);
      e = launch_chained(k_norm_join<T>, grid, 256, 0, s, 1, a.sums, static_cast<int>(p.parts), n.dim, to);
    }
    return e;
  }));
}

}  // namespace

}  // namespace gm

extern "C" gm_status gm_norm_forward(const gm_norm* n, void* stream, void* x_out, int64_t x_out_ld, void* y, int64_t y_ld,
                                     float* stats) {
  gm::NvtxRange range("gm_norm_forward");
  gm_status rc = gm::check_norm(n, true);
  if (rc == GM_OK) rc = gm::check_rows(*n, x_out, x_out_ld);
  if (rc == GM_OK) rc = gm::check_rows(*n, y, y_ld);
  if (rc != GM_OK) return rc;
  if ((y && !n->before) || !gm::aligned(stats, 16)) return GM_ERR_INVALID_ARG;
  if (x_out == n->x && x_out && x_out_ld != n->x_ld && n->n_rows > 1) return GM_ERR_INVALID_ARG;
  if (n->n_rows > 0 && ((n->before && !y) || (n->f && !x_out) || (!x_out && !y))) return GM_ERR_INVALID_ARG;
  if (n->n_rows == 0) return GM_OK;
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  return gm::norm_forward(*n, static_cast<cudaStream_t>(stream), x_out, x_out_ld, y, y_ld, stats);
}

extern "C" gm_status gm_norm_backward(const gm_norm* n, const gm_layer_config* cfg, void* stream, const float* stats,
                                      const void* gx, int64_t gx_ld, const void* gy, int64_t gy_ld,
                                      const gm_norm_grads* grads) {
  gm::NvtxRange range("gm_norm_backward");
  gm_status rc = gm::check_norm(n, false);
  if (rc != GM_OK) return rc;
  if (!grads) return GM_ERR_INVALID_ARG;
  const gm_norm_grads& o = *grads;
  const struct { const void* p; int64_t ld; } rows[] = {{gx, gx_ld}, {gy, gy_ld}, {o.x, o.x_ld}, {o.f, o.f_ld}};
  for (const auto& r : rows) {
    rc = gm::check_rows(*n, r.p, r.ld);
    if (rc != GM_OK) return rc;
  }
  if (n->gate_kind == GM_GATE_MATRIX) rc = gm::check_rows(*n, o.gate, o.gate_ld);
  if (rc != GM_OK) return rc;
  const int64_t es = gm::elem_bytes(n->type);
  for (const void* p : {o.gate, o.after, o.after_bias, o.before, o.before_bias})
    if (!gm::aligned(p, es)) return GM_ERR_INVALID_ARG;
  if ((o.f && !n->f && n->n_rows > 0) || (o.gate && n->gate_kind == GM_GATE_NONE) || (o.after && !n->after) ||
      (o.after_bias && !n->after_bias) || (o.before && !n->before) || (o.before_bias && !n->before_bias) || (gy && !n->before))
    return GM_ERR_INVALID_ARG;
  if (!o.x && !o.f && !o.gate && !o.after && !o.after_bias && !o.before && !o.before_bias) return GM_ERR_INVALID_ARG;
  if (!gm::aligned(stats, 16) || (n->n_rows > 0 && !stats)) return GM_ERR_INVALID_ARG;
  gm_layer_config c = {};
  if (cfg) c = *cfg;
  if (c.workspace && (!gm::aligned(c.workspace, 256) || c.workspace_bytes < 0)) return GM_ERR_INVALID_ARG;
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  return gm::norm_backward(*n, c, static_cast<cudaStream_t>(stream), stats, gx, gx_ld, gy, gy_ld, o);
}

extern "C" gm_status gm_norm_workspace(const gm_norm* n, int64_t* bytes) {
  if (!bytes) return GM_ERR_INVALID_ARG;
  const gm_status rc = gm::check_norm(n, false);
  if (rc != GM_OK) return rc;
  *bytes = 0;
  if (n->n_rows == 0) return GM_OK;
  const int sms = gm::sm_count(gm::kMostBlocks);
  if (sms <= 0) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  *bytes = static_cast<int64_t>(gm::NormPlan(*n, sms).a.used);
  return GM_OK;
}
