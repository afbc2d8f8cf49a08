// gm_norm.cu -- the norms around a residual with its gate and scale (include/gm_layers.h), forward and
// backward.
//
// Every element is read and written once: a group of threads holds a row in registers, the row's means are the
// group's sums. Memory should bound it; what stands in the way is the instructions an element takes, so what depends
// on the column alone (after * gate, before) is formed once, and what depends on the row alone (1 / size, the
// scale, the means) is gathered into factors of the row. The backward pass also sums over rows (gradients of
// weights, of a gate that is a vector): a thread keeps its columns from row to row and adds them up in
// shared memory, and the blocks' sums are joined by a second kernel in a fixed order, so no value is
// added atomically. Two sums serve all where the gate is a vector or none: with A_j = sum over rows of dx n(f), B_j of dx,
//   dafter = scale gate A, dgate = scale (after A + after_bias B), dafter_bias = scale gate B.
// Rows longer than a block holds (kHeldDim) are walked several times instead, their weights read again each time: 4096 x 12288
// bf16 rms 214 us forward (60 at a copy's rate) and 578 backward (89), 2048 x 16384 138 and 402.
//
// 8192 x 4096 bf16, rms, after, gate vector: forward 47 us for 268 MB, 5.7 TB/s or 85 % of what a copy reaches; backward 78 us
// for 403 MB, 5.2 TB/s or 76 %, and 7 us to join the blocks' sums. 24 % of the warps fit (registers); what they wait for is
// divided between memory, the sums' exchanges and shared memory. The general form, with twice the instructions an element: layer norm
// with biases 97 and 131 us (four sums one after another), a matrix of gates 78 and 143. One row of 4096: 6 us, a launch and three
// trips to memory.
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gm_device.cuh"
#include "gm_host.h"
#include "gm_layers.h"
#include "gm_loss.h"
#include "gm_umma.cuh"

namespace gm {

namespace {

constexpr int kPer = 8;         // elements of a row a thread holds together: 16 bytes of a 16-bit type
constexpr int kHeldDim = 8192;  // of a row held by at most 512 threads, 16 elements each
constexpr int kLongBlock = 512;
constexpr int kSmThreads = 512;  // of the forward pass on an SM: by registers
constexpr int kSums = 4;        // over rows, at most
enum { kSumBefore, kSumA, kSumBeforeBias, kSumB };

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
  for (int i = 0; i < kPer; i += 2) {
    if constexpr (TYPE == GM_LOSS_F32) {
      v[i] = __uint_as_float(r.w[i]), v[i + 1] = __uint_as_float(r.w[i + 1]);
    } else if constexpr (TYPE == GM_LOSS_BF16) {
      v[i] = __uint_as_float(r.w[i / 2] << 16), v[i + 1] = __uint_as_float(r.w[i / 2] & 0xffff0000u);
    } else {
      const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i / 2]));
      v[i] = x.x, v[i + 1] = x.y;
    }
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
    for (int i = 0; i < kPer; i += 2) {
      if constexpr (TYPE == GM_LOSS_BF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v[i], v[i + 1]);
        r.w[i / 2] = *reinterpret_cast<const uint32_t*>(&x);
      } else {
        const __half2 x = __floats2half2_rn(v[i], v[i + 1]);
        r.w[i / 2] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
  }
  return r;
}

// Columns of a thread: VEC (rows and vectors start and end on 16 bytes): 8 consecutive ones; else one
// of every `group`, so that a warp's loads of single elements lie together.
template <bool VEC>
__device__ __forceinline__ int column(int t, int group, int i) {
  return VEC ? t * kPer + i : t + i * group;
}
// t: the thread's place in its group, plus kPer * group (VEC: group) for the next turn of a long row.
template <int TYPE, bool VEC>
__device__ __forceinline__ Raw<TYPE> load(const void* row, int t, int group, int dim) {
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
      const int c = column<false>(t, group, i);
      if (c >= dim) continue;
      if constexpr (TYPE == GM_LOSS_F32) r.w[i] = static_cast<const uint32_t*>(row)[c];
      else r.w[i / 2] |= static_cast<uint32_t>(static_cast<const uint16_t*>(row)[c]) << (i & 1 ? 16 : 0);
    }
  }
  return r;
}
template <int TYPE, bool VEC>
__device__ __forceinline__ void store(void* row, int t, int group, int dim, const float (&v)[kPer]) {
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
      const int c = column<false>(t, group, i);
      if (c >= dim) continue;
      if constexpr (TYPE == GM_LOSS_F32) static_cast<uint32_t*>(row)[c] = r.w[i];
      else static_cast<uint16_t*>(row)[c] = static_cast<uint16_t>(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2]);
    }
  }
}
// Row i of a matrix. SHORT: rows are less than 4 GB apart, so that one multiplication of 32 bits does.
template <int TYPE, bool SHORT, class P>
__device__ __forceinline__ P* row_at(P* m, int64_t ld, int64_t i) {
  using Byte = std::conditional_t<std::is_const<P>::value, const char, char>;
  constexpr int kBytes = TYPE == GM_LOSS_F32 ? 4 : 2;
  if constexpr (SHORT) return static_cast<Byte*>(m) + static_cast<uint64_t>(static_cast<uint32_t>(i)) * static_cast<uint32_t>(ld * kBytes);
  else return static_cast<Byte*>(m) + i * ld * kBytes;
}

// Threads that work on a row. A group of one warp needs no barrier; the others meet at one of their own, and the sums' places
// alternate, so that one barrier a sum is enough.
template <int N>
struct Sums {
  float v[N];
};
struct Group {
  int size, id, t;
  float* sh;  // [2][2][16] of this group
  int turn = 0;
  __device__ __forceinline__ Group(int size, float* all) : size(size), id(threadIdx.x / size), t(threadIdx.x % size) {
    sh = all + id * 64;
  }
  template <int N>  // 1 or 2 sums over the group's threads, known to each
  __device__ __forceinline__ Sums<N> sum(Sums<N> s) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) s.v[k] += __shfl_xor_sync(kFull, s.v[k], d);
    if (size > 32) {
      float* at = sh + 32 * turn;
      turn ^= 1;
      if ((t & 31) == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) at[16 * k + (t >> 5)] = s.v[k];
      }
      asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(size) : "memory");
      const int warps = size >> 5, lane = t & 15;  // at most 16
#pragma unroll
      for (int k = 0; k < N; ++k) s.v[k] = lane < warps ? at[16 * k + lane] : 0.f;
#pragma unroll
      for (int d = 8; d > 0; d >>= 1)
#pragma unroll
        for (int k = 0; k < N; ++k) s.v[k] += __shfl_xor_sync(kFull, s.v[k], d);
    }
    return s;
  }
};

// Eight of a thread's columns: where they are, and which of them lie in the row.
template <int TYPE, bool VEC>
struct Columns {
  int t, group, dim;
  __device__ __forceinline__ void get(const void* p, float (&v)[kPer]) const { unpack<TYPE>(load<TYPE, VEC>(p, t, group, dim), v); }
  __device__ __forceinline__ Raw<TYPE> raw(const void* p) const { return load<TYPE, VEC>(p, t, group, dim); }
  __device__ __forceinline__ void put(void* p, const float (&v)[kPer]) const { store<TYPE, VEC>(p, t, group, dim, v); }
  // rows of whole 16 bytes: the same for all that lie in one 16
  __device__ __forceinline__ bool inside(int i) const {
    return column<VEC>(t, group, !VEC ? i : TYPE == GM_LOSS_F32 ? i & 4 : 0) < dim;
  }
  // The same from the row's last columns where these lie past its end (their weights are 0): no load then waits for a
  // comparison. For rows of whole pieces.
  __device__ __forceinline__ Raw<TYPE> raw_or_last(const void* p) const {
    Raw<TYPE> r;
    const uint4* q = static_cast<const uint4*>(p) + min(t, dim / kPer - 1) * (kWords<TYPE> / 4);
#pragma unroll
    for (int h = 0; h < kWords<TYPE> / 4; ++h) {
      const uint4 x = q[h];
      r.w[4 * h] = x.x, r.w[4 * h + 1] = x.y, r.w[4 * h + 2] = x.z, r.w[4 * h + 3] = x.w;
    }
    return r;
  }
};
// LEAN: no means taken off, no biases, a gate that is a vector or none: half the instructions of the general form
// (8192 x 4096 bf16 backward: 78 us, 131 with layer norm and biases).
__device__ __forceinline__ bool is_matrix(const gm_norm& n) { return n.gate_kind == GM_GATE_MATRIX; }

// What depends on the column alone: h = after * gate (that of a matrix comes with the row), hc = after_bias * gate,
// before (as it is in memory) and its bias.
template <int TYPE, bool VEC, bool LEAN>
struct Weights {
  float h[kPer], hc[LEAN ? 1 : kPer];
  Raw<TYPE> before, before_bias;
  __device__ __forceinline__ void read(const gm_norm& n, const Columns<TYPE, VEC>& c) {
    // columns past the end have weights of 0
#pragma unroll
    for (int i = 0; i < kPer; ++i) h[i] = n.f && c.inside(i) ? 1.f : 0.f;
    if (n.after) c.get(n.after, h);
    if constexpr (!LEAN) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) hc[i] = 0.f;
      if (n.after_bias) c.get(n.after_bias, hc);
    }
    if (n.gate_kind == GM_GATE_VECTOR) {
      float g[kPer];
      c.get(n.gate, g);
#pragma unroll
      for (int i = 0; i < kPer; ++i) h[i] *= g[i];
      if constexpr (!LEAN) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) hc[i] *= g[i];
      }
    }
    before = before_bias = Raw<TYPE>{};
    if (n.before) before = c.raw(n.before);
    if (!LEAN && n.before_bias) before_bias = c.raw(n.before_bias);
  }
  // x' from x and f less its mean; factor: scale / size of f; g: the row's gates, of a matrix
  __device__ __forceinline__ void update(const gm_norm& n, float (&x)[kPer], const float (&f)[kPer], float factor, const float (&g)[kPer]) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      if constexpr (LEAN) {
        x[i] = fmaf(f[i] * h[i], factor, x[i]);
      } else {
        const float p = fmaf(f[i] * h[i], factor, hc[i] * n.scale);
        x[i] = is_matrix(n) ? fmaf(p, g[i], x[i]) : x[i] + p;
      }
    }
  }
};

// The weights of a thread's columns, read once and kept; by the general form with 16 columns a thread, whose registers they
// would fill, at each use, from L1. That form does not ask for the next row either. Backward, 4096 x 8192 layer norm with biases:
// bf16 156 us, f32 276; with all kept (spilled) 199 and 551. Forward and backward 275 bf16; walked, as longer rows are, 932 (8192 x 4104).
// The general backward form is at its 128 registers all the same: it spills 56 to 256 bytes in f32, 100 in 16 bits with 16
// columns a thread of rows off 16-byte boundaries.
template <int TYPE, bool VEC, int NV, bool LEAN>
struct Kept {
  static constexpr bool kAll = LEAN || NV == 1;
  Weights<TYPE, VEC, LEAN> w[kAll ? NV : 1];
  __device__ __forceinline__ void read(const gm_norm& n, const Columns<TYPE, VEC> (&c)[NV]) {
    if constexpr (kAll) {
#pragma unroll
      for (int k = 0; k < NV; ++k) w[k].read(n, c[k]);
    }
  }
  __device__ __forceinline__ Weights<TYPE, VEC, LEAN> of(const gm_norm& n, const Columns<TYPE, VEC> (&c)[NV], int k) const {
    if constexpr (kAll) {
      return w[k];
    } else {
      Weights<TYPE, VEC, LEAN> x;
      x.read(n, c[k]);
      return x;
    }
  }
};

template <bool LEAN>
__device__ __forceinline__ void less(float (&v)[kPer], float mean) {
  if constexpr (!LEAN) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] -= mean;
  }
}

struct NormArgs {
  gm_norm n;
  float inv_dim;
  void *x_out, *y;
  int64_t x_out_ld, y_ld;
  float4* stats;
};

// Mean and 1 / size of a row: sum(g) gives the sum of g(value) over its elements.
template <bool LEAN, class SUM>
__device__ __forceinline__ float2 statistics(const gm_norm& n, float inv_dim, SUM&& sum) {
  float mean = 0.f;
  if (!LEAN && n.norm == GM_NORM_LAYER) mean = sum([](float v) { return v; }) * inv_dim;
  const float square = sum([mean](float v) { return LEAN ? v * v : (v - mean) * (v - mean); }) * inv_dim;
  return make_float2(mean, 1.f / sqrtf(square + n.eps));
}

// ---- forward -------------------------------------------------------------------------------------
// A row in registers: NV turns of 8 columns a thread.
template <int TYPE, bool VEC, int NV, bool LEAN>
__global__ void __launch_bounds__(512, 1) k_norm_forward(const NormArgs a, int group) {
  __shared__ float sh[16 * 64];
  chain_wait();
  Group g(group, sh);
  const gm_norm& n = a.n;
  const int dim = static_cast<int>(n.dim), groups = blockDim.x / group;
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + g.id;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  Columns<TYPE, VEC> c[NV];
  Kept<TYPE, VEC, NV, LEAN> w;
#pragma unroll
  for (int k = 0; k < NV; ++k) c[k] = Columns<TYPE, VEC>{g.t + k * (VEC ? group : group * kPer), group, dim};
  w.read(n, c);
  constexpr auto at = [](auto* m, int64_t ld, int64_t i) { return row_at<TYPE, LEAN>(m, ld, i); };
  Raw<TYPE> x_next[NV], f_next[NV], gate_next[NV];
  auto ask = [&](int64_t i) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x_next[k] = c[k].raw(at(n.x, n.x_ld, i));
      if (n.f) f_next[k] = c[k].raw(at(n.f, n.f_ld, i));
      if (!LEAN && is_matrix(n)) gate_next[k] = c[k].raw(at(n.gate, n.gate_ld, i));
    }
  };
  if (row < n.n_rows && w.kAll) ask(row);
  for (; row < n.n_rows; row += step) {
    if (!w.kAll) ask(row);
    float2 of_f = make_float2(0.f, 1.f), of_x = make_float2(0.f, 1.f);
    float x[NV][kPer], f[NV][kPer];
    Raw<TYPE> gates[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      gates[k] = gate_next[k];
      unpack<TYPE>(x_next[k], x[k]);
      if (n.f) unpack<TYPE>(f_next[k], f[k]);
    }
    if (row + step < n.n_rows && w.kAll) ask(row + step);
    auto over = [&](const float (&v)[NV][kPer]) {
      return [&](auto&& of) {
        Sums<1> s = {{0.f}};
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int i = 0; i < kPer; ++i) s.v[0] += LEAN || c[k].inside(i) ? of(v[k][i]) : 0.f;
        return g.sum(s).v[0];
      };
    };
    if (n.f) {
      if (n.after) of_f = statistics<LEAN>(n, a.inv_dim, over(f));
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float gate[kPer];
        if (!LEAN && is_matrix(n)) unpack<TYPE>(gates[k], gate);
        less<LEAN>(f[k], of_f.x);
        w.of(n, c, k).update(n, x[k], f[k], n.scale * of_f.y, gate);
      }
    }
    if (a.x_out) {
#pragma unroll
      for (int k = 0; k < NV; ++k) c[k].put(at(a.x_out, a.x_out_ld, row), x[k]);
    }
    if (a.y) {
      of_x = statistics<LEAN>(n, a.inv_dim, over(x));
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float b[kPer];
        const Weights<TYPE, VEC, LEAN> own = w.of(n, c, k);
        unpack<TYPE>(own.before, b);
        less<LEAN>(x[k], of_x.x);
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[k][i] = x[k][i] * of_x.y * b[i];
        if constexpr (!LEAN) {
          unpack<TYPE>(own.before_bias, b);
#pragma unroll
          for (int i = 0; i < kPer; ++i) x[k][i] += b[i];
        }
        c[k].put(at(a.y, a.y_ld, row), x[k]);
      }
    }
    if (a.stats && g.t == 0) a.stats[row] = make_float4(of_f.x, of_f.y, of_x.x, of_x.y);
  }
}

// Rows longer than that: a block walks its row once for each sum and once to write it. What it reads again
// comes from L2. x is read for the last time before x_out is written, which may be the same memory.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(kLongBlock) k_norm_forward_long(const NormArgs a) {
  constexpr bool LEAN = false;
  __shared__ float sh[64];
  chain_wait();
  Group g(kLongBlock, sh);
  const gm_norm& n = a.n;
  const int dim = static_cast<int>(n.dim);
  for (int64_t row = blockIdx.x; row < n.n_rows; row += gridDim.x) {
    auto at_row = [&](auto* m, int64_t ld) { return row_at<TYPE, false>(m, ld, row); };
    float2 of_f = make_float2(0.f, 1.f), of_x = make_float2(0.f, 1.f);
    auto walk = [&](auto&& body) {
      for (int at = 0; at < dim; at += kLongBlock * kPer)
        body(Columns<TYPE, VEC>{g.t + (VEC ? at / kPer : at), kLongBlock, dim});
    };
    auto total = [&](auto&& values) {
      return [&](auto&& of) {
        Sums<1> s = {{0.f}};
        walk([&](const Columns<TYPE, VEC>& c) {
          float v[kPer];
          values(c, v);
#pragma unroll
          for (int i = 0; i < kPer; ++i) s.v[0] += c.inside(i) ? of(v[i]) : 0.f;
        });
        return g.sum(s).v[0];
      };
    };
    Weights<TYPE, VEC, LEAN> w;
    auto updated = [&](const Columns<TYPE, VEC>& c, float (&x)[kPer]) {
      c.get(at_row(n.x, n.x_ld), x);
      w.read(n, c);
      if (!n.f) return;
      float f[kPer], gate[kPer];
      c.get(at_row(n.f, n.f_ld), f);
      less<LEAN>(f, of_f.x);
      if (is_matrix(n)) c.get(at_row(n.gate, n.gate_ld), gate);
      w.update(n, x, f, n.scale * of_f.y, gate);
    };
    if (n.after) of_f = statistics<LEAN>(n, a.inv_dim, total([&](const Columns<TYPE, VEC>& c, float (&v)[kPer]) { c.get(at_row(n.f, n.f_ld), v); }));
    if (a.y) of_x = statistics<LEAN>(n, a.inv_dim, total(updated));
    walk([&](const Columns<TYPE, VEC>& c) {
      float x[kPer], b[kPer];
      updated(c, x);
      if (a.x_out) c.put(at_row(a.x_out, a.x_out_ld), x);
      if (!a.y) return;
      less<LEAN>(x, of_x.x);
      unpack<TYPE>(w.before, b);
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = x[i] * of_x.y * b[i];
      unpack<TYPE>(w.before_bias, b);
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] += b[i];
      c.put(at_row(a.y, a.y_ld), x);
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

// Eight columns of a row as they are in memory.
template <int TYPE>
struct RowIn {
  Raw<TYPE> x, f, gx, gy, gate;
};

// A thread's eight columns of one row on the way back. What sums over rows is handed to add(which, values). Columns past the
// row's end have weights, and so all terms of a row's sums, of 0.
template <int TYPE, bool VEC, bool LEAN>
struct Back {
  const BackArgs& a;
  const Weights<TYPE, VEC, LEAN>& w;
  const RowIn<TYPE>& in;
  float4 st;
  // x: x' less its mean; d = gy * before; the row's sums of d x and of d
  template <class ADD>
  __device__ __forceinline__ void start(float (&x)[kPer], float (&d)[kPer], Sums<2>& s, ADD&& add) const {
    unpack<TYPE>(in.x, x);
    if (a.n.f) {
      float f[kPer], gate[kPer];
      unpack<TYPE>(in.f, f);
      less<LEAN>(f, st.x);
      if (!LEAN && is_matrix(a.n)) unpack<TYPE>(in.gate, gate);
      w.update(a.n, x, f, a.n.scale * st.y, gate);
    }
    less<LEAN>(x, st.z);
    if (!a.gy) return;
    float t[kPer];
    unpack<TYPE>(in.gy, d);
    if constexpr (!LEAN) add(kSumBeforeBias, d, 1.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = d[i] * x[i];
    add(kSumBefore, t, st.w);
    float b[kPer];
    unpack<TYPE>(w.before, b);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s.v[0] = fmaf(b[i], t[i], s.v[0]);
      d[i] *= b[i];
      if constexpr (!LEAN) s.v[1] += d[i];
    }
  }
  // dx, in place of d. mean: of d n(x') and of d
  __device__ __forceinline__ void to_x(const float (&x)[kPer], float (&d)[kPer], Sums<2> mean) const {
    float gx[kPer];
    unpack<TYPE>(in.gx, gx);
    if (!a.gy) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) d[i] = gx[i];
      return;
    }
    const float k = -mean.v[0] * st.w * st.w, m = -mean.v[1] * st.w;
#pragma unroll
    for (int i = 0; i < kPer; ++i) d[i] = fmaf(x[i], k, fmaf(d[i], st.w, LEAN ? gx[i] : gx[i] + m));
  }
  // e = gate * after * dx, in place of dx; f less its mean; the row's sums of e f and of e
  template <class ADD, class GATE>
  __device__ __forceinline__ void past_gate(float (&d)[kPer], float (&f)[kPer], Sums<2>& s, ADD&& add, GATE&& gate_out) const {
    const gm_norm& n = a.n;
    unpack<TYPE>(in.f, f);
    less<LEAN>(f, st.x);
    if (!LEAN && is_matrix(n)) {
      float t[kPer], gate[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        t[i] = fmaf(f[i] * st.y, w.h[i], w.hc[LEAN ? 0 : i]) * (n.scale * d[i]);
      }
      gate_out(t);
      unpack<TYPE>(in.gate, gate);
#pragma unroll
      for (int i = 0; i < kPer; ++i) d[i] *= gate[i];
    }
    float t[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) t[i] = d[i] * f[i];
    add(kSumA, t, st.y);
    if constexpr (!LEAN) add(kSumB, d, 1.f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s.v[0] = fmaf(w.h[i], t[i], s.v[0]);
      d[i] *= w.h[i];
      if constexpr (!LEAN) s.v[1] += d[i];
    }
  }
  // df, in place of e. mean: of e n(f) and of e
  __device__ __forceinline__ void to_f(float (&e)[kPer], const float (&f)[kPer], Sums<2> mean) const {
    const float r = a.n.scale * st.y, k = -mean.v[0] * r * st.y, m = -mean.v[1] * r;
#pragma unroll
    for (int i = 0; i < kPer; ++i) e[i] = fmaf(f[i], k, LEAN ? e[i] * r : fmaf(e[i], r, m));
  }
};
// The means that a row's two sums give; unit: what n() divided by, inverted. Without a norm: none.
template <bool LEAN>
__device__ __forceinline__ Sums<2> means_of(const gm_norm& n, Group& g, Sums<2> s, float inv_dim, float unit) {
  if constexpr (LEAN) s.v[0] = g.sum(Sums<1>{{s.v[0]}}).v[0];
  else s = g.sum(s);
  s.v[0] *= inv_dim * unit, s.v[1] *= inv_dim;
  if (LEAN || n.norm != GM_NORM_LAYER) s.v[1] = 0.f;
  return s;
}

// Rows held by a group: NV turns of 8 columns a thread, the next row under way. The sums over rows are kept in shared
// memory, each thread's own columns.
// ONE: a block has one group, so that a row's address is the same for all its threads.
constexpr int kMostThreads = 512;
template <int TYPE, bool VEC, int NV, bool LEAN, bool ONE>
__global__ void __launch_bounds__(kMostThreads, 1) k_norm_backward(const BackArgs a, int group) {
  __shared__ float sh[16 * 64];
  extern __shared__ float4 acc[];  // [sum][turn][2][kMostThreads]
  chain_wait();
  Group g(group, sh);
  const gm_norm& n = a.n;
  const int dim = static_cast<int>(n.dim), groups = ONE ? 1 : blockDim.x / group;
  constexpr int kHere = LEAN ? 2 : 4;
  int64_t row = ONE ? static_cast<int64_t>(blockIdx.x) : static_cast<int64_t>(blockIdx.x) * groups + g.id;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  Columns<TYPE, VEC> c[NV];
  Kept<TYPE, VEC, NV, LEAN> w;
#pragma unroll
  for (int k = 0; k < NV; ++k) c[k] = Columns<TYPE, VEC>{g.t + k * (VEC ? group : group * kPer), group, dim};
  w.read(n, c);
  constexpr auto at = [](auto* m, int64_t ld, int64_t i) { return row_at<TYPE, LEAN>(m, ld, i); };
  if (a.sums) {
#pragma unroll
    for (int s = 0; s < 2 * NV * kHere; ++s) acc[s * kMostThreads + threadIdx.x] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  auto adder = [&](int k) {
    return [&, k](int which, const float (&v)[kPer], float by) {
      if (!a.sums) return;
      float4* at = acc + 2 * (which * NV + k) * kMostThreads + threadIdx.x;
      float4 x = at[0], y = at[kMostThreads];
      x.x = fmaf(v[0], by, x.x), x.y = fmaf(v[1], by, x.y), x.z = fmaf(v[2], by, x.z), x.w = fmaf(v[3], by, x.w);
      y.x = fmaf(v[4], by, y.x), y.y = fmaf(v[5], by, y.y), y.z = fmaf(v[6], by, y.z), y.w = fmaf(v[7], by, y.w);
      at[0] = x, at[kMostThreads] = y;
    };
  };
  auto get = [&](int k, const void* p) { return LEAN ? c[k].raw_or_last(p) : c[k].raw(p); };
  RowIn<TYPE> next[NV];  // gx, wanted last, waits in L2
  float4 st_next;
  auto ask = [&](int64_t i) {
    st_next = a.stats[i];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      next[k].x = get(k, at(n.x, n.x_ld, i));
      if (n.f) next[k].f = get(k, at(n.f, n.f_ld, i));
      if (a.gy) next[k].gy = get(k, at(a.gy, a.gy_ld, i));
      if (!LEAN && is_matrix(n)) next[k].gate = get(k, at(n.gate, n.gate_ld, i));
      if (VEC && a.gx && c[k].inside(0))
        asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(at(a.gx, a.gx_ld, i)) + c[k].t * kPer * (TYPE == GM_LOSS_F32 ? 4 : 2)));
    }
  };
  if (row < n.n_rows && w.kAll) ask(row);
  for (; row < n.n_rows; row += step) {
    if (!w.kAll) ask(row);
    RowIn<TYPE> in[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      in[k] = next[k];
      if (a.gx) in[k].gx = get(k, at(a.gx, a.gx_ld, row));
      else in[k].gx = Raw<TYPE>{};
    }
    const float4 st = st_next;
    if (row + step < n.n_rows && w.kAll) ask(row + step);
    using B = Back<TYPE, VEC, LEAN>;
    float x[NV][kPer], d[NV][kPer];
    Sums<2> s = {{0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < NV; ++k) B{a, w.of(n, c, k), in[k], st}.start(x[k], d[k], s, adder(k));
    if (a.need_x) {
      if (a.gy) s = means_of<LEAN>(a.n, g, s, a.inv_dim, st.w);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        B{a, w.of(n, c, k), in[k], st}.to_x(x[k], d[k], s);
        if (a.o.x) c[k].put(at(a.o.x, a.o.x_ld, row), d[k]);
      }
      if (n.f) {
        s = Sums<2>{{0.f, 0.f}};
#pragma unroll
        for (int k = 0; k < NV; ++k)
          B{a, w.of(n, c, k), in[k], st}.past_gate(d[k], x[k], s, adder(k), [&](const float (&v)[kPer]) {
            if (a.o.gate) c[k].put(at(a.o.gate, a.o.gate_ld, row), v);
          });
        if (a.o.f) {
          s = n.after ? means_of<LEAN>(a.n, g, s, a.inv_dim, st.y) : Sums<2>{{0.f, 0.f}};
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            B{a, w.of(n, c, k), in[k], st}.to_f(d[k], x[k], s);
            c[k].put(at(a.o.f, a.o.f_ld, row), d[k]);
          }
        }
      }
    }
  }
  if (!a.sums) return;
  __syncthreads();
  if (g.id != 0) return;  // one group adds the others' in their order
  float* out = a.sums + static_cast<int64_t>(blockIdx.x) * kSums * n.dim;
#pragma unroll
  for (int s = 0; s < kHere; ++s)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float v[kPer] = {};
      for (int j = 0; j < groups; ++j) {
        const float4* at = acc + 2 * (s * NV + k) * kMostThreads + j * group + g.t;
        const float4 x = at[0], y = at[kMostThreads];
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (c[k].inside(i)) out[s * n.dim + column<VEC>(c[k].t, group, i)] = v[i];
    }
}

// Eight columns of a row of the long ones, and their weights.
template <int TYPE, bool VEC, bool LEAN>
__device__ __forceinline__ void read_long(const BackArgs& a, const Columns<TYPE, VEC>& c, int64_t row, RowIn<TYPE>& in,
                                          Weights<TYPE, VEC, LEAN>& w) {
  const gm_norm& n = a.n;
  auto get = [&](const void* m, int64_t ld) { return c.raw(row_at<TYPE, false>(m, ld, row)); };
  in = RowIn<TYPE>{};
  in.x = get(n.x, n.x_ld);
  if (n.f) in.f = get(n.f, n.f_ld);
  if (a.gy) in.gy = get(a.gy, a.gy_ld);
  if (a.gx) in.gx = get(a.gx, a.gx_ld);
  if (is_matrix(n)) in.gate = get(n.gate, n.gate_ld);
  w.read(n, c);
}

// Rows longer than that: a block walks its row three times and leaves the row's means, by which
// k_norm_columns sums over rows.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(kLongBlock) k_norm_backward_long(const BackArgs a) {
  constexpr bool LEAN = false;
  __shared__ float sh[64];
  chain_wait();
  Group g(kLongBlock, sh);
  const gm_norm& n = a.n;
  const int dim = static_cast<int>(n.dim);
  for (int64_t row = blockIdx.x; row < n.n_rows; row += gridDim.x) {
    const float4 st = a.stats[row];
    auto at_row = [&](void* m, int64_t ld) { return row_at<TYPE, false>(m, ld, row); };
    Sums<2> mean_x = {{0.f, 0.f}}, mean_f = {{0.f, 0.f}}, s = {{0.f, 0.f}}, unused = {{0.f, 0.f}};
    auto none = [](int, const float (&)[kPer], float) {};
    float x[kPer], d[kPer];
    auto walk = [&](auto&& body) {
      for (int at = 0; at < dim; at += kLongBlock * kPer) {
        const Columns<TYPE, VEC> c{g.t + (VEC ? at / kPer : at), kLongBlock, dim};
        RowIn<TYPE> in;
        Weights<TYPE, VEC, LEAN> w;
        read_long(a, c, row, in, w);
        body(Back<TYPE, VEC, LEAN>{a, w, in, st}, c);
      }
    };
    if (a.gy) {
      walk([&](const auto& b, const auto&) { b.start(x, d, s, none); });
      mean_x = means_of<LEAN>(a.n, g, s, a.inv_dim, st.w);
    }
    if (n.after && a.o.f) {
      s = Sums<2>{{0.f, 0.f}};
      walk([&](const auto& b, const auto&) {
        b.start(x, d, unused, none);
        b.to_x(x, d, mean_x);
        b.past_gate(d, x, s, none, [](const float (&)[kPer]) {});
      });
      mean_f = means_of<LEAN>(a.n, g, s, a.inv_dim, st.y);
    }
    walk([&](const auto& b, const auto& c) {
      b.start(x, d, unused, none);
      b.to_x(x, d, mean_x);
      if (a.o.x) c.put(at_row(a.o.x, a.o.x_ld), d);
      if (!n.f) return;
      b.past_gate(d, x, unused, none, [&](const float (&v)[kPer]) {
        if (a.o.gate) c.put(at_row(a.o.gate, a.o.gate_ld), v);
      });
      if (!a.o.f) return;
      b.to_f(d, x, mean_f);
      c.put(at_row(a.o.f, a.o.f_ld), d);
    });
    if (g.t == 0) a.means[row] = make_float4(mean_x.v[0], mean_x.v[1], mean_f.v[0], mean_f.v[1]);
  }
}

// Sums over rows of long rows: a block takes 32 * kPer columns of a range of rows, its 8 warps every eighth.
constexpr int kColumnWarps = 8, kColumns = 32 * kPer;
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(32 * kColumnWarps) k_norm_columns(const BackArgs a, int64_t rows_a_block) {
  constexpr bool LEAN = false;
  __shared__ float sh[kSums][kColumns];
  chain_wait();
  const gm_norm& n = a.n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int col0 = blockIdx.x * kColumns;
  const Columns<TYPE, VEC> c{(VEC ? col0 / kPer : col0) + lane, 32, static_cast<int>(n.dim)};
  float acc[kSums][kPer];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[s][i] = 0.f;
  auto add = [&](int which, const float (&v)[kPer], float by) {
#pragma unroll
    for (int s = 0; s < kSums; ++s)
      if (s == which) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[s][i] = fmaf(v[i], by, acc[s][i]);
      }
  };
  const int64_t first = blockIdx.y * rows_a_block, end = min(n.n_rows, first + rows_a_block);
  for (int64_t row = first + warp; row < end; row += kColumnWarps) {
    RowIn<TYPE> in;
    Weights<TYPE, VEC, LEAN> w;
    read_long(a, c, row, in, w);
    const Back<TYPE, VEC, LEAN> b{a, w, in, a.stats[row]};
    float x[kPer], d[kPer];
    Sums<2> unused = {{0.f, 0.f}};
    b.start(x, d, unused, add);
    if (!a.need_x || !n.f) continue;
    const float4 m = a.means[row];
    b.to_x(x, d, Sums<2>{{m.x, m.y}});
    b.past_gate(d, x, unused, add, [](const float (&)[kPer]) {});
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

// The blocks' sums joined, and the gradients that they give: 32 columns a block, its 32 warps every 32nd part.
// blockIdx.y: before with its bias, or what comes from A and B.
template <int TYPE>
__global__ void __launch_bounds__(1024) k_norm_join(const BackArgs a, int parts, bool biases) {
  __shared__ float sh[2][32][33];
  chain_wait();
  const gm_norm& n = a.n;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = blockIdx.y;
  int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float x[2] = {0.f, 0.f};
  if (col < n.dim) {
    const float* p = a.sums + first * n.dim + col;
#pragma unroll 4
    for (int k = warp; k < parts; k += 32) {
      x[0] += p[static_cast<int64_t>(k) * kSums * n.dim];
      if (biases) x[1] += p[(static_cast<int64_t>(k) * kSums + 2) * n.dim];
    }
  }
  sh[0][warp][lane] = x[0], sh[1][warp][lane] = x[1];
  __syncthreads();
  // a warp a column, its lanes the parts
  x[0] = warp_reduce_sum(sh[0][lane][warp]);
  x[1] = biases ? warp_reduce_sum(sh[1][lane][warp]) : 0.f;
  col = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane != 0 || col >= n.dim) return;
  auto set = [&](void* out, float v) {
    if (!out) return;
    if constexpr (TYPE == GM_LOSS_F32) static_cast<float*>(out)[col] = v;
    else static_cast<uint16_t*>(out)[col] = static_cast<uint16_t>(round16<TYPE>(v));
  };
  auto of = [&](const void* p, float none) {
    if (!p) return none;
    if constexpr (TYPE == GM_LOSS_F32) return static_cast<const float*>(p)[col];
    else return lower16(static_cast<const uint16_t*>(p)[col], TYPE == GM_LOSS_BF16);
  };
  if (first == 0) {
    set(a.o.before, x[0]);
    set(a.o.before_bias, x[1]);
  } else {
    const bool vector = n.gate_kind == GM_GATE_VECTOR;
    const float by = n.scale * (vector ? of(n.gate, 1.f) : 1.f);
    set(a.o.after, by * x[0]);
    set(a.o.after_bias, by * x[1]);
    if (vector) set(a.o.gate, n.scale * fmaf(of(n.after, 1.f), x[0], of(n.after_bias, 0.f) * x[1]));
  }
}

// ---- host ----------------------------------------------------------------------------------------
gm_status check_norm(const gm_norm* n) {
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

// How a row is held: lean rows of 512 and more with 16 columns a thread where they are of 16 bits, others with 8.
// The others with 16 where a block does not hold them else.
struct Form {
  bool vec, lean, held;
  int turns, group;
  Form(const gm_norm& n, bool vec, std::initializer_list<int64_t> lds) : vec(vec) {
    const int wide = n.type == GM_LOSS_F32 ? 1 : 2;
    lean = vec && n.dim % kPer == 0 && n.dim >= 512 && n.dim <= kHeldDim / 2 * wide && n.norm == GM_NORM_RMS && !n.after_bias && !n.before_bias &&
           n.gate_kind != GM_GATE_MATRIX;
    for (int64_t ld : lds) lean = lean && ld * elem_bytes(n.type) <= UINT32_MAX;
    turns = lean ? wide : n.dim > kHeldDim / 2 ? 2 : 1;
    held = n.dim <= kHeldDim;
    group = static_cast<int>(up(div_up(n.dim, kPer * turns), 32));
  }
};
// f(type, rows by 16 bytes, lean, turns) with constants
template <class F>
cudaError_t by_form(const gm_norm& n, const Form& form, F&& f) {
  using std::integral_constant;
  using Yes = std::true_type;
  using No = std::false_type;
  using One = integral_constant<int, 1>;
  using Two = integral_constant<int, 2>;
  auto with = [&](auto t) {
    if (form.lean) return f(t, Yes(), Yes(), integral_constant<int, t == GM_LOSS_F32 ? 1 : 2>());
    auto turned = [&](auto v) { return form.turns == 1 ? f(t, v, No(), One()) : f(t, v, No(), Two()); };
    return form.vec ? turned(Yes()) : turned(No());
  };
  return n.type == GM_LOSS_F32    ? with(integral_constant<int, GM_LOSS_F32>())
         : n.type == GM_LOSS_BF16 ? with(integral_constant<int, GM_LOSS_BF16>())
                                  : with(integral_constant<int, GM_LOSS_F16>());
}

gm_status done(cudaError_t e) { return cudaGetLastError() != cudaSuccess || e != cudaSuccess ? GM_ERR_CUDA : GM_OK; }

gm_status norm_forward(const gm_norm& n, cudaStream_t s, void* x_out, int64_t x_out_ld, void* y, int64_t y_ld, float* stats) {
  const int sms = sm_count(kMostBlocks);
  if (sms <= 0) return done(cudaErrorUnknown);
  const Form form(n, Sixteen(n)(x_out, x_out_ld)(y, y_ld).ok, {n.x_ld, n.f_ld, x_out_ld, y_ld});
  const NormArgs a{n, 1.f / static_cast<float>(n.dim), x_out, y, x_out_ld, y_ld, reinterpret_cast<float4*>(stats)};
  return done(by_form(n, form, [&](auto t, auto v, auto l, auto turns) {
    constexpr int T = t, N = turns;
    constexpr bool V = v, L = l;
    if (!form.held) return launch_chained(k_norm_forward_long<T, V>, grid_for(n.n_rows, 1), kLongBlock, 0, s, 1, a);
    const int group = form.group, block = std::max(group, 128) / group * group;
    const unsigned grid = grid_for(n.n_rows, block / group, int64_t(sms) * std::max(1, kSmThreads / block));
    return launch_chained(k_norm_forward<T, V, N, L>, grid, block, 0, s, 1, a, group);
  }));
}

// How a backward call is cut, and where its workspace lies.
struct NormPlan {
  Arena a;
  int block = 0;
  int64_t parts, rows_a_part = 0;  // of the sums over rows
  size_t o_sums, o_means = 0;
  NormPlan(const gm_norm& n, const Form& form, int sms) {
    if (!form.held) {
      const int64_t slabs = div_up(n.dim, kColumns);
      parts = std::max<int64_t>(1, std::min<int64_t>(div_up(4 * sms, slabs), div_up(n.n_rows, 4 * kColumnWarps)));
      rows_a_part = div_up(n.n_rows, parts);
      parts = div_up(n.n_rows, rows_a_part);
      o_means = a.add(n.n_rows * 16);
    } else {
      block = std::max(form.group, 256) / form.group * form.group;
      parts = std::min<int64_t>(div_up(n.n_rows, block / form.group), int64_t(sms) * (512 / block));
    }
    o_sums = a.add(parts * kSums * n.dim * 4);
  }
};

gm_status norm_backward(const gm_norm& n, const gm_layer_config& cfg, cudaStream_t s, const float* stats, const void* gx,
                        int64_t gx_ld, const void* gy, int64_t gy_ld, const gm_norm_grads& o) {
  const int sms = sm_count(kMostBlocks);
  if (sms <= 0) return done(cudaErrorUnknown);
  const int64_t es = elem_bytes(n.type);
  const bool vector = n.gate_kind == GM_GATE_VECTOR;
  if (n.n_rows == 0) {
    for (void* p : {o.after, o.after_bias, o.before, o.before_bias, vector ? o.gate : nullptr})
      if (p && cudaMemsetAsync(p, 0, n.dim * es, s) != cudaSuccess) {
        cudaGetLastError();
        return GM_ERR_CUDA;
      }
    return GM_OK;
  }
  Sixteen all(n);
  all(gx, gx_ld)(gy, gy_ld)(o.x, o.x_ld)(o.f, o.f_ld)(vector ? nullptr : o.gate, o.gate_ld);
  const Form form(n, all.ok, {n.x_ld, n.f_ld, gx_ld, gy_ld, o.x_ld, o.f_ld});
  NormPlan p(n, form, sms);
  const gm_status rc = p.a.open(cfg.workspace, cfg.workspace_bytes, s);
  if (rc != GM_OK) return rc;
  const bool sums = o.before || o.before_bias || o.after || o.after_bias || (vector && o.gate);
  BackArgs a{n, o, 1.f / static_cast<float>(n.dim), reinterpret_cast<const float4*>(stats), gx, gy, gx_ld, gy_ld};
  a.need_x = o.x || o.f || o.gate || o.after || o.after_bias;
  a.sums = sums ? p.a.at<float>(p.o_sums) : nullptr;
  a.means = form.held ? nullptr : p.a.at<float4>(p.o_means);
  return done(by_form(n, form, [&](auto t, auto v, auto l, auto turns) {
    constexpr int T = t, N = turns;
    constexpr bool V = v, L = l;
    cudaError_t e = cudaSuccess;
    if (!form.held) {
      if (a.need_x) e = launch_chained(k_norm_backward_long<T, V>, grid_for(n.n_rows, 1), kLongBlock, 0, s, 1, a);
      if (e == cudaSuccess && sums) {
        const dim3 grid(static_cast<unsigned>(div_up(n.dim, kColumns)), static_cast<unsigned>(p.parts));
        e = launch_chained(k_norm_columns<T, V>, grid, 32 * kColumnWarps, 0, s, 1, a, p.rows_a_part);
      }
    } else {
      constexpr int kBytes = (L ? 2 : 4) * 2 * 16 * N;  // of a thread
      auto* k = k_norm_backward<T, V, N, L, false>;
      if constexpr (L) {
        if (p.block == form.group) k = k_norm_backward<T, V, N, L, true>;
      }
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes * kMostThreads);
      const size_t smem = sums ? size_t(kBytes) * kMostThreads : 0;
      if (e == cudaSuccess) e = launch_chained(k, static_cast<unsigned>(p.parts), p.block, smem, s, 1, a, form.group);
    }
    if (e == cudaSuccess && sums) {
      const dim3 grid(static_cast<unsigned>(div_up(n.dim, 32)), n.f ? 2 : 1);
      e = launch_chained(k_norm_join<T>, grid, 1024, 0, s, 1, a, static_cast<int>(p.parts), !L);
    }
    return e;
  }));
}

}  // namespace

}  // namespace gm

extern "C" gm_status gm_norm_forward(const gm_norm* n, void* stream, void* x_out, int64_t x_out_ld, void* y, int64_t y_ld,
                                     float* stats) {
  gm::NvtxRange range("gm_norm_forward");
  gm_status rc = gm::check_norm(n);
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
  gm_status rc = gm::check_norm(n);
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
  const gm_status rc = gm::check_norm(n);
  if (rc != GM_OK) return rc;
  *bytes = 0;
  if (n->n_rows == 0) return GM_OK;
  const int sms = gm::sm_count(gm::kMostBlocks);
  if (sms <= 0) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  // which form a call takes depends on its other arrays too
  const gm::Form lean(*n, true, {}), general(*n, false, {});
  *bytes = static_cast<int64_t>(std::max(gm::NormPlan(*n, lean, sms).a.used, gm::NormPlan(*n, general, sms).a.used));
  return GM_OK;
}
