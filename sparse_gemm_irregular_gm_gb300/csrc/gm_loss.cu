// gm_loss.cu -- losses over a large class table (include/gm_losses.h): the host
// driver and the kernels around the tensor-core products of gm_loss_prod.cu.
//
// Forward, for each piece of the classes (usually one): the product reduces Z = H W^T to a
// maximum and sums of exponentials for each row and half tile, a second kernel joins them.
// Backward, for each piece of the classes: the product again, its end writing the piece of
// G = dloss/dZ, then dH += G W_piece and dW_piece = G^T H. What is stored of Z's size has a bound.
#include "gm_loss.h"

#include <algorithm>
#include <atomic>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <nvtx3/nvToolsExt.h>

#include "gm_device.cuh"
#include "gm_umma.cuh"

namespace gm {

namespace {

__device__ int g_loss_status;

// Reads and clears in one step: what other streams' kernels set meanwhile is either told now or kept.
__global__ void k_take_status(int* __restrict__ taken) { *taken = atomicExch(&g_loss_status, 0); }

// ---- operands that TMA cannot read in place ------------------------------------------
// f32: three bf16 planes, x = x0 + x1 + x2 with x0 the nearest bf16 of x and so on, which
// keeps all 24 bits; an infinity stands in the third plane alone, which meets only the other operand's
// first, its sign and size (in the first it would meet low planes that are 0: NaN where the product is
// infinite); 16-bit types: one plane, copied. Rows are padded with zeros to ld, a
// multiple of 8: a thread writes 8 elements of each plane at once. VEC: the rows of src start
// on 16-byte boundaries. Bound by memory: 126425 x 1320 f32, 1.67 GB in and out, 245 us (6.8 TB/s);
// 489196 x 437 f16, 0.86 GB, 132 us (6.5 TB/s).
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

template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) k_pack(const void* __restrict__ src, int64_t rows, int dim, int64_t src_ld,
                                              uint16_t* __restrict__ dst, int ld) {
  chain_wait();
  const unsigned per_row = static_cast<unsigned>(ld) / 8;
  const int64_t n = rows * ld, pieces = rows * per_row, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += stride) {
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

// ---- the teacher's rows -----------------------------------------------------------------
// The largest of values, to which NaN gives way. 64-bit ones by their bits as signed integers, those below
// 0 turned over (2048 rows of 2500 values: 294 us for k_teacher with maxima in fp64, 92 so).
__device__ __forceinline__ float key_of(float x) { return x; }
__device__ __forceinline__ int64_t key_of(double x) {
  const int64_t b = __double_as_longlong(x), size = b & INT64_MAX, inf = int64_t(0x7ff) << 52;
  return size > inf ? INT64_MIN : b < 0 ? b ^ INT64_MAX : b;
}
__device__ __forceinline__ float value_of(float k) { return k; }
__device__ __forceinline__ double value_of(int64_t k) {  // of what is less than any value: -inf
  return k == INT64_MIN ? -INFINITY : __longlong_as_double(k < 0 ? k ^ INT64_MAX : k);
}
__device__ __forceinline__ float larger(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ int64_t larger(int64_t x, int64_t y) { return x > y ? x : y; }
template <class V>
using Key = decltype(key_of(V()));

template <int W, class K>
__device__ __forceinline__ K group_max(K x, K* sh) {  // every thread of the W warps gets the result
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x = larger(x, __shfl_xor_sync(kFull, x, d));
  if constexpr (W > 1) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sh[0];
#pragma unroll
    for (int w = 1; w < W; ++w) x = larger(x, sh[w]);
  }
  return x;
}
template <int W>
__device__ __forceinline__ float group_sum(float x, float* sh) {
  x = warp_reduce_sum(x);
  if constexpr (W > 1) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = x;
    __syncthreads();
    x = sh[0];
#pragma unroll
    for (int w = 1; w < W; ++w) x += sh[w];
  }
  return x;
}
template <int W>
__device__ __forceinline__ bool group_or(bool x) {
  if constexpr (W > 1) return __syncthreads_or(x) != 0;
  else return __any_sync(kFull, x);
}

// q = softmax of a row's stored values / T; base[row] = sum q log q. Bound by the latency
// of a row's loads: a warp a row where rows are short; rows over kLongRow entries are
// left to the whole block afterwards. The rows of a block lie a grid apart, since long rows
// of a graph's product are neighbours. A value counts by its distance to the row's largest, taken in
// the values' own type (64-bit ones may be large and close). From there on fp32: a thread sums at most 32
// terms of a short row and one in 1024 of a long one (1024 of a row over 2^20 classes), and an fp64 log
// or sum costs more here than the loads do (8192 rows of 128 entries: 142 us with them, 8 without;
// 1500 ragged rows, the longest of some 47,000 entries: 30 us).
constexpr int kLongRow = 1024, kTeacherWarps = 32;

template <class V, class R, class C>
struct TeacherArgs {
  const R* rp;
  const C* col;
  const V* val;
  int64_t n_rows, n_cls, nnz;
  float inv_t;
  int64_t* start;
  int32_t* len;
  int2* ents;
  float* base;
  int* status;
  const int* falls;  // k_falls's, [n_falls]; null: few rows, each block looks by itself
  int n_falls;
};

// Whether any row pointer is smaller than the one before it: the block's threads look at every
// (blocks * threads)th. Up to kLookAlone rows every block of k_teacher looks at all of them, 0.4 us of 3.2
// at 4 rows and 1.3 of 5.6 at 4096; then k_falls does once, 2.1 us at 4097 rows and 3.6 at 100,000.
template <class R>
__device__ __forceinline__ bool rows_fall(const R* __restrict__ rp, int64_t n_rows, int64_t block, int64_t blocks) {
  bool falls = false;
#pragma unroll 4
  for (int64_t i = block * blockDim.x + threadIdx.x; i < n_rows; i += blocks * blockDim.x) falls |= rp[i] > rp[i + 1];
  return __syncthreads_or(falls) != 0;
}
constexpr int kFallsBlocks = 64;
constexpr int64_t kLookAlone = 4096;  // rows
template <class R>
__global__ void __launch_bounds__(1024) k_falls(const R* __restrict__ rp, int64_t n_rows, int* __restrict__ out) {
  chain_wait();
  const bool falls = rows_fall(rp, n_rows, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) out[blockIdx.x] = falls;
}
// Whether a row starts before the end of an earlier one, so that its entries are that one's too: then it
// is left alone. Asked of all rows when a row pointer falls. A whole warp. Not inlined, so that its
// registers do not cost k_teacher its second block on an SM (512 rows of 64 entries: 3.6 -> 6.8 us).
template <class R>
__device__ __noinline__ bool starts_inside(const R* rp, int64_t nnz, int64_t row, int64_t lo) {
  int64_t most = 0;
  for (int64_t i = threadIdx.x & 31; i < row; i += 32) {
    const int64_t first = static_cast<int64_t>(rp[i]), last = static_cast<int64_t>(rp[i + 1]);
    if (first >= 0 && last >= first && last <= nnz && last > most) most = last;
  }
  return __any_sync(kFull, lo < most);
}

template <int W, class V, class R, class C>
__device__ __forceinline__ void teacher_row(const TeacherArgs<V, R, C>& a, int64_t row, int64_t lo, int64_t hi,
                                            bool shared, Key<V>* sh_max, float* sh) {
  constexpr int kGroup = 32 * W;
  const int lane = threadIdx.x % kGroup;
  bool bad = lo < 0 || hi < lo || hi > a.nnz || shared;
  V m = 0;
  float sum = 0.f, b = 0.f;
  if (!bad) {
    bool wrong = false;
    Key<V> most = key_of(static_cast<V>(-INFINITY));
#pragma unroll 4
    for (int64_t i = lo + lane; i < hi; i += kGroup) {
      const int64_t c = static_cast<int64_t>(a.col[i]);
      if (c < 0 || c >= a.n_cls || (i > lo && static_cast<int64_t>(a.col[i - 1]) >= c)) wrong = true;
      most = larger(most, key_of(a.val[i]));
    }
    bad = group_or<W>(wrong);
    m = value_of(group_max<W>(most, sh_max));
    if (m == -INFINITY) m = 0;  // every exponential is 0, or NaN
  }
  auto below = [&](V x) { return static_cast<float>(x - m) * a.inv_t; };
  // a NaN value leaves the maximum alone and makes the sum NaN, so the row counts as one with entries
  if (!bad) {
#pragma unroll 4
    for (int64_t i = lo + lane; i < hi; i += kGroup) sum += expf(below(a.val[i]));
    sum = group_sum<W>(sum, sh);
  }
  const bool any = !bad && sum != 0.f;
  if (any) {
    const float log_sum = logf(sum), inv = 1.f / sum;
#pragma unroll 4
    for (int64_t i = lo + lane; i < hi; i += kGroup) {
      const float v = below(a.val[i]), q = expf(v) * inv;
      a.ents[i] = make_int2(static_cast<int>(a.col[i]), __float_as_int(q));
      if (q > 0.f || q != q) b += q * (v - log_sum);
    }
    b = group_sum<W>(b, sh);
  }
  if (lane == 0) {
    a.start[row] = lo;
    a.len[row] = any ? static_cast<int32_t>(hi - lo) : 0;
    a.base[row] = bad ? NAN : b;
    if (bad) atomicOr(a.status, kLossBadTeacher);
  }
}

template <class V, class R, class C>
__global__ void __launch_bounds__(32 * kTeacherWarps, 2) k_teacher(const TeacherArgs<V, R, C> a) {
  __shared__ Key<V> sh_max[kTeacherWarps];
  __shared__ float sh[kTeacherWarps];
  __shared__ unsigned s_long;
  const int warp = threadIdx.x >> 5;
  chain_wait();
  const bool falls = a.falls ? __syncthreads_or(static_cast<int>(threadIdx.x) < a.n_falls && a.falls[threadIdx.x]) != 0
                             : rows_fall(a.rp, a.n_rows, 0, 1);
  for (int64_t row0 = blockIdx.x; row0 < a.n_rows; row0 += int64_t(gridDim.x) * kTeacherWarps) {
    if (threadIdx.x == 0) s_long = 0;
    __syncthreads();
    const int64_t row = row0 + int64_t(warp) * gridDim.x;
    if (row < a.n_rows) {
      const int64_t lo = static_cast<int64_t>(a.rp[row]), hi = static_cast<int64_t>(a.rp[row + 1]);
      const bool shared = falls && lo < hi && starts_inside(a.rp, a.nnz, row, lo);
      if (!shared && lo >= 0 && hi <= a.nnz && hi - lo > kLongRow) {
        if ((threadIdx.x & 31) == 0) atomicOr(&s_long, 1u << warp);
      } else {
        teacher_row<1>(a, row, lo, hi, shared, sh_max, sh);
      }
    }
    __syncthreads();
    for (unsigned left = s_long; left; left &= left - 1) {
      const int64_t r = row0 + int64_t(__ffs(left) - 1) * gridDim.x;
      teacher_row<kTeacherWarps>(a, r, static_cast<int64_t>(a.rp[r]), static_cast<int64_t>(a.rp[r + 1]), false, sh_max, sh);
      __syncthreads();
    }
    __syncthreads();
  }
}

// This lane's part of a call's `lost` (gm_loss_prod.cu): not 0 where a product gave up. A warp that writes
// results reads all of it, early, and asks once it has its sums. lost null: kernels that wait for nothing.
__device__ __forceinline__ uint64_t lost_word(const uint8_t* lost) {
  static_assert(kMostBlocks == 8 * 32, "a word a lane");
  return lost ? reinterpret_cast<const uint64_t*>(lost)[threadIdx.x & 31] : 0;
}

// ---- joining the half tiles of a row -----------------------------------------------------
struct JoinArgs {
  float4* carry;  // [row]: the sums so far, of a piece that is not the last; null: results
  const float4* part;
  int64_t n_parts, n_rows;
  Targets tgt;
  const float* z_t;
  const int32_t* ent_len;  // null: no teacher
  const float* base;
  float inv_t;
  float *loss, *lse, *kl, *lse_t;
  int* status;
  const uint8_t* lost;
};
// Bound by the latency of its loads: 4 of them in flight a thread (2000 rows, 1024 half tiles,
// 33 MB: 22 us with one, 9 with four).
template <int ROWS>  // rows of a block; 256 / ROWS threads a row
__global__ void __launch_bounds__(256) k_join(const JoinArgs a) {
  constexpr int kSub = 256 / ROWS;
  chain_wait();
  const int rl = threadIdx.x % ROWS, sub = threadIdx.x / ROWS;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + rl;
  const bool dis = a.ent_len != nullptr;
  const uint64_t lost_here = threadIdx.x < 32 ? lost_word(a.lost) : 0;  // the warp with sub 0
  float m = -INFINITY, s1 = 0.f, st = 0.f, zq = 0.f;
  auto add = [&](float4 o) {
    const float mn = fmaxf(m, o.x), ref = mn == -INFINITY ? 0.f : mn;
    s1 = s1 * ex2((m - ref) * kLog2e) + o.y * ex2((o.x - ref) * kLog2e);
    if (dis) {
      const float c = kLog2e * a.inv_t;
      st = st * ex2((m - ref) * c) + o.z * ex2((o.x - ref) * c);
      zq += o.w;
    }
    m = mn;
  };
  if (row < a.n_rows) {
    const float4* p = a.part + row;
    int64_t i = sub;
    for (; i + 3 * kSub < a.n_parts; i += 4 * kSub) {
      float4 o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = p[(i + q * kSub) * a.n_rows];
#pragma unroll
      for (int q = 0; q < 4; ++q) add(o[q]);
    }
    for (; i < a.n_parts; i += kSub) add(p[i * a.n_rows]);
  }
  __shared__ float4 sh[256];
  for (int d = kSub / 2; d > 0; d >>= 1) {
    if (sub >= d && sub < 2 * d) sh[threadIdx.x] = make_float4(m, s1, st, zq);
    __syncthreads();
    if (sub < d) add(sh[threadIdx.x + d * ROWS]);
    __syncthreads();
  }
  const bool lost = __any_sync(kFull, lost_here != 0);
  if (sub != 0 || row >= a.n_rows) return;
  if (a.carry) {
    a.carry[row] = make_float4(m, s1, st, zq);
    return;
  }
  if (a.tgt.t) {
    const float l = lost ? NAN : m + logf(s1);
    const int64_t t = check_target(a.tgt, raw_target(a.tgt, row));
    a.lse[row] = l;
    a.loss[row] = t == -1 ? 0.f : t == -2 ? NAN : l - a.z_t[row];
    if (t == -2) atomicOr(a.status, kLossBadTarget);
  }
  if (dis) {
    const float l = lost ? NAN : m * a.inv_t + logf(st);
    a.lse_t[row] = l;
    a.kl[row] = a.ent_len[row] > 0 ? a.base[row] - zq * a.inv_t + l : a.base[row];  // no entries: 0, or NaN
  }
}

// ---- weights of the rows, for the scales of G in f16 -------------------------------------------
// Bits of the largest (0: none) and of the smallest above 0 (infinity: none), one block: 2 us at 777
// rows, its launch.
__global__ void __launch_bounds__(1024) k_weights(int64_t n, const RowGrads r, unsigned* __restrict__ out) {
  chain_wait();
  float most = 0.f, least = INFINITY;
  for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
    const float x = weight_of(row_coef(r, row_raw(r, i)));
    most = fmaxf(most, x);  // NaN gives way
    if (x > 0.f) least = fminf(least, x);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    most = fmaxf(most, __shfl_xor_sync(kFull, most, d));
    least = fminf(least, __shfl_xor_sync(kFull, least, d));
  }
  __shared__ float sh[2][32];
  if ((threadIdx.x & 31) == 0) sh[0][threadIdx.x >> 5] = most, sh[1][threadIdx.x >> 5] = least;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) most = fmaxf(most, sh[0][w]), least = fminf(least, sh[1][w]);
    out[0] = __float_as_uint(most), out[1] = __float_as_uint(least);
  }
}

// dh = the splits' sums (of a lost product: NaN), rounded. SUB threads share the splits of an element (fixed order): 1
// where there are few splits of many elements, 8 where it is the other way round (7 x 80 elements
// of 304 splits: 28 -> 5 us).
template <int SUB>
__global__ void __launch_bounds__(256) k_sum_splits(const float* __restrict__ acc, int splits, int64_t split_stride,
                                                    int64_t rows, int64_t dim, int64_t acc_ld, void* __restrict__ out,
                                                    int64_t out_ld, int type, const uint8_t* __restrict__ lost) {
  constexpr int kCols = 256 / SUB;
  __shared__ float sh[SUB][kCols];
  chain_wait();
  const int64_t n = rows * dim, stride = static_cast<int64_t>(gridDim.x) * kCols;
  const int col = threadIdx.x % kCols, sub = threadIdx.x / kCols;
  const uint64_t lost_here = sub == 0 ? lost_word(lost) : 0;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kCols; i0 < n; i0 += stride) {
    const int64_t i = i0 + col;
    const int64_t r = i / dim, c = i - r * dim;
    float x = 0.f;
    if (i < n) {
      const float* p = acc + r * acc_ld + c;
#pragma unroll 4
      for (int s = sub; s < splits; s += SUB) x += p[s * split_stride];
    }
    if constexpr (SUB > 1) {
      __syncthreads();
      sh[sub][col] = x;
      __syncthreads();
      if (sub != 0) continue;
#pragma unroll
      for (int s = 1; s < SUB; ++s) x += sh[s][col];
    }
    const bool gone = __any_sync(kFull, lost_here != 0);  // a warp has one sub where SUB is over 1
    if (i >= n) continue;
    if (gone) x = NAN;
    const int64_t o = r * out_ld + c;
    if (type == GM_LOSS_F32) static_cast<float*>(out)[o] = x;
    else if (type == GM_LOSS_BF16) static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(x);
    else static_cast<__half*>(out)[o] = __float2half_rn(x);
  }
}

// ---- host -----------------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn() {
  static const EncodeTiled fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// Matrix of `planes` planes of rows x cols elements of 2 bytes (4: fp32), ld elements a row.
struct Operand {
  const void* p;
  int64_t rows, cols, ld, plane;
  int planes;
  int bytes = 2;
};
// Boxes of box_rows rows of row_bytes (128 or 64), swizzled over that width; elements outside read as 0.
bool encode(CUtensorMap* m, const Operand& o, int box_rows, int row_bytes = 128) {
  const EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(o.planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * o.bytes, static_cast<cuuint64_t>(o.plane) * o.bytes};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(row_bytes / o.bytes), static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(m, o.bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_UINT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void*>(o.p), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
            row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

constexpr int64_t kMostIndex = (int64_t(1) << 31) - 256;  // tile coordinates are int32
constexpr int64_t kDefaultCap = int64_t(512) << 20;  // of G; f16: of each of the two sets of planes (Scales)
constexpr int64_t kStatsCap = int64_t(512) << 20;    // of a forward call's row statistics

struct Call {
  gm_logits z = {};
  const gm_csr* teacher = nullptr;  // null: cross entropy alone
  int64_t nnz = -1;                 // the teacher's entries, -1 without one
  int32_t value_type = 0, index_type = 0;
  float temperature = 1.f;
  const gm_labels* labels = nullptr;
  int64_t cap = 0;                  // 0: the default
  int32_t flags = 0;
  void* workspace = nullptr;
  int64_t workspace_bytes = 0;
  cudaStream_t s = nullptr;
  int sms = 0;
  int* status = nullptr;
};

// One workspace block, carved in order.
struct Arena {
  DevBuf<unsigned char> buf;  // from the hooks, unless the caller brought memory
  unsigned char* p = nullptr;
  size_t used = 0;
  gm_status open(const Call& c) {
    if (c.workspace) {
      if (static_cast<int64_t>(used) > c.workspace_bytes) return GM_ERR_WORKSPACE;
      p = static_cast<unsigned char*>(c.workspace);
      return GM_OK;
    }
    if (!buf.alloc(used, c.s)) return GM_ERR_OOM;
    p = buf.p;
    return GM_OK;
  }
  size_t add(int64_t bytes) {
    const size_t at = used;
    used += static_cast<size_t>(up(bytes, 256));
    return at;
  }
  template <class T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(p + off);
  }
};

// The call's own words: lost (ProdArgs), and the report of a checked call.
struct Words {
  size_t lost = 0, status = 0;
  void plan(Arena& a) {
    lost = a.add(kMostBlocks);
    status = a.add(4);
  }
};

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

int64_t elem_bytes(int32_t type) { return type == GM_LOSS_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }


gm_status check(Call& c, const gm_logits* z, const gm_labels* labels, const gm_loss_config* cfg, void* stream) {
  if (!z) return GM_ERR_INVALID_ARG;
  c.z = *z;
  if (c.z.n_rows < 0 || c.z.n_classes < 1 || c.z.dim < 1) return GM_ERR_INVALID_ARG;
  if (c.z.n_rows > kMostIndex || c.z.n_classes > kMostIndex || c.z.dim > (int64_t(1) << 24)) return GM_ERR_INDEX_OVERFLOW;
  if (c.z.type != GM_LOSS_F32 && c.z.type != GM_LOSS_BF16 && c.z.type != GM_LOSS_F16) return GM_ERR_INVALID_ARG;
  const int64_t es = elem_bytes(c.z.type);
  if (!c.z.w || !aligned(c.z.w, es) || (c.z.n_rows > 0 && (!c.z.h || !aligned(c.z.h, es)))) return GM_ERR_INVALID_ARG;
  if (c.z.h_ld < c.z.dim || c.z.w_ld < c.z.dim) return GM_ERR_INVALID_ARG;
  if (c.z.h_ld > (int64_t(1) << 36) || c.z.w_ld > (int64_t(1) << 36)) return GM_ERR_INDEX_OVERFLOW;
  c.labels = labels;
  if (labels && ((c.z.n_rows > 0 && !labels->target) || (labels->target32 != 0 && labels->target32 != 1) ||
                 !aligned(labels->target, labels->target32 ? 4 : 8)))
    return GM_ERR_INVALID_ARG;
  if (cfg) {
    if (cfg->workspace_cap_bytes < 0 || (cfg->flags & ~GM_LOSS_CHECK)) return GM_ERR_INVALID_ARG;
    c.cap = cfg->workspace_cap_bytes;
    c.flags = cfg->flags;
    if (cfg->workspace && (!aligned(cfg->workspace, 256) || cfg->workspace_bytes < 0)) return GM_ERR_INVALID_ARG;
    c.workspace = cfg->workspace;
    c.workspace_bytes = cfg->workspace_bytes;
  }
  c.s = static_cast<cudaStream_t>(stream);
  return GM_OK;
}

gm_status check_teacher(Call& c, const gm_csr* t, int32_t value_type, int32_t index_type, float temperature) {
  if (!t) return GM_ERR_INVALID_ARG;
  if (t->n_rows != c.z.n_rows || t->n_cols != c.z.n_classes) return GM_ERR_DIM_MISMATCH;
  if (value_type != GM_VALUE_F64 && value_type != GM_VALUE_F32) return GM_ERR_INVALID_ARG;
  if (index_type & ~(GM_INDEX_ROWPTR32 | GM_INDEX_COL64)) return GM_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(kLog2e / temperature)) return GM_ERR_INVALID_ARG;
  if (t->nnz < 0 || !t->row_ptr || (t->nnz > 0 && (!t->col_idx || !t->vals))) return GM_ERR_INVALID_ARG;
  if (!aligned(t->row_ptr, index_type & GM_INDEX_ROWPTR32 ? 4 : 8) ||
      !aligned(t->col_idx, index_type & GM_INDEX_COL64 ? 8 : 4) || !aligned(t->vals, value_type == GM_VALUE_F64 ? 8 : 4))
    return GM_ERR_INVALID_ARG;
  c.teacher = t;
  c.nnz = t->nnz;
  c.value_type = value_type;
  c.index_type = index_type;
  c.temperature = temperature;
  return GM_OK;
}

// SMs of the current device (at most kMostBlocks), looked up once a device.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  n = std::min(n, kMostBlocks);
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Device facts and a clear error state; GM_ERR_CUDA leaves a pending error to its owner.
gm_status begin(Call& c) {
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  void* st = nullptr;
  c.sms = sm_count();
  if (c.sms <= 0 || cudaGetSymbolAddress(&st, g_loss_status) != cudaSuccess) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  c.status = static_cast<int*>(st);
  return GM_OK;
}

gm_status status_of(int bits) {
  if (bits & kLossTimeout) return GM_ERR_DEVICE_TIMEOUT;
  return bits ? GM_ERR_BAD_INDEX : GM_OK;
}

// A checked call reports to a word of its own: it neither tells of other calls' rows nor keeps theirs from
// gm_loss_status.
gm_status own_status(Call& c, int* word) {
  if (!(c.flags & GM_LOSS_CHECK)) return GM_OK;
  c.status = word;
  if (cudaMemsetAsync(word, 0, 4, c.s) == cudaSuccess) return GM_OK;
  cudaGetLastError();
  return GM_ERR_CUDA;
}

gm_status finish(const Call& c, bool launched, const int* word = nullptr) {
  if (cudaGetLastError() != cudaSuccess || !launched) return GM_ERR_CUDA;
  if (!(c.flags & GM_LOSS_CHECK)) return GM_OK;
  int bits = 0;
  if ((word && cudaMemcpyAsync(&bits, word, 4, cudaMemcpyDeviceToHost, c.s) != cudaSuccess) ||
      cudaStreamSynchronize(c.s) != cudaSuccess) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  return status_of(bits);
}

Targets targets_of(const Call& c) {
  if (!c.labels) return Targets{nullptr, true, 0, c.z.n_classes};
  return Targets{c.labels->target, c.labels->target32 == 0, c.labels->ignore_index, c.z.n_classes};
}

// H or W as a 16-bit operand, in place or laid out in workspace.
struct Source {
  const void* p;
  int64_t rows, dim, ld;
  int32_t type;
  bool packed;
  size_t off = 0;
  Source(const void* p, int64_t rows, int64_t dim, int64_t ld, int32_t type)
      : p(p), rows(rows), dim(dim), ld(ld), type(type) {
    packed = type == GM_LOSS_F32 || !aligned(p, 16) || (rows > 1 && ld % 8 != 0);
    if (rows <= 1) this->ld = up(dim, 8);
    if (packed) this->ld = up(dim, 8);
    src_ld = ld;
  }
  int64_t src_ld;
  int planes() const { return type == GM_LOSS_F32 ? 3 : 1; }
  void plan(Arena& a) {
    if (packed) off = a.add(planes() * rows * ld * 2);
  }
  Operand ready(const Arena& a, cudaStream_t s) const {
    Operand o{p, rows, dim, ld, rows * ld, planes()};
    if (packed) {
      o.p = a.at<uint16_t>(off);
      const unsigned grid = grid_for(rows * ld / 8, 256);
      uint16_t* dst = a.at<uint16_t>(off);
      const int d = static_cast<int>(dim), l = static_cast<int>(ld);
      const bool vec = aligned(p, 16) && (rows <= 1 || src_ld % 4 == 0);
      launch_chained(type != GM_LOSS_F32 ? k_pack<false, false> : vec ? k_pack<true, true> : k_pack<true, false>, grid,
                     256, 0, s, 1, p, rows, d, src_ld, dst, l);
    }
    return o;
  }
};

struct TeacherPlan {
  size_t start = 0, len = 0, ents = 0, base = 0, falls = 0;
  void plan(Arena& a, const Call& c) {
    if (c.nnz < 0) return;
    start = a.add(c.z.n_rows * 8);
    len = a.add(c.z.n_rows * 4);
    base = a.add(c.z.n_rows * 4);
    falls = a.add(kFallsBlocks * 4);
    ents = a.add(c.nnz * 8);
  }
  template <class V, class R, class C>
  void run(const Arena& a, const Call& c) const {
    // rows a block: as many as its warps only when every SM then still has blocks
    const int64_t blocks = std::min<int64_t>(c.z.n_rows, std::max<int64_t>(div_up(c.z.n_rows, kTeacherWarps), 2 * c.sms));
    int* falls_at = nullptr;
    unsigned n_falls = 0;
    if (c.z.n_rows > kLookAlone) {
      falls_at = a.at<int>(falls);
      n_falls = static_cast<unsigned>(std::min<int64_t>(kFallsBlocks, div_up(c.z.n_rows, kLookAlone)));
      launch_chained(k_falls<R>, n_falls, 1024, 0, c.s, 1, static_cast<const R*>(c.teacher->row_ptr), c.z.n_rows, falls_at);
    }
    const TeacherArgs<V, R, C> args{static_cast<const R*>(c.teacher->row_ptr), static_cast<const C*>(c.teacher->col_idx),
                                    static_cast<const V*>(c.teacher->vals), c.z.n_rows, c.z.n_classes, c.nnz,
                                    1.f / c.temperature, a.at<int64_t>(start), a.at<int32_t>(len), a.at<int2>(ents),
                                    a.at<float>(base), c.status, falls_at, static_cast<int>(n_falls)};
    launch_chained(k_teacher<V, R, C>, static_cast<unsigned>(blocks), 32 * kTeacherWarps, 0, c.s, 1, args);
  }
  template <class V>
  void run_indices(const Arena& a, const Call& c) const {
    const bool r32 = c.index_type & GM_INDEX_ROWPTR32, c64 = c.index_type & GM_INDEX_COL64;
    if (r32 && c64) run<V, int32_t, int64_t>(a, c);
    else if (r32) run<V, int32_t, int32_t>(a, c);
    else if (c64) run<V, int64_t, int64_t>(a, c);
    else run<V, int64_t, int32_t>(a, c);
  }
  void launch(const Arena& a, const Call& c) const {
    if (!c.teacher) return;
    if (c.value_type == GM_VALUE_F64) run_indices<double>(a, c);
    else run_indices<float>(a, c);
  }
};

// Stages (64 elements each) of a row of Z summed in TMEM at a time: 1024 elements leave an error
// under 4e-7 of the row's log-sum; summing every stage apart would read TMEM 16 times as often.
constexpr int kChunk = 16;

void set_logits_args(ProdArgs& g, const Call& c, const Arena& a, const TeacherPlan& t) {
  g.tgt = targets_of(c);
  g.status = c.status;
  g.planes = c.z.type == GM_LOSS_F32 ? 3 : 1;
  g.bf16 = c.z.type != GM_LOSS_F16;
  g.chunk = kChunk;
  g.inv_t = 1.f / c.temperature;
  g.c_t = kLog2e / c.temperature;
  if (c.teacher) {
    g.ent_start = a.at<int64_t>(t.start);
    g.ent_len = a.at<int32_t>(t.len);
    g.ents = a.at<int2>(t.ents);
  }
}

// Row tiles walked together: their rows of H stay in L2 while the class table streams by once.
int group_of(int64_t m_tiles, int64_t tile_rows, int64_t dim, int planes) {
  const int64_t bytes = tile_rows * dim * 2 * planes;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(m_tiles, (int64_t(40) << 20) / bytes)));
}

// Few rows go to kernels that read W once as it lies, instead of the tensor cores.
bool skinny(const Call& c) { return c.z.n_rows <= skinny_rows(c.z.type) && c.z.dim <= kSkinnyDim; }
// Elements of a load of matrices whose rows start at p, ld elements apart: 16 bytes, 4, or one element.
int skinny_vec(const void* p, int64_t ld, int64_t dim, int64_t rows, int64_t es) {
  if (rows <= 1) ld = dim;
  if (aligned(p, 16) && ld * es % 16 == 0 && dim * es % 16 == 0) return static_cast<int>(16 / es);
  return es == 2 && aligned(p, 4) && ld % 2 == 0 && dim % 2 == 0 ? 2 : 1;
}
SkinnyArgs skinny_args(const Call& c, const Arena& a, const TeacherPlan& t) {
  SkinnyArgs g = {};
  g.h = c.z.h;
  g.w = c.z.w;
  g.h_ld = c.z.h_ld;
  g.w_ld = c.z.w_ld;
  g.dim = c.z.dim;
  g.n_cls = c.z.n_classes;
  g.n = static_cast<int>(c.z.n_rows);
  g.tgt = targets_of(c);
  g.inv_t = 1.f / c.temperature;
  g.c_t = kLog2e / c.temperature;
  g.status = c.status;
  if (c.teacher) {
    g.ent_start = a.at<int64_t>(t.start);
    g.ent_len = a.at<int32_t>(t.len);
    g.ents = a.at<int2>(t.ents);
  }
  return g;
}

// How a forward call is cut, and where its workspace lies.
struct ForwardPlan {
  Arena a;
  Source h, w;
  TeacherPlan t;
  int blocks = 0;  // of the kernel for few rows; 0: the product
  Words own;
  int cg, bn;
  int64_t n_tiles;      // of a row tile, in all
  int64_t piece_tiles;  // of a piece of the classes
  int64_t n_parts;      // [0]: with several pieces, the sums of those before; then half tiles
  size_t o_part, o_zt;
  explicit ForwardPlan(const Call& c)
      : h(c.z.h, c.z.n_rows, c.z.dim, c.z.h_ld, c.z.type), w(c.z.w, c.z.n_classes, c.z.dim, c.z.w_ld, c.z.type) {
    const int64_t n = c.z.n_rows;
    own.plan(a);
    cg = n > 128 ? 2 : 1;
    bn = prod_logits_cols(cg, h.planes());
    n_tiles = div_up(c.z.n_classes, bn);
    const int64_t most = std::max<int64_t>(1, kStatsCap / (n * 32)), pieces = div_up(n_tiles, most);
    piece_tiles = div_up(n_tiles, pieces);
    n_parts = 2 * piece_tiles + (pieces > 1);
    if (skinny(c)) {
      n_parts = blocks = skinny_most_blocks(c.z.n_classes, c.sms);
    } else {
      h.plan(a);
      w.plan(a);
    }
    t.plan(a, c);
    o_part = a.add(n_parts * n * 16);
    o_zt = a.add(n * 4);
  }
};

gm_status forward(Call& c, float* kl, float* lse_t, float* loss, float* lse) {
  gm_status rc = begin(c);
  if (rc != GM_OK) return rc;
  const int64_t n = c.z.n_rows;
  if (n == 0) return finish(c, true);
  ForwardPlan p(c);
  Arena& a = p.a;
  rc = a.open(c);
  if (rc != GM_OK) return rc;
  uint8_t* lost = a.at<uint8_t>(p.own.lost);
  int* word = a.at<int>(p.own.status);
  rc = own_status(c, word);
  if (rc != GM_OK) return rc;
  const TeacherPlan& t = p.t;
  float4* part = a.at<float4>(p.o_part);
  float* z_t = a.at<float>(p.o_zt);
  JoinArgs j = {};
  j.n_rows = n;
  j.tgt = targets_of(c);
  j.z_t = z_t;
  j.ent_len = c.teacher ? a.at<int32_t>(t.len) : nullptr;
  j.base = c.teacher ? a.at<float>(t.base) : nullptr;
  j.inv_t = 1.f / c.temperature;
  j.loss = loss;
  j.lse = lse;
  j.kl = kl;
  j.lse_t = lse_t;
  j.status = c.status;
  j.lost = p.blocks ? nullptr : lost;
  // few rows: a block each, so that their half tiles are read by many threads; more: 2 a block,
  // a whole 32-byte sector (512 rows, 8192 half tiles: 45 -> 18 us); many: 8, a 128-byte line
  auto join = [&](const float4* first, int64_t parts, float4* carry) {
    j.part = first;
    j.n_parts = parts;
    j.carry = carry;
    const unsigned blocks1 = static_cast<unsigned>(n), blocks2 = static_cast<unsigned>(div_up(n, 2)),
                   blocks8 = static_cast<unsigned>(div_up(n, 8));
    return (n <= 2 * c.sms    ? launch_chained(k_join<1>, blocks1, 256, 0, c.s, 1, j)
            : n <= 16 * c.sms ? launch_chained(k_join<2>, blocks2, 256, 0, c.s, 1, j)
                              : launch_chained(k_join<8>, blocks8, 256, 0, c.s, 1, j)) == cudaSuccess;
  };
  bool ok;
  if (p.blocks) {
    t.launch(a, c);
    SkinnyArgs g = skinny_args(c, a, t);
    g.part = part;
    g.z_t = z_t;
    const int vec = skinny_vec(g.w, g.w_ld, g.dim, g.n_cls, elem_bytes(c.z.type));
    ok = launch_skinny(g, c.z.type, false, vec, &p.blocks, c.s) == cudaSuccess && join(part, p.blocks, nullptr);
  } else {
    const Operand oh = p.h.ready(a, c.s), ow = p.w.ready(a, c.s);
    t.launch(a, c);
    ProdMaps maps;
    if (!encode(&maps.a, oh, prod_box_rows_a()) || !encode(&maps.b, ow, prod_box_rows_b(p.cg, p.bn))) return GM_ERR_CUDA;
    maps.o = maps.a;  // not used
    ProdArgs g = {};
    set_logits_args(g, c, a, t);
    g.m = n;
    g.m_tiles = static_cast<int>(div_up(n, 128 * p.cg));
    g.splits = 1;
    g.k_blocks = g.k_per_split = static_cast<int>(div_up(c.z.dim, 64));
    g.group = group_of(g.m_tiles, 128 * p.cg, c.z.dim, g.planes);
    const bool pieces = p.piece_tiles < p.n_tiles;
    g.part = part + (pieces ? n : 0);
    g.part_ld = n;
    g.z_t = z_t;
    g.lost = lost;
    ok = true;
    for (int64_t t0 = 0; ok && t0 < p.n_tiles; t0 += p.piece_tiles) {
      const int64_t tiles = std::min(p.piece_tiles, p.n_tiles - t0);
      const bool first = t0 == 0, last = t0 + tiles == p.n_tiles;
      g.n_tiles = static_cast<int>(tiles);
      g.cls0 = t0 * p.bn;
      g.b_row0 = static_cast<int>(g.cls0);
      g.n = std::min(tiles * p.bn, c.z.n_classes - g.cls0);
      g.lost_first = first;
      ok = launch_prod(Prod::kStats, p.cg, p.bn, maps, g, c.sms, c.s) == cudaSuccess &&
           join(first ? g.part : part, 2 * tiles + !first, last ? nullptr : part);
    }
  }
  return finish(c, ok, word);
}

struct Grads {
  const float *lse_t, *g_kl, *lse, *g_loss, *g_lse;
  void* dh;
  int64_t dh_ld;
  void* dw;
  int64_t dw_ld;
};

// Where a gradient goes: by TMA where its rows start and end on 16-byte boundaries (a store
// drops what lies outside the map by 16 bytes, not by elements).
bool set_result(CUtensorMap* m, ProdArgs& g, void* out, int64_t rows, int64_t dim, int64_t ld, int32_t type) {
  const int es = static_cast<int>(elem_bytes(type));
  g.out = out;
  g.out_ld = ld;
  g.out_type = type;
  // half a tile of 64 columns of 2 bytes is less than a box
  g.by_tma = aligned(out, 16) && (rows <= 1 || ld * es % 16 == 0) && dim * es % 16 == 0 && (es == 4 || dim > 64);
  if (!g.by_tma) return true;
  if (rows <= 1) ld = up(dim, 16 / es);
  return encode(m, Operand{out, rows, dim, ld, rows * ld, 1, es}, 32);
}

void sum_splits(const Call& c, const float* acc, int splits, int64_t acc_ld, const Grads& q, const uint8_t* lost) {
  const int64_t n = c.z.n_rows * c.z.dim, stride = c.z.n_rows * acc_ld;
  const bool many = splits >= 16;
  launch_chained(many ? k_sum_splits<8> : k_sum_splits<1>, grid_for(n, many ? 32 : 256), 256, 0, c.s, 1, acc, splits, stride,
                 c.z.n_rows, c.z.dim, acc_ld, q.dh, q.dh_ld, static_cast<int>(c.z.type), lost);
}

// How a backward call is cut, and where its workspace lies.
struct BackwardPlan {
  Arena a;
  Source h, w;
  TeacherPlan t;
  int planes, g_planes, g_sets, bn_h, bn_w, cg_h, cg_w;
  int64_t width;   // classes of a piece; rows of G are as long
  int64_t splits;  // of dH's sum along a piece's classes
  bool dh_direct;  // dH needs no sum over pieces or splits
  int64_t acc_ld;
  int blocks = 0;  // of the kernel for few rows; 0: the products
  Words own;
  size_t o_weights = 0, o_g = 0, o_acc = 0;
  explicit BackwardPlan(const Call& c)
      : h(c.z.h, c.z.n_rows, c.z.dim, c.z.h_ld, c.z.type), w(c.z.w, c.z.n_classes, c.z.dim, c.z.w_ld, c.z.type) {
    const int64_t n = c.z.n_rows, cls = c.z.n_classes, dim = c.z.dim;
    own.plan(a);
    planes = c.z.type == GM_LOSS_F32 ? 3 : 1;
    if (skinny(c)) {
      blocks = skinny_most_blocks(cls, c.sms);
      t.plan(a, c);
      o_acc = a.add(blocks * n * dim * 4);
      return;
    }
    g_planes = planes == 3 ? 3 : n <= 128 ? 2 : 1;
    g_sets = c.z.type == GM_LOSS_F16 ? 2 : 1;  // see Scales
    const int64_t cap = c.cap ? c.cap : g_sets * kDefaultCap, g_bytes = n * 2 * g_planes * g_sets;  // of a class
    // pieces of the classes: as few as the bound on G allows, of about equal width
    const int64_t most = std::max<int64_t>(256, cap / g_bytes / 256 * 256);
    const int64_t n_pieces = div_up(cls, most);
    width = std::min<int64_t>(most, up(div_up(cls, n_pieces), 256));
    // tiles of dH: split along the classes when they are fewer than the SMs
    bn_h = prod_sums_cols(dim, n, planes);
    bn_w = prod_sums_cols(dim, cls, planes);
    cg_h = bn_h == 256 && n > 128 ? 2 : 1;
    cg_w = bn_w == 256 && cls > 128 ? 2 : 1;
    const int64_t dh_tiles = div_up(n, 128 * cg_h) * div_up(dim, bn_h);
    const int64_t kb = div_up(std::min(width, cls), 64);
    splits = std::max<int64_t>(1, std::min<int64_t>(c.sms / cg_h / dh_tiles, kb / 8));
    splits = div_up(kb, div_up(kb, splits));
    dh_direct = n_pieces == 1 && splits == 1;
    acc_ld = up(dim, 32);
    h.plan(a);
    w.plan(a);
    t.plan(a, c);
    o_weights = a.add(8);
    o_g = a.add(g_bytes * width);
    o_acc = dh_direct ? 0 : a.add(splits * n * acc_ld * 4);
  }
};

gm_status backward(Call& c, const Grads& q) {
  gm_status rc = begin(c);
  if (rc != GM_OK) return rc;
  const int64_t n = c.z.n_rows, cls = c.z.n_classes, dim = c.z.dim, es = elem_bytes(c.z.type);
  if (n == 0) {
    bool ok = true;
    if (q.dw) ok = cudaMemset2DAsync(q.dw, q.dw_ld * es, 0, dim * es, cls, c.s) == cudaSuccess;
    return finish(c, ok);
  }
  BackwardPlan p(c);
  Arena& a = p.a;
  rc = a.open(c);
  if (rc != GM_OK) return rc;
  uint8_t* lost = a.at<uint8_t>(p.own.lost);
  int* word = a.at<int>(p.own.status);
  rc = own_status(c, word);
  if (rc != GM_OK) return rc;
  const TeacherPlan& t = p.t;
  const RowGrads row{targets_of(c), q.lse,   q.g_loss, q.g_lse, c.teacher ? a.at<int32_t>(t.len) : nullptr,
                     q.lse_t,       q.g_kl, 1.f / c.temperature};
  if (p.blocks) {
    t.launch(a, c);
    SkinnyArgs g = skinny_args(c, a, t);
    g.row = row;
    g.dh = q.dh;
    g.dw = q.dw;
    g.dw_ld = q.dw_ld;
    g.acc = a.at<float>(p.o_acc);
    int vec = skinny_vec(g.w, g.w_ld, dim, cls, es);
    if (q.dw) vec = std::min(vec, skinny_vec(q.dw, q.dw_ld, dim, cls, es));
    const bool ok = launch_skinny(g, c.z.type, true, vec, &p.blocks, c.s) == cudaSuccess;
    if (ok && q.dh) sum_splits(c, g.acc, p.blocks, dim, q, nullptr);
    return finish(c, ok, word);
  }
  const int planes = p.planes, bn_h = p.bn_h, bn_w = p.bn_w, cg_h = p.cg_h, cg_w = p.cg_w;
  const int64_t width = p.width, g_ld = p.width, splits = p.splits, acc_ld = p.acc_ld;
  const bool dh_direct = p.dh_direct;
  const size_t o_g = p.o_g, o_acc = p.o_acc;
  const Operand oh = p.h.ready(a, c.s), ow = p.w.ready(a, c.s);
  t.launch(a, c);
  ProdArgs base = {};
  set_logits_args(base, c, a, t);
  base.row = row;
  base.g_planes = p.g_planes;
  base.lost = lost;
  if (c.z.type == GM_LOSS_F16) {
    unsigned* weights = a.at<unsigned>(p.o_weights);
    launch_chained(k_weights, 1, 1024, 0, c.s, 1, n, base.row, weights);
    base.weights = weights;
    // classes * 2^-25 / 2^(13 - near) <= 2^-11; with 2^27 classes and more no two exponents are near
    base.near = 27;
    while (base.near > 0 && (cls >> (27 - base.near)) > 0) --base.near;
  }
  uint16_t* g_mem = a.at<uint16_t>(o_g);
  bool ok = true;
  for (int64_t c0 = 0; ok && c0 < cls; c0 += width) {
    const int64_t wid = std::min(width, cls - c0);
    const Operand og{g_mem, n, wid, g_ld, n * g_ld, p.g_planes * p.g_sets};
    ProdMaps maps;
    {
      const int cg = n > 128 ? 2 : 1;
      const int bn = prod_logits_cols(cg, planes);
      if (!encode(&maps.a, oh, prod_box_rows_a()) || !encode(&maps.b, ow, prod_box_rows_b(cg, bn)) ||
          !encode(&maps.o, og, 32, prod_grad_row_bytes(planes, base.chunk, static_cast<int>(div_up(dim, 64)))))
        return GM_ERR_CUDA;
      ProdArgs g = base;
      g.m = n;
      g.n = wid;
      g.m_tiles = static_cast<int>(div_up(n, 128 * cg));
      g.n_tiles = static_cast<int>(div_up(wid, bn));
      g.splits = 1;
      g.k_blocks = g.k_per_split = static_cast<int>(div_up(dim, 64));
      g.group = group_of(g.m_tiles, 128 * cg, dim, planes);
      g.b_row0 = static_cast<int>(c0);
      g.cls0 = c0;
      g.lost_first = c0 == 0;
      ok = launch_prod(Prod::kGrad, cg, bn, maps, g, c.sms, c.s) == cudaSuccess;
    }
    if (ok && q.dh) {
      Operand piece = ow;  // the piece's rows alone: past them reads 0
      piece.rows = c0 + wid;
      if (!encode(&maps.a, og, prod_box_rows_a()) || !encode(&maps.b, piece, 64)) return GM_ERR_CUDA;
      ProdArgs g = base;
      g.m = n;
      g.n = dim;
      g.m_tiles = static_cast<int>(div_up(n, 128 * cg_h));
      g.n_tiles = static_cast<int>(div_up(dim, bn_h));
      g.k_blocks = static_cast<int>(div_up(wid, 64));
      g.k_per_split = static_cast<int>(div_up(g.k_blocks, splits));
      g.splits = static_cast<int>(div_up(g.k_blocks, g.k_per_split));
      g.group = 1;
      g.b_row0 = static_cast<int>(c0);
      bool set;
      if (dh_direct) {
        set = set_result(&maps.o, g, q.dh, n, dim, q.dh_ld, c.z.type);
      } else {
        g.acc = g.by_tma = true;
        g.acc_add = c0 > 0;
        set = encode(&maps.o, Operand{a.at<float>(o_acc), n, dim, acc_ld, n * acc_ld, static_cast<int>(splits), 4}, 32);
      }
      if (!set) return GM_ERR_CUDA;
      ok = launch_prod(Prod::kDh, cg_h, bn_h, maps, g, c.sms, c.s) == cudaSuccess;
    }
    if (ok && q.dw) {
      if (!encode(&maps.a, og, 64) || !encode(&maps.b, oh, 64)) return GM_ERR_CUDA;
      ProdArgs g = base;
      g.m = wid;
      g.n = dim;
      g.m_tiles = static_cast<int>(div_up(wid, 128 * cg_w));
      g.n_tiles = static_cast<int>(div_up(dim, bn_w));
      g.splits = 1;
      g.k_blocks = g.k_per_split = static_cast<int>(div_up(n, 64));
      g.group = 1;
      if (!set_result(&maps.o, g, static_cast<char*>(q.dw) + c0 * q.dw_ld * es, wid, dim, q.dw_ld, c.z.type))
        return GM_ERR_CUDA;
      ok = launch_prod(Prod::kDw, cg_w, bn_w, maps, g, c.sms, c.s) == cudaSuccess;
    }
  }
  if (ok && q.dh && !dh_direct)
    sum_splits(c, a.at<float>(o_acc), static_cast<int>(splits), acc_ld, q, lost);
  return finish(c, ok, word);
}

gm_status check_grads(const Call& c, const Grads& q) {
  if (!q.dh && !q.dw) return GM_ERR_INVALID_ARG;
  const int64_t es = elem_bytes(c.z.type);
  if ((q.dh && (q.dh_ld < c.z.dim || !aligned(q.dh, es))) || (q.dw && (q.dw_ld < c.z.dim || !aligned(q.dw, es))))
    return GM_ERR_INVALID_ARG;
  if (c.z.n_rows == 0) return GM_OK;
  if (c.labels && (!q.lse || !q.g_loss)) return GM_ERR_INVALID_ARG;
  if (c.teacher && (!q.lse_t || !q.g_kl)) return GM_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(q.lse), static_cast<const void*>(q.lse_t),
                        static_cast<const void*>(q.g_loss), static_cast<const void*>(q.g_lse),
                        static_cast<const void*>(q.g_kl)})
    if (!aligned(p, 4)) return GM_ERR_INVALID_ARG;
  return GM_OK;
}

}  // namespace

}  // namespace gm

extern "C" gm_status gm_xent_forward(const gm_logits* z, const gm_labels* labels, const gm_loss_config* cfg,
                                     void* stream, float* loss, float* lse) {
  gm::NvtxRange range("gm_xent_forward");
  gm::Call c;
  if (!labels) return GM_ERR_INVALID_ARG;
  const gm_status rc = gm::check(c, z, labels, cfg, stream);
  if (rc != GM_OK) return rc;
  if (c.z.n_rows > 0 && (!loss || !lse || !gm::aligned(loss, 4) || !gm::aligned(lse, 4))) return GM_ERR_INVALID_ARG;
  return gm::forward(c, nullptr, nullptr, loss, lse);
}

extern "C" gm_status gm_xent_backward(const gm_logits* z, const gm_labels* labels, const gm_loss_config* cfg,
                                      void* stream, const float* lse, const float* grad_loss, const float* grad_lse,
                                      void* dh, int64_t dh_ld, void* dw, int64_t dw_ld) {
  gm::NvtxRange range("gm_xent_backward");
  gm::Call c;
  if (!labels) return GM_ERR_INVALID_ARG;
  gm_status rc = gm::check(c, z, labels, cfg, stream);
  if (rc != GM_OK) return rc;
  const gm::Grads q{nullptr, nullptr, lse, grad_loss, grad_lse, dh, dh_ld, dw, dw_ld};
  rc = gm::check_grads(c, q);
  return rc != GM_OK ? rc : gm::backward(c, q);
}

extern "C" gm_status gm_distill_forward(const gm_logits* z, const gm_csr* teacher, int32_t value_type,
                                        int32_t index_type, float temperature, const gm_labels* labels,
                                        const gm_loss_config* cfg, void* stream, float* kl, float* lse_t, float* loss,
                                        float* lse) {
  gm::NvtxRange range("gm_distill_forward");
  gm::Call c;
  gm_status rc = gm::check(c, z, labels, cfg, stream);
  if (rc == GM_OK) rc = gm::check_teacher(c, teacher, value_type, index_type, temperature);
  if (rc != GM_OK) return rc;
  if (!labels && (loss || lse)) return GM_ERR_INVALID_ARG;
  if (c.z.n_rows > 0 && (!kl || !lse_t || (labels && (!loss || !lse)))) return GM_ERR_INVALID_ARG;
  for (const float* p : {kl, lse_t, loss, lse})
    if (!gm::aligned(p, 4)) return GM_ERR_INVALID_ARG;
  return gm::forward(c, kl, lse_t, loss, lse);
}

extern "C" gm_status gm_distill_backward(const gm_logits* z, const gm_csr* teacher, int32_t value_type,
                                         int32_t index_type, float temperature, const gm_labels* labels,
                                         const gm_loss_config* cfg, void* stream, const float* lse_t,
                                         const float* grad_kl, const float* lse, const float* grad_loss,
                                         const float* grad_lse, void* dh, int64_t dh_ld, void* dw, int64_t dw_ld) {
  gm::NvtxRange range("gm_distill_backward");
  gm::Call c;
  gm_status rc = gm::check(c, z, labels, cfg, stream);
  if (rc == GM_OK) rc = gm::check_teacher(c, teacher, value_type, index_type, temperature);
  if (rc != GM_OK) return rc;
  const gm::Grads q{lse_t, grad_kl, lse, grad_loss, grad_lse, dh, dh_ld, dw, dw_ld};
  rc = gm::check_grads(c, q);
  return rc != GM_OK ? rc : gm::backward(c, q);
}

extern "C" gm_status gm_loss_workspace(const gm_logits* z, int64_t teacher_nnz, int32_t backward,
                                       const gm_loss_config* cfg, int64_t* bytes) {
  if (!bytes || (backward != 0 && backward != 1)) return GM_ERR_INVALID_ARG;
  gm::Call c;
  const gm_status rc = gm::check(c, z, nullptr, cfg, nullptr);
  if (rc != GM_OK) return rc;
  *bytes = 0;
  if (c.z.n_rows == 0) return GM_OK;
  c.nnz = teacher_nnz < 0 ? -1 : teacher_nnz;
  c.sms = gm::sm_count();
  if (c.sms <= 0) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  *bytes = static_cast<int64_t>(backward ? gm::BackwardPlan(c).a.used : gm::ForwardPlan(c).a.used);
  return GM_OK;
}

extern "C" gm_status gm_loss_status(void* stream) {
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  gm::DevBuf<int> taken;
  if (!taken.alloc(1, s)) return GM_ERR_OOM;
  (gm::k_take_status<<<1, 1, 0, s>>>(taken.p), gm::note_launch());
  int bits = 0;
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemcpyAsync(&bits, taken.p, 4, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  return gm::status_of(bits);
}
