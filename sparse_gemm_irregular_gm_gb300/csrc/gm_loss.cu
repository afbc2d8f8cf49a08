// gm_loss.cu -- losses over a large class table (include/gm_losses.h): the host
// driver and the kernels around the tensor-core products of gm_loss_prod.cu.
//
// Forward: one product reduces Z = H W^T to a maximum and sums of exponentials for
// each row and half tile, a second kernel joins them. Backward, for each piece of the
// classes: the product again, its end writing the piece of G = dloss/dZ, then
// dH += G W_piece and dW_piece = G^T H. Nothing of the size of Z is ever stored.
#include "gm_loss.h"

#include <algorithm>
#include <cmath>
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <nvtx3/nvToolsExt.h>

#include "gm_device.cuh"
#include "gm_umma.cuh"

namespace gm {

namespace {

__device__ int g_loss_status;

// ---- operands that TMA cannot read in place ------------------------------------------
// f32: three bf16 planes, x = x0 + x1 + x2 with x0 the nearest bf16 of x and so on, which
// keeps all 24 bits; 16-bit types: one plane, copied. Rows are padded with zeros to ld.
__global__ void k_pack(const void* __restrict__ src, int64_t rows, int64_t dim, int64_t src_ld, bool f32,
                       uint16_t* __restrict__ dst, int64_t ld) {
  const int64_t n = rows * ld, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t r = i / ld, c = i - r * ld;
    if (!f32) {
      dst[i] = c < dim ? static_cast<const uint16_t*>(src)[r * src_ld + c] : 0;
      continue;
    }
    float x = c < dim ? static_cast<const float*>(src)[r * src_ld + c] : 0.f;
    const bool finite = fabsf(x) <= 3.4e38f;
    for (int p = 0; p < 3; ++p) {
      const __nv_bfloat16 b = __float2bfloat16_rn(x);
      dst[p * n + i] = __bfloat16_as_ushort(b);
      x = finite ? x - __bfloat162float(b) : 0.f;  // infinities and NaN stand in the first plane
    }
  }
}

// ---- the teacher's rows -----------------------------------------------------------------
template <class T>
__device__ T block_reduce(T x, T* sh, bool maximum) {  // 128 threads; every thread gets the result
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const T y = __shfl_xor_sync(kFull, x, d);
    x = maximum ? (y > x ? y : x) : x + y;
  }
  __syncthreads();
  if (lane == 0) sh[warp] = x;
  __syncthreads();
  x = sh[0];
  for (int w = 1; w < 4; ++w) x = maximum ? (sh[w] > x ? sh[w] : x) : x + sh[w];
  return x;
}

// q = softmax of each row's stored values / T, one block a row; base[row] = sum q log q.
template <class V, class R, class C>
__global__ void __launch_bounds__(128) k_teacher(const R* __restrict__ rp, const C* __restrict__ col,
                                                 const V* __restrict__ val, int64_t n_rows, int64_t n_cls, int64_t nnz,
                                                 float inv_t, int64_t* __restrict__ start, int32_t* __restrict__ len,
                                                 int2* __restrict__ ents, float* __restrict__ base,
                                                 int* __restrict__ status) {
  __shared__ double sh_d[4];
  __shared__ float sh_f[4];
  for (int64_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
    const int64_t lo = static_cast<int64_t>(rp[row]), hi = static_cast<int64_t>(rp[row + 1]);
    bool bad = lo < 0 || hi < lo || hi > nnz;
    float m = -INFINITY;
    if (!bad) {
      int wrong = 0;
      for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
        const int64_t c = static_cast<int64_t>(col[i]);
        if (c < 0 || c >= n_cls || (i > lo && static_cast<int64_t>(col[i - 1]) >= c)) wrong = 1;
        m = fmaxf(m, static_cast<float>(val[i] * inv_t));
      }
      bad = __syncthreads_or(wrong) != 0;
      m = block_reduce(m, sh_f, true);
    }
    double sum = 0.0, log_sum = 0.0, b = 0.0;
    // a NaN value leaves the maximum alone and makes the sum NaN, so the row counts as one with entries
    bool any = false;
    if (!bad) {
      for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
        const float v = static_cast<float>(val[i] * inv_t);
        sum += v == -INFINITY ? 0.0 : static_cast<double>(expf(v - m));
      }
      sum = block_reduce(sum, sh_d, false);
      any = sum != 0.0;
    }
    if (any) {
      log_sum = log(sum);
      const float inv = static_cast<float>(1.0 / sum);
      for (int64_t i = lo + threadIdx.x; i < hi; i += blockDim.x) {
        const float v = static_cast<float>(val[i] * inv_t);
        const float q = v == -INFINITY ? 0.f : expf(v - m) * inv;
        ents[i] = make_int2(static_cast<int>(col[i]), __float_as_int(q));
        if (q > 0.f || q != q) b += static_cast<double>(q) * (static_cast<double>(v) - m - log_sum);
      }
      b = block_reduce(b, sh_d, false);
    }
    if (threadIdx.x == 0) {
      start[row] = lo;
      len[row] = any ? static_cast<int32_t>(hi - lo) : 0;
      base[row] = bad ? NAN : static_cast<float>(b);
      if (bad) atomicOr(status, kLossBadTeacher);
    }
  }
}

// ---- joining the half tiles of a row -----------------------------------------------------
struct JoinArgs {
  const float4* part;
  int64_t n_parts, n_rows;
  Targets tgt;
  const float* z_t;
  const int32_t* ent_len;  // null: no teacher
  const float* base;
  float inv_t;
  float *loss, *lse, *kl, *lse_t;
  int* status;
};
template <int ROWS>  // rows of a block; 256 / ROWS threads a row
__global__ void __launch_bounds__(256) k_join(const JoinArgs a) {
  constexpr int kSub = 256 / ROWS;
  const int rl = threadIdx.x % ROWS, sub = threadIdx.x / ROWS;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + rl;
  const bool dis = a.ent_len != nullptr;
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
  if (row < a.n_rows)
    for (int64_t p = sub; p < a.n_parts; p += kSub) add(a.part[p * a.n_rows + row]);
  __shared__ float4 sh[256];
  for (int d = kSub / 2; d > 0; d >>= 1) {
    if (sub >= d && sub < 2 * d) sh[threadIdx.x] = make_float4(m, s1, st, zq);
    __syncthreads();
    if (sub < d) add(sh[threadIdx.x + d * ROWS]);
    __syncthreads();
  }
  if (sub != 0 || row >= a.n_rows) return;
  const bool lost = (*a.status & kLossTimeout) != 0;
  if (a.tgt.t) {
    const float l = lost ? NAN : m + logf(s1);
    const int64_t t = row_target(a.tgt, row);
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

// ---- what the backward pass needs of a row -------------------------------------------------
__global__ void k_row_grads(int64_t n, Targets tgt, const float* __restrict__ lse, const float* __restrict__ g_loss,
                            const float* __restrict__ g_lse, const int32_t* __restrict__ ent_len,
                            const float* __restrict__ lse_t, const float* __restrict__ g_kl, float inv_t,
                            float4* __restrict__ row_c, float* __restrict__ row_gl, unsigned* __restrict__ g_max,
                            int* __restrict__ status) {
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; r < n; r += stride) {
    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
    float gl = 0.f;
    if (tgt.t) {
      const int64_t t = row_target(tgt, r);
      gl = t >= 0 ? g_loss[r] : 0.f;
      c.x = lse[r];
      c.y = gl + (g_lse ? g_lse[r] : 0.f);
      if (t == -2) atomicOr(status, kLossBadTarget);
    }
    if (ent_len) {
      c.z = lse_t[r];
      c.w = ent_len[r] > 0 ? g_kl[r] * inv_t : 0.f;
    }
    row_c[r] = c;
    row_gl[r] = gl;
    // no product of the row's weights and probabilities is larger
    if (g_max) atomicMax(g_max, __float_as_uint(fabsf(c.y) + fabsf(gl) + fabsf(c.w)));
  }
}

// dh = the splits' sums, rounded
__global__ void k_sum_splits(const float* __restrict__ acc, int splits, int64_t split_stride, int64_t rows, int64_t dim,
                             int64_t acc_ld, void* __restrict__ out, int64_t out_ld, int type,
                             const unsigned* __restrict__ g_max, const int* __restrict__ status) {
  const int64_t n = rows * dim, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const float inv = (*status & kLossTimeout) ? NAN : 1.f / g_scale_of(g_max);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += stride) {
    const int64_t r = i / dim, c = i - r * dim;
    float x = 0.f;
    for (int s = 0; s < splits; ++s) x += acc[s * split_stride + r * acc_ld + c];
    x *= inv;
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

// 16-bit matrix of `planes` planes of rows x cols, ld elements a row.
struct Operand {
  const uint16_t* p;
  int64_t rows, cols, ld, plane;
  int planes;
};
// Boxes of box_rows rows of 64 elements, 128-byte swizzle; elements outside read as 0.
bool encode(CUtensorMap* m, const Operand& o, int box_rows) {
  const EncodeTiled fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(o.cols), static_cast<cuuint64_t>(o.rows),
                              static_cast<cuuint64_t>(o.planes)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(o.ld) * 2, static_cast<cuuint64_t>(o.plane) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<uint16_t*>(o.p), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }

// One workspace block, carved in order.
struct Arena {
  DevBuf<unsigned char> buf;
  size_t used = 0;
  size_t add(int64_t bytes) {
    const size_t at = used;
    used += static_cast<size_t>(up(bytes, 256));
    return at;
  }
  template <class T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(buf.p + off);
  }
};

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

int64_t elem_bytes(int32_t type) { return type == GM_LOSS_F32 ? 4 : 2; }
bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int64_t kMostIndex = (int64_t(1) << 31) - 256;  // tile coordinates are int32
constexpr int64_t kDefaultCap = int64_t(256) << 20;

struct Call {
  gm_logits z;
  const gm_csr* teacher;  // null: cross entropy alone
  int32_t value_type = 0, index_type = 0;
  float temperature = 1.f;
  const gm_labels* labels;
  int64_t cap = kDefaultCap;
  int32_t flags = 0;
  cudaStream_t s = nullptr;
  int sms = 0;
  int* status = nullptr;
};

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
    if (cfg->workspace_cap_bytes) c.cap = cfg->workspace_cap_bytes;
    c.flags = cfg->flags;
  }
  c.s = static_cast<cudaStream_t>(stream);
  return GM_OK;
}

gm_status check_teacher(Call& c, const gm_csr* t, int32_t value_type, int32_t index_type, float temperature) {
  if (!t) return GM_ERR_INVALID_ARG;
  if (t->n_rows != c.z.n_rows || t->n_cols != c.z.n_classes) return GM_ERR_DIM_MISMATCH;
  if (value_type != GM_VALUE_F64 && value_type != GM_VALUE_F32) return GM_ERR_INVALID_ARG;
  if (index_type & ~(GM_INDEX_ROWPTR32 | GM_INDEX_COL64)) return GM_ERR_INVALID_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature)) return GM_ERR_INVALID_ARG;
  if (t->nnz < 0 || !t->row_ptr || (t->nnz > 0 && (!t->col_idx || !t->vals))) return GM_ERR_INVALID_ARG;
  if (!aligned(t->row_ptr, index_type & GM_INDEX_ROWPTR32 ? 4 : 8) ||
      !aligned(t->col_idx, index_type & GM_INDEX_COL64 ? 8 : 4) || !aligned(t->vals, value_type == GM_VALUE_F64 ? 8 : 4))
    return GM_ERR_INVALID_ARG;
  c.teacher = t;
  c.value_type = value_type;
  c.index_type = index_type;
  c.temperature = temperature;
  return GM_OK;
}

// Device facts and a clear error state; GM_ERR_CUDA leaves a pending error to its owner.
gm_status begin(Call& c) {
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  int dev = 0;
  void* st = nullptr;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaGetSymbolAddress(&st, g_loss_status) != cudaSuccess) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  c.status = static_cast<int*>(st);
  return GM_OK;
}

gm_status finish(const Call& c, bool launched) {
  if (cudaGetLastError() != cudaSuccess || !launched) return GM_ERR_CUDA;
  return c.flags & GM_LOSS_CHECK ? gm_loss_status(c.s) : GM_OK;
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
    Operand o{static_cast<const uint16_t*>(p), rows, dim, ld, rows * ld, planes()};
    if (packed) {
      o.p = a.at<uint16_t>(off);
      k_pack<<<grid_for(rows * ld, 256), 256, 0, s>>>(p, rows, dim, src_ld, type == GM_LOSS_F32, a.at<uint16_t>(off), ld);
      note_launch();
    }
    return o;
  }
};

struct TeacherPlan {
  size_t start = 0, len = 0, ents = 0, base = 0;
  void plan(Arena& a, const Call& c) {
    if (!c.teacher) return;
    start = a.add(c.z.n_rows * 8);
    len = a.add(c.z.n_rows * 4);
    base = a.add(c.z.n_rows * 4);
    ents = a.add(c.teacher->nnz * 8);
  }
  template <class V, class R, class C>
  void run(const Arena& a, const Call& c) const {
    const int64_t blocks = std::min<int64_t>(c.z.n_rows, int64_t(c.sms) * 64);
    k_teacher<V, R, C><<<static_cast<unsigned>(blocks), 128, 0, c.s>>>(
        static_cast<const R*>(c.teacher->row_ptr), static_cast<const C*>(c.teacher->col_idx),
        static_cast<const V*>(c.teacher->vals), c.z.n_rows, c.z.n_classes, c.teacher->nnz, 1.f / c.temperature,
        a.at<int64_t>(start), a.at<int32_t>(len), a.at<int2>(ents), a.at<float>(base), c.status);
    note_launch();
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

void set_logits_args(ProdArgs& g, const Call& c, const Arena& a, const TeacherPlan& t) {
  g.tgt = targets_of(c);
  g.status = c.status;
  g.planes = c.z.type == GM_LOSS_F32 ? 3 : 1;
  g.bf16 = c.z.type != GM_LOSS_F16;
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

gm_status forward(Call& c, float* kl, float* lse_t, float* loss, float* lse) {
  gm_status rc = begin(c);
  if (rc != GM_OK) return rc;
  const int64_t n = c.z.n_rows;
  if (n == 0) return finish(c, true);
  const int cg = n > 128 ? 2 : 1, bn = 256;
  const int64_t n_tiles = div_up(c.z.n_classes, bn), n_parts = 2 * n_tiles;
  Arena a;
  Source h(c.z.h, n, c.z.dim, c.z.h_ld, c.z.type), w(c.z.w, c.z.n_classes, c.z.dim, c.z.w_ld, c.z.type);
  TeacherPlan t;
  h.plan(a);
  w.plan(a);
  t.plan(a, c);
  const size_t o_part = a.add(n_parts * n * 16), o_zt = a.add(n * 4);
  if (!a.buf.alloc(a.used, c.s)) return GM_ERR_OOM;
  const Operand oh = h.ready(a, c.s), ow = w.ready(a, c.s);
  t.launch(a, c);
  ProdMaps maps;
  if (!encode(&maps.a, oh, prod_box_rows_a()) || !encode(&maps.b, ow, prod_box_rows_b(cg, bn))) return GM_ERR_CUDA;
  ProdArgs g = {};
  set_logits_args(g, c, a, t);
  g.m = n;
  g.n = c.z.n_classes;
  g.m_tiles = static_cast<int>(div_up(n, 128 * cg));
  g.n_tiles = static_cast<int>(n_tiles);
  g.splits = 1;
  g.k_blocks = g.k_per_split = static_cast<int>(div_up(c.z.dim, 64));
  g.group = group_of(g.m_tiles, 128 * cg, c.z.dim, g.planes);
  g.part = a.at<float4>(o_part);
  g.part_ld = n;
  g.z_t = a.at<float>(o_zt);
  bool ok = launch_prod(Prod::kStats, cg, bn, maps, g, c.sms, c.s) == cudaSuccess;
  JoinArgs j = {};
  j.part = g.part;
  j.n_parts = n_parts;
  j.n_rows = n;
  j.tgt = g.tgt;
  j.z_t = g.z_t;
  j.ent_len = g.ent_len;
  j.base = c.teacher ? a.at<float>(t.base) : nullptr;
  j.inv_t = 1.f / c.temperature;
  j.loss = loss;
  j.lse = lse;
  j.kl = kl;
  j.lse_t = lse_t;
  j.status = c.status;
  if (ok) {
    // few rows: a block each, so that their half tiles are read by many threads
    if (n <= 4 * c.sms) k_join<1><<<static_cast<unsigned>(n), 256, 0, c.s>>>(j);
    else k_join<32><<<static_cast<unsigned>(div_up(n, 32)), 256, 0, c.s>>>(j);
    note_launch();
  }
  return finish(c, ok);
}

struct Grads {
  const float *lse_t, *g_kl, *lse, *g_loss, *g_lse;
  void* dh;
  int64_t dh_ld;
  void* dw;
  int64_t dw_ld;
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
  const int planes = c.z.type == GM_LOSS_F32 ? 3 : 1;
  // pieces of the classes: as few as the bound on G allows, of about equal width
  const int64_t most = std::max<int64_t>(256, c.cap / (n * 2 * planes) / 256 * 256);
  const int64_t n_pieces = div_up(cls, most);
  const int64_t width = std::min<int64_t>(most, up(div_up(cls, n_pieces), 256));
  const int64_t g_ld = width;
  // tiles of dH: split along the classes when they are fewer than the SMs
  const int bn_d = dim > 128 ? 256 : dim > 64 ? 128 : 64;
  const int cg_h = bn_d == 256 && n > 128 ? 2 : 1, cg_w = bn_d == 256 ? 2 : 1;
  const int64_t dh_tiles = div_up(n, 128 * cg_h) * div_up(dim, bn_d);
  const int64_t kb = div_up(std::min(width, cls), 64);
  int64_t splits = std::max<int64_t>(1, std::min<int64_t>(c.sms / cg_h / dh_tiles, kb / 8));
  splits = div_up(kb, div_up(kb, splits));
  const bool dh_direct = n_pieces == 1 && splits == 1;
  const int64_t acc_ld = up(dim, 32);

  Arena a;
  Source h(c.z.h, n, dim, c.z.h_ld, c.z.type), w(c.z.w, cls, dim, c.z.w_ld, c.z.type);
  TeacherPlan t;
  h.plan(a);
  w.plan(a);
  t.plan(a, c);
  const size_t o_rc = a.add(n * 16), o_gl = a.add(n * 4), o_max = a.add(4), o_g = a.add(planes * n * g_ld * 2);
  const size_t o_acc = q.dh && !dh_direct ? a.add(splits * n * acc_ld * 4) : 0;
  if (!a.buf.alloc(a.used, c.s)) return GM_ERR_OOM;
  const Operand oh = h.ready(a, c.s), ow = w.ready(a, c.s);
  t.launch(a, c);
  ProdArgs base = {};
  set_logits_args(base, c, a, t);
  unsigned* g_max = nullptr;
  if (c.z.type == GM_LOSS_F16) {
    g_max = a.at<unsigned>(o_max);
    if (cudaMemsetAsync(g_max, 0, 4, c.s) != cudaSuccess) return GM_ERR_CUDA;
  }
  k_row_grads<<<grid_for(n, 256), 256, 0, c.s>>>(n, base.tgt, q.lse, q.g_loss, q.g_lse, base.ent_len, q.lse_t, q.g_kl,
                                                 1.f / c.temperature, a.at<float4>(o_rc), a.at<float>(o_gl), g_max,
                                                 c.status);
  note_launch();
  base.g_max = g_max;
  uint16_t* g_mem = a.at<uint16_t>(o_g);
  bool ok = true;
  for (int64_t c0 = 0; ok && c0 < cls; c0 += width) {
    const int64_t wid = std::min(width, cls - c0);
    const Operand og{g_mem, n, wid, g_ld, n * g_ld, planes};
    ProdMaps maps;
    {
      const int cg = n > 128 ? 2 : 1;
      if (!encode(&maps.a, oh, prod_box_rows_a()) || !encode(&maps.b, ow, prod_box_rows_b(cg, 256))) return GM_ERR_CUDA;
      ProdArgs g = base;
      g.m = n;
      g.n = wid;
      g.m_tiles = static_cast<int>(div_up(n, 128 * cg));
      g.n_tiles = static_cast<int>(div_up(wid, 256));
      g.splits = 1;
      g.k_blocks = g.k_per_split = static_cast<int>(div_up(dim, 64));
      g.group = group_of(g.m_tiles, 128 * cg, dim, planes);
      g.b_row0 = static_cast<int>(c0);
      g.cls0 = c0;
      g.row_c = a.at<float4>(o_rc);
      g.row_gl = a.at<float>(o_gl);
      g.g = g_mem;
      g.g_ld = g_ld;
      g.g_plane = og.plane;
      ok = launch_prod(Prod::kGrad, cg, 256, maps, g, c.sms, c.s) == cudaSuccess;
    }
    if (ok && q.dh) {
      Operand piece = ow;  // the piece's rows alone: past them reads 0
      piece.rows = c0 + wid;
      if (!encode(&maps.a, og, prod_box_rows_a()) || !encode(&maps.b, piece, 64)) return GM_ERR_CUDA;
      ProdArgs g = base;
      g.m = n;
      g.n = dim;
      g.m_tiles = static_cast<int>(div_up(n, 128 * cg_h));
      g.n_tiles = static_cast<int>(div_up(dim, bn_d));
      g.k_blocks = static_cast<int>(div_up(wid, 64));
      g.k_per_split = static_cast<int>(div_up(g.k_blocks, splits));
      g.splits = static_cast<int>(div_up(g.k_blocks, g.k_per_split));
      g.group = 1;
      g.b_row0 = static_cast<int>(c0);
      if (dh_direct) {
        g.out = q.dh;
        g.out_ld = q.dh_ld;
        g.out_type = c.z.type;
      } else {
        g.acc = a.at<float>(o_acc);
        g.acc_ld = acc_ld;
        g.acc_split = n * acc_ld;
        g.acc_add = c0 > 0;
      }
      ok = launch_prod(Prod::kDh, cg_h, bn_d, maps, g, c.sms, c.s) == cudaSuccess;
    }
    if (ok && q.dw) {
      if (!encode(&maps.a, og, 64) || !encode(&maps.b, oh, 64)) return GM_ERR_CUDA;
      ProdArgs g = base;
      g.m = wid;
      g.n = dim;
      g.m_tiles = static_cast<int>(div_up(wid, 128 * cg_w));
      g.n_tiles = static_cast<int>(div_up(dim, bn_d));
      g.splits = 1;
      g.k_blocks = g.k_per_split = static_cast<int>(div_up(n, 64));
      g.group = 1;
      g.out = static_cast<char*>(q.dw) + c0 * q.dw_ld * es;
      g.out_ld = q.dw_ld;
      g.out_type = c.z.type;
      ok = launch_prod(Prod::kDw, cg_w, bn_d, maps, g, c.sms, c.s) == cudaSuccess;
    }
  }
  if (ok && q.dh && !dh_direct) {
    k_sum_splits<<<grid_for(n * dim, 256), 256, 0, c.s>>>(a.at<float>(o_acc), static_cast<int>(splits), n * acc_ld, n,
                                                          dim, acc_ld, q.dh, q.dh_ld, c.z.type, g_max, c.status);
    note_launch();
  }
  return finish(c, ok);
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
  gm::Call c = {};
  c.cap = gm::kDefaultCap;
  c.temperature = 1.f;
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
  gm::Call c = {};
  c.cap = gm::kDefaultCap;
  c.temperature = 1.f;
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
  gm::Call c = {};
  c.cap = gm::kDefaultCap;
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
  gm::Call c = {};
  c.cap = gm::kDefaultCap;
  gm_status rc = gm::check(c, z, labels, cfg, stream);
  if (rc == GM_OK) rc = gm::check_teacher(c, teacher, value_type, index_type, temperature);
  if (rc != GM_OK) return rc;
  const gm::Grads q{lse_t, grad_kl, lse, grad_loss, grad_lse, dh, dh_ld, dw, dw_ld};
  rc = gm::check_grads(c, q);
  return rc != GM_OK ? rc : gm::backward(c, q);
}

extern "C" gm_status gm_loss_status(void* stream) {
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int bits = 0;
  if (cudaMemcpyFromSymbolAsync(&bits, gm::g_loss_status, 4, 0, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  if (bits) {
    const int zero = 0;
    if (cudaMemcpyToSymbolAsync(gm::g_loss_status, &zero, 4, 0, cudaMemcpyHostToDevice, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess) {
      cudaGetLastError();
      return GM_ERR_CUDA;
    }
  }
  if (bits & gm::kLossTimeout) return GM_ERR_DEVICE_TIMEOUT;
  return bits ? GM_ERR_BAD_INDEX : GM_OK;
}
