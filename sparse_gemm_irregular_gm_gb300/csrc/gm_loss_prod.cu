// gm_loss_prod.cu -- the matrix products of the losses over a class table, each
// with its own end: Z = H W^T reduced to row statistics, Z again turned into
// G = dloss/dZ, dH = G W and dW = G^T H.
//
// One persistent kernel: blocks (or pairs of blocks) walk the tiles of the result.
// Warp 0 loads operand tiles with TMA into a ring of 64-deep stages, one lane of warp
// 1 issues tcgen05 products into one of two TMEM accumulators, and warps 4-11 read
// the other accumulator: a thread holds one row, 32 columns at a time, so the row
// reductions need no shuffles.
#include "gm_device.cuh"
#include "gm_loss.h"
#include "gm_umma.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gm {

namespace {

constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;
constexpr int kBK = 64;  // summed elements a stage: one 128-byte swizzled row

// Order of the plane products of split fp32 operands (x = x0 + x1 + x2, bf16 each, by
// falling size): the small ones first, so that they meet a small accumulator; x1 y2,
// x2 y1 and x2 y2 lie under 2^-24 of x y and are left out.
__device__ __constant__ const int kPlaneA[6] = {2, 0, 1, 1, 0, 0};
__device__ __constant__ const int kPlaneB[6] = {0, 2, 1, 0, 1, 0};

template <int CG, int BN>
struct Shape {
  static constexpr int kABytes = 128 * 128;            // this block's 128 rows of A
  static constexpr int kBRows = BN / CG;               // its rows (columns) of B
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kStages = 196608 / kStage > 8 ? 8 : 196608 / kStage;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + 512;
};

struct Tile {
  int m, n, split;
};
__device__ __forceinline__ Tile tile_at(const ProdArgs& g, int t) {
  const int mn = g.m_tiles * g.n_tiles;
  Tile r;
  r.split = t / mn;
  t -= r.split * mn;
  const int per = g.group * g.n_tiles;
  const int grp = t / per;
  t -= grp * per;
  const int rows = min(g.group, g.m_tiles - grp * g.group);
  r.n = t / rows;
  r.m = grp * g.group + t - r.n * rows;
  return r;
}

// First entry of [lo, hi) whose class is at least cls.
__device__ __forceinline__ int64_t first_entry(const int2* e, int64_t lo, int64_t hi, int64_t cls) {
  while (lo < hi) {
    const int64_t mid = (lo + hi) >> 1;
    if (e[mid].x < cls) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t pack2(float a, float b, bool bf16) {
  if (bf16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
  const __half2 r = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Teacher entries of a row, in step with the columns.
struct Walk {
  const int2* e;
  int64_t at, end;
  int2 next;
  __device__ __forceinline__ void start(const ProdArgs& g, int64_t row, int64_t cls) {
    e = g.ents;
    at = end = 0;
    if (row < g.m) {
      const int64_t lo = g.ent_start[row];
      end = lo + g.ent_len[row];
      at = first_entry(e, lo, end, cls);
    }
    next = at < end ? e[at] : make_int2(INT32_MAX, 0);
  }
  __device__ __forceinline__ void step() {
    ++at;
    next = at < end ? e[at] : make_int2(INT32_MAX, 0);
  }
};

// ---- row statistics of half a tile -------------------------------------------------
template <int BN, bool LAB, bool DIS>
__device__ __forceinline__ void end_stats(const ProdArgs& g, uint32_t tmem, int64_t row, int n_tile, int half) {
  constexpr int kCols = BN / 2;
  const int64_t cls = g.cls0 + int64_t(n_tile) * BN + half * kCols;  // class of the first column
  const int64_t end = g.cls0 + g.n;
  float m = -INFINITY, s1 = 0.f, st = 0.f, zq = 0.f;
  int64_t t = -1;
  if (LAB && row < g.m) t = row_target(g.tgt, row);
  Walk w;
  if (DIS) w.start(g, row, cls);
#pragma unroll 1
  for (int c = 0; c < kCols; c += 32) {
    const int64_t k0 = cls + c;
    if (k0 >= end) break;
    float v[32];
    __syncwarp();
    tmem_load32(tmem + half * kCols + c, v);
    tmem_load_wait(v);
    if (k0 + 32 > end) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (k0 + j >= end) v[j] = -INFINITY;
    }
    float mx = v[0];
#pragma unroll
    for (int j = 1; j < 32; ++j) mx = fmaxf(mx, v[j]);
    const float mn = fmaxf(m, mx);
    const float ref = mn == -INFINITY ? 0.f : mn;
    if (LAB) {
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        a0 += ex2(fmaf(v[j], kLog2e, -ref * kLog2e));
        a1 += ex2(fmaf(v[j + 1], kLog2e, -ref * kLog2e));
      }
      s1 = s1 * ex2((m - ref) * kLog2e) + (a0 + a1);
    }
    if (DIS) {
      float a0 = 0.f, a1 = 0.f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {
        a0 += ex2(fmaf(v[j], g.c_t, -ref * g.c_t));
        a1 += ex2(fmaf(v[j + 1], g.c_t, -ref * g.c_t));
      }
      st = st * ex2((m - ref) * g.c_t) + (a0 + a1);
    }
    m = mn;
    if (LAB) {
      const int rel = t >= k0 && t < k0 + 32 ? static_cast<int>(t - k0) : -1;
      if (__any_sync(kFull, rel >= 0)) {
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == rel) z = v[j];
        if (rel >= 0) g.z_t[row] = z;
      }
    }
    if (DIS) {
      while (__any_sync(kFull, w.next.x < k0 + 32)) {
        const int rel = w.next.x < k0 + 32 ? static_cast<int>(w.next.x - k0) : -1;
        float z = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == rel) z = v[j];
        if (rel >= 0) {
          const float q = __int_as_float(w.next.y);
          if (q > 0.f || q != q) zq += q * z;
          w.step();
        }
      }
    }
  }
  if (row < g.m) g.part[(int64_t(n_tile) * 2 + half) * g.part_ld + row] = make_float4(m, s1, st, zq);
}

// ---- gradient of the logits ----------------------------------------------------------
// G_ij = a_i e^(z - lse) - gl_i [j = t_i] + b_i (e^(z / T - lse_T) - q_ij), rounded to 16 bits as
// the operand of the two products after it (times a power of two in f16, whose range
// is too short for small probabilities times small weights); fp32 operands keep it in
// three bf16 planes, 24 bits.
template <int BN, bool LAB, bool DIS>
__device__ __forceinline__ void end_grad(const ProdArgs& g, uint32_t tmem, int64_t row, int n_tile, int half) {
  constexpr int kCols = BN / 2;
  const int64_t col0 = int64_t(n_tile) * BN + half * kCols;
  const int64_t cls = g.cls0 + col0;
  const bool in = row < g.m;
  float4 rc = make_float4(0.f, 0.f, 0.f, 0.f);
  float gl = 0.f;
  int64_t t = -1;
  if (in) {
    rc = g.row_c[row];
    if (LAB) {
      gl = g.row_gl[row];
      t = row_target(g.tgt, row);
    }
  }
  const float scale = g_scale_of(g.g_max);
  const float a = rc.y * scale, b = rc.w * scale;
  gl *= scale;
  Walk w;
  if (DIS) w.start(g, row, cls);
  if (cls >= g.cls0 + g.n) return;
#pragma unroll 1
  for (int c = 0; c < kCols; c += 32) {
    const int64_t k0 = cls + c;
    float v[32];
    __syncwarp();
    tmem_load32(tmem + half * kCols + c, v);
    tmem_load_wait(v);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float r = 0.f;
      if (LAB) r = a != 0.f ? a * ex2((v[j] - rc.x) * kLog2e) : 0.f;
      if (DIS) r += b != 0.f ? b * ex2(fmaf(v[j], g.inv_t, -rc.z) * kLog2e) : 0.f;
      v[j] = r;
    }
    if (LAB) {
      const int rel = t >= k0 && t < k0 + 32 ? static_cast<int>(t - k0) : -1;
      if (__any_sync(kFull, rel >= 0)) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == rel) v[j] -= gl;
      }
    }
    if (DIS) {
      while (__any_sync(kFull, w.next.x < k0 + 32)) {
        const int rel = w.next.x < k0 + 32 ? static_cast<int>(w.next.x - k0) : -1;
        const float q = b != 0.f ? b * __int_as_float(w.next.y) : 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == rel) v[j] -= q;
        if (rel >= 0) w.step();
      }
    }
    if (!in) continue;
    uint16_t* dst = g.g + row * g.g_ld + col0 + c;
#pragma unroll 1
    for (int p = 0; p < g.planes; ++p) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint4 x;
        x.x = pack2(v[8 * q + 0], v[8 * q + 1], g.bf16);
        x.y = pack2(v[8 * q + 2], v[8 * q + 3], g.bf16);
        x.z = pack2(v[8 * q + 4], v[8 * q + 5], g.bf16);
        x.w = pack2(v[8 * q + 6], v[8 * q + 7], g.bf16);
        reinterpret_cast<uint4*>(dst)[q] = x;
      }
      if (p + 1 < g.planes) {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] -= __bfloat162float(__float2bfloat16_rn(v[j]));
        dst += g.g_plane;
      }
    }
  }
}

// ---- results of the gradient products ---------------------------------------------------
template <int BN>
__device__ __forceinline__ void end_sum(const ProdArgs& g, uint32_t tmem, int64_t row, int n_tile, int split,
                                        int half) {
  constexpr int kCols = BN / 2;
  const int64_t col0 = int64_t(n_tile) * BN + half * kCols;
  const float inv = g.acc ? 1.f : 1.f / g_scale_of(g.g_max);
#pragma unroll 1
  for (int c = 0; c < kCols; c += 32) {
    const int64_t col = col0 + c;
    if (col >= g.n) break;
    float v[32];
    __syncwarp();
    tmem_load32(tmem + half * kCols + c, v);
    tmem_load_wait(v);
    if (row >= g.m) continue;
    const int64_t left = g.n - col;
    if (g.acc) {  // acc_ld is a multiple of 4 and covers whole chunks
      float4* dst = reinterpret_cast<float4*>(g.acc + split * g.acc_split + row * g.acc_ld + col);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float4 x = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
        if (g.acc_add) {
          const float4 o = dst[q];
          x = make_float4(x.x + o.x, x.y + o.y, x.z + o.z, x.w + o.w);
        }
        dst[q] = x;
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= inv;
    const int es = g.out_type == GM_LOSS_F32 ? 4 : 2;
    char* base = static_cast<char*>(g.out) + (row * g.out_ld + col) * es;
    if (left >= 32 && (reinterpret_cast<uintptr_t>(base) & 15) == 0) {
      if (es == 4) {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          reinterpret_cast<float4*>(base)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      } else {
        const bool bf = g.out_type == GM_LOSS_BF16;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4 x;
          x.x = pack2(v[8 * q + 0], v[8 * q + 1], bf);
          x.y = pack2(v[8 * q + 2], v[8 * q + 3], bf);
          x.z = pack2(v[8 * q + 4], v[8 * q + 5], bf);
          x.w = pack2(v[8 * q + 6], v[8 * q + 7], bf);
          reinterpret_cast<uint4*>(base)[q] = x;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (j >= left) continue;
        if (es == 4) reinterpret_cast<float*>(base)[j] = v[j];
        else if (g.out_type == GM_LOSS_BF16) reinterpret_cast<__nv_bfloat16*>(base)[j] = __float2bfloat16_rn(v[j]);
        else reinterpret_cast<__half*>(base)[j] = __float2half_rn(v[j]);
      }
    }
  }
}

template <Prod KIND, int CG, int BN, bool LAB, bool DIS>
__global__ void __launch_bounds__(kThreads, 1) k_prod(const __grid_constant__ CUtensorMap map_a,
                                                      const __grid_constant__ CUtensorMap map_b, const ProdArgs g) {
  using S = Shape<CG, BN>;
  constexpr bool kAmn = KIND == Prod::kDw;                        // G^T: rows of G run along the result's rows
  constexpr bool kBmn = KIND == Prod::kDw || KIND == Prod::kDh;   // H and W with the summed dimension outside
  extern __shared__ unsigned char smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + S::kStages * S::kStage;
  const uint32_t full = bars, empty = bars + 8 * S::kStages, tfull = empty + 8 * S::kStages, tempty = tfull + 16,
                 spare = tempty + 16;
  __shared__ int s_abort;
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  constexpr uint32_t kCols = 2 * BN;

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, kEpiWarps * CG);
    }
    mbar_init(spare, 1);
    mbar_init_fence();
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
  }
  if (warp == 1) tmem_alloc<CG>(smem_addr(&s_tmem), kCols);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem;

  const int n_tiles = g.m_tiles * g.n_tiles * g.splits;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;
  const int n_pairs = g.planes == 1 ? 1 : 6;
  volatile int* abort = &s_abort;

  if (warp == 0 && lane == 0) {
    // ---- loads
    int st = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int t = first; ok && t < n_tiles; t += stride) {
      const Tile tl = tile_at(g, t);
      const int kb0 = tl.split * g.k_per_split, kb1 = min(g.k_blocks, kb0 + g.k_per_split);
      const int m0 = tl.m * 128 * CG + static_cast<int>(rank) * 128;
      const int n0 = tl.n * BN + static_cast<int>(rank) * S::kBRows;
      for (int p = 0; ok && p < n_pairs; ++p) {
        const int pa = n_pairs == 1 ? 0 : kPlaneA[p], pb = n_pairs == 1 ? 0 : kPlaneB[p];
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(empty + 8 * st, ph ^ 1, abort)) {
            ok = false;
            break;
          }
          const uint32_t a = base + st * S::kStage, b = a + S::kABytes;
          const uint32_t bar = CG == 2 ? map_to_rank(full + 8 * st, 0) : full + 8 * st;
          if (rank == 0) mbar_expect_tx(full + 8 * st, CG * S::kStage);
          if constexpr (!kAmn) {
            tma_load_3d<CG>(a, &map_a, kb * kBK, g.a_row0 + m0, pa, bar);
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) tma_load_3d<CG>(a + i * 8192, &map_a, m0 + i * 64, g.a_row0 + kb * kBK, pa, bar);
          }
          if constexpr (!kBmn) {
            tma_load_3d<CG>(b, &map_b, kb * kBK, g.b_row0 + n0, pb, bar);
          } else {
#pragma unroll
            for (int i = 0; i < S::kBRows / 64; ++i)
              tma_load_3d<CG>(b + i * 8192, &map_b, n0 + i * 64, g.b_row0 + kb * kBK, pb, bar);
          }
          ++issued;
          if (++st == S::kStages) st = 0, ph ^= 1;
        }
      }
    }
    // A block that gave up leaves only once the loads it issued have landed (the waits
    // are bounded as well); rank 0's barriers count both blocks' loads.
    if (!ok && rank == 0) {
      int no_abort = 0;
      for (int i = 0; i < S::kStages && i < issued; ++i) {
        if (--st < 0) st = S::kStages - 1, ph ^= 1;
        mbar_wait(full + 8 * st, ph, &no_abort);
      }
    }
  } else if (warp == 1 && lane == 0 && rank == 0) {
    // ---- products
    const uint32_t idesc = instr_desc(g.bf16, kAmn, kBmn, 128 * CG, BN);
    int st = 0, buf = 0;
    uint32_t ph = 0, bph = 0;
    bool ok = true;
    for (int t = first; ok && t < n_tiles; t += stride) {
      const int split = t / (g.m_tiles * g.n_tiles);
      const int kb0 = split * g.k_per_split, kb1 = min(g.k_blocks, kb0 + g.k_per_split);
      const int steps = (kb1 - kb0) * n_pairs;
      if (!mbar_wait(tempty + 8 * buf, bph ^ 1, abort)) break;
      tc_fence_after();
      for (int i = 0; i < steps; ++i) {
        if (!mbar_wait(full + 8 * st, ph, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = base + st * S::kStage, b = a + S::kABytes;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t da = kAmn ? smem_desc(a + k * 2048, 8192, 1024) : smem_desc(a + k * 32, 16, 1024);
          const uint64_t db = kBmn ? smem_desc(b + k * 2048, 8192, 1024) : smem_desc(b + k * 32, 16, 1024);
          tc_mma_f16<CG>(tmem + buf * BN, da, db, idesc, (i | k) != 0);
        }
        tc_commit<CG>(empty + 8 * st);
        if (++st == S::kStages) st = 0, ph ^= 1;
      }
      if (!ok) break;
      tc_commit<CG>(tfull + 8 * buf);
      if (++buf == 2) buf = 0, bph ^= 1;
    }
    if (*abort) {  // the products still running read this block's shared memory
      int no_abort = 0;
      tc_commit<CG>(spare);
      mbar_wait(spare, 0, &no_abort);
    }
  } else if (warp >= kEpiWarp0) {
    // ---- results
    const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
    int buf = 0;
    uint32_t bph = 0;
    for (int t = first; t < n_tiles; t += stride) {
      const Tile tl = tile_at(g, t);
      if (!__all_sync(kFull, mbar_wait(tfull + 8 * buf, bph, abort))) break;
      tc_fence_after();
      const int64_t row = int64_t(tl.m) * 128 * CG + rank * 128 + quad * 32 + lane;
      const uint32_t acc = tmem + (static_cast<uint32_t>(quad * 32) << 16) + buf * BN;
      if constexpr (KIND == Prod::kStats) end_stats<BN, LAB, DIS>(g, acc, row, tl.n, half);
      else if constexpr (KIND == Prod::kGrad) end_grad<BN, LAB, DIS>(g, acc, row, tl.n, half);
      else end_sum<BN>(g, acc, row, tl.n, tl.split, half);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2) mbar_arrive_cluster(map_to_rank(tempty + 8 * buf, 0));
        else mbar_arrive(tempty + 8 * buf);
      }
      if (++buf == 2) buf = 0, bph ^= 1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, kCols);
  if (threadIdx.x == 0 && s_abort) atomicOr(g.status, kLossTimeout);
}

template <Prod KIND, int CG, int BN, bool LAB, bool DIS>
cudaError_t launch_one(const ProdMaps& maps, const ProdArgs& a, int num_sms, cudaStream_t s) {
  using S = Shape<CG, BN>;
  auto* k = k_prod<KIND, CG, BN, LAB, DIS>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = int64_t(a.m_tiles) * a.n_tiles * a.splits;
  const int groups = static_cast<int>(tiles < num_sms / CG ? tiles : num_sms / CG);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(groups * CG));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CG;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k, maps.a, maps.b, a);
  note_launch();
  return e;
}

template <Prod KIND, int CG, int BN>
cudaError_t launch_modes(const ProdMaps& maps, const ProdArgs& a, int num_sms, cudaStream_t s) {
  const bool lab = a.tgt.t != nullptr, dis = a.ents != nullptr || a.ent_len != nullptr;
  if (lab && dis) return launch_one<KIND, CG, BN, true, true>(maps, a, num_sms, s);
  if (dis) return launch_one<KIND, CG, BN, false, true>(maps, a, num_sms, s);
  return launch_one<KIND, CG, BN, true, false>(maps, a, num_sms, s);
}

}  // namespace

int prod_box_rows_a() { return 128; }
int prod_box_rows_b(int cg, int bn) { return bn / cg; }

cudaError_t launch_prod(Prod kind, int cg, int bn, const ProdMaps& maps, const ProdArgs& a, int num_sms,
                        cudaStream_t s) {
  switch (kind) {
    case Prod::kStats:
      return cg == 2 ? launch_modes<Prod::kStats, 2, 256>(maps, a, num_sms, s)
                     : launch_modes<Prod::kStats, 1, 256>(maps, a, num_sms, s);
    case Prod::kGrad:
      return cg == 2 ? launch_modes<Prod::kGrad, 2, 256>(maps, a, num_sms, s)
                     : launch_modes<Prod::kGrad, 1, 256>(maps, a, num_sms, s);
    case Prod::kDh:
      if (bn == 256)
        return cg == 2 ? launch_one<Prod::kDh, 2, 256, false, false>(maps, a, num_sms, s)
                       : launch_one<Prod::kDh, 1, 256, false, false>(maps, a, num_sms, s);
      return bn == 128 ? launch_one<Prod::kDh, 1, 128, false, false>(maps, a, num_sms, s)
                       : launch_one<Prod::kDh, 1, 64, false, false>(maps, a, num_sms, s);
    case Prod::kDw:
      if (bn == 256)
        return cg == 2 ? launch_one<Prod::kDw, 2, 256, false, false>(maps, a, num_sms, s)
                       : launch_one<Prod::kDw, 1, 256, false, false>(maps, a, num_sms, s);
      return bn == 128 ? launch_one<Prod::kDw, 1, 128, false, false>(maps, a, num_sms, s)
                       : launch_one<Prod::kDw, 1, 64, false, false>(maps, a, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gm
