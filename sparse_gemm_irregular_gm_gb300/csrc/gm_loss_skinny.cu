// gm_loss_skinny.cu -- the losses for one row of H, or up to 8 of fp32: reading the class table
// is the work, the tensor cores' tiles of 128 rows would be mostly empty, and fp32 operands
// would have to be laid out in three planes first.
//
// fp32 arithmetic on the table as it lies in memory, whatever its type and alignment.
// H stays in shared memory; a warp takes R classes at a time, so that one read of H serves
// R rows of W. Forward: one pass over W. Backward: one pass that forms the logits again,
// G in fp32, writes dW and sums dH, so W comes from HBM once and dW goes there once; the
// second look at a tile's classes, for dH, finds them in L2 while all SMs' tiles fit there (rows
// up to some 8 KB; past that W is read twice).
//
// Measured, kernels of a call, us, these / the products:
//                              forward        backward
//   f32   1 x 4096 x 131072    333 / 1539    1037 / 2481
//   f32   8 x 4096 x 131072    844 / 1366    1629 / 2300
//   f32   1 x 80 x 400000       37 /  164      74 /  303
//   f32   8 x 305 x 29546       25 /   37      68 /   85
//   bf16  1 x 64 x 400000       33 /   21      79 /   89
//   bf16  1 x 1024 x 32768      16 /   16      47 /   53
//   bf16  1 x 2650 x 26281      46 /   86     178 /  170
//   bf16  1 x 4096 x 131072    198 /  218     609 /  560
// fp32 operands are faster here at every size measured. 16-bit ones need no layout for the products where
// their rows lie on 16-byte boundaries: with one row they lose 58 % (dim 64) to gain 46 % forward and lie
// within 22 % backward, and they come here; with 8 rows (both calls: 428 / 274 at 8 x 2650 x 26281,
// 1783 / 708 at 8 x 4096 x 131072) they do not. 2 to 7 have not been measured. The forward pass of
// 1 x 4096 x 131072 f32 runs at 95 % of the measured copy rate; the backward pass waits at its tiles'
// barriers.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gm_device.cuh"
#include "gm_loss.h"
#include "gm_umma.cuh"

namespace gm {

namespace {

// ---- loads and stores of VEC consecutive elements ---------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float x, float* p) { *p = x; }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16* p) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float x, __half* p) { *p = __float2half_rn(x); }

template <int BYTES>
struct Raw;
template <>
struct Raw<2> { using type = uint16_t; };
template <>
struct Raw<4> { using type = uint32_t; };
template <>
struct Raw<16> { using type = uint4; };

template <class T, int VEC>
struct Piece {
  using R = typename Raw<VEC * sizeof(T)>::type;
  union {
    R raw;
    T x[VEC];
  };
  __device__ __forceinline__ Piece() {}
  __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const R*>(p)); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<R*>(p) = raw; }
  __device__ __forceinline__ void zero() { raw = R{}; }
  __device__ __forceinline__ float get(int i) const { return to_f32(x[i]); }
  __device__ __forceinline__ void set(int i, float v) { from_f32(v, &x[i]); }
};

// Classes a warp takes at a time, at most: their logits with N rows fill at most a warp's lanes.
// How many it does take (SkinnyArgs.take) is cut in the backward pass so that a block's last turn is
// as full as the others: 1 x 2650 x 26281 f32 had two turns of 103 blocks and none of 49, 517 us
// instead of 322. Without the backward pass's barriers it costs more than it saves (137 -> 164 us
// forward, 4 x 1240 x 144605 f32).
template <int N>
constexpr int kClasses = N == 8 ? 4 : 8;

// H in shared memory, fp32: [row][quarter of a piece][piece][up to 4], so that lanes with
// neighbouring pieces read neighbouring 16 bytes.
template <int VEC>
__device__ __forceinline__ int h_at(int row, int d, int pieces) {
  constexpr int kIn = VEC < 4 ? VEC : 4, kQ = VEC / kIn;
  const int p = d / VEC, e = d % VEC;
  return ((row * kQ + e / kIn) * pieces + p) * kIn + e % kIn;
}
template <int VEC>
__device__ __forceinline__ void read_h(const float* hs, int row, int piece, int pieces, float (&v)[VEC]) {
  constexpr int kIn = VEC < 4 ? VEC : 4, kQ = VEC / kIn;
#pragma unroll
  for (int q = 0; q < kQ; ++q) {
    const float* p = hs + ((row * kQ + q) * pieces + piece) * kIn;
    if constexpr (kIn == 4) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      v[4 * q] = x.x, v[4 * q + 1] = x.y, v[4 * q + 2] = x.z, v[4 * q + 3] = x.w;
    } else if constexpr (kIn == 2) {
      const float2 x = *reinterpret_cast<const float2*>(p);
      v[0] = x.x, v[1] = x.y;
    } else {
      v[0] = *p;
    }
  }
}

template <class T, int N, int VEC>
__device__ __forceinline__ void stage_h(const SkinnyArgs& a, float* hs, int pieces) {
  const T* h = static_cast<const T*>(a.h);
  for (int i = threadIdx.x; i < N * pieces * VEC; i += blockDim.x) {
    const int row = i / (pieces * VEC), d = i - row * pieces * VEC;
    hs[h_at<VEC>(row, d, pieces)] = row < a.n && d < a.dim ? to_f32(h[row * a.h_ld + d]) : 0.f;
  }
}

// A warp's way through its classes: batches of `take` (at most R), `step` apart, up to j_end. The next piece of
// each row is always under way, across the ends of rows and batches too, since a batch's end is a
// chain of shuffles and exponentials that would leave the memory idle.
template <class T, int N, int VEC, bool CUT>  // CUT: take may be less than R
struct Classes {
  static constexpr int R = kClasses<N>;
  const T* w;
  int64_t ld, j_end, step, j;  // j: batch of the piece under way
  int take, pieces, turns, turn, lane;
  Piece<T, VEC> ahead[R];
  __device__ __forceinline__ Classes(const SkinnyArgs& a, int64_t first, int64_t end, int64_t step, int pieces)
      : w(static_cast<const T*>(a.w)), ld(a.w_ld), j_end(end), step(step), j(first), take(a.take), pieces(pieces),
        turns((pieces + 31) / 32), turn(0), lane(threadIdx.x & 31) {
    fetch();
  }
  __device__ __forceinline__ void fetch() {
    const int p = turn * 32 + lane;
    const T* x = w + j * ld + int64_t(p) * VEC;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (p < pieces && (!CUT || r < take) && j + r < j_end) ahead[r].load(x + r * ld);
      else ahead[r].zero();
    }
  }
  // Logits of the batch with every row: value r * N + n, in lanes [v * 32 / (R N), (v + 1) * 32 / (R N)).
  // Sums run over D / 32 products a lane, then the lanes pairwise.
  __device__ __forceinline__ float logits(const float* hs) {
    float acc[R * N];
#pragma unroll
    for (int i = 0; i < R * N; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int t = 0; t < turns; ++t) {
      Piece<T, VEC> x[R];
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = ahead[r];
      const int p = min(t * 32 + lane, pieces - 1);
      if (++turn == turns) turn = 0, j += step;
      fetch();
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float h[VEC];
        read_h<VEC>(hs, n, p, pieces, h);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int e = 0; e < VEC; ++e) acc[r * N + n] = fmaf(x[r].get(e), h[e], acc[r * N + n]);
      }
    }
    // each step halves the values a lane holds, then the lanes that hold the same one add up
#pragma unroll
    for (int off = 16, count = R * N; off > 0; off >>= 1) {
      const bool up = lane & off;
      if (count > 1) {
        count >>= 1;
#pragma unroll
        for (int i = 0; i < R * N / 2; ++i) {
          if (i >= count) break;
          const float send = up ? acc[i] : acc[i + count], keep = up ? acc[i + count] : acc[i];
          acc[i] = keep + __shfl_xor_sync(kFull, send, off);
        }
      } else {
        acc[0] += __shfl_xor_sync(kFull, acc[0], off);
      }
    }
    return acc[0];
  }
};

// Lane n < N walks the teacher's entries of row n; classes come in rising order.
struct SkinnyWalk {
  int64_t at, end;
  int2 next;
  __device__ __forceinline__ void start(const SkinnyArgs& a, int n, int64_t cls) {
    at = end = 0;
    if (a.ent_len && n < a.n) {
      const int64_t first = a.ent_start[n];
      int64_t lo = first, hi = end = first + a.ent_len[n];
      while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (a.ents[mid].x < cls) lo = mid + 1;
        else hi = mid;
      }
      at = lo;
    }
    get(a);
  }
  __device__ __forceinline__ void get(const SkinnyArgs& a) { next = at < end ? a.ents[at] : make_int2(INT32_MAX, 0); }
};

__device__ __forceinline__ void merge(float& m, float& s1, float& st, float m2, float s12, float st2, float c_t) {
  const float mn = fmaxf(m, m2), ref = mn == -INFINITY ? 0.f : mn;
  s1 = s1 * ex2((m - ref) * kLog2e) + s12 * ex2((m2 - ref) * kLog2e);
  st = st * ex2((m - ref) * c_t) + st2 * ex2((m2 - ref) * c_t);
  m = mn;
}

constexpr int kForwardWarps = 8;

template <class T, int N, int VEC>
__global__ void __launch_bounds__(32 * kForwardWarps) k_skinny_stats(const SkinnyArgs a) {
  constexpr int R = kClasses<N>, kPer = 32 / (R * N);
  extern __shared__ __align__(16) float hs[];
  __shared__ float4 parts[kForwardWarps][N];
  const int pieces = static_cast<int>((a.dim + VEC - 1) / VEC);
  chain_wait();
  stage_h<T, N, VEC>(a, hs, pieces);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane / kPer / N, n = lane / kPer % N;
  const int64_t t = a.tgt.t && n < a.n ? check_target(a.tgt, raw_target(a.tgt, n)) : -1;
  const int64_t j_first = (int64_t(blockIdx.x) * kForwardWarps + warp) * a.per_warp;
  const int64_t j_end = min(a.n_cls, j_first + a.per_warp);
  SkinnyWalk w;
  w.start(a, lane, j_first);
  Classes<T, N, VEC, false> cls(a, j_first, j_end, R, pieces);
  float m = -INFINITY, s1 = 0.f, st = 0.f, zq = 0.f;
  for (int64_t j0 = j_first; j0 < j_end; j0 += R) {
    const float z = cls.logits(hs);
    if (j0 + r < j_end) {
      const float mn = fmaxf(m, z), ref = mn == -INFINITY ? 0.f : mn;
      s1 = s1 * ex2((m - ref) * kLog2e) + ex2((z - ref) * kLog2e);
      st = st * ex2((m - ref) * a.c_t) + ex2((z - ref) * a.c_t);
      m = mn;
      if (t == j0 + r) a.z_t[n] = z;
    }
    const int64_t stop = min(j0 + R, j_end);
    while (__any_sync(kFull, w.next.x < stop)) {
      const bool mine = w.next.x < stop;
      const float zs = __shfl_sync(kFull, z, mine ? (static_cast<int>(w.next.x - j0) * N + lane) * kPer : 0);
      if (mine) {
        const float q = __int_as_float(w.next.y);
        if (q > 0.f || q != q) zq += q * zs;
        ++w.at;
        w.get(a);
      }
    }
  }
#pragma unroll
  for (int off = N * kPer; off < 32; off <<= 1)
    merge(m, s1, st, __shfl_xor_sync(kFull, m, off), __shfl_xor_sync(kFull, s1, off), __shfl_xor_sync(kFull, st, off), a.c_t);
  const float zq_n = __shfl_sync(kFull, zq, n);
  if (r == 0 && lane % kPer == 0) parts[warp][n] = make_float4(m, s1, st, zq_n);
  __syncthreads();
  if (threadIdx.x < a.n) {
    float4 x = parts[0][threadIdx.x];
    for (int k = 1; k < kForwardWarps; ++k) {
      const float4 y = parts[k][threadIdx.x];
      merge(x.x, x.y, x.z, y.x, y.y, y.z, a.c_t);
      x.w += y.w;
    }
    a.part[int64_t(blockIdx.x) * a.n + threadIdx.x] = x;
  }
}

// ---- backward ---------------------------------------------------------------------------------
constexpr int kOwn = 8;  // columns of D a thread holds dH sums of, for every row

template <int N, int THREADS>
constexpr int kTile = THREADS / 32 * kClasses<N>;  // classes of a tile: one turn of every warp

template <class T, int N, int VEC, int THREADS>
__global__ void __launch_bounds__(THREADS) k_skinny_grads(const SkinnyArgs a) {
  constexpr int R = kClasses<N>, kPer = 32 / (R * N), kT = kTile<N, THREADS>, kGroups = kOwn / VEC;
  const int take = a.take, turn = take * (THREADS / 32);  // classes of a warp, of the block at a time
  constexpr int Q = 4;  // classes taken together when dW and dH are formed
  extern __shared__ __align__(16) float hs[];
  __shared__ __align__(16) float gs[kT][N];
  const int pieces = static_cast<int>((a.dim + VEC - 1) / VEC);
  chain_wait();
  stage_h<T, N, VEC>(a, hs, pieces);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r = lane / kPer / N, n = lane / kPer % N;
  RowCoef rc = {0.f, 0.f, 0.f, 0.f, 0.f, -1};
  if (n < a.n) {
    rc = row_coef(a.row, row_raw(a.row, n));
    if (blockIdx.x == 0 && rc.t == -2) atomicOr(a.status, kLossBadTarget);
  }
  const bool live = rc.a != 0.f || rc.b != 0.f || rc.gl != 0.f;
  const int64_t j_first = int64_t(blockIdx.x) * a.per_block, j_end = min(a.n_cls, j_first + a.per_block);
  // threads that own the same columns take the tile's classes in turn
  const int cols = min(pieces, THREADS), slices = THREADS / cols;
  const int slice = threadIdx.x / cols, col = threadIdx.x - slice * cols;
  const bool owns = slice < slices;
  float dh[kGroups][N][VEC];
#pragma unroll
  for (int k = 0; k < kGroups; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) dh[k][i][e] = 0.f;
  SkinnyWalk w;  // a warp's classes rise by tiles; entries of the classes between are passed over
  w.start(a, lane, j_first + warp * take);
  Classes<T, N, VEC, true> cls(a, j_first + warp * take, j_end, turn, pieces);
  for (int64_t j0 = j_first; j0 < j_end; j0 += turn) {
    const int64_t jw = j0 + warp * take;
    if (jw < j_end) {
      const float z = cls.logits(hs);
      float g = 0.f;
      if (r < take && jw + r < j_end && live) {
        if (a.tgt.t) g = rc.a * ex2((z - rc.lse) * kLog2e);
        if (a.ent_len) g = fmaf(rc.b, ex2(fmaf(z, a.inv_t, -rc.lse_t) * kLog2e), g);
        if (rc.t == jw + r) g -= rc.gl;
      }
      const int64_t stop = min(jw + take, j_end);
      for (;;) {
        const bool mine = w.next.x < stop;
        const unsigned any = __ballot_sync(kFull, mine);
        if (!any) break;
        // the lane that walks row i hands its entry to the lanes that hold its logit
        const int c = mine && w.next.x >= jw ? static_cast<int>(w.next.x - jw) : -1;
        const int c_n = __shfl_sync(kFull, c, n);
        const float q_n = __shfl_sync(kFull, __int_as_float(w.next.y), n);
        if (c_n == r && live) g -= rc.b * q_n;
        if (mine) {
          ++w.at;
          w.get(a);
        }
      }
      if (lane % kPer == 0 && r < take) gs[warp * take + r][n] = jw + r < j_end ? g : 0.f;
    }
    __syncthreads();
    const int tile = static_cast<int>(min(int64_t(turn), j_end - j0));
    if (owns) {
      for (int c0 = slice * Q; c0 < tile; c0 += slices * Q) {
        float g[Q][N];
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
          for (int i = 0; i < N; ++i) g[q][i] = c0 + q < tile ? gs[c0 + q][i] : 0.f;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) {
          const int p = col + k * THREADS;
          if (p >= pieces) break;
          Piece<T, VEC> x[Q];
          if (a.dh) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              if (c0 + q < tile) x[q].load(static_cast<const T*>(a.w) + (j0 + c0 + q) * a.w_ld + int64_t(p) * VEC);
              else x[q].zero();
            }
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
              for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int e = 0; e < VEC; ++e) dh[k][i][e] = fmaf(g[q][i], x[q].get(e), dh[k][i][e]);
          }
          if (a.dw) {
            float y[Q][VEC];
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
              for (int e = 0; e < VEC; ++e) y[q][e] = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) {
              float h[VEC];
              read_h<VEC>(hs, i, p, pieces, h);
#pragma unroll
              for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int e = 0; e < VEC; ++e) y[q][e] = fmaf(g[q][i], h[e], y[q][e]);
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
              if (c0 + q >= tile) break;
              Piece<T, VEC> o;
#pragma unroll
              for (int e = 0; e < VEC; ++e) o.set(e, y[q][e]);
              o.store(static_cast<T*>(a.dw) + (j0 + c0 + q) * a.dw_ld + int64_t(p) * VEC);
            }
          }
        }
      }
    }
    __syncthreads();
  }
  if (!a.dh) return;
  // the slices' sums into the first one's, in order; H is no longer needed
  for (int s = 0; s < slices; ++s) {
    __syncthreads();
    if (owns && slice == s) {
#pragma unroll
      for (int k = 0; k < kGroups; ++k) {
        const int p = col + k * THREADS;
        if (p >= pieces) break;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            float* x = hs + (i * pieces + p) * VEC + e;
            *x = s ? *x + dh[k][i][e] : dh[k][i][e];
          }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n * a.dim; i += THREADS) {
    const int row = i / static_cast<int>(a.dim), d = i - row * static_cast<int>(a.dim);
    a.acc[(int64_t(blockIdx.x) * a.n + row) * a.dim + d] = hs[row * pieces * VEC + d];
  }
}

// As many blocks as are resident at once, but none without work of its own; the workspace was
// planned for `most`. The attribute belongs to the kernel on its device, not to the call: every call sets
// the most its instance can ask for, so that threads with rows of other lengths do not take it back.
template <class K>
cudaError_t fit_grid(K* k, int threads, int rows, size_t smem, int64_t work, int most, int* blocks) {
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(rows * kSkinnyDim * 4));
  int per_sm = 0, dev = 0, sms = 0;
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, threads, smem);
  if (e == cudaSuccess) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) return cudaErrorLaunchOutOfResources;
  const int64_t n = work < int64_t(per_sm) * sms ? work : int64_t(per_sm) * sms;
  *blocks = static_cast<int>(n < most ? n : most);
  return cudaSuccess;
}

template <class T, int N, int VEC>
cudaError_t run_forward(SkinnyArgs a, int* blocks, cudaStream_t s) {
  auto* k = k_skinny_stats<T, N, VEC>;
  const size_t smem = size_t(N) * ((a.dim + VEC - 1) / VEC) * VEC * 4;
  const int64_t batch = kForwardWarps * kClasses<N>;
  const cudaError_t e = fit_grid(k, 32 * kForwardWarps, N, smem, (a.n_cls + batch - 1) / batch, *blocks, blocks);
  if (e != cudaSuccess) return e;
  const int64_t warps = int64_t(*blocks) * kForwardWarps, each = (a.n_cls + warps - 1) / warps;
  a.per_warp = (each + kClasses<N> - 1) / kClasses<N> * kClasses<N>;
  return launch_chained(k, *blocks, 32 * kForwardWarps, smem, s, 1, a);
}
template <class T, int N, int VEC, int THREADS>
cudaError_t run_backward(SkinnyArgs a, int* blocks, cudaStream_t s) {
  auto* k = k_skinny_grads<T, N, VEC, THREADS>;
  const size_t smem = size_t(N) * ((a.dim + VEC - 1) / VEC) * VEC * 4;
  constexpr int kT = kTile<N, THREADS>;
  const cudaError_t e = fit_grid(k, THREADS, N, smem, (a.n_cls + kT - 1) / kT, *blocks, blocks);
  if (e != cudaSuccess) return e;
  a.per_block = (a.n_cls + *blocks - 1) / *blocks;
  const int64_t turns = (a.per_block + kT - 1) / kT, share = turns * (THREADS / 32);
  a.take = static_cast<int>((a.per_block + share - 1) / share);
  return launch_chained(k, *blocks, THREADS, smem, s, 1, a);
}

template <class T, int N, int VEC>
cudaError_t run_vec(const SkinnyArgs& a, bool backward, int* blocks, cudaStream_t s) {
  if (!backward) return run_forward<T, N, VEC>(a, blocks, s);
  return a.dim <= 256 * kOwn ? run_backward<T, N, VEC, 256>(a, blocks, s) : run_backward<T, N, VEC, 512>(a, blocks, s);
}
template <class T>
cudaError_t run_16(const SkinnyArgs& a, bool backward, int vec, int* blocks, cudaStream_t s) {
  return vec == 8   ? run_vec<T, 1, 8>(a, backward, blocks, s)
         : vec == 2 ? run_vec<T, 1, 2>(a, backward, blocks, s)
                    : run_vec<T, 1, 1>(a, backward, blocks, s);
}
template <int N>
cudaError_t run_32(const SkinnyArgs& a, bool backward, int vec, int* blocks, cudaStream_t s) {
  return vec == 4 ? run_vec<float, N, 4>(a, backward, blocks, s) : run_vec<float, N, 1>(a, backward, blocks, s);
}

}  // namespace

int skinny_most_blocks(int64_t n_cls, int sms) {
  const int64_t least = (n_cls + 31) / 32;  // a block takes 32 classes at least
  return static_cast<int>(least < 8 * sms ? least : 8 * sms);
}

int skinny_rows(int type) { return type == GM_LOSS_F32 ? 8 : 1; }

cudaError_t launch_skinny(const SkinnyArgs& a, int type, bool backward, int vec, int* blocks, cudaStream_t s) {
  if (type == GM_LOSS_BF16) return run_16<__nv_bfloat16>(a, backward, vec, blocks, s);
  if (type == GM_LOSS_F16) return run_16<__half>(a, backward, vec, blocks, s);
  return a.n <= 1   ? run_32<1>(a, backward, vec, blocks, s)
         : a.n <= 4 ? run_32<4>(a, backward, vec, blocks, s)
                    : run_32<8>(a, backward, vec, blocks, s);
}

}  // namespace gm
