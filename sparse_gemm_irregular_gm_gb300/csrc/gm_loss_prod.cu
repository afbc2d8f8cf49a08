// gm_loss_prod.cu -- the matrix products of the losses over a class table, each
// with its own end: Z = H W^T reduced to row statistics, Z again turned into
// G = dloss/dZ, dH = G W and dW = G^T H.
//
// One persistent kernel: blocks (or pairs of blocks) walk the tiles of the result.
// Warp 0 loads operand tiles with TMA into a ring of 64-deep stages, one lane of warp
// 1 issues tcgen05 products into one of two TMEM accumulators, and warps from 4 on read
// the other accumulator, 8 a tile: a thread holds one row, 32 columns at a time, so the row
// reductions need no shuffles. Results of 16 or 32 bits go through shared memory and
// out by TMA, 128 bytes a row at a time.
//
// Why tiles of 256 by 256 over two blocks: a stage then brings 32 KB to an SM for 512 cycles of
// products, the 64 bytes a cycle that L2 gives an SM; a 128 by 256 tile a block would need 96.
// Measured, bf16, 2048 x 1024 x 65536 (2.75e11 operations each): statistics 136 us, the tensor
// cores 95 % busy while tiles run; G 146; dH 154 (64 of 76 pairs have a tile); dW 151. Back to back
// (8192 x 4096 x 131072) the power cap bounds them: 1.71 PFLOP/s. With dim 256 or less the
// bytes of G bound the gradients: dH of 512 x 256 x 262144 66 us, 78 % of the DRAM rate.
#include "gm_device.cuh"
#include "gm_loss.h"
#include "gm_umma.cuh"

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gm {

namespace {

constexpr int kEpiWarp0 = 4, kEpiWarps = 8;  // first warp that reads results, warps that read one tile
// Registers a thread where sums are held in registers (kParts, kSplit): the warps that load
// and issue give theirs up to those that read results. 128 * 56 + 256 * 224 = 384 * 168, what a
// block is launched with; launch_one checks that it is.
constexpr int kLaunchRegs = 168, kIssueRegs = 56, kResultRegs = 224;
static_assert(128 * kIssueRegs + 256 * kResultRegs <= 384 * kLaunchRegs, "more registers than the launch brings");
constexpr int kBK = 64;  // summed elements a stage: one 128-byte swizzled row

// How a tile's sum is kept.
//   kWhole: in TMEM from the first stage to the last. The tensor cores cut each sum to
//     24 bits instead of rounding it, so the error grows with the number of stages: 3.3e-7
//     of a row's log-sum at dim 1024, 1.6e-6 at 4096 (the fp32 form: 4e-8).
//   kParts: in TMEM over `chunk` stages, the parts added in registers, rounded: for logits of
//     long rows, whose error goes into the losses as it is.
//   kSplit: fp32 operands as three bf16 planes a stage, six products of planes a stage, in TMEM
//     over one stage, the stages added in registers.
//   kSplitWhole: the same, but in TMEM to the end: logits of at most two stages.
//   kTwo: 16-bit operands, but G in two planes: gradients of few rows (see g_planes).
enum { kWhole = 0, kParts = 1, kSplit = 2, kSplitWhole = 3, kTwo = 4 };
constexpr int kWholeBlocks = 2;
template <int ACC>
constexpr bool three_planes = ACC == kSplit || ACC == kSplitWhole;
template <int ACC>
constexpr int kPlanesA = three_planes<ACC> ? 3 : ACC == kTwo ? 2 : 1;
template <int ACC>
constexpr int kPlanesB = three_planes<ACC> ? 3 : 1;
template <int ACC>
constexpr int kPairs = three_planes<ACC> ? 6 : kPlanesA<ACC>;  // products of planes a stage
template <int ACC>
constexpr bool in_registers = ACC == kParts || ACC == kSplit;

// Products of planes of split operands (x = x0 + x1 + x2 by falling size), the small ones
// first, so that they meet a small accumulator; x1 y2, x2 y1 and x2 y2 lie under 2^-24
// of x y and are left out.
template <int ACC>
__device__ __forceinline__ constexpr int pair_a(int p) {
  return ACC == kTwo ? 1 - p : !three_planes<ACC> ? 0 : p == 0 ? 2 : p == 1 ? 0 : p == 2 ? 1 : p == 3 ? 1 : 0;
}
template <int ACC>
__device__ __forceinline__ constexpr int pair_b(int p) {
  return !three_planes<ACC> ? 0 : p == 0 ? 0 : p == 1 ? 2 : p == 2 ? 1 : p == 3 ? 0 : p == 4 ? 1 : 0;
}

// Groups of 8 warps that read results. What is done with a logit (an exponential, a maximum,
// a sum) is a chain of latencies that 2 warps a scheduler do not cover: with one group the
// statistics of 512 x 256 x 1048576 took 332 us, the tensor cores 37 % busy. Two groups take
// the tiles in turn, one accumulator each. Sums held in registers leave room for one group;
// the gradients' results are only moved.
template <Prod KIND, int ACC>
constexpr int kGroups = !in_registers<ACC> && (KIND == Prod::kStats || KIND == Prod::kGrad) ? 2 : 1;

template <Prod KIND, int CG, int BN, int ACC>
struct Shape {
  static constexpr int kThreads = 128 + 256 * kGroups<KIND, ACC>;
  static constexpr int kABytes = 128 * 128;            // a plane of this block's 128 rows of A
  static constexpr int kBRows = BN / CG;               // its rows (columns) of B
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStage = kPlanesA<ACC> * kABytes + kPlanesB<ACC> * kBBytes;
  static constexpr int kMost = 196608 / kStage;        // 32 KB of the block's 227 hold results on their way out
  static constexpr int kStages = kMost > 8 ? 8 : kMost;
  static constexpr int kBox = 4096 / kGroups<KIND, ACC>;  // a warp's results on their way out
  static constexpr int kOut = 32768;
  static constexpr size_t kSmem = 1024 + size_t(kStages) * kStage + kOut + 512;
  static_assert(kStages >= 2, "two stages at least");
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

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  } else {
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&r);
  }
}

// Rounds pairs of values to 16 bits; REST: leaves in v what the rounding took.
template <bool BF16, bool REST>
__device__ __forceinline__ void round16(float (&v)[32], uint32_t (&x)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    x[j] = pack2<BF16>(v[2 * j], v[2 * j + 1]);
    if constexpr (REST) {
      float a, b;
      if constexpr (BF16) {
        a = __uint_as_float(x[j] << 16), b = __uint_as_float(x[j] & 0xffff0000u);
      } else {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
        a = y.x, b = y.y;
      }
      v[2 * j] -= a, v[2 * j + 1] -= b;
    }
  }
}

// Teacher entries of a row, in step with the columns; one entry read ahead.
struct Walk {
  const int2* e;
  int64_t at, end;
  int2 next, after;
  __device__ __forceinline__ int2 get(int64_t i) const { return i < end ? e[i] : make_int2(INT32_MAX, 0); }
  __device__ __forceinline__ void start(const ProdArgs& g, int64_t row, int64_t cls) {
    e = g.ents;
    at = end = 0;
    if (row < g.m) {
      const int64_t lo = g.ent_start[row];
      end = lo + g.ent_len[row];
      at = first_entry(e, lo, end, cls);
    }
    next = get(at);
    after = get(at + 1);
  }
  __device__ __forceinline__ void step() {
    ++at;
    next = after;
    after = get(at + 1);
  }
};

// What a thread looks up of its row: read a tile ahead, used before the tile's sums are there.
// COEF: the row's weights, for its G or for the scale of it.
template <Prod KIND, bool LAB, bool DIS, bool COEF>
struct RowState {
  Walk w;
  RowCoef c;
  static __device__ __forceinline__ RowRaw read(const ProdArgs& g, int64_t row) {
    RowRaw x = {};
    if (row < g.m) {
      if constexpr (KIND == Prod::kStats && LAB) x.t = raw_target(g.tgt, row);
      if constexpr (COEF) x = (KIND == Prod::kGrad || g.weights) ? row_raw(g.row, row) : x;
    }
    return x;
  }
  __device__ __forceinline__ void start(const ProdArgs& g, const RowRaw& x, int64_t row, int64_t cls, bool first) {
    c = RowCoef{0.f, 0.f, 0.f, 0.f, 0.f, -1};
    if (row < g.m) {
      if constexpr (KIND == Prod::kStats && LAB) c.t = check_target(g.tgt, x.t);
      if constexpr (COEF) {
        if (KIND == Prod::kGrad || g.weights) c = row_coef(g.row, x);
        if (LAB && first && c.t == -2) atomicOr(g.status, kLossBadTarget);
      }
    }
    if constexpr (DIS) w.start(g, row, cls);
  }
};

// The sums of a thread's row, 32 columns at a time: from TMEM (AHEAD: the next 32 under way
// while these are used), or from registers.
// DONE is called once the last columns are read: the accumulator is free again.
template <int COLS, bool AHEAD, class DONE>
struct FromTmem {
  uint32_t at;
  DONE& done;
  float ahead[AHEAD ? 32 : 1];
  __device__ __forceinline__ FromTmem(uint32_t addr, DONE& d) : at(addr), done(d) {
    if constexpr (AHEAD) tmem_load32(at, ahead);
  }
  template <int C>
  __device__ __forceinline__ void get(float (&v)[32]) {
    if constexpr (AHEAD) {
      tmem_load_wait(ahead);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = ahead[j];
      if constexpr (C + 32 < COLS) {
        __syncwarp();
        tmem_load32(at + C + 32, ahead);
      }
    } else {
      __syncwarp();
      tmem_load32(at + C, v);
      tmem_load_wait(v);
    }
    if constexpr (C + 32 >= COLS) done();
  }
};
template <int COLS>
struct Held {
  float acc[COLS];
  template <int C>
  __device__ __forceinline__ void get(float (&v)[32]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] = acc[C + j];
  }
};

template <class Src>
constexpr bool kHeld = false;
template <int COLS>
constexpr bool kHeld<Held<COLS>> = true;

// Calls f with 0, 32, 64, ... below COLS as compile-time constants.
template <int COLS, int C = 0, class F>
__device__ __forceinline__ void each_32(F&& f) {
  if constexpr (C < COLS) {
    f(std::integral_constant<int, C>{});
    each_32<COLS, C + 32>(f);
  }
}

// ---- row statistics of half a tile -------------------------------------------------
template <int BN, bool LAB, bool DIS, class Src>
__device__ __forceinline__ void end_stats(const ProdArgs& g, Src& src, RowState<Prod::kStats, LAB, DIS, false>& rs, int64_t row,
                                          int n_tile, int half) {
  constexpr int kCols = BN / 2;
  const int64_t cls = g.cls0 + int64_t(n_tile) * BN + half * kCols;  // class of the first column
  const int64_t end = g.cls0 + g.n;
  float m = -INFINITY, s1 = 0.f, st = 0.f, zq = 0.f;
  const int64_t t = rs.c.t;
  each_32<kCols>([&](auto cc) {
    constexpr int c = decltype(cc)::value;
    const int64_t k0 = cls + c;
    float v[32];
    src.template get<c>(v);
    if (k0 >= end) return;
    if (k0 + 32 > end) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (k0 + j >= end) v[j] = -INFINITY;
    }
    float m0 = fmaxf(v[0], v[1]), m1 = fmaxf(v[2], v[3]);
#pragma unroll
    for (int j = 4; j < 32; j += 4) {
      m0 = fmaxf(m0, fmaxf(v[j], v[j + 1]));
      m1 = fmaxf(m1, fmaxf(v[j + 2], v[j + 3]));
    }
    const float mn = fmaxf(m, fmaxf(m0, m1));
    const float ref = mn == -INFINITY ? 0.f : mn;
    if (LAB) {
      float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 32; ++j) a[j & 3] += ex2(fmaf(v[j], kLog2e, -ref * kLog2e));
      s1 = s1 * ex2((m - ref) * kLog2e) + ((a[0] + a[1]) + (a[2] + a[3]));
    }
    if (DIS) {
      float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < 32; ++j) a[j & 3] += ex2(fmaf(v[j], g.c_t, -ref * g.c_t));
      st = st * ex2((m - ref) * g.c_t) + ((a[0] + a[1]) + (a[2] + a[3]));
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
      Walk& w = rs.w;
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
  });
  if (row < g.m) g.part[(int64_t(n_tile) * 2 + half) * g.part_ld + row] = make_float4(m, s1, st, zq);
}

// ---- results on their way out ------------------------------------------------------------
// A warp's 32 rows of 128 bytes (64: NARROW) in shared memory, 16-byte pieces swizzled as the
// TMA store expects them, so that neither side meets a bank twice.
template <bool NARROW>
struct Outbox {
  uint32_t buf;
  int lane;
  __device__ __forceinline__ void open() {  // the last store has read the buffer
    if (lane == 0) tma_wait_read();
    __syncwarp();
  }
  __device__ __forceinline__ void put(int piece, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    if constexpr (NARROW) st_shared_v4(buf + lane * 64 + ((piece ^ ((lane >> 1) & 3)) << 4), a, b, c, d);
    else st_shared_v4(buf + lane * 128 + ((piece ^ (lane & 7)) << 4), a, b, c, d);
  }
  // 32 columns of 16 bits; the values become what rounding took of them with rest.
  __device__ __forceinline__ void put16(int piece0, float (&v)[32], bool bf16, bool rest, uint32_t keep) {
    uint32_t x[16];
    if (bf16) {
      if (rest) round16<true, true>(v, x);
      else round16<true, false>(v, x);
    } else {
      if (rest) round16<false, true>(v, x);
      else round16<false, false>(v, x);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) put(piece0 + q, keep & x[4 * q], keep & x[4 * q + 1], keep & x[4 * q + 2], keep & x[4 * q + 3]);
  }
  // 32 columns in f16 at another scale: their values, or what rounding takes of them.
  __device__ __forceinline__ void put_half(int piece0, const float (&v)[32], float scale, bool rest, uint32_t keep) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[8 * q + 2 * j] * scale, b = v[8 * q + 2 * j + 1] * scale;
        x[j] = pack2<false>(a, b);
        if (rest) {
          const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
          x[j] = pack2<false>(a - y.x, b - y.y);
        }
        x[j] &= keep;
      }
      put(piece0 + q, x[0], x[1], x[2], x[3]);
    }
  }
  __device__ __forceinline__ void put32(const float (&v)[32]) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      put(q, __float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
          __float_as_uint(v[4 * q + 3]));
  }
  __device__ __forceinline__ void send(const CUtensorMap* m, int x, int y, int z, bool add) {
    async_proxy_fence();
    __syncwarp();
    if (lane == 0) {
      if (add) tma_add_3d(m, buf, x, y, z);
      else tma_store_3d(m, buf, x, y, z);
      tma_commit();
    }
  }
  // The same by plain stores, for rows that do not start on 16-byte boundaries: the warp
  // writes a row's columns together.
  __device__ __forceinline__ void copy(void* out, int64_t ld, int es, int64_t row0, int64_t rows, int64_t col0,
                                       int64_t cols) {
    __syncwarp();
    const int n = static_cast<int>(min(int64_t(32), rows - row0));
    const bool in0 = es == 4 ? lane < cols : 2 * lane < cols, in1 = 2 * lane + 1 < cols;
    char* p = static_cast<char*>(out) + (row0 * ld + col0) * es + lane * 4;
    const int64_t step = ld * es;
#pragma unroll 1
    for (int r0 = 0; r0 < n; r0 += 16) {
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        x[i] = ld_shared_u32(buf + (r0 + i) * 128 + (((lane >> 2) ^ (i & 7)) << 4) + (lane & 3) * 4);
#pragma unroll
      for (int i = 0; i < 16; ++i, p += step) {
        const bool row = r0 + i < n;
        if (es == 4) {
          if (row && in0) *reinterpret_cast<uint32_t*>(p) = x[i];
        } else {
          if (row && in0) reinterpret_cast<uint16_t*>(p)[0] = static_cast<uint16_t>(x[i]);
          if (row && in1) reinterpret_cast<uint16_t*>(p)[1] = static_cast<uint16_t>(x[i] >> 16);
        }
      }
    }
    __syncwarp();
  }
};

// ---- gradient of the logits ----------------------------------------------------------
// G_ij = a_i e^(z - lse) - gl_i [j = t_i] + b_i (e^(z / T - lse_T) - q_ij), rounded to 16 bits as
// the operand of the two products after it (in f16 times a power of two, see Scales); fp32 operands keep it in
// three bf16 planes, 24 bits. In 16 bits the factors go into the exponent.
template <bool LAB, bool DIS, bool FINE>
struct GradRow {
  float a, b, gl, x1, xt, s1, st;
  bool live;
  __device__ __forceinline__ GradRow(const RowCoef& c, float scale) {
    a = c.a * scale, b = c.b * scale, gl = c.gl * scale;
    live = a != 0.f || b != 0.f || gl != 0.f;
    if (FINE) {
      x1 = c.lse, xt = c.lse_t;
    } else {  // 0 as a factor: 2^-inf
      x1 = __log2f(fabsf(a)) - c.lse * kLog2e, xt = __log2f(fabsf(b)) - c.lse_t * kLog2e;
      s1 = copysignf(1.f, a), st = copysignf(1.f, b);
    }
  }
  __device__ __forceinline__ void of(float (&v)[32], const ProdArgs& g, int64_t t, int64_t k0, Walk& w) const {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      float r = 0.f;
      if (FINE) {
        if (LAB) r = a * ex2((v[j] - x1) * kLog2e);
        if (DIS) r = fmaf(b, ex2(fmaf(v[j], g.inv_t, -xt) * kLog2e), r);
      } else {
        if (LAB) r = s1 * ex2(fmaf(v[j], kLog2e, x1));
        if (DIS) r = fmaf(st, ex2(fmaf(v[j], g.c_t, xt)), r);
      }
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
        const float q = b * __int_as_float(w.next.y);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (j == rel) v[j] -= q;
        if (rel >= 0) w.step();
      }
    }
  }
};

template <int BN, bool LAB, bool DIS, int ACC, class Src>
__device__ __forceinline__ void end_grad(const ProdArgs& g, const CUtensorMap* map_o, Src& src,
                                         RowState<Prod::kGrad, LAB, DIS, true>& rs, int64_t row, int n_tile, int half,
                                         Outbox<!kHeld<Src>> box) {
  constexpr int kCols = BN / 2;
  constexpr bool FINE = ACC != kWhole, kHalf = !three_planes<ACC>;  // kHalf: may be f16
  const int64_t col0 = int64_t(n_tile) * BN + half * kCols;
  const int64_t cls = g.cls0 + col0;
  const int64_t row0 = row - box.lane;
  float own = 1.f, to_all = NAN;  // the row's scale; from it to the one of all rows, NaN where that is the same for all
  if constexpr (kHalf) {
    const Scales scales(g);
    own = scales.of(rs.c);
    if (scales.apart) to_all = scales.all / own;
  }
  const GradRow<LAB, DIS, FINE> gr(rs.c, own);
  const uint32_t keep = gr.live ? 0xffffffffu : 0u;  // a row without weight is 0 whatever its logits are
  const int first = kHalf && to_all == to_all ? -g.g_planes : 0;  // planes under 0: those of the scale of all rows
  if constexpr (!kHeld<Src>) {
    each_32<kCols>([&](auto cc) {
      constexpr int c = decltype(cc)::value;
      float v[32];
      src.template get<c>(v);
      gr.of(v, g, rs.c.t, cls + c, rs.w);
#pragma unroll 1
      for (int p = first; p < g.g_planes; ++p) {
        box.open();
        if (kHalf && p < 0) box.put_half(0, v, to_all, p != first, keep);
        else box.put16(0, v, FINE || g.bf16, p + 1 < g.g_planes, keep);
        if (row0 < g.m && col0 + c < g.n)
          box.send(map_o, static_cast<int>(col0 + c), static_cast<int>(row0), p < 0 ? p - 2 * first : p, false);
      }
    });
  } else {
    each_32<kCols>([&](auto cc) {
      constexpr int c = decltype(cc)::value;
      float v[32];
      src.template get<c>(v);
      gr.of(v, g, rs.c.t, cls + c, rs.w);
#pragma unroll
      for (int j = 0; j < 32; ++j) src.acc[c + j] = v[j];
    });
#pragma unroll 1
    for (int p = first; p < g.g_planes; ++p) {
      const int plane = p < 0 ? p - 2 * first : p;
      each_32<kCols>([&](auto cc) {
        constexpr int c = decltype(cc)::value;
        float v[32];
        src.template get<c>(v);
        if constexpr (c % 64 == 0) box.open();
        if (kHalf && p < 0) box.put_half(c % 64 == 0 ? 0 : 4, v, to_all, p != first, keep);
        else box.put16(c % 64 == 0 ? 0 : 4, v, g.bf16, p + 1 < g.g_planes, keep);
        if constexpr (c % 64 == 32) {
          if (row0 < g.m && col0 + c - 32 < g.n)
            box.send(map_o, static_cast<int>(col0 + c - 32), static_cast<int>(row0), plane, false);
        }
        if (p >= 0 && p + 1 < g.g_planes) {
#pragma unroll
          for (int j = 0; j < 32; ++j) src.acc[c + j] = v[j];
        }
      });
    }
  }
}

// ---- results of the gradient products ---------------------------------------------------
template <int BN, class Src>
__device__ __forceinline__ void end_sum(const ProdArgs& g, const CUtensorMap* map_o, Src& src, int64_t row, int n_tile,
                                        int split, int half, float inv, Outbox<false> box) {
  constexpr int kCols = BN / 2;
  const int64_t col0 = int64_t(n_tile) * BN + half * kCols;
  const int64_t row0 = row - box.lane;
  const bool sums = g.acc;
  const bool wide = sums || g.out_type == GM_LOSS_F32;
  const bool bf = g.out_type == GM_LOSS_BF16;
  each_32<kCols>([&](auto cc) {
    constexpr int c = decltype(cc)::value;
    float v[32];
    src.template get<c>(v);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= inv;
    // 32 columns of 4 bytes or 64 of 2 fill the box; half a tile of 32 columns sends what it has
    constexpr bool kPair = kCols >= 64;
    constexpr int first = kPair ? c / 64 * 64 : c;
    const int64_t col = col0 + (wide ? c : first);
    if (wide) {
      box.open();
      box.put32(v);
    } else {
      if (c == first) box.open();
      box.put16(c == first ? 0 : 4, v, bf, false, 0xffffffffu);
      if (kPair && c % 64 == 0) return;
    }
    if (row0 >= g.m || col >= g.n) return;
    if (g.by_tma) {
      box.send(map_o, static_cast<int>(col), static_cast<int>(row0), split, g.acc_add);
    } else {
      const int64_t most = wide || !kPair ? 32 : 64;
      box.copy(g.out, g.out_ld, wide ? 4 : 2, row0, g.m, col, min(most, g.n - col));
    }
  });
}

template <Prod KIND, int CG, int BN, bool LAB, bool DIS, int ACC>
__global__ void __launch_bounds__((Shape<KIND, CG, BN, ACC>::kThreads), 1) k_prod(const __grid_constant__ CUtensorMap map_a,
                                                      const __grid_constant__ CUtensorMap map_b,
                                                      const __grid_constant__ CUtensorMap map_o, const ProdArgs g) {
  using S = Shape<KIND, CG, BN, ACC>;
  constexpr bool kAmn = KIND == Prod::kDw;                        // G^T: rows of G run along the result's rows
  constexpr bool kBmn = KIND == Prod::kDw || KIND == Prod::kDh;   // H and W with the summed dimension outside
  extern __shared__ unsigned char smem_raw[];
  const uint32_t base = (smem_addr(smem_raw) + 1023u) & ~1023u;
  const uint32_t out = base + S::kStages * S::kStage;
  const uint32_t bars = out + S::kOut;
  const uint32_t full = bars, empty = bars + 8 * S::kStages, tfull = empty + 8 * S::kStages, tempty = tfull + 16,
                 spare = tempty + 16;
  __shared__ int s_abort;
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;
  constexpr uint32_t kTmemCols = 2 * BN;

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
  if (warp == 1) tmem_alloc<CG>(smem_addr(&s_tmem), kTmemCols);
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  chain_wait();

  const int n_tiles = g.m_tiles * g.n_tiles * g.splits;
  const int first = blockIdx.x / CG, stride = gridDim.x / CG;
  const int chunk = !in_registers<ACC> ? (1 << 30) : ACC == kSplit ? 1 : g.chunk;  // stages an accumulator takes
  volatile int* abort = &s_abort;

  if (warp < kEpiWarp0) {
    if constexpr (in_registers<ACC>) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == 0) {
      // ---- loads
      const bool one = elect_one();
      int a_plane = 0;  // dW's planes of G
      if constexpr (KIND == Prod::kDw && !three_planes<ACC>) a_plane = Scales(g).apart ? g.g_planes : 0;
      int st = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; ok && t < n_tiles; t += stride) {
        const Tile tl = tile_at(g, t);
        const int kb0 = tl.split * g.k_per_split, kb1 = min(g.k_blocks, kb0 + g.k_per_split);
        const int m0 = tl.m * 128 * CG + static_cast<int>(rank) * 128;
        const int n0 = tl.n * BN + static_cast<int>(rank) * S::kBRows;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!__all_sync(kFull, mbar_wait(empty + 8 * st, ph ^ 1, abort))) {
            ok = false;
            break;
          }
          if (one) {
            const uint32_t bar = CG == 2 ? map_to_rank(full + 8 * st, 0) : full + 8 * st;
            if (rank == 0) mbar_expect_tx(full + 8 * st, CG * S::kStage);
#pragma unroll
            for (int p = 0; p < kPlanesA<ACC>; ++p) {
              const uint32_t a = base + st * S::kStage + p * S::kABytes;
              if constexpr (!kAmn) {
                tma_load_3d<CG>(a, &map_a, kb * kBK, m0, p, bar);
              } else {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  tma_load_3d<CG>(a + i * 8192, &map_a, m0 + i * 64, kb * kBK, a_plane + p, bar);
              }
            }
#pragma unroll
            for (int p = 0; p < kPlanesB<ACC>; ++p) {
              const uint32_t b = base + st * S::kStage + kPlanesA<ACC> * S::kABytes + p * S::kBBytes;
              if constexpr (!kBmn) {
                tma_load_3d<CG>(b, &map_b, kb * kBK, g.b_row0 + n0, p, bar);
              } else {
#pragma unroll
                for (int i = 0; i < S::kBRows / 64; ++i)
                  tma_load_3d<CG>(b + i * 8192, &map_b, n0 + i * 64, g.b_row0 + kb * kBK, p, bar);
              }
            }
          }
          __syncwarp();
          ++issued;
          if (++st == S::kStages) st = 0, ph ^= 1;
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
    } else if (warp == 1 && rank == 0) {
      // ---- products. The tensor cores wait for this loop when it is slow: the tile's
      // buffer is waited for outside it, and a stage's operands are a constant away from
      // the first one's descriptors.
      const bool one = elect_one();
      const uint32_t idesc = instr_desc(g.bf16, kAmn, kBmn, 128 * CG, BN);
      const uint32_t b0 = base + kPlanesA<ACC> * S::kABytes;
      const uint64_t desc_a = kAmn ? smem_desc(base, 8192, 1024) : smem_desc(base, 16, 1024);
      const uint64_t desc_b = kBmn ? smem_desc(b0, 8192, 1024) : smem_desc(b0, 16, 1024);
      constexpr int kStepA = (kAmn ? 2048 : 32) >> 4, kStepB = (kBmn ? 2048 : 32) >> 4;  // 16 summed elements further
      int st = 0, buf = 0;
      uint32_t ph = 0, bph = 0;
      bool ok = true;
      for (int t = first; ok && t < n_tiles; t += stride) {
        const int split = t / (g.m_tiles * g.n_tiles);
        const int kb0 = split * g.k_per_split, steps = min(g.k_blocks, kb0 + g.k_per_split) - kb0;
        for (int i0 = 0; ok && i0 < steps; i0 += chunk) {
          if (!__all_sync(kFull, mbar_wait(tempty + 8 * buf, bph ^ 1, abort))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int n = min(chunk, steps - i0);
          const uint32_t d = tmem + buf * BN;
          for (int i = 0; i < n; ++i) {
            if (!__all_sync(kFull, mbar_wait(full + 8 * st, ph, abort))) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (one) {
#pragma unroll
              for (int p = 0; p < kPairs<ACC>; ++p) {
                const int pa = pair_a<ACC>(p), pb = pair_b<ACC>(p);
                const uint64_t da = desc_a + ((st * S::kStage + pa * S::kABytes) >> 4);
                const uint64_t db = desc_b + ((st * S::kStage + pb * S::kBBytes) >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  tc_mma_f16<CG>(d, da + k * kStepA, db + k * kStepB, idesc, (i | p | k) != 0);
              }
              tc_commit<CG>(empty + 8 * st);
            }
            __syncwarp();
            if (++st == S::kStages) st = 0, ph ^= 1;
          }
          if (!ok) break;
          if (one) tc_commit<CG>(tfull + 8 * buf);
          __syncwarp();
          if (++buf == 2) buf = 0, bph ^= 1;
        }
      }
      if (*abort) {  // the products still running read this block's shared memory
        int no_abort = 0;
        if (one) tc_commit<CG>(spare);
        __syncwarp();
        mbar_wait(spare, 0, &no_abort);
      }
    }
  } else {
    if constexpr (in_registers<ACC>) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kResultRegs));
    // ---- results
    constexpr int kCols = BN / 2;
    constexpr int kTurns = kGroups<KIND, ACC>;
    const int quad = warp & 3, half = ((warp - kEpiWarp0) >> 2) & 1;
    const int turn = kTurns == 2 ? (warp - kEpiWarp0) >> 3 : 0;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    Outbox<kTurns == 2 && KIND == Prod::kGrad> box{out + (warp - kEpiWarp0) * S::kBox, lane};
    int buf = turn;
    uint32_t bph = 0;
    auto ready = [&] {
      const bool ok = __all_sync(kFull, mbar_wait(tfull + 8 * buf, bph, abort));
      tc_fence_after();
      return ok;
    };
    auto done = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 2) mbar_arrive_cluster(map_to_rank(tempty + 8 * buf, 0));
        else mbar_arrive(tempty + 8 * buf);
      }
      if (kTurns == 2) bph ^= 1;  // a group keeps to one accumulator
      else if (++buf == 2) buf = 0, bph ^= 1;
    };
    using Row = RowState<KIND, LAB, DIS, KIND == Prod::kGrad || (KIND == Prod::kDh && !three_planes<ACC>)>;
    auto row_of = [&](const Tile& x) { return int64_t(x.m) * 128 * CG + rank * 128 + quad * 32 + lane; };
    Tile tl = {0, 0, 0};
    RowRaw raw = {};
    if (first + turn * stride < n_tiles) {
      tl = tile_at(g, first + turn * stride);
      raw = Row::read(g, row_of(tl));
    }
    Tile next = tl;
    for (int t = first + turn * stride; t < n_tiles; t += kTurns * stride, tl = next) {
      const int64_t row = row_of(tl);
      Row rs;
      rs.start(g, raw, row, g.cls0 + int64_t(tl.n) * BN + half * kCols, tl.n == 0 && half == 0);
      if (t + kTurns * stride < n_tiles) {
        next = tile_at(g, t + kTurns * stride);
        raw = Row::read(g, row_of(next));
      }
      auto finish = [&](auto& src) {
        if constexpr (KIND == Prod::kStats) end_stats<BN, LAB, DIS>(g, src, rs, row, tl.n, half);
        else if constexpr (KIND == Prod::kGrad) end_grad<BN, LAB, DIS, ACC>(g, &map_o, src, rs, row, tl.n, half, box);
        else {
          float inv = 1.f;  // of the scale of G
          if constexpr (!three_planes<ACC>) inv = 1.f / (KIND == Prod::kDh ? Scales(g).of(rs.c) : Scales(g).all);
          end_sum<BN>(g, &map_o, src, row, tl.n, tl.split, half, inv, box);
        }
      };
      if constexpr (!in_registers<ACC>) {
        if (!ready()) break;
        FromTmem<kCols, kTurns == 1, decltype(done)> src(tmem + lanes + buf * BN + half * kCols, done);
        finish(src);
      } else {
        const int kb0 = tl.split * g.k_per_split, steps = min(g.k_blocks, kb0 + g.k_per_split) - kb0;
        Held<kCols> src;
#pragma unroll
        for (int j = 0; j < kCols; ++j) src.acc[j] = 0.f;
        bool ok = true;
#pragma unroll 1
        for (int i = 0; i < steps; i += chunk) {
          if (!ready()) {
            ok = false;
            break;
          }
          each_32<kCols>([&](auto cc) {
            constexpr int c = decltype(cc)::value;
            float v[32];
            __syncwarp();
            tmem_load32(tmem + lanes + buf * BN + half * kCols + c, v);
            tmem_load_wait(v);
#pragma unroll
            for (int j = 0; j < 32; ++j) src.acc[c + j] += v[j];
          });
          done();
        }
        if (!ok) break;
        finish(src);
      }
    }
    if (lane == 0) tma_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_free<CG>(tmem, kTmemCols);
  // The report may be read and cleared at any time, by other calls too; what later kernels of this
  // call go by stays in its workspace.
  if (threadIdx.x == 0) {
    const int gave_up = s_abort;
    if (gave_up) atomicOr(g.status, kLossTimeout);
    if (g.lost_first)
      for (int i = blockIdx.x; i < kMostBlocks; i += gridDim.x) g.lost[i] = i == static_cast<int>(blockIdx.x) && gave_up;
    else if (gave_up) g.lost[blockIdx.x] = 1;
  }
}

template <Prod KIND, int CG, int BN, bool LAB, bool DIS, int ACC>
cudaError_t launch_one(const ProdMaps& maps, const ProdArgs& a, int num_sms, cudaStream_t s) {
  using S = Shape<KIND, CG, BN, ACC>;
  auto* k = k_prod<KIND, CG, BN, LAB, DIS, ACC>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (e != cudaSuccess) return e;
  if (in_registers<ACC>) {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, k);
    if (e != cudaSuccess) return e;
    if (at.numRegs != kLaunchRegs) return cudaErrorLaunchOutOfResources;
  }
  const int64_t tiles = int64_t(a.m_tiles) * a.n_tiles * a.splits;
  const int groups = static_cast<int>(tiles < num_sms / CG ? tiles : num_sms / CG);
  return launch_chained(k, static_cast<unsigned>(groups * CG), S::kThreads, S::kSmem, s, CG, maps.a, maps.b, maps.o, a);
}

template <Prod KIND, int CG, int BN, int ACC>
cudaError_t launch_modes(const ProdMaps& maps, const ProdArgs& a, int num_sms, cudaStream_t s) {
  const bool lab = a.tgt.t != nullptr, dis = a.ent_len != nullptr;
  if (lab && dis) return launch_one<KIND, CG, BN, true, true, ACC>(maps, a, num_sms, s);
  if (dis) return launch_one<KIND, CG, BN, false, true, ACC>(maps, a, num_sms, s);
  return launch_one<KIND, CG, BN, true, false, ACC>(maps, a, num_sms, s);
}

template <Prod KIND>
cudaError_t launch_logits(int cg, const ProdMaps& maps, const ProdArgs& a, int num_sms, cudaStream_t s) {
  if (a.planes == 3 && a.k_blocks <= kWholeBlocks)
    return cg == 2 ? launch_modes<KIND, 2, 256, kSplitWhole>(maps, a, num_sms, s)
                   : launch_modes<KIND, 1, 128, kSplitWhole>(maps, a, num_sms, s);
  if (a.planes == 3)
    return cg == 2 ? launch_modes<KIND, 2, 256, kSplit>(maps, a, num_sms, s)
                   : launch_modes<KIND, 1, 128, kSplit>(maps, a, num_sms, s);
  if (a.chunk < a.k_blocks)
    return cg == 2 ? launch_modes<KIND, 2, 256, kParts>(maps, a, num_sms, s)
                   : launch_modes<KIND, 1, 256, kParts>(maps, a, num_sms, s);
  return cg == 2 ? launch_modes<KIND, 2, 256, kWhole>(maps, a, num_sms, s)
                 : launch_modes<KIND, 1, 256, kWhole>(maps, a, num_sms, s);
}

template <Prod KIND>
cudaError_t launch_sums(int cg, int bn, const ProdMaps& maps, const ProdArgs& a, int num_sms, cudaStream_t s) {
  if (a.planes == 3)
    return cg == 2     ? launch_one<KIND, 2, 256, false, false, kSplit>(maps, a, num_sms, s)
           : bn == 128 ? launch_one<KIND, 1, 128, false, false, kSplit>(maps, a, num_sms, s)
                       : launch_one<KIND, 1, 64, false, false, kSplit>(maps, a, num_sms, s);
  if (a.g_planes == 2)
    return bn == 128  ? launch_one<KIND, 1, 128, false, false, kTwo>(maps, a, num_sms, s)
           : bn == 64 ? launch_one<KIND, 1, 64, false, false, kTwo>(maps, a, num_sms, s)
           : KIND == Prod::kDw && cg == 2 ? launch_one<Prod::kDw, 2, 256, false, false, kTwo>(maps, a, num_sms, s)
                                          : launch_one<KIND, 1, 256, false, false, kTwo>(maps, a, num_sms, s);
  if (bn == 256) {
    if constexpr (KIND == Prod::kDw) {  // dH of at most 128 rows has two planes of G
      if (cg == 1) return launch_one<KIND, 1, 256, false, false, kWhole>(maps, a, num_sms, s);
    }
    return launch_one<KIND, 2, 256, false, false, kWhole>(maps, a, num_sms, s);
  }
  return bn == 128 ? launch_one<KIND, 1, 128, false, false, kWhole>(maps, a, num_sms, s)
                   : launch_one<KIND, 1, 64, false, false, kWhole>(maps, a, num_sms, s);
}

}  // namespace

int prod_box_rows_a() { return 128; }
int prod_box_rows_b(int cg, int bn) { return bn / cg; }

int prod_logits_cols(int cg, int planes) { return planes == 3 && cg == 1 ? 128 : 256; }
int prod_sums_cols(int64_t dim, int64_t rows, int planes) {
  const int bn = dim > 128 ? 256 : dim > 64 ? 128 : 64;
  return planes == 3 && rows <= 128 ? (bn < 128 ? bn : 128) : bn;
}

int prod_grad_row_bytes(int planes, int chunk, int k_blocks) {
  const bool held = planes == 3 ? k_blocks > kWholeBlocks : chunk < k_blocks;
  return held ? 128 / kGroups<Prod::kGrad, kParts> : 128 / kGroups<Prod::kGrad, kWhole>;
}

cudaError_t launch_prod(Prod kind, int cg, int bn, const ProdMaps& maps, const ProdArgs& a, int num_sms,
                        cudaStream_t s) {
  switch (kind) {
    case Prod::kStats: return launch_logits<Prod::kStats>(cg, maps, a, num_sms, s);
    case Prod::kGrad: return launch_logits<Prod::kGrad>(cg, maps, a, num_sms, s);
    case Prod::kDh: return launch_sums<Prod::kDh>(cg, bn, maps, a, num_sms, s);
    case Prod::kDw: return launch_sums<Prod::kDw>(cg, bn, maps, a, num_sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace gm
