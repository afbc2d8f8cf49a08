// gm_draw.cu -- a class drawn from each row of logits (include/gm_sampling.h).
//
// A row is read from memory once, into the shared memory of a block or of a cluster of blocks, and
// everything else works there: its maximum; for top-k and top-p a border found digit by digit (below),
// never a sort; the kept weights' sum; the class at which u is passed. Nothing is written but the results.
//
// Borders. Classes are compared by D, the distance of their ordered bits from the row's largest: 16 bits, or 32 of
// f32. A histogram of D's upper 11 bits (counts for top-k, sums of weights for top-p) shows the digit in
// which the border lies, one of the next 11 bits within that digit its next, until D is
// known; of the classes that have just that D the first so many are kept, in class order.
//
// Weights are integers: w = 2^(t), t = (z - max) log2(e) / T <= 0, as a multiple of 2^-B with B such that all of a row
// add up in 64 bits. So sums are exact, in any order, and every pass sees the same ones.
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "gm_device.cuh"
#include "gm_host.h"
#include "gm_loss.h"
#include "gm_sampling.h"
#include "gm_umma.cuh"

namespace gm {

namespace {

using u64 = unsigned long long;

constexpr int kBins = 2048;
constexpr int kMostCluster = 8;
constexpr int kPer = 8;  // classes a thread takes at a time: 16 bytes of a 16-bit type
constexpr int kTable = 33;

struct DrawArgs {
  const void* z;
  int64_t ld;
  int n_classes, part;     // classes of a row, of a block (a multiple of kPer)
  int bits;                // B
  bool held;               // the block's part lies in shared memory
  gm_draw_rule rule;
  const float* u;
  int64_t* index;
  float* logprob;
  int32_t* kept;
};

// ---- ordered bits of a logit ----------------------------------------------------------------------
// Larger logits have larger keys; -0 has 0's, a NaN of either sign the largest of all.
template <int TYPE>
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
  if constexpr (TYPE == GM_LOSS_F32) {
    const uint32_t size = bits & 0x7fffffffu;
    if (size > 0x7f800000u) return 0xffffffffu;
    if (size == 0) return 0x80000000u;
    return bits & 0x80000000u ? ~bits : bits | 0x80000000u;
  } else {
    constexpr uint32_t inf = TYPE == GM_LOSS_BF16 ? 0x7f80u : 0x7c00u;
    const uint32_t size = bits & 0x7fffu;
    if (size > inf) return 0xffffu;
    if (size == 0) return 0x8000u;
    return bits & 0x8000u ? 0xffffu - bits : bits | 0x8000u;
  }
}
template <int TYPE>
constexpr uint32_t kInfKey = TYPE == GM_LOSS_F32 ? 0xff800000u : TYPE == GM_LOSS_BF16 ? 0xff80u : 0xfc00u;
template <int TYPE>
constexpr uint32_t kNoneKey = TYPE == GM_LOSS_F32 ? 0x007fffffu : TYPE == GM_LOSS_BF16 ? 0x007fu : 0x03ffu;  // -inf's
template <int TYPE>
__device__ __forceinline__ float value_of(uint32_t key) {
  if constexpr (TYPE == GM_LOSS_F32) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
  } else {
    const uint32_t b = key & 0x8000u ? key & 0x7fffu : 0xffffu - key;
    if constexpr (TYPE == GM_LOSS_BF16) return __uint_as_float(b << 16);
    else return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
  }
}
// Key of the smallest logit that is at least x.
template <int TYPE>
__device__ __forceinline__ uint32_t key_from(double x) {
  const float f = __double2float_ru(x);
  if constexpr (TYPE == GM_LOSS_F32) return key_of<TYPE>(__float_as_uint(f));
  else if constexpr (TYPE == GM_LOSS_BF16) return key_of<TYPE>(__bfloat16_as_ushort(__float2bfloat16_ru(f)));
  else return key_of<TYPE>(__half_as_ushort(__float2half_ru(f)));
}

// ---- weights ---------------------------------------------------------------------------------------
// t = (z - max) * (c + c_low) is formed to 48 bits or so: the difference with its rounding error, the product with its
// own. Its fraction f in [-1/2, 1/2], in units of 2^-31, is split into the nearest 32nd, whose power is in a table of
// 31-bit integers, and a rest g with |g| <= 1/64, whose 2^g - 1 = g ln 2 + (g ln 2)^2 / 2 + ... is at
// most 0.011, so that fp32 gives it to 2^-31. About 30 instructions; exact at t = 0.
struct Weigher {
  float top, c, c_low;
  uint32_t top_key;
  int bits;
  const uint32_t* table;
  __device__ __forceinline__ u64 operator()(uint32_t key, float z) const {
    if (key == top_key) return u64(1) << bits;
    const float d = z - top;
    const float t = __fmul_rn(d, c);  // a product of its own: its error is taken from it below
    if (!(t > -static_cast<float>(bits) - 2.f)) return 0;
    const float b = d - z;
    const float d_low = (z - (d - b)) - (top + b);
    const float t_low = fmaf(d, c, -t) + fmaf(d, c_low, d_low * c);
    const float whole = rintf(t);
    const uint32_t x = static_cast<uint32_t>(__float2int_rn((t - whole) * 2147483648.f)) +
                       static_cast<uint32_t>(__float2int_rn(t_low * 2147483648.f)) + (1u << 30) + (1u << 25);
    const uint32_t j = min(x >> 26, static_cast<uint32_t>(kTable - 1));
    const float g = static_cast<float>(static_cast<int>(x - (j << 26)) - (1 << 25)) * 4.656612873077393e-10f;  // 2^-31
    const float l = g * 0.693147180559945f;
    const float q = l * fmaf(l, fmaf(l, fmaf(l, 0.0416666667f, 0.1666666667f), 0.5f), 1.f);
    const uint32_t p = table[j];
    const uint32_t m = p + static_cast<uint32_t>(__float2int_rn(static_cast<float>(p) * q));
    const int shift = bits - 31 + static_cast<int>(whole);
    if (shift >= 0) return u64(m) << shift;
    return shift < -32 ? 0 : (u64(m) + (u64(1) << (-shift - 1))) >> -shift;
  }
};

// ---- sums over the block and the cluster --------------------------------------------------------------
struct Share {  // what a block tells the others of its part
  u64 sum;      // weights of the classes above the border
  uint32_t ties, above;
};
struct Shared {
  uint32_t table[kTable + 1];
  Share told[kMostCluster];
  u64 told_top[kMostCluster];
  u64 warp_sum[33];
  uint32_t warp_top[33], warp_ties[33], warp_above[33];
  uint32_t low[kBins], high[kBins];  // counts, or the two words of sums
  u64 before;                        // what lies above the digit found
  uint32_t digit;
  u64 in_digit;
};

__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void put_remote_u64(void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(map_to_rank(smem_addr(p), rank)), "l"(v) : "memory");
}

template <int TYPE>
struct Row {
  Shared& sh;
  const DrawArgs& a;
  int blocks, rank;       // of the cluster
  const void* data;       // of this block's part: class c at element c + phase
  int n, phase;           // classes of the part, their first one's place within 16 bytes
  __device__ __forceinline__ void meet() const {
    if (blocks > 1) cluster_sync_all();
    else __syncthreads();
  }
  __device__ __forceinline__ int pieces() const { return (phase + n + kPer - 1) / kPer; }
  // Keys of a piece; outside the part: none's.
  __device__ __forceinline__ void keys(int piece, uint32_t (&k)[kPer]) const {
    const int c0 = piece * kPer - phase;
    uint32_t w[8];
    if (a.held || (c0 >= 0 && c0 + kPer <= n)) {
      const uint4* p = static_cast<const uint4*>(data);
      if constexpr (TYPE == GM_LOSS_F32) {
        const uint4 x = p[2 * piece], y = p[2 * piece + 1];
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
      } else {
        const uint4 x = p[piece];
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        k[i] = key_of<TYPE>(TYPE == GM_LOSS_F32 ? w[i] : i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i) k[i] = c0 + i >= 0 && c0 + i < n ? key_of<TYPE>(element(c0 + i)) : kNoneKey<TYPE>;
    }
  }
  __device__ __forceinline__ uint32_t element(int c) const {  // of the part, in memory or held
    if constexpr (TYPE == GM_LOSS_F32) return static_cast<const uint32_t*>(data)[phase + c];
    else return static_cast<const uint16_t*>(data)[phase + c];
  }
  // f(key) for every class, in any order
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    for (int p = threadIdx.x; p < pieces(); p += blockDim.x) {
      uint32_t k[kPer];
      keys(p, k);
#pragma unroll
      for (int i = 0; i < kPer; ++i) f(k[i]);
    }
  }

  // One digit of a border. The histogram has been filled; target(total) is what the border's sum is to reach. Finds the
  // first digit at which the sum from digit 0 on, and `before` it, is at least the target.
  template <bool MASS, class T>
  __device__ __forceinline__ void find(u64 before, T&& target) const {
    meet();  // histograms are complete
    const int per = kBins / blockDim.x;  // blockDim.x: 128 .. 1024
    const int b0 = threadIdx.x * per;
    u64 mine = 0;
    auto bin = [&](int b) {
      u64 x = 0;
      for (int r = 0; r < blocks; ++r) {
        if (blocks > 1) x += MASS ? u64(remote_u32(&sh.low[b], r)) + (u64(remote_u32(&sh.high[b], r)) << 32) : remote_u32(&sh.low[b], r);
        else x += MASS ? u64(sh.low[b]) + (u64(sh.high[b]) << 32) : sh.low[b];
      }
      return x;
    };
    for (int i = 0; i < per; ++i) mine += bin(b0 + i);
    u64 total;
    u64 at = before + block_exclusive_scan(mine, sh.warp_sum, &total);
    const double goal = target(before + total);
    const bool last = threadIdx.x == blockDim.x - 1;
    // a thread's bins hold the border when the sum before them falls short of it and the sum with them does not; the last
    // one's do where rounding leaves no other
    if (static_cast<double>(at) < goal && (static_cast<double>(at + mine) >= goal || last)) {
      for (int i = 0; i < per; ++i) {
        const u64 x = bin(b0 + i);
        if (static_cast<double>(at + x) >= goal || (i == per - 1)) {
          sh.digit = b0 + i;
          sh.before = at;
          sh.in_digit = x;
          break;
        }
        at += x;
      }
    }
    meet();  // found, and the histograms are read
  }
  __device__ __forceinline__ void clear() const {
    for (int i = threadIdx.x; i < kBins; i += blockDim.x) sh.low[i] = sh.high[i] = 0;
    __syncthreads();
  }
};

// Classes kept: those with D < d, and of those with D = d the first `ties`.
struct Border {
  uint32_t d;
  int64_t ties;
};

template <int TYPE>
__global__ void __launch_bounds__(1024) k_draw(const __grid_constant__ DrawArgs a) {
  extern __shared__ __align__(16) unsigned char part_mem[];
  __shared__ Shared sh;
  constexpr int kBytes = TYPE == GM_LOSS_F32 ? 4 : 2;
  constexpr int kDigits = TYPE == GM_LOSS_F32 ? 3 : 2;
  uint32_t blocks;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(blocks));
  const uint32_t rank = blocks > 1 ? cluster_rank() : 0;
  const int64_t row_i = blockIdx.x / blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (threadIdx.x < kTable)
    sh.table[threadIdx.x] = static_cast<uint32_t>(__double2ll_rn(2147483648.0 * exp2((static_cast<int>(threadIdx.x) - 16) * 0.03125)));
  chain_wait();

  // ---- the part of the row, and its largest key
  const int first = static_cast<int>(min(int64_t(rank) * a.part, int64_t(a.n_classes)));
  const int n = min(a.part, a.n_classes - first);
  const char* src = static_cast<const char*>(a.z) + (row_i * a.ld + first) * kBytes;
  const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(src) % (kPer * kBytes) / kBytes);
  Row<TYPE> row{sh, a, static_cast<int>(blocks), static_cast<int>(rank), a.held ? static_cast<const void*>(part_mem) : src - phase * kBytes, n, phase};
  uint32_t top = 0;
  if (a.held) {
    // whole pieces as they lie; the ends by elements, and none's logit around them
    const char* base = src - phase * kBytes;
    for (int p = threadIdx.x; p < row.pieces(); p += blockDim.x) {
      const int c0 = p * kPer - phase;
      uint4 x[kBytes / 2];
      if (c0 >= 0 && c0 + kPer <= n) {
#pragma unroll
        for (int h = 0; h < kBytes / 2; ++h) x[h] = __ldcs(reinterpret_cast<const uint4*>(base) + p * (kBytes / 2) + h);
      } else {
        uint32_t w[2 * kBytes];
#pragma unroll
        for (int i = 0; i < 2 * kBytes; ++i) w[i] = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const bool in = c0 + i >= 0 && c0 + i < n;
          if constexpr (TYPE == GM_LOSS_F32) {
            w[i] = in ? reinterpret_cast<const uint32_t*>(src)[c0 + i] : 0xff800000u;
          } else {
            const uint32_t v = in ? reinterpret_cast<const uint16_t*>(src)[c0 + i] : TYPE == GM_LOSS_BF16 ? 0xff80u : 0xfc00u;
            w[i / 2] |= v << (i & 1 ? 16 : 0);
          }
        }
#pragma unroll
        for (int h = 0; h < kBytes / 2; ++h) x[h] = make_uint4(w[4 * h], w[4 * h + 1], w[4 * h + 2], w[4 * h + 3]);
      }
#pragma unroll
      for (int h = 0; h < kBytes / 2; ++h) {
        reinterpret_cast<uint4*>(part_mem)[p * (kBytes / 2) + h] = x[h];
        const uint32_t w[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (TYPE == GM_LOSS_F32) top = max(top, key_of<TYPE>(w[i]));
          else top = max(top, max(key_of<TYPE>(w[i] & 0xffffu), key_of<TYPE>(w[i] >> 16)));
        }
      }
    }
  } else {
    row.each([&](uint32_t k) { top = max(top, k); });
  }
  for (int i = threadIdx.x; i < kBins; i += blockDim.x) sh.low[i] = sh.high[i] = 0;
  top = __reduce_max_sync(kFull, top);
  if (lane == 0) sh.warp_top[warp] = top;
  __syncthreads();
  top = sh.warp_top[lane < warps ? lane : 0];
  top = __reduce_max_sync(kFull, top);
  if (blocks > 1) {
    if (threadIdx.x < blocks) put_remote_u64(&sh.told_top[rank], threadIdx.x, top);
    cluster_sync_all();
    for (int r = 0; r < blocks; ++r) top = max(top, static_cast<uint32_t>(sh.told_top[r]));
  }

  // ---- the row's rule
  const float temp = a.rule.temperature ? a.rule.temperature[row_i] : a.rule.all_temperature;
  const float top_p = a.rule.top_p ? a.rule.top_p[row_i] : a.rule.all_top_p;
  const float min_p = a.rule.min_p ? a.rule.min_p[row_i] : a.rule.all_min_p;
  int64_t top_k = a.rule.top_k ? a.rule.top_k[row_i] : a.rule.all_top_k;
  const float u = a.u[row_i];
  const double c = temp > 0.f ? 1.4426950408889634 / static_cast<double>(temp) : 0.0;
  const float c_high = static_cast<float>(c);
  const bool fine = top > kNoneKey<TYPE> && top <= kInfKey<TYPE> && u >= 0.f && u < 1.f && temp >= 0.f && temp < INFINITY &&
                    c_high < INFINITY && top_k >= 0 && top_p >= 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f;
  if (!fine) {  // the same for every block of the row
    if (rank == 0 && threadIdx.x == 0) {
      a.index[row_i] = -1;
      a.logprob[row_i] = NAN;
      a.kept[row_i] = 0;
    }
    return;
  }
  if (temp == 0.f) top_k = 1;
  const float top_z = value_of<TYPE>(top);
  const Weigher weigh{top_z, c_high, static_cast<float>(c - static_cast<double>(c_high)), top, a.bits, sh.table};

  // what is not -inf, and passes min-p
  Border border{top - kNoneKey<TYPE> - 1, INT64_MAX};
  uint32_t by_min = border.d;
  if (min_p > 0.f && temp > 0.f && top < kInfKey<TYPE>) {
    const uint32_t least = key_from<TYPE>(static_cast<double>(top_z) + static_cast<double>(temp) * log(static_cast<double>(min_p)));
    by_min = min(by_min, top - min(top, least));
  } else if (min_p > 0.f) {
    by_min = 0;  // T = 0, or +inf: w is 1 or 0
  }

  // ---- top-k
  if (top_k > 0 && top_k < a.n_classes) {
    u64 before = 0;
    uint32_t lo = 0;  // digits found so far
#pragma unroll 1
    for (int g = 0; g < kDigits; ++g) {
      const int shift = TYPE == GM_LOSS_F32 ? (g == 0 ? 21 : g == 1 ? 10 : 0) : (g == 0 ? 5 : 0);
      const int shift0 = TYPE == GM_LOSS_F32 ? (g == 1 ? 21 : 10) : 5;  // of the digit before
      if (g > 0) row.clear();
      row.each([&](uint32_t k) {
        const uint32_t d = top - k;
        if (g == 0 || (d >> shift0) == (lo >> shift0)) atomicAdd(&sh.low[(d - lo) >> shift], 1u);
      });
      row.template find<false>(before, [&](u64) { return static_cast<double>(top_k); });
      lo += sh.digit << shift;
      before = sh.before;
    }
    if (lo <= border.d) border = Border{lo, top_k - static_cast<int64_t>(before)};
    if (top_p < 1.f) row.clear();
  }

  // ---- top-p
  if (top_p < 1.f) {
    u64 before = 0;
    uint32_t lo = 0;
    double goal = 0.0;
    // of the classes at the border itself only `ties` count, which one thread adds at once where they are not all
    const bool all = border.ties == INT64_MAX;
    const u64 w_border = weigh(top - border.d, value_of<TYPE>(top - border.d));
    auto add = [&](uint32_t at, u64 w) {
      const uint32_t l = static_cast<uint32_t>(w), old = atomicAdd(&sh.low[at], l);
      const uint32_t h = static_cast<uint32_t>(w >> 32) + (old + l < old);
      if (h) atomicAdd(&sh.high[at], h);
    };
#pragma unroll 1
    for (int g = 0; g < kDigits; ++g) {
      const int shift = TYPE == GM_LOSS_F32 ? (g == 0 ? 21 : g == 1 ? 10 : 0) : (g == 0 ? 5 : 0);
      const int shift0 = TYPE == GM_LOSS_F32 ? (g == 1 ? 21 : 10) : 5;
      if (g > 0) row.clear();
      row.each([&](uint32_t k) {
        const uint32_t d = top - k;
        if (d > border.d || (d == border.d && !all)) return;
        if (g > 0 && (d >> shift0) != (lo >> shift0)) return;
        const u64 w = weigh(k, value_of<TYPE>(k));
        if (w) add((d - lo) >> shift, w);
      });
      if (!all && rank == 0 && threadIdx.x == 0 && (g == 0 || (border.d >> shift0) == (lo >> shift0)))
        add((border.d - lo) >> shift, w_border * static_cast<u64>(border.ties));
      row.template find<true>(before, [&](u64 total) {
        if (g == 0) goal = fmax(static_cast<double>(top_p) * static_cast<double>(total), 1.0);
        return goal;
      });
      lo += sh.digit << shift;
      before = sh.before;
    }
    // so many of the classes with this very D
    const u64 w = weigh(top - lo, value_of<TYPE>(top - lo)), have = w ? sh.in_digit / w : 0;
    u64 ties = w ? static_cast<u64>(ceil((goal - static_cast<double>(before)) / static_cast<double>(w))) : 1;
    ties = max(u64(1), min(ties, max(have, u64(1))));
    if (lo < border.d || static_cast<int64_t>(ties) < border.ties) border = Border{lo, static_cast<int64_t>(ties)};
  }

  // ---- min-p
  if (by_min < border.d) border = Border{by_min, INT64_MAX};

  // ---- sums of what is kept, by warps: a warp takes pieces that follow one another
  const int per_warp = (row.pieces() + warps - 1) / warps;
  const int p0 = min(warp * per_warp, row.pieces()), p1 = min(p0 + per_warp, row.pieces());
  const u64 w_tie = weigh(top - border.d, value_of<TYPE>(top - border.d));
  u64 sum = 0;
  uint32_t ties = 0, above = 0;
  for (int p = p0 + lane; p < p1; p += 32) {
    uint32_t k[kPer];
    row.keys(p, k);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t d = top - k[i];
      if (d < border.d) sum += weigh(k[i], value_of<TYPE>(k[i])), ++above;
      else if (d == border.d) ++ties;
    }
  }
  sum = warp_reduce_sum(sum);
  ties = __reduce_add_sync(kFull, ties);
  above = __reduce_add_sync(kFull, above);
  if (lane == 0) sh.warp_sum[warp] = sum, sh.warp_ties[warp] = ties, sh.warp_above[warp] = above;
  __syncthreads();
  Share mine = {0, 0, 0};
  u64 sum_before = 0;  // of this warp, in its block
  uint32_t ties_before = 0;
  for (int w = 0; w < warps; ++w) {
    if (w == warp) sum_before = mine.sum, ties_before = mine.ties;
    mine.sum += sh.warp_sum[w], mine.ties += sh.warp_ties[w], mine.above += sh.warp_above[w];
  }
  u64 total = mine.sum;
  int64_t all_ties = mine.ties, kept = mine.above;
  if (blocks > 1) {
    if (threadIdx.x < blocks) {
      put_remote_u64(&sh.told[rank].sum, threadIdx.x, mine.sum);
      put_remote_u64(&sh.told[rank].ties, threadIdx.x, (u64(mine.above) << 32) | mine.ties);
    }
    cluster_sync_all();
    total = 0, all_ties = kept = 0;
    for (int r = 0; r < blocks; ++r) {
      if (r == rank) sum_before += total, ties_before += static_cast<uint32_t>(all_ties);
      total += sh.told[r].sum, all_ties += sh.told[r].ties, kept += sh.told[r].above;
    }
  }
  const int64_t most = min(border.ties, all_ties);
  total += static_cast<u64>(most) * w_tie;
  kept += most;
  const double goal = static_cast<double>(u) * static_cast<double>(total);
  auto tied = [&](int64_t before, int64_t n_ties) {  // of n_ties after `before` others, how many are kept
    return static_cast<u64>(max(int64_t(0), min(most - before, n_ties)));
  };
  sum_before += static_cast<u64>(min(most, int64_t(ties_before))) * w_tie;
  sum += tied(ties_before, ties) * w_tie;
  if (!(static_cast<double>(sum_before) <= goal && static_cast<double>(sum_before + sum) > goal)) return;

  // ---- the one warp in which the sum passes u: 32 pieces at a time, then the lane, then the class
  int64_t tie = ties_before;
  u64 at = sum_before;
  for (int p = p0; p < p1; p += 32) {
    uint32_t k[kPer];
    u64 own = 0;
    uint32_t own_ties = 0;
    const bool in = p + lane < p1;
    if (in) {
      row.keys(p + lane, k);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const uint32_t d = top - k[i];
        if (d < border.d) own += weigh(k[i], value_of<TYPE>(k[i]));
        else if (d == border.d) ++own_ties;
      }
    }
    const uint32_t ties_to = warp_inclusive_scan(own_ties);
    int64_t tie_at = tie + ties_to - own_ties;
    own += tied(tie_at, own_ties) * w_tie;
    const u64 to = warp_inclusive_scan(own);
    const unsigned passed = __ballot_sync(kFull, static_cast<double>(at + to) > goal);
    if (!passed) {
      at += __shfl_sync(kFull, to, 31);
      tie += __shfl_sync(kFull, ties_to, 31);
      continue;
    }
    if (lane != __ffs(passed) - 1) return;
    at += to - own;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t d = top - k[i];
      u64 w = 0;
      if (d < border.d) w = weigh(k[i], value_of<TYPE>(k[i]));
      else if (d == border.d) w = tied(tie_at, 1) * w_tie, ++tie_at;
      at += w;
      if (w && static_cast<double>(at) > goal) {
        a.index[row_i] = first + (p + lane) * kPer - phase + i;
        const double log_w = k[i] == top ? 0.0 : (static_cast<double>(value_of<TYPE>(k[i])) - static_cast<double>(top_z)) / static_cast<double>(temp);
        a.logprob[row_i] = static_cast<float>(log_w - log(ldexp(static_cast<double>(total), -a.bits)));
        a.kept[row_i] = static_cast<int32_t>(kept);
        return;
      }
    }
    return;
  }
}

// ---- host ---------------------------------------------------------------------------------------------
constexpr int64_t kMostClasses = int64_t(1) << 24;
constexpr int kHeldBytes = 196608;  // of a row in a block's shared memory

template <int TYPE>
cudaError_t launch(DrawArgs& a, int64_t n_rows, int sms, cudaStream_t s) {
  const int64_t es = TYPE == GM_LOSS_F32 ? 4 : 2, n = a.n_classes;
  const cudaError_t e = cudaFuncSetAttribute(k_draw<TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldBytes);
  if (e != cudaSuccess) return e;
  // blocks of a row: until it fits, or the SMs have work
  int blocks = 1;
  auto part = [&] { return up(div_up(n, blocks), kPer); };
  while (blocks < kMostCluster && ((part() + kPer) * es > kHeldBytes || (n_rows * blocks * 2 <= sms && part() > 8192))) blocks *= 2;
  a.part = static_cast<int>(part());
  a.held = (part() + kPer) * es <= kHeldBytes;
  if (n_rows * blocks > INT32_MAX) return cudaErrorInvalidValue;  // more bytes than any device has
  const int64_t threads = std::min<int64_t>(1024, std::max<int64_t>(128, up(div_up(part(), 4 * kPer), 128)));
  int block = 128;  // a power of two: bins are shared out evenly
  while (block < threads) block *= 2;
  return launch_chained(k_draw<TYPE>, static_cast<unsigned>(n_rows * blocks), block, a.held ? static_cast<size_t>((part() + kPer) * es) : 0,
                        s, blocks, a);
}

}  // namespace

}  // namespace gm

extern "C" gm_status gm_draw(const void* logits, int64_t n_rows, int64_t n_classes, int64_t ld, int32_t type,
                             const gm_draw_rule* rule, const float* u, void* stream, int64_t* index, float* logprob,
                             int32_t* kept) {
  using namespace gm;
  NvtxRange range("gm_draw");
  if (n_rows < 0 || n_classes < 1 || !rule) return GM_ERR_INVALID_ARG;
  if (n_rows > kMostIndex || n_classes > kMostClasses || ld > kMostLd) return GM_ERR_INDEX_OVERFLOW;
  if (type != GM_LOSS_F32 && type != GM_LOSS_BF16 && type != GM_LOSS_F16) return GM_ERR_INVALID_ARG;
  if (ld < n_classes || !aligned(logits, elem_bytes(type)) || !aligned(index, 8)) return GM_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(u), static_cast<const void*>(logprob), static_cast<const void*>(kept),
                        static_cast<const void*>(rule->temperature), static_cast<const void*>(rule->top_k),
                        static_cast<const void*>(rule->top_p), static_cast<const void*>(rule->min_p)})
    if (!aligned(p, 4)) return GM_ERR_INVALID_ARG;
  const float t = rule->all_temperature;
  if (!rule->temperature && t != 0.f && (!(t > 0.f) || !std::isfinite(t) || !std::isfinite(kLog2e / t))) return GM_ERR_INVALID_ARG;
  if (!rule->top_k && rule->all_top_k < 0) return GM_ERR_INVALID_ARG;
  if (!rule->top_p && !(rule->all_top_p >= 0.f && rule->all_top_p <= 1.f)) return GM_ERR_INVALID_ARG;
  if (!rule->min_p && !(rule->all_min_p >= 0.f && rule->all_min_p <= 1.f)) return GM_ERR_INVALID_ARG;
  if (n_rows > 0 && (!logits || !u || !index || !logprob || !kept)) return GM_ERR_INVALID_ARG;
  if (n_rows == 0) return GM_OK;
  if (cudaPeekAtLastError() != cudaSuccess) return GM_ERR_CUDA;
  const int sms = sm_count(kMostBlocks);
  if (sms <= 0) {
    cudaGetLastError();
    return GM_ERR_CUDA;
  }
  DrawArgs a = {};
  a.z = logits;
  a.ld = ld;
  a.n_classes = static_cast<int>(n_classes);
  // a row's weights, at most 2^B each, add up to less than 2^63
  a.bits = 46;
  while ((int64_t(1) << (62 - a.bits)) < n_classes) --a.bits;
  a.rule = *rule;
  a.u = u;
  a.index = index;
  a.logprob = logprob;
  a.kept = kept;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == GM_LOSS_F32    ? launch<GM_LOSS_F32>(a, n_rows, sms, s)
                        : type == GM_LOSS_BF16 ? launch<GM_LOSS_BF16>(a, n_rows, sms, s)
                                               : launch<GM_LOSS_F16>(a, n_rows, sms, s);
  return cudaGetLastError() != cudaSuccess || e != cudaSuccess ? GM_ERR_CUDA : GM_OK;
}
