// gm_draw.cu -- a class drawn from each row of logits (include/gm_sampling.h).
//
// A row is read from memory once, into the shared memory of a block or of a cluster of blocks where it fits (beside the
// counts up to 36856 classes a block; else its later passes read it from L2), and everything else works there: its maximum; for
// top-k and top-p a border found by histograms, never a sort; the kept weights' sum; the class at which u is passed. Nothing is
// written but the results.
//
// Borders. Classes are compared by D, the distance of their ordered bits from the row's largest: 16 bits, or 32 of
// f32. A border is a D and how many of the classes that have just that D are kept, in class order.
//   Long rows of 16 bits (KEYS): how often each of the 65536 values occurs is counted while the row is read, 128 KB of
//   16-bit counts. Counts, and sums of counts times weights, of 1024 lines of 64 values then lead to the border: a weight is
//   computed for each value that occurs, not for each class, and looked up when classes are summed.
//   Others: a histogram of D's upper 11 bits shows the digit in which the border lies, one of the next
//   11 bits within that digit its next, until D is known.
//
// Bound by latency, far from memory's rate: with counts an SM has one row, whose warps wait for shared memory and at barriers
// with nothing beside them (LSU 26 % busy, DRAM 7 %, 43 % of the warps). 256 x 131072 bf16 with top-p 101 us (67 MB; plain 8240),
// of a row's clocks 36 % reading and counting, 19 % the search, 25 % the sums; 1 x 131072 with all four rules 15 us back to
// back, 19 alone.
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

constexpr float kLog2eLow = 1.92596299e-8f;  // log2(e) - kLog2e

constexpr int kMostCluster = 8;
// Classes that are compared each with each: so many steps of each thread, where a search would take its rounds over the
// cluster. 1 x 131072, top-k and top-p, us: 50 classes 19 (search 27), 128: 21 (27), 256: 27 (27.5); 64 rows: 29 (39), 31 (39),
// 37 (40), and 512 classes 47 (40).
constexpr int kFew = 256;
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
// A logit's place: 16 bits, or 32 of f32, that grow as logits fall. The bits of positive ones are turned over, of negative
// ones less 1, which brings -0 to 0's place and leaves the others apart. NaN lies before inf's place or after -inf's. Two
// 16-bit ones at a time.
__device__ __forceinline__ uint32_t place_pair(uint32_t w) {
  const uint32_t m = (w >> 15) & 0x00010001u;
  return (w ^ ((0x00010001u - m) * 0x7fffu)) - m;
}
template <int TYPE>
__device__ __forceinline__ uint32_t place_of(uint32_t bits) {
  if constexpr (TYPE == GM_LOSS_F32) {
    const uint32_t m = bits >> 31;
    return (bits ^ ((1u - m) * 0x7fffffffu)) - m;
  } else {
    return place_pair(bits) & 0xffffu;
  }
}
template <int TYPE>
constexpr uint32_t kInfBits = TYPE == GM_LOSS_F32 ? 0x7f800000u : TYPE == GM_LOSS_BF16 ? 0x7f80u : 0x7c00u;
template <int TYPE>
constexpr uint32_t kZero = TYPE == GM_LOSS_F32 ? 0x7fffffffu : 0x7fffu;  // 0's place
template <int TYPE>
constexpr uint32_t kInfPlace = kZero<TYPE> - kInfBits<TYPE>;
template <int TYPE>
constexpr uint32_t kNonePlace = kZero<TYPE> + kInfBits<TYPE>;  // -inf's
template <int TYPE>
__device__ __forceinline__ float value_of(uint32_t place) {
  const uint32_t size = place <= kZero<TYPE> ? kZero<TYPE> - place : place - kZero<TYPE>;
  const float x = TYPE == GM_LOSS_F32    ? __uint_as_float(size)
                  : TYPE == GM_LOSS_BF16 ? __uint_as_float(size << 16)
                                         : __half2float(__ushort_as_half(static_cast<unsigned short>(size)));
  return place <= kZero<TYPE> ? x : -x;
}
// Place of the smallest logit that is at least x + y + y_low.
template <int TYPE>
__device__ __forceinline__ uint32_t place_from(float x, float y, float y_low) {
  float f = x + y;
  const float b = f - x;
  const float rest = (x - (f - b)) + (y - b) + y_low;  // what the sum's rounding took
  if (rest > 0.f) f = nextafterf(f, INFINITY);
  if constexpr (TYPE == GM_LOSS_F32) return place_of<TYPE>(__float_as_uint(f));
  else if constexpr (TYPE == GM_LOSS_BF16) return place_of<TYPE>(__bfloat16_as_ushort(__float2bfloat16_ru(f)));
  else return place_of<TYPE>(__half_as_ushort(__float2half_ru(f)));
}

// The whole part of f * n for f in [0, 1], and whether something is left: in integers, since 64-bit floating point is
// 1 / 70 as fast as 32-bit here (all threads of a block dividing by T so took 5 us).
__device__ __forceinline__ u64 whole_times(float f, u64 n, bool& left) {
  const uint32_t bits = __float_as_uint(f) & 0x7fffffffu, e = bits >> 23;  // -0 is 0
  const u64 m = e ? (bits & 0x7fffffu) | 0x800000u : bits;
  const int s = e ? 150 - static_cast<int>(e) : 149;  // f = m 2^-s, 23 <= s
  const u64 lo = m * n, hi = __umul64hi(m, n);
  if (s >= 128) {
    left = (lo | hi) != 0;
    return 0;
  }
  if (s >= 64) {
    const u64 w = hi >> (s - 64);
    left = lo != 0 || (w << (s - 64)) != hi;
    return w;
  }
  left = (lo & ((u64(1) << s) - 1)) != 0;
  return (hi << (64 - s)) | (lo >> s);
}

// ---- weights ---------------------------------------------------------------------------------------
// 2^(31 + f / 2^31) for f in [-2^30, 2^30], to 2^-28 of itself: the nearest 32nd of f's range, whose power
// is in a table of 32-bit integers, and a rest g with |g| <= 1/64, whose 2^g - 1 = g ln 2 + (g ln 2)^2 / 2 + ... is at
// most 0.011, so that fp32 gives it to 2^-31. Exact at 0.
// 2^(31 + (j - 16) / 32), rounded
__constant__ uint32_t kPowers[kTable] = {
    1518500250u, 1551751076u, 1585730000u, 1620452965u, 1655936265u, 1692196547u,
    1729250827u, 1767116489u, 1805811301u, 1845353420u, 1885761398u, 1927054196u,
    1969251188u, 2012372174u, 2056437387u, 2101467502u, 2147483648u, 2194507417u,
    2242560872u, 2291666561u, 2341847524u, 2393127307u, 2445529972u, 2499080105u,
    2553802834u, 2609723834u, 2666869345u, 2725266179u, 2784941738u, 2845924021u,
    2908241642u, 2971923842u, 3037000500u};
__device__ __forceinline__ uint32_t power(int f, const uint32_t* table) {
  const uint32_t x = static_cast<uint32_t>(f) + (1u << 30) + (1u << 25);
  const uint32_t j = min(x >> 26, static_cast<uint32_t>(kTable - 1));
  const float g = static_cast<float>(static_cast<int>(x - (j << 26)) - (1 << 25)) * 4.656612873077393e-10f;  // 2^-31
  const float l = g * 0.693147180559945f;
  const float q = l * fmaf(l, fmaf(l, fmaf(l, 0.0416666667f, 0.1666666667f), 0.5f), 1.f);
  const uint32_t p = table[j];
  return p + static_cast<uint32_t>(__float2int_rn(static_cast<float>(p) * q));
}
// w of a logit. t = (z - max) * (c + c_low) is formed to 48 bits or so: the difference with its rounding error, the product
// with its own.
struct Weigher {
  float top, c, c_low;
  uint32_t top_place;
  int bits;
  const uint32_t* table;
  __device__ __forceinline__ u64 operator()(uint32_t place, float z) const {
    if (place == top_place) return u64(1) << bits;
    const float d = z - top;
    const float t = __fmul_rn(d, c);  // a product of its own: its error is taken from it below
    if (!(t > -static_cast<float>(bits) - 2.f)) return 0;
    const float b = d - z;
    const float d_low = (z - (d - b)) - (top + b);
    const float t_low = fmaf(d, c, -t) + fmaf(d, c_low, d_low * c);
    const float whole = rintf(t);
    const uint32_t m = power(__float2int_rn((t - whole) * 2147483648.f) + __float2int_rn(t_low * 2147483648.f), table);
    const int shift = bits - 31 + static_cast<int>(whole);
    if (shift >= 0) return u64(m) << shift;
    return shift < -32 ? 0 : (u64(m) + (u64(1) << (-shift - 1))) >> -shift;
  }
};

// A value in two parts.
struct Pair {
  float x, low;
};
__device__ __forceinline__ Pair sum_of(float a, float b) {
  const float s = a + b, t = s - a;
  return Pair{s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair times(Pair a, float x, float x_low) {
  const float p = __fmul_rn(a.x, x);
  return sum_of(p, fmaf(a.x, x, -p) + fmaf(a.x, x_low, a.low * x));
}
constexpr float kLn2 = 0.693147180559945f, kLn2Low = -1.9046543e-9f;
// ln(m / 2^31 * 2^e) for m in [2^31, 2^32), to about 2^-28: log2f, put right by how far its power is from m.
__device__ __forceinline__ Pair log_of(uint32_t m, int e, const uint32_t* table) {
  const float y = log2f(static_cast<float>(m) * 4.656612873077393e-10f);  // 2^-31; in [0, 1]
  const float whole = rintf(y);
  const uint32_t p = power(__float2int_rn((y - whole) * 2147483648.f), table);
  const float off = static_cast<float>(static_cast<int64_t>(m) - (static_cast<int64_t>(p) << static_cast<int>(whole))) / static_cast<float>(m);
  Pair l = sum_of(static_cast<float>(e), y);
  l.low = fmaf(off, 1.44269504f, l.low);
  return times(l, kLn2, kLn2Low);
}
__device__ __forceinline__ Pair log_of(float x, const uint32_t* table) {  // 0 < x, finite
  const uint32_t bits = __float_as_uint(x), e = bits >> 23, m = e ? (bits & 0x7fffffu) | 0x800000u : bits;
  const int z = __clz(m);
  return log_of(m << z, (e ? static_cast<int>(e) - 150 : -149) + 31 - z, table);
}
__device__ __forceinline__ Pair log_of(u64 n, int e, const uint32_t* table) {  // ln(n 2^e), n > 0
  const int z = __clzll(static_cast<long long>(n));
  return log_of(static_cast<uint32_t>((n << z) >> 32), e + 63 - z, table);
}

// ---- sums over the block and the cluster --------------------------------------------------------------
constexpr int kGroups = 64;                          // of bins, or of lines: the first step of a search
constexpr int kBins = 2048, kGroupBins = kBins / kGroups;
constexpr int kLine = 64, kLines = 65536 / kLine, kGroupLines = kLines / kGroups;
constexpr int kWeights = 16384;                      // KEYS: weights that take the counts' place
constexpr int kCountBytes = 65536 * 2;               // KEYS: counts of all values, in front of the held part

struct Share {  // what a block tells the others of its part
  u64 sum;      // weights of the classes above the border
  uint32_t ties, above;
};
// Classes kept: those with D < d, and of those with D = d the first `ties`.
struct Border {
  uint32_t d;
  int64_t ties;
  __device__ __forceinline__ bool all() const { return ties == INT64_MAX; }
};
template <bool KEYS>
struct Shared {
  uint32_t table[kTable + 1];
  Share told[kMostCluster];
  u64 told_ends[kMostCluster], told_off[kMostCluster];
  Border border;
  uint32_t cut;                    // the few largest: those with D up to this, where there are few
  uint32_t n_few;
  uint32_t digit;                  // !KEYS: D's digits found so far
  bool found;
  u64 before, goal;
  u64 warp_sum[32];
  uint32_t warp_top[32], warp_last[32], warp_ties[32], warp_above[32];
  u64 coarse[kMostCluster][kGroups];
  alignas(16) uint32_t bins[KEYS ? 2 : 2 * kBins];  // !KEYS: histograms
  alignas(16) u64 line[KEYS ? kLines : 1];
  int n_lines;                     // lines that hold anything
  uint16_t lines[KEYS ? kLines : 1];
};

__device__ __forceinline__ uint32_t remote_u32(const void* p, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ u64 remote_u64(const void* p, uint32_t rank) {
  u64 v;
  asm volatile("ld.shared::cluster.b64 %0, [%1];" : "=l"(v) : "r"(map_to_rank(smem_addr(p), rank)) : "memory");
  return v;
}
__device__ __forceinline__ void put_remote_u64(void* p, uint32_t rank, u64 v) {
  asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(map_to_rank(smem_addr(p), rank)), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_remote_u32(void* p, uint32_t rank, uint32_t v) {
  uint32_t was;
  asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(was) : "r"(map_to_rank(smem_addr(p), rank)), "r"(v) : "memory");
  return was;
}
// f(rank) for every block of the row, all under way before the first is used; their sum.
template <class F>
__device__ __forceinline__ u64 from_each(int blocks, F&& f) {
  decltype(f(0)) v[kMostCluster];
#pragma unroll
  for (int r = 0; r < kMostCluster; ++r) v[r] = r < blocks ? f(r) : 0;
  u64 sum = 0;
#pragma unroll
  for (int r = 0; r < kMostCluster; ++r) sum += v[r];
  return sum;
}

// A warp's way to the place at which a sum reaches the goal: the sum before what was found so far, the sum of all, and
// that of what was found.
struct Search {
  u64 before, total, goal, in;
  // the first lane at which `before` and the sum of v up to and with it reach the goal (the last, where there is none)
  __device__ __forceinline__ uint32_t step(u64 v) {
    const u64 to = warp_inclusive_scan(v);
    const unsigned at = __ballot_sync(kFull, before + to >= goal);
    const int l = at ? __ffs(at) - 1 : 31;
    before += __shfl_sync(kFull, to - v, l);
    in = __shfl_sync(kFull, v, l);
    return l;
  }
  // the same of two values a lane
  __device__ __forceinline__ uint32_t step2(u64 a, u64 b) {
    const uint32_t l = step(a + b);
    const u64 first = __shfl_sync(kFull, a, l);
    if (before + first >= goal) {
      in = first;
      return 2 * l;
    }
    before += first, in -= first;
    return 2 * l + 1;
  }
};

template <int TYPE, bool KEYS>
struct Row {
  static constexpr int kWords = TYPE == GM_LOSS_F32 ? 8 : 4;  // of a piece
  Shared<KEYS>& sh;
  const DrawArgs& a;
  uint32_t* counts;       // KEYS: of the values at each place, two a word
  uint32_t *low, *high;   // histograms: counts, or the two words of sums
  int blocks, rank;       // of the cluster
  const void* data;       // of this block's part, from piece 0 on: places where they are held, else logits
  int n, phase;           // classes of the part, their first one's element in piece 0
  __device__ __forceinline__ void meet() const {
    if (blocks > 1) cluster_sync_all();
    else __syncthreads();
  }
  __device__ __forceinline__ int pieces() const { return (phase + n + kPer - 1) / kPer; }
  // Places of a piece; outside the part: none's.
  __device__ __forceinline__ void places(int piece, uint32_t (&q)[kPer]) const {
    uint32_t w[kWords];
    if (a.held) {
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const uint4 x = static_cast<const uint4*>(data)[piece * (kWords / 4) + h];
        w[4 * h] = x.x, w[4 * h + 1] = x.y, w[4 * h + 2] = x.z, w[4 * h + 3] = x.w;
      }
    } else {
      read(data, piece, w);
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) q[i] = TYPE == GM_LOSS_F32 ? w[i % kWords] : i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu;
  }
  // A piece of the row in memory, as places: 16 bytes at a time, the ends by elements. base: of piece 0.
  __device__ __forceinline__ void read(const void* base, int piece, uint32_t (&w)[kWords]) const {
    const int c0 = piece * kPer - phase;
    if (c0 >= 0 && c0 + kPer <= n) {
#pragma unroll
      for (int h = 0; h < kWords / 4; ++h) {
        const uint4 x = static_cast<const uint4*>(base)[piece * (kWords / 4) + h];
        w[4 * h] = x.x, w[4 * h + 1] = x.y, w[4 * h + 2] = x.z, w[4 * h + 3] = x.w;
      }
    } else {
      constexpr uint32_t none = kZero<TYPE> + 1 + kInfBits<TYPE>;  // -inf's bits
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const bool in = c0 + i >= 0 && c0 + i < n;
        const int at = piece * kPer + i;
        if constexpr (TYPE == GM_LOSS_F32) w[i] = in ? static_cast<const uint32_t*>(base)[at] : none;
        else w[i / 2] |= (in ? static_cast<const uint16_t*>(base)[at] : none) << (i & 1 ? 16 : 0);
      }
    }
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = TYPE == GM_LOSS_F32 ? place_of<TYPE>(w[i]) : place_pair(w[i]);
  }
  // f(place) for every class, in any order
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    for (int p = threadIdx.x; p < pieces(); p += blockDim.x) {
      uint32_t q[kPer];
      places(p, q);
#pragma unroll
      for (int i = 0; i < kPer; ++i) f(q[i]);
    }
  }
  __device__ __forceinline__ uint32_t count_at(uint32_t place) const {
    return reinterpret_cast<const uint16_t*>(counts)[place];
  }

  // A group's sum goes to every block; t: lane or thread, one for each block.
  __device__ __forceinline__ void tell(int g, u64 sum, int t) const {
    if (t >= blocks) return;
    if (blocks > 1) put_remote_u64(&sh.coarse[rank][g], t, sum);
    else sh.coarse[0][g] = sum;
  }
  // One warp: the group in which the goal is reached. goal_of: from the sum of all.
  template <class G>
  __device__ __forceinline__ uint32_t group(Search& s, G&& goal_of) const {
    const int lane = threadIdx.x & 31;
    const u64 x = from_each(blocks, [&](int r) { return sh.coarse[r][2 * lane]; });
    const u64 y = from_each(blocks, [&](int r) { return sh.coarse[r][2 * lane + 1]; });
    s.total = s.before + warp_reduce_sum(x + y);
    s.goal = goal_of(s.total);
    return s.step2(x, y);
  }

  // !KEYS: a digit of the border, from the histogram that the block's threads have filled. One warp calls
  // then(search, digit), whose results all threads may read afterwards.
  template <bool MASS, class G, class F>
  __device__ __forceinline__ void digit(u64 before, G&& goal_of, F&& then) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    __syncthreads();
    for (int g = warp; g < kGroups; g += warps) {
      const int b = g * kGroupBins + lane;
      tell(g, warp_reduce_sum(MASS ? u64(low[b]) + (u64(high[b]) << 32) : u64(low[b])), lane);
    }
    meet();
    if (warp == 0) {
      Search s{before, 0, 0, 0};
      const uint32_t g = group(s, goal_of), b = g * kGroupBins + lane;
      const u64 x = from_each(blocks, [&](int r) {
        if (blocks == 1) return MASS ? u64(low[b]) + (u64(high[b]) << 32) : u64(low[b]);
        return MASS ? u64(remote_u32(&low[b], r)) + (u64(remote_u32(&high[b], r)) << 32) : u64(remote_u32(&low[b], r));
      });
      const uint32_t d = g * kGroupBins + s.step(x);
      then(s, d);
    }
    meet();  // histograms and sums are read
  }
  __device__ __forceinline__ void clear() const {
    for (int i = threadIdx.x; i < kBins; i += blockDim.x) low[i] = high[i] = 0;
    __syncthreads();
  }

  // KEYS: the border's D, from the counts of values from place `top` to last_d further on. value(D, count): what so many
  // classes of it add; COUNTS: their number. One warp calls then(search, D); D says nothing where all together fall short of
  // the goal.
  template <bool COUNTS, class V, class G, class F>
  __device__ __forceinline__ void border_of(uint32_t top, uint32_t last_d, V&& value, G&& goal_of, F&& then) const {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int line0 = static_cast<int>(top / kLine), line1 = static_cast<int>(min(top + last_d, 0xffffu) / kLine);
    auto of_line = [&](uint32_t line, uint32_t even, uint32_t odd, u64& x, u64& y) {
      const uint32_t d = line * kLine + 2 * lane - top;  // wraps for values above the largest, whose counts are 0
      x = even ? value(d, even) : 0, y = odd ? value(d + 1, odd) : 0;
    };
    // four lines at a time: eight lanes read one. Weights are formed of lines that hold anything, which the warps then share.
    if constexpr (!COUNTS) {
      if (threadIdx.x == 0) sh.n_lines = 0;
      __syncthreads();
    }
    for (int l = 4 * warp; l < kLines; l += 4 * warps) {
      if constexpr (COUNTS) {
        const uint4 c = reinterpret_cast<const uint4*>(counts)[l * 8 + lane];
        uint32_t n_ = 0;
#pragma unroll
        for (const uint32_t w : {c.x, c.y, c.z, c.w}) n_ += (w & 0xffffu) + (w >> 16);
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) n_ += __shfl_xor_sync(kFull, n_, d);
        if ((lane & 7) == 0) sh.line[l + lane / 8] = n_;
      } else {
        if (lane < 4) sh.line[l + lane] = 0;
        if (l + 3 < line0 || l > line1) continue;
        const uint4 c = reinterpret_cast<const uint4*>(counts)[l * 8 + lane];
        const unsigned some = __ballot_sync(kFull, (c.x | c.y | c.z | c.w) != 0);
        if (lane < 4 && (some >> (8 * lane) & 0xffu) && l + lane >= line0 && l + lane <= line1)
          sh.lines[atomicAdd(&sh.n_lines, 1)] = static_cast<uint16_t>(l + lane);
      }
    }
    if constexpr (!COUNTS) {
      __syncthreads();
      for (int i = warp; i < sh.n_lines; i += warps) {
        const int l = sh.lines[i];
        const uint32_t word = counts[l * 32 + lane];
        u64 x, y;
        of_line(l, word & 0xffffu, word >> 16, x, y);
        x = warp_reduce_sum(x + y);
        if (lane == 0) sh.line[l] = x;
      }
    }
    __syncthreads();
    if (threadIdx.x < kGroups) {
      u64 sum = 0;
#pragma unroll
      for (int i = 0; i < kGroupLines; ++i) sum += sh.line[threadIdx.x * kGroupLines + i];
      for (int r = 0; r < blocks; ++r) tell(threadIdx.x, sum, r);
    }
    meet();
    if (warp == 0) {
      Search s{0, 0, 0, 0};
      const uint32_t g = group(s, goal_of);
      const bool reached = s.total >= s.goal;  // else there is no line to look into
      const u64 x = !reached ? 0 : from_each(blocks, [&](int r) {
        if (lane >= kGroupLines) return u64(0);
        return blocks == 1 ? sh.line[g * kGroupLines + lane] : remote_u64(&sh.line[g * kGroupLines + lane], r);
      });
      const uint32_t line = g * kGroupLines + (reached ? s.step(x) : 0);  // one of the group's: its sums reach the goal
      const u64 both = !reached ? 0 : from_each(blocks, [&](int r) {
        const uint32_t w = blocks == 1 ? counts[line * 32 + lane] : remote_u32(&counts[line * 32 + lane], r);
        return u64(w & 0xffffu) | (u64(w >> 16) << 32);
      });
      u64 even, odd;
      of_line(line, static_cast<uint32_t>(both), static_cast<uint32_t>(both >> 32), even, odd);
      then(s, reached ? line * kLine + s.step2(even, odd) - top : 0);
    }
    meet();  // lines and sums are read
  }
};

template <int TYPE, bool KEYS>
__global__ void __launch_bounds__(1024) k_draw(const __grid_constant__ DrawArgs a) {
  extern __shared__ __align__(16) unsigned char dynamic_mem[];
  __shared__ Shared<KEYS> sh;
  using R = Row<TYPE, KEYS>;
  constexpr int kBytes = TYPE == GM_LOSS_F32 ? 4 : 2, kWords = R::kWords;
  constexpr int kDigits = TYPE == GM_LOSS_F32 ? 3 : 2;
  uint32_t* counts = reinterpret_cast<uint32_t*>(dynamic_mem);
  unsigned char* part_mem = dynamic_mem + (KEYS ? kCountBytes : 0);
  uint32_t blocks;
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(blocks));
  const uint32_t rank = blocks > 1 ? cluster_rank() : 0;
  if (blocks > 1) cluster_arrive();  // waited for before another block's shared memory is used: it must have started
  const int64_t row_i = blockIdx.x / blocks;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (threadIdx.x < kTable) sh.table[threadIdx.x] = kPowers[threadIdx.x];
  if (threadIdx.x == 0) sh.n_few = 0;
  if constexpr (KEYS) {
    for (int i = threadIdx.x; i < kCountBytes / 16; i += blockDim.x) reinterpret_cast<uint4*>(counts)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  } else {
    for (int i = threadIdx.x; i < 2 * kBins; i += blockDim.x) sh.bins[i] = 0;
  }
  chain_wait();

  // the row's rule
  const float temp = a.rule.temperature ? a.rule.temperature[row_i] : a.rule.all_temperature;
  const float top_p = a.rule.top_p ? a.rule.top_p[row_i] : a.rule.all_top_p;
  const float min_p = a.rule.min_p ? a.rule.min_p[row_i] : a.rule.all_min_p;
  int64_t top_k = a.rule.top_k ? a.rule.top_k[row_i] : a.rule.all_top_k;
  const float u = a.u[row_i];

  // ---- the part of the row, and the places of its largest and smallest
  const int first = static_cast<int>(min(int64_t(rank) * a.part, int64_t(a.n_classes)));
  const int n = min(a.part, a.n_classes - first);
  const char* src = static_cast<const char*>(a.z) + (row_i * a.ld + first) * kBytes;
  const int phase = static_cast<int>(reinterpret_cast<uintptr_t>(src) % (kPer * kBytes) / kBytes);
  src -= phase * kBytes;  // piece 0
  uint32_t* const bins = KEYS ? counts : sh.bins;
  const R row{sh, a, counts, bins, bins + kBins, static_cast<int>(blocks), static_cast<int>(rank), a.held ? static_cast<const void*>(part_mem) : src, n, phase};
  const int pieces = row.pieces();
  uint32_t top = 0xffffffffu, last = 0, n_counted = 0;
  constexpr int kAhead = TYPE == GM_LOSS_F32 ? 2 : 4;  // pieces of a thread under way
  for (int p0 = threadIdx.x; p0 < pieces; p0 += kAhead * blockDim.x) {
    uint32_t w[kAhead][kWords];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (p0 + j * static_cast<int>(blockDim.x) < pieces) row.read(src, p0 + j * blockDim.x, w[j]);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int p = p0 + j * blockDim.x;
      if (p >= pieces) break;
      if (a.held) {
#pragma unroll
        for (int h = 0; h < kWords / 4; ++h)
          reinterpret_cast<uint4*>(part_mem)[p * (kWords / 4) + h] =
              make_uint4(w[j][4 * h], w[j][4 * h + 1], w[j][4 * h + 2], w[j][4 * h + 3]);
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t x = w[j][i];
        if constexpr (TYPE == GM_LOSS_F32) {
          top = min(top, x), last = max(last, x);
        } else {  // two at a time, taken apart at the end
          top = __vminu2(top, x), last = __vmaxu2(last, x);
        }
        if constexpr (KEYS) {
          if (x != kNonePlace<TYPE> * 0x10001u) {  // two masked classes
            n_counted += 2;
            atomicAdd(&counts[(x & 0xffffu) >> 1], 1u + (x & 1u) * 0xffffu);
            atomicAdd(&counts[x >> 17], 1u + (x >> 16 & 1u) * 0xffffu);
          }
        }
      }
    }
  }
  if constexpr (TYPE != GM_LOSS_F32) top = min(top & 0xffffu, top >> 16), last = max(last & 0xffffu, last >> 16);
  top = __reduce_min_sync(kFull, top);
  last = __reduce_max_sync(kFull, last);
  if (lane == 0) sh.warp_top[warp] = top, sh.warp_last[warp] = last;
  __syncthreads();
  top = __reduce_min_sync(kFull, sh.warp_top[lane < warps ? lane : 0]);
  last = __reduce_max_sync(kFull, sh.warp_last[lane < warps ? lane : 0]);
  if (blocks > 1) {
    cluster_wait();  // all blocks run; the reading of the row lies between
    if (threadIdx.x < blocks) put_remote_u64(&sh.told_ends[rank], threadIdx.x, (u64(last) << 32) | top);
    cluster_sync_all();
    for (int r = 0; r < blocks; ++r) {
      top = min(top, static_cast<uint32_t>(sh.told_ends[r]));
      last = max(last, static_cast<uint32_t>(sh.told_ends[r] >> 32));
    }
  }

  // KEYS: counts serve while none has passed 16 bits, which their sum would show: a carry takes 65536 away and adds 1 or
  // nothing. Else, with tens of thousands of equal logits, the row is searched by digits.
  bool by_counts = KEYS;
  if (KEYS && a.part > 65535) {
    int off = static_cast<int>(n_counted);
    for (int i = threadIdx.x; i < kCountBytes / 16; i += blockDim.x) {
      const uint4 c = reinterpret_cast<const uint4*>(counts)[i];
#pragma unroll
      for (const uint32_t w : {c.x, c.y, c.z, c.w}) off -= static_cast<int>((w & 0xffffu) + (w >> 16));
    }
    off = __reduce_add_sync(kFull, off);
    if (lane == 0) sh.warp_above[warp] = off;
    __syncthreads();
    off = __reduce_add_sync(kFull, lane < warps ? sh.warp_above[lane] : 0);
    if (blocks > 1) {
      if (threadIdx.x < blocks) put_remote_u64(&sh.told_off[rank], threadIdx.x, off != 0);
      cluster_sync_all();
      for (int r = 0; r < blocks; ++r) off |= static_cast<int>(sh.told_off[r]);
    }
    by_counts = off == 0;
    __syncthreads();
    if (!by_counts) row.clear();
  }

  // log2(e) / T in two parts
  const float c_high = temp > 0.f ? kLog2e / temp : 0.f;
  const float c_low = temp > 0.f ? (fmaf(-c_high, temp, kLog2e) + kLog2eLow) / temp : 0.f;
  const bool fine = top < kNonePlace<TYPE> && top >= kInfPlace<TYPE> && last <= kNonePlace<TYPE> && u >= 0.f && u < 1.f && temp >= 0.f &&
                    temp < INFINITY && c_high < INFINITY && top_k >= 0 && top_p >= 0.f && top_p <= 1.f && min_p >= 0.f && min_p <= 1.f;
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
  const Weigher weigh{top_z, c_high, c_low, top, a.bits, sh.table};
  // the row's results: a class, its place, the sum of what is kept, how many that are
  auto answer = [&](int64_t index, uint32_t place, u64 sum, int64_t n_kept) {
    const Pair l = log_of(sum, -a.bits, sh.table);
    Pair w = {0.f, 0.f};
    if (place != top) {
      const Pair d = sum_of(value_of<TYPE>(place), -top_z);
      w.x = d.x / temp;
      w.low = (fmaf(-w.x, temp, d.x) + d.low) / temp;
    }
    a.index[row_i] = index;
    const Pair x = sum_of(w.x, -l.x);
    a.logprob[row_i] = x.x + (x.low + (w.low - l.low));
    a.kept[row_i] = static_cast<int32_t>(n_kept);
  };
  auto weight = [&](uint32_t d) { return weigh(top + d, value_of<TYPE>(top + d)); };

  // what is not -inf, and passes min-p
  Border border{kNonePlace<TYPE> - top - 1, INT64_MAX};
  uint32_t by_min = border.d;
  if (min_p > 0.f && temp > 0.f && top > kInfPlace<TYPE>) {
    Pair l = times(log_of(min_p, sh.table), temp, 0.f);
    if (!(l.x > -INFINITY)) l = Pair{-INFINITY, 0.f};  // T ln(min_p) past fp32, whose parts would be inf - inf: nothing falls short
    const uint32_t from = place_from<TYPE>(top_z, l.x, l.low);
    by_min = min(by_min, max(from, top) - top);
  } else if (min_p > 0.f) {
    by_min = 0;  // T = 0, or +inf: w is 1 or 0
  }
  // The few classes with D up to `cut`, the rule's kept ones among them: the row's first block takes them as a list and
  // compares each with each, a thread a class.
  auto of_few = [&](uint32_t cut) {
    u64* list = KEYS ? sh.line : reinterpret_cast<u64*>(sh.bins);  // place and class; then weights
    u64* w_few = list + kFew;
    for (int p = threadIdx.x; p < pieces; p += blockDim.x) {
      uint32_t q[kPer];
      row.places(p, q);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (q[i] - top > cut) continue;
        const u64 x = (u64(q[i]) << 32) | static_cast<uint32_t>(first + p * kPer - phase + i);
        if (blocks == 1) list[atomicAdd(&sh.n_few, 1u)] = x;
        else put_remote_u64(&list[add_remote_u32(&sh.n_few, 0, 1u)], 0, x);
      }
    }
    row.meet();
    if (rank != 0) return;
    const int m = static_cast<int>(sh.n_few), i = threadIdx.x;
    const u64 x = i < m ? list[i] : ~u64(0);
    const uint32_t place = static_cast<uint32_t>(x >> 32);
    const u64 w = i < m ? weigh(place, value_of<TYPE>(place)) : 0;
    if (i < m) w_few[i] = w;
    auto sum_all = [&](u64 v) {  // over the block
      v = warp_reduce_sum(v);
      __syncthreads();
      if (lane == 0) sh.warp_sum[warp] = v;
      __syncthreads();
      return warp_reduce_sum(lane < warps ? sh.warp_sum[lane] : u64(0));
    };
    __syncthreads();
    int n_before = 0;
    u64 before = 0;
    if (i < m) {
#pragma unroll 4
      for (int j = 0; j < m; ++j)
        if (list[j] < x) ++n_before, before += w_few[j];  // equal places: by class
    }
    bool kept_here = i < m && (top_k == 0 || n_before < top_k);
    const u64 all = sum_all(kept_here ? w : 0);
    if (top_p < 1.f) {
      bool left;
      const u64 whole = whole_times(top_p, all, left);
      kept_here = kept_here && (n_before == 0 || before < whole + left);
    }
    kept_here = kept_here && place - top <= by_min;
    const u64 total = sum_all(kept_here ? w : 0);
    const int n_kept = __syncthreads_count(kept_here);
    if (i < m) w_few[i] = kept_here ? w : 0;
    __syncthreads();
    bool left;
    const u64 goal = whole_times(u, total, left);
    if (!kept_here) return;
    u64 upto = 0;
#pragma unroll 4
    for (int j = 0; j < m; ++j)
      if (static_cast<uint32_t>(list[j]) <= static_cast<uint32_t>(x)) upto += w_few[j];
    if (upto > goal && upto - w <= goal) answer(static_cast<uint32_t>(x), place, total, n_kept);
  };
  constexpr bool kLong = TYPE == GM_LOSS_F32;
  auto shift_of = [](int g) { return kLong ? (g == 0 ? 21 : g == 1 ? 10 : 0) : (g == 0 ? 5 : 0); };

  // ---- top-k
  if (top_k > 0 && top_k < a.n_classes) {
    auto goal = [&](u64) { return static_cast<u64>(top_k); };
    const u64 few = min(kFew, static_cast<int>(blockDim.x));
    if (KEYS && by_counts) {
      row.template border_of<true>(top, 0xffffu, [](uint32_t, uint32_t count) { return u64(count); }, goal, [&](const Search& s, uint32_t d) {
        const bool all = s.total < s.goal;  // masked classes are not all counted
        if (all) d = 0xffffffffu;
        if (lane == 0) sh.border = Border{d, top_k - static_cast<int64_t>(s.before)}, sh.cut = d, sh.found = (all ? s.total : s.before + s.in) <= few;
      });
    } else {
      uint32_t d = 0;
      u64 before = 0;
#pragma unroll 1
      for (int g = 0; g < kDigits; ++g) {
        const int shift = shift_of(g), done = g > 0 ? shift_of(g - 1) : 0;
        if (g > 0) row.clear();
        row.each([&](uint32_t q) {
          const uint32_t x = q - top;
          if (g == 0 || (x >> done) == (d >> done)) atomicAdd(&row.low[(x - d) >> shift], 1u);
        });
        row.template digit<false>(before, goal, [&](const Search& s, uint32_t x) {
          if (lane == 0) {
            sh.border = Border{d + (x << shift), top_k - static_cast<int64_t>(s.before)}, sh.before = s.before;
            sh.cut = d + (x << shift) + ((1u << shift) - 1), sh.found = s.before + s.in <= few;
          }
        });
        if (sh.found) break;
        d = sh.border.d, before = sh.before;
      }
    }
    if (sh.found) {
      of_few(min(sh.cut, border.d));
      return;
    }
    if (!by_counts && top_p < 1.f) row.clear();
    if (sh.border.d <= border.d) border = sh.border;
  }

  // ---- top-p
  if (top_p < 1.f) {
    // the classes at a border of top-k, of which only some count, come after all others and are not in the sums
    const Border old = border;
    const u64 extra = old.all() ? 0 : weight(old.d) * static_cast<u64>(old.ties);
    auto goal = [&](u64 total) {
      bool left;
      const u64 w = whole_times(top_p, total + extra, left);
      return max(w + left, u64(1));
    };
    // so many of the classes with this very D
    auto at = [&](const Search& s, uint32_t d) {
      const bool stays = s.total < s.goal;  // all others fall short
      if (stays) d = old.d;
      const u64 w = weight(d), from = stays ? s.total : s.before;
      const u64 ties = w ? max(u64(1), (s.goal - from + w - 1) / w) : 1;
      if (lane == 0) sh.border = Border{d, static_cast<int64_t>(ties)};
    };
    if (KEYS && by_counts) {
      row.template border_of<false>(top, old.d, [&](uint32_t x, uint32_t count) {
        return x < old.d || (x == old.d && old.all()) ? weight(x) * count : u64(0);
      }, goal, at);
    } else {
      auto add = [&](uint32_t bin, u64 w) {
        const uint32_t l = static_cast<uint32_t>(w), was = atomicAdd(&row.low[bin], l);
        const uint32_t h = static_cast<uint32_t>(w >> 32) + (was + l < was);
        if (h) atomicAdd(&row.high[bin], h);
      };
      uint32_t d = 0;
      u64 before = 0, reach = 0;
#pragma unroll 1
      for (int g = 0; g < kDigits; ++g) {
        const int shift = shift_of(g), done = g > 0 ? shift_of(g - 1) : 0;
        if (g > 0) row.clear();
        row.each([&](uint32_t q) {
          const uint32_t x = q - top;
          if (x > old.d || (x == old.d && !old.all())) return;
          if (g > 0 && (x >> done) != (d >> done)) return;
          const u64 w = weigh(q, value_of<TYPE>(q));
          if (w) add((x - d) >> shift, w);
        });
        row.template digit<true>(before, [&](u64 total) { return g == 0 ? goal(total) : reach; }, [&](const Search& s, uint32_t x) {
          const bool stays = s.total < s.goal;
          if (stays || g == kDigits - 1) at(s, d + (x << shift));
          if (lane == 0) sh.digit = d + (x << shift), sh.before = s.before, sh.goal = s.goal, sh.found = stays;
        });
        if (sh.found) break;
        d = sh.digit, before = sh.before, reach = sh.goal;
      }
    }
    if (sh.border.d < border.d || sh.border.ties < border.ties) border = sh.border;
  }

  // ---- min-p
  if (by_min < border.d) border = Border{by_min, INT64_MAX};

  // KEYS: the weights of the values that occur in this part, in place of their counts, by D: those up to the border and a
  // 0 after it; where the border lies further on, those nearest to the largest, those nearest to the border, backwards
  // from it, and that of 0. What else lies between, beyond 64 powers of two from either, is rare; `sparse` where there is any.
  // A class at the border has its mark in place of a weight.
  constexpr u64 kTie = u64(1) << 54;  // a thread sums at most 64 weights of 2^46
  const u64* weights = reinterpret_cast<const u64*>(counts);
  constexpr uint32_t kNear = kWeights / 2, kOfZero = kWeights - 2, kNothing = kWeights - 1;
  const bool whole = border.d + 2 <= kWeights;
  uint32_t above = 0, ties = 0;
  bool sparse = false;
  if (KEYS && by_counts) {
    ties = row.count_at(top + border.d);
    // classes above the border, eight places at a time
    uint32_t n_above = 0;
    bool between = false;
    const uint32_t end = top + border.d;  // not this
    for (uint32_t i = top / 8 + threadIdx.x; i * 8 < end; i += blockDim.x) {
      const uint4 c = reinterpret_cast<const uint4*>(counts)[i];
      if ((c.x | c.y | c.z | c.w) == 0) continue;
      const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t q = i * 8 + j, m = j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu, d = q - top;
        if (q >= end) continue;
        n_above += m;
        between = between || (m && !whole && d >= kNear && end - q >= kNear - 2 && q != kZero<TYPE>);
      }
    }
    n_above = __reduce_add_sync(kFull, n_above);
    if (lane == 0) sh.warp_above[warp] = n_above;
    auto d_of = [&](uint32_t i) { return whole || i < kNear ? i : border.d - (i - kNear); };
    u64 occurs = 0;
    const uint32_t entries = whole ? border.d : kOfZero;
    for (uint32_t i = threadIdx.x, j = 0; i < entries; i += blockDim.x, ++j)
      if (row.count_at(top + d_of(i))) occurs |= u64(1) << j;
    sparse = __syncthreads_or(between);
    for (uint32_t i = threadIdx.x, j = 0; i < entries; i += blockDim.x, ++j)
      if (occurs >> j & 1) reinterpret_cast<u64*>(counts)[i] = weight(d_of(i));
    above = __reduce_add_sync(kFull, lane < warps ? sh.warp_above[lane] : 0u);
    __syncthreads();
    if (threadIdx.x == 0) {
      reinterpret_cast<u64*>(counts)[whole ? border.d : kNear] = kTie;
      reinterpret_cast<u64*>(counts)[whole ? border.d + 1 : kNothing] = 0;
      if (!whole) reinterpret_cast<u64*>(counts)[kOfZero] = weigh(kZero<TYPE>, 0.f);
    }
    __syncthreads();
  }

  // ---- sums of what is kept, by warps: a warp takes pieces that follow one another
  const int per_warp = (pieces + warps - 1) / warps;
  const int p0 = min(warp * per_warp, pieces), p1 = min(p0 + per_warp, pieces);
  const u64 w_tie = weight(border.d);
  // weights above the border of a piece, and how many classes are at it
  auto sum_piece = [&](int p, uint32_t& n_ties, uint32_t& n_above) {
    uint32_t q[kPer];
    row.places(p, q);
    u64 x = 0;
    if (KEYS && by_counts && !sparse) {
      if (whole) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x += weights[min(q[i] - top, border.d + 1)];
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const uint32_t d = q[i] - top;
          x += weights[d < kNear ? d : d > border.d ? kNothing : min(kNear + border.d - d, kOfZero)];
        }
      }
      n_ties += static_cast<uint32_t>(x / kTie);
      return x % kTie;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint32_t d = q[i] - top;
      n_ties += d == border.d;
      if (d < border.d) ++n_above, x += weigh(q[i], value_of<TYPE>(q[i]));
    }
    return x;
  };
  u64 sum = 0;
  uint32_t warp_ties = 0, warp_above = 0;
  for (int p = p0 + lane; p < p1; p += 32) sum += sum_piece(p, warp_ties, warp_above);
  sum = warp_reduce_sum(sum);
  warp_ties = __reduce_add_sync(kFull, warp_ties);
  if (!by_counts) warp_above = __reduce_add_sync(kFull, warp_above);
  if (lane == 0) {
    sh.warp_sum[warp] = sum, sh.warp_ties[warp] = warp_ties;
    if (!by_counts) sh.warp_above[warp] = warp_above;
  }
  __syncthreads();
  u64 sum_before, total;  // of this warp in its block, of the block
  uint32_t ties_before;
  {
    const u64 x = lane < warps ? sh.warp_sum[lane] : 0;
    const uint32_t t = lane < warps ? sh.warp_ties[lane] : 0;
    const u64 x_to = warp_inclusive_scan(x);
    const uint32_t t_to = warp_inclusive_scan(t);
    sum_before = __shfl_sync(kFull, x_to - x, warp), ties_before = __shfl_sync(kFull, t_to - t, warp);
    total = __shfl_sync(kFull, x_to, 31), ties = __shfl_sync(kFull, t_to, 31);
    if (!by_counts) above = __reduce_add_sync(kFull, lane < warps ? sh.warp_above[lane] : 0u);
  }
  int64_t all_ties = ties, kept = above;
  u64 part_from = 0, part_sum = total;  // of the row's sum: before this block's part, of the part
  int64_t part_ties = ties, part_ties_from = 0;
  if (blocks > 1) {
    if (threadIdx.x < blocks) {
      put_remote_u64(&sh.told[rank].sum, threadIdx.x, total);
      put_remote_u64(&sh.told[rank].ties, threadIdx.x, (u64(above) << 32) | ties);
    }
    cluster_sync_all();
    total = 0, all_ties = kept = 0;
    for (int r = 0; r < blocks; ++r) {
      if (r == rank) part_from = total, part_ties_from = all_ties;
      total += sh.told[r].sum, all_ties += sh.told[r].ties, kept += sh.told[r].above;
    }
  }
  const int64_t most = min(border.ties, all_ties);
  total += static_cast<u64>(most) * w_tie;
  kept += most;
  bool left;
  const u64 goal = whole_times(u, total, left);  // more than u * total: more than its whole part
  auto tied = [&](int64_t before, int64_t n_ties) {  // of n_ties after `before` others, how many are kept
    return static_cast<u64>(max(int64_t(0), min(most - before, n_ties)));
  };
  part_sum += tied(part_ties_from, part_ties) * w_tie;
  part_from += tied(0, part_ties_from) * w_tie;
  if (part_from > goal || part_from + part_sum <= goal) return;  // in another block's part
  sum_before += part_from + tied(part_ties_from, ties_before) * w_tie;
  sum += tied(part_ties_from + ties_before, warp_ties) * w_tie;

  // ---- the one warp in which the sum passes u: 32 pieces at a time, then the lane, then the class
  if (sum_before > goal || sum_before + sum <= goal) return;
  int64_t tie = part_ties_from + ties_before;
  u64 at = sum_before;
  for (int p = p0; p < p1; p += 32) {
    u64 own = 0;
    uint32_t own_ties = 0, unused = 0;
    if (p + lane < p1) own = sum_piece(p + lane, own_ties, unused);
    __syncwarp();
    const uint32_t ties_to = warp_inclusive_scan(own_ties);
    int64_t tie_at = tie + ties_to - own_ties;
    own += tied(tie_at, own_ties) * w_tie;
    const u64 to = warp_inclusive_scan(own);
    const unsigned passed = __ballot_sync(kFull, at + to > goal);
    if (!passed) {
      at += __shfl_sync(kFull, to, 31);
      tie += __shfl_sync(kFull, ties_to, 31);
      continue;
    }
    if (lane != __ffs(passed) - 1) return;
    at += to - own;
    uint32_t q[kPer];
    row.places(p + lane, q);
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      uint32_t place = q[0];  // q[i], in registers
#pragma unroll
      for (int j = 1; j < kPer; ++j) place = i == j ? q[j] : place;
      const uint32_t d = place - top;
      u64 w = 0;
      if (d < border.d) w = weigh(place, value_of<TYPE>(place));
      else if (d == border.d) w = tied(tie_at, 1) * w_tie, ++tie_at;
      at += w;
      if (w && at > goal) {
        answer(first + (p + lane) * kPer - phase + i, place, total, kept);
        return;
      }
    }
    return;
  }
}

// ---- host ---------------------------------------------------------------------------------------------
constexpr int64_t kMostClasses = int64_t(1) << 24;
constexpr int kHeldBytes = 204800;          // of a block's shared memory: counts, and its part of the row
constexpr int64_t kSharedBytes = 90112;     // of a part, of which two lie in an SM's shared memory
// Rows of 16 bits are searched by counts of all values, or by digits. Counting takes one atomic a class, and 128 KB to clear and
// to walk, so that an SM has one row at a time; digits take up to two atomics, and for top-p a weight, a class. us, counts /
// digits: top-p at 512 x 8192: 62 / 42, 12288: 64 / 75, 20000: 70 / 101, 131072: 175 / 474; top-k = 50 at 20000: 54 / 35,
// 50000: 73 / 73, 131072: 138 / 184; 1 x 131072: top-p 23 / 31, top-k 19 / 19. Without either there is no border: at
// 512 x 131072 364 / 296.
constexpr int64_t kLeastShared = 12288;   // with top-p
constexpr int64_t kLeastCounted = 49152;  // with top-k alone

// Threads of a block that has `part` classes, `bytes` of them, where an SM gets `rows` of such blocks: the 1024 that its
// registers hold, shared between the rows, 8 to 32 classes a thread: a block's steps wait for one another, so that blocks
// side by side fill an SM better than threads of one. By powers of two, of which two, four or eight blocks
// fill it. 2000 x 12288 bf16, top-k = 50: 84 us with 512 threads, 134 with 768 (one block an SM); 300 x 8192 top-p: 35 with 512,
// 64 with 128.
int64_t threads_for(int64_t part, int64_t bytes, int64_t rows) {
  auto power_from = [](int64_t x) {
    int64_t p = 128;
    while (p < x && p < 1024) p *= 2;
    return p;
  };
  if (bytes > kSharedBytes) return power_from(div_up(part, kPer));
  const int64_t least = std::min<int64_t>(power_from(div_up(part, 4 * kPer)), 512), most = power_from(div_up(part, kPer));
  int64_t threads = most;
  while (threads > least && threads * rows > 1024) threads /= 2;
  return threads;
}

template <int TYPE, bool KEYS>
cudaError_t launch_as(DrawArgs& a, int64_t n_rows, int sms, cudaStream_t s) {
  const int64_t es = TYPE == GM_LOSS_F32 ? 4 : 2, n = a.n_classes, room = kHeldBytes - (KEYS ? kCountBytes : 0);
  const cudaError_t e = cudaFuncSetAttribute(k_draw<TYPE, KEYS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeldBytes);
  if (e != cudaSuccess) return e;
  // Blocks of a row: until it fits, or the SMs have work. 131072 bf16 by 1, 2, 4, 8 blocks, us: one row 48, 36, 27, 26;
  // 40 rows 48, 38, 45, 59.
  int blocks = 1;
  auto part = [&] { return up(div_up(n, blocks), kPer); };
  while (blocks < kMostCluster && ((!KEYS && (part() + kPer) * es > room) || (n_rows * blocks * 2 <= sms && part() > 8192))) blocks *= 2;
  if (n_rows * blocks > INT32_MAX) return cudaErrorInvalidValue;  // more bytes than any device has
  a.part = static_cast<int>(part());
  a.held = (part() + kPer) * es <= room;
  const int64_t threads = KEYS ? 1024 : threads_for(part(), (part() + kPer) * es, div_up(n_rows * blocks, sms));
  const size_t smem = (KEYS ? kCountBytes : 0) + (a.held ? static_cast<size_t>((part() + kPer) * es) : 0);
  return launch_chained(k_draw<TYPE, KEYS>, static_cast<unsigned>(n_rows * blocks), static_cast<unsigned>(threads), smem, s, blocks, a);
}

template <int TYPE>
cudaError_t launch(DrawArgs& a, int64_t n_rows, int sms, cudaStream_t s) {
  if constexpr (TYPE != GM_LOSS_F32) {
    const bool warm = a.rule.temperature || a.rule.all_temperature != 0.f, by_share = a.rule.top_p || a.rule.all_top_p < 1.f;
    const bool border = by_share || a.rule.top_k || a.rule.all_top_k > 0;
    if (warm && border && a.n_classes >= (by_share ? kLeastShared : kLeastCounted)) return launch_as<TYPE, true>(a, n_rows, sms, s);
  }
  return launch_as<TYPE, false>(a, n_rows, sms, s);
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
