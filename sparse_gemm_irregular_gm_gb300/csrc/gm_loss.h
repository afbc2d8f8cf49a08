// gm_loss.h -- shared by the translation units of the losses over a large class
// table (gm_loss.cu: kernels that read rows and entries, host driver;
// gm_loss_prod.cu: the tensor-core products).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gm_internal.h"
#include "gm_losses.h"

namespace gm {

// Launches k so that its start overlaps the end of the kernel before it; k calls chain_wait
// (gm_umma.cuh). cluster: blocks of a cluster.
template <class... P, class... A>
cudaError_t launch_chained(void (*k)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, unsigned cluster,
                           A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k, static_cast<A&&>(args)...);
  note_launch();
  return e;
}

constexpr float kLog2e = 1.4426950408889634f;

// Bits of a status word: the device's, which gm_loss_status reads, or a checked call's own.
enum : int {
  kLossTimeout = 1,    // a bounded wait inside a kernel gave up
  kLossBadTarget = 2,  // a target outside [0, n_classes) that is not the ignored one
  kLossBadTeacher = 4  // a malformed teacher row: see gm_distill_forward
};

constexpr int kMostBlocks = 256;  // of a product; a word of 8 a lane says whether any gave up

// Products the kernel makes and what it does with a finished tile.
enum class Prod {
  kStats,  // Z = H W^T: each row's maximum and sums of exponentials over half a tile's columns
  kGrad,   // Z = H W^T again: G = dloss/dZ in 16 bits (three planes of bf16 for fp32 operands)
  kDh,     // G W
  kDw      // G^T H
};

// Where a row's target stands.
struct Targets {
  const void* t;    // null: no labels
  bool is64;
  int64_t ignore;
  int64_t n_cls;
};

__device__ __forceinline__ int64_t check_target(const Targets& t, int64_t v) {  // -1: ignored, -2: out of range
  return v == t.ignore ? -1 : (v >= 0 && v < t.n_cls) ? v : -2;
}

// What a backward call is given of each row.
struct RowGrads {
  Targets tgt;
  const float *lse, *g_loss, *g_lse;  // with labels; g_lse may be null
  const int32_t* ent_len;             // null: no teacher
  const float *lse_t, *g_kl;
  float inv_t;
};
// The row's values as they are in memory, read well before they are used.
struct RowRaw {
  int64_t t;
  float lse, g_loss, g_lse, lse_t, g_kl;
  int32_t len;
};
__device__ __forceinline__ int64_t raw_target(const Targets& t, int64_t row) {
  return t.is64 ? static_cast<const int64_t*>(t.t)[row] : static_cast<const int32_t*>(t.t)[row];
}
__device__ __forceinline__ RowRaw row_raw(const RowGrads& r, int64_t row) {
  RowRaw x = {0, 0.f, 0.f, 0.f, 0.f, 0.f, 0};
  if (r.tgt.t) {
    x.t = raw_target(r.tgt, row);
    x.lse = r.lse[row];
    x.g_loss = r.g_loss[row];
    if (r.g_lse) x.g_lse = r.g_lse[row];
  }
  if (r.ent_len) {
    x.len = r.ent_len[row];
    x.lse_t = r.lse_t[row];
    x.g_kl = r.g_kl[row];
  }
  return x;
}
// G_ij = a e^(z - lse) - gl [j = t] + b (e^(z / T - lse_t) - q)
struct RowCoef {
  float lse, a, gl, lse_t, b;
  int64_t t;
};
__device__ __forceinline__ RowCoef row_coef(const RowGrads& r, const RowRaw& x) {
  RowCoef c = {0.f, 0.f, 0.f, 0.f, 0.f, -1};
  if (r.tgt.t) {
    c.t = check_target(r.tgt, x.t);
    c.gl = c.t >= 0 ? x.g_loss : 0.f;
    c.lse = x.lse;
    c.a = c.t == -2 ? 0.f : c.gl + x.g_lse;  // an ignored row has an lse like any other
  }
  if (r.ent_len) {
    c.lse_t = x.lse_t;
    c.b = x.len > 0 ? x.g_kl * r.inv_t : 0.f;
  }
  return c;
}

// What the finished tile of a product is combined with.
struct ProdArgs {
  // tiles: m_tiles * n_tiles * splits, in groups of `group` row tiles, the column tiles
  // of a group one after another, its row tiles innermost
  int m_tiles, n_tiles, splits, group;
  int k_blocks;      // blocks of 64 along the summed dimension
  int k_per_split;   // blocks of a split
  int chunk;         // blocks summed in TMEM at a time (16-bit logits)
  int planes;        // 1, or 3: each fp32 operand is the sum of three bf16 planes
  // Planes of G: 3 of bf16 with fp32 operands; with 16-bit ones 1, rounded, or for at most 128 rows
  // 2, value and remainder: there the gradients' products wait for W and dW, a second product
  // a stage costs no time, and a gradient is then rounded once, like the plain form's.
  int g_planes;
  bool bf16;
  int b_row0;        // first row of W's map
  int64_t m, n;      // rows and columns of the result
  int* status;
  uint8_t* lost;     // [kMostBlocks] of this call: 1 where a block gave up
  bool lost_first;   // the call's first product: writes all of them
  // kStats, kGrad
  int64_t cls0;      // class of column 0
  Targets tgt;
  const int64_t* ent_start;  // teacher: first entry of each row, its entries, their class and probability
  const int32_t* ent_len;
  const int2* ents;
  float inv_t, c_t;  // 1 / T, log2(e) / T
  float4* part;      // [half tile][row]: max, sum e^(z - max), sum e^((z - max) / T), sum q z
  int64_t part_ld;
  float* z_t;        // [row] logit of the target
  RowGrads row;
  const unsigned* weights;  // f16: bits of the largest and the smallest of the rows' weights (null: no scale)
  int near;                 // exponents that weights of one scale may lie apart
  // kDh, kDw
  bool acc;          // the map of results is one of fp32 partial sums (by split), added to with acc_add
  bool acc_add;
  bool by_tma;       // results go out by their map; else by plain stores to out
  void* out;
  int64_t out_ld;
  int out_type;      // GM_LOSS_*
};

// Scales of G in f16, whose range is too short for small probabilities times small weights: powers
// of two that bring the largest |G| possible, a row's weight, into [2^13, 2^14). What lies under
// 2^-14 then loses bits, at most half of 2^-24 each: 2^-38 of the weight. While all rows' weights lie
// within 2^near of the largest, its scale serves them all; near is such that the classes of a row
// together lose no more than 2^-11 of its weight, f16's own rounding. Otherwise G is kept twice: with a
// scale for each row for dH, whose rows are sums of their own, and with the largest weight's for dW.
__device__ __forceinline__ float weight_of(const RowCoef& c) { return fabsf(c.a) + fabsf(c.gl) + fabsf(c.b); }
__device__ __forceinline__ float scale_for(float weight) {
  if (!(weight > 0.0f) || !(weight < 3.0e38f)) return 1.0f;
  int e;
  frexpf(weight, &e);
  e = 14 - e;
  return ldexpf(1.0f, e < -100 ? -100 : e > 100 ? 100 : e);
}
struct Scales {
  float all = 1.0f;
  bool apart = false;
  __device__ __forceinline__ explicit Scales(const ProdArgs& g) {
    if (!g.weights) return;
    const unsigned most = g.weights[0], least = g.weights[1];
    all = scale_for(__uint_as_float(most));
    apart = static_cast<int>(most >> 23) - static_cast<int>(least >> 23) > g.near;
  }
  __device__ __forceinline__ float of(const RowCoef& c) const { return apart ? scale_for(weight_of(c)) : all; }
};

struct ProdMaps {
  CUtensorMap a, b, o;  // operands, result, boxes of 32 rows (kGrad: of
                        // prod_grad_row_bytes; kDh, kDw with by_tma: of 128 bytes)
};
// Box height of the operands' maps (rows of a K-major box; MN-major boxes are 64 by 64).
int prod_box_rows_a();
int prod_box_rows_b(int cg, int bn);
// Columns of a tile: of the logits' products, and of the gradients' ones (rows: of their result).
int prod_logits_cols(int cg, int planes);
int prod_sums_cols(int64_t dim, int64_t rows, int planes);
int prod_grad_row_bytes(int planes, int chunk, int k_blocks);
// Launches a product; cg: blocks a tile (1: 128 rows, 2: 256), bn: columns of a tile (64, 128 or 256).
cudaError_t launch_prod(Prod kind, int cg, int bn, const ProdMaps& maps, const ProdArgs& a, int num_sms,
                        cudaStream_t s);

// ---- few rows (gm_loss_skinny.cu) --------------------------------------------------------
constexpr int64_t kSkinnyDim = 4096;  // elements of a row of H at most: H and the sums of dH fit a block
int skinny_rows(int type);            // rows at most
struct SkinnyArgs {
  const void *h, *w;
  int64_t h_ld, w_ld, dim, n_cls;
  int n;
  // set by the launch: classes of a warp (forward), of a block (backward), of a warp at a time
  int64_t per_warp, per_block;
  int take;
  Targets tgt;
  const int64_t* ent_start;     // teacher; ent_len null: none
  const int32_t* ent_len;
  const int2* ents;
  float inv_t, c_t;
  int* status;
  float4* part;                 // forward: [block][row]
  float* z_t;
  RowGrads row;                 // backward
  void *dh, *dw;                // null: not wanted (dh: whether acc is written)
  int64_t dw_ld;
  float* acc;                   // [block][row][dim]
};
// Blocks of a launch at most, for the workspace.
int skinny_most_blocks(int64_t n_cls, int sms);
// vec: elements of a load of W (and store of dW): 16 bytes, 4 or one element, as rows allow.
// *blocks: at most so many, then how many there are.
cudaError_t launch_skinny(const SkinnyArgs& a, int type, bool backward, int vec, int* blocks, cudaStream_t s);

}  // namespace gm
