// gm_host.h -- host helpers shared by the dense operators (gm_loss.cu, gm_linear.cu, gm_norm.cu,
// gm_draw.cu): rounding, alignment, one call's workspace, device facts, TMA maps.
#pragma once

#include <algorithm>
#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stdint.h>

#include "gm_internal.h"
#include "gm_losses.h"

namespace gm {

inline int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
inline int64_t div_up(int64_t x, int64_t m) { return (x + m - 1) / m; }
inline int64_t elem_bytes(int32_t type) { return type == GM_LOSS_F32 ? 4 : 2; }
inline bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

constexpr int64_t kMostIndex = (int64_t(1) << 31) - 256;  // tile coordinates are int32
constexpr int64_t kMostLd = int64_t(1) << 36;

// One workspace block, carved in order.
struct Arena {
  DevBuf<unsigned char> buf;  // from the hooks, unless the caller brought memory
  unsigned char* p = nullptr;
  size_t used = 0;
  gm_status open(void* workspace, int64_t workspace_bytes, cudaStream_t s) {
    if (workspace) {
      if (static_cast<int64_t>(used) > workspace_bytes) return GM_ERR_WORKSPACE;
      p = static_cast<unsigned char*>(workspace);
      return GM_OK;
    }
    if (!buf.alloc(used, s)) return GM_ERR_OOM;
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

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

// SMs of the current device (at most `most`), looked up once a device; 0: the lookup failed.
inline int sm_count(int most) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n <= 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  }
  return std::min(n, most);
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiled encode_fn() {
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
inline bool encode(CUtensorMap* m, const Operand& o, int box_rows, int row_bytes = 128) {
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

}  // namespace gm
