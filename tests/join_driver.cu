// What k_linear_join makes of a product's parts, beside a `lost` array that a test fills (a product that gives up cannot be had on demand).
#include "gm_linear.cu"

extern "C" int join_parts(const float* acc, int splits, int64_t rows, int64_t outs, int64_t acc_ld, int act, const float* residual,
                          float* y, float* z, const uint8_t* lost) {
  using namespace gm;
  LinearEnd e = {};
  e.act = act;
  e.residual = residual;
  e.residual_ld = outs;
  e.keep = z != nullptr;
  e.z = z;
  e.z_ld = outs;
  const cudaError_t rc = launch_chained(k_linear_join, grid_for(rows * (acc_ld / 4), 256), 256, 0, nullptr, 1, acc, splits, rows, outs, acc_ld, e,
                                        static_cast<void*>(y), outs, static_cast<int>(GM_LOSS_F32), outs % 4 == 0, lost);
  return rc == cudaSuccess ? static_cast<int>(cudaDeviceSynchronize()) : static_cast<int>(rc);
}
