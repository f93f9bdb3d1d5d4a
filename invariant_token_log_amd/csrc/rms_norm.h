// Internal launchers of the root-mean-square norm (not part of the C ABI).
// Arguments are checked by the callers in token_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace itl {

constexpr int64_t kMaxNorm = 65536;  // longest row

struct NormRows {
  const void* x;
  int64_t ld_x;
  const void* residual;  // or null
  int64_t ld_r;
  void* sum;  // or null
  int64_t ld_s;
};

// y (of dtype, or 8-bit rows with scale when q8) and rstd (or null); weight
// null (q8 only): no norm.
void launch_rms_norm(int dtype, const NormRows& rows, const void* weight, int64_t n, int64_t h,
                     float eps, void* y, int64_t ld_y, float* scale, float* rstd, bool q8,
                     hipStream_t s);

// Partial rows of the weight gradient.
int64_t norm_bwd_blocks(int64_t n, int64_t h);

void launch_rms_norm_bwd(int dtype, const void* s, int64_t ld_s, const void* weight,
                         const float* rstd, const void* dy, int64_t ld_dy, const void* ds,
                         int64_t ld_ds, int64_t n, int64_t h, void* dx, int64_t ld_dx,
                         void* dweight, float* partial, hipStream_t stream);

}  // namespace itl
