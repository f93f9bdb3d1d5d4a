// Internal launchers of the layer norm (not part of the C ABI).  Arguments are
// checked by the callers in layer_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dropout.h"
#include "rms_norm.h"  // NormRows, kMaxNorm

namespace itl {

// drop null: none.  mean, rstd: fp32 [n] or null.  bias null: none.
void launch_layer_norm(int dtype, const NormRows& rows, const Drop* drop, const void* weight,
                       const void* bias, int64_t n, int64_t h, float eps, void* y, int64_t ld_y,
                       float* mean, float* rstd, hipStream_t s);

struct LayerNormGrad {
  const void* s;
  int64_t ld_s;
  const void* weight;
  const float* mean;
  const float* rstd;
  const void* dy;
  int64_t ld_dy;
  const void* ds;  // or null
  int64_t ld_ds;
  const Drop* drop;  // or null
  void* dx;
  int64_t ld_dx;
  void* dres;  // with drop: the gradient before dropout's, or null
  int64_t ld_dres;
  void* dweight;  // or null
  void* dbias;    // or null
};

// Partial rows (of 2 h floats each) of the weight's and bias's gradients.
int64_t layer_norm_bwd_blocks(int dtype, int64_t n, int64_t h);

void launch_layer_norm_bwd(int dtype, const LayerNormGrad& g, int64_t n, int64_t h, float* partial,
                           hipStream_t s);

}  // namespace itl
