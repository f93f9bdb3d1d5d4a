// Internal launcher of the 8-bit LM head (not part of the C ABI).  Arguments
// are checked by the callers in token_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace itl {

constexpr int kQ8Tile = 128;  // vocabulary columns per statistic tile
constexpr int64_t kMaxQ8Stride = int64_t{1} << 23;  // bytes between operand rows

// Tile statistics [n, T] (T = ceil(v / kQ8Tile), row-major), the target logits of
// the active rows and, unless z is null, the unscaled logits [n, ld_z] fp32
// of the 8-bit head: logits = (hidden weight^T) hs[r] ws[j]; hidden [n, ld_h]
// and weight [v, ld_w] e4m3, 16-byte aligned rows, h a multiple of 64.  pw
// null: no entropy moment.  scratch: q8_fwd_scratch_bytes(n, h) bytes.
void launch_q8_partials(const uint8_t* hidden, int64_t ld_h, const float* hs,
                        const uint8_t* weight, int64_t ld_w, const float* ws, int64_t n, int64_t h,
                        int64_t v, Targets targets, int64_t ignore, float* pm, float* ps,
                        float* pt, float inv_t, float* pw, float* z, int64_t ld_z, char* scratch,
                        hipStream_t s);

int64_t q8_fwd_scratch_bytes(int64_t n, int64_t h);

}  // namespace itl
