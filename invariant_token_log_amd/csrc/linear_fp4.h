// Internal launcher of the 4-bit LM head (not part of the C ABI).  Arguments
// are checked by the callers in token_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace itl {

// A 4-bit weight (fp4.h): [v, ld_d] and [v, ld_s] bytes, data rows 16-byte
// aligned.
struct Fp4Weight {
  const uint8_t* data;
  int64_t ld_d;
  const uint8_t* scales;
  int64_t ld_s;
};

// Bytes between the weight's rows, elements between the hidden rows, at most.
constexpr int64_t kMaxFp4Stride = int64_t{1} << 23;
constexpr int64_t kMaxHiddenStride = int64_t{1} << 25;

// launch_linear_partials on a 4-bit weight, the same bits as on the bf16 weight
// that it stands for.  hb: linear_fwd_blocked_bytes(n, h) bytes.
void launch_fp4_partials(const uint16_t* hidden, int64_t ld_h, const Fp4Weight& w, int64_t n,
                         int64_t h, int64_t v, Targets targets, int64_t ignore, float* pm,
                         float* ps, float* pt, float inv_t, int32_t round_bf16, float* pw, void* z,
                         int32_t z_bf16, int64_t ld_z, uint16_t* hb, hipStream_t s);

}  // namespace itl
