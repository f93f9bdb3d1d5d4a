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

// Up to this many rows the products read the 4-bit rows themselves, 97 us for
// every 64 at V = 151936, H = 4096; more rows take the bf16 kernels on a decoded
// copy, 256 us and 450 for every 512 (448 rows: 680 us against 716, 512 rows: 776
// against 744).
constexpr int64_t kFp4Direct = 448;

// The decoded copy, K32-blocked with round_up(v, 256) rows (those past v
// zeros), as launch_linear_partials takes it (wblk): exact.
int64_t fp4_decoded_bytes(int64_t v, int64_t h);
void launch_fp4_decode(const Fp4Weight& w, int64_t v, int64_t h, uint16_t* out, hipStream_t s);

// launch_linear_partials on a 4-bit weight, the same bits as on its decoded
// copy.
void launch_fp4_partials(const uint16_t* hidden, int64_t ld_h, const Fp4Weight& w, int64_t n,
                         int64_t h, int64_t v, Targets targets, int64_t ignore, float* pm,
                         float* ps, float* pt, float inv_t, int32_t round_bf16, float* pw, void* z,
                         int32_t z_bf16, int64_t ld_z, hipStream_t s);

}  // namespace itl
