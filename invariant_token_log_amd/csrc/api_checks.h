// Host-side argument checks and workspace helpers of token_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>

#include "invariant_logp.h"
#include "launch.h"

namespace itl {

constexpr size_t kWsAlign = 256;

inline size_t ws_round(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }

inline bool ws_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && have >= need && reinterpret_cast<uintptr_t>(ws) % kWsAlign == 0);
}

inline int dtype_size(int32_t dtype) { return dtype == LOGP_F32 ? 4 : 2; }

inline bool known_dtype(int32_t dtype) {
  return dtype == LOGP_F32 || dtype == LOGP_BF16 || dtype == LOGP_F16;
}

// Rows whose start and stride are multiples of 16 bytes.
inline bool rows_aligned16(const void* p, int64_t ld, int size) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * size) % 16 == 0;
}

// Chunks a lane holds of a tile of w columns, or 0 for a width that is not
// offered for the type.
inline int tile_chunks(int32_t dtype, int32_t w) {
  const int per = dtype == LOGP_F32 ? 256 : 512;
  if (w < per || w % per) return 0;
  const int c = w / per;
  return (c == 1 || c == 2 || c == 4 || c == 8 || c == 16) ? c : 0;
}

// A temperature is usable when it is finite, > 0 and its reciprocal rounded
// to fp32 is finite too.
inline float reciprocal_temperature(float t) {
  return static_cast<float>(1.0 / static_cast<double>(t));
}
inline bool usable_temperature(float t) {
  return std::isfinite(t) && t > 0.0f && std::isfinite(reciprocal_temperature(t));
}

inline int32_t launch_status() {
  return hipGetLastError() == hipSuccess ? LOGP_OK : LOGP_ERR_HIP;
}

}  // namespace itl
