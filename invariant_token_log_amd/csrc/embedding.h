// Internal launchers of the embedding (not part of the C ABI).  Arguments are
// checked by the callers in layer_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace itl {

constexpr int64_t kMaxEmbedTokens = int64_t{1} << 24;  // of a gradient
constexpr int64_t kMaxEmbedWidth = int64_t{1} << 24;

// out[i] = rne(scale table[tokens[i]]); zeros for `ignore`, NaN for any other
// token outside [0, v).
void launch_embedding(int dtype, const void* table, int64_t ld_t, int64_t v, int64_t h,
                      Targets tokens, int64_t n, int64_t ignore, float scale, void* out,
                      int64_t ld_o, hipStream_t s);

// The same from 4-bit rows (fp4.h); out of out_dtype.
void launch_embedding_fp4(const uint8_t* data, int64_t ld_d, const uint8_t* scales, int64_t ld_s,
                          int64_t v, int64_t h, Targets tokens, int64_t n, int64_t ignore,
                          float scale, int out_dtype, void* out, int64_t ld_o, hipStream_t s);

// dtable[t] = rne([dtable[t] +] scale sum of dy[i] over i with tokens[i] = t, in
// ascending i).  dy of dtype, dtable fp32 or of dtype (f32_out).  Without
// accumulate every row of dtable [v, ld_t] is written, with it the rows of the
// given tokens alone.  ws: embedding_bwd_bytes(...) bytes.
int64_t embedding_bwd_bytes(int64_t n, int64_t v, int64_t h);
void launch_embedding_bwd(int dtype, const void* dy, int64_t ld_y, Targets tokens, int64_t n,
                          int64_t v, int64_t h, int64_t ignore, float scale, bool f32_out,
                          bool accumulate, void* dtable, int64_t ld_t, char* ws, hipStream_t s);

}  // namespace itl
