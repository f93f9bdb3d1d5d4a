// Internal launchers of the token operators (not part of the C ABI).
// Arguments are checked by the callers in token_api.hip before any of these
// runs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace itl {

constexpr int kMaxTokens = 256;  // given tokens a row
constexpr int kMaxTop = 64;      // alternatives a row (one a lane)
constexpr int kMaxEntries = kMaxTokens + kMaxTop;

// The given tokens of every row: [n, m] int64 or int32, contiguous.
struct TokenView {
  const void* p;
  int32_t is32;
  int64_t m;
  int64_t ignore;
  __host__ __device__ __forceinline__ int64_t at(int64_t r, int64_t i) const {
    return is32 ? static_cast<int64_t>(static_cast<const int32_t*>(p)[r * m + i])
                : static_cast<const int64_t*>(p)[r * m + i];
  }
};

// The alternatives whose gradient comes in: [n, k] ids, -1 = none.
struct TopView {
  const int64_t* ids;
  int64_t k;
};

struct TokenOut {
  float* logp;       // [n, m]
  float* lse;        // [n] or null
  float* ent;        // [n] or null
  float* top_logp;   // [n, k]
  int64_t* top_ids;  // [n, k]
};

// Group maxima of one streamed row.
int64_t token_groups(int chunks, int64_t ntiles);

// Row-major [n, T] tile statistics of the streamed logits (pw null: no
// entropy moment) and, unless gm is null, the order keys of the group maxima
// [n, token_groups].
void launch_token_partials(int dtype, bool vec, int chunks, const void* logits, int64_t ld,
                           int64_t n, int64_t v, const TokenView& tok, int ntiles, float* pm,
                           float* ps, float* pw, uint32_t* gm, hipStream_t s);

// Merge, alternatives and outputs.  head_tile 256 or 128: gm is the [n, T]
// table of an LM head's tile maxima (x then holds fp32 or, at 256, bf16
// logits); 0: the streamed rows' keys.  x null: m = 1, top_k = 0, and pt
// holds the token's logit.
void launch_token_finish(int dtype, bool vec, int head_tile, const void* x, int64_t ld,
                         float inv_t, const float* pt, int64_t n, int64_t v, const TokenView& tok,
                         int ntiles, const float* pm, const float* ps, const float* pw,
                         const void* gm, int64_t groups, int top_k, const TokenOut& out,
                         hipStream_t s);

// Gradient of the logits (ent null: no entropy term; grad null: zero).
void launch_token_bwd(int dtype, bool vec, const void* logits, int64_t ld, int64_t n, int64_t v,
                      const TokenView& tok, const TopView& alt, const float* lse,
                      const float* grad, const float* grad_top, const float* ent,
                      const float* gent, void* dlogits, int64_t ld_out, hipStream_t s);

// act[r] = -1 (active) or -2 (padding row); gsum[r] (unless null) = the sum
// of the row's entry gradients.
void launch_token_rows(int64_t n, const TokenView& tok, const TopView& alt, const float* grad,
                       const float* grad_top, int32_t* act, float* gsum, hipStream_t s);

// What the fused backward adds to dz at the entries' columns.
struct TokenDz {
  TokenView tok;
  TopView alt;
  const float* logp;      // [n, m] from the forward
  const float* top_logp;  // [n, k] from the forward
  const float* grad;
  const float* grad_top;
  const float* gsum;
};
void launch_token_dz(const TokenDz& t, int64_t n, int64_t v, float inv_t, const float* ent,
                     const float* gent, int64_t c0, int64_t cols, uint16_t* dz, hipStream_t s);

}  // namespace itl
