// C ABI of the embedding, dropout, the layer norm and 4-bit rows
// (include/invariant_layers.h): argument checks (all before any HIP call) and
// launches.
#include "invariant_layers.h"

#include "api_checks.h"
#include "dropout.h"
#include "embedding.h"
#include "fp4.h"
#include "layer_norm.h"

namespace {

using itl::known_dtype;
using itl::rows_aligned16;

int32_t check_drop(double p, int64_t draw, int64_t first_row) {
  if (!(p >= 0.0 && p <= 1.0) || draw < 0 || draw >= (int64_t{1} << 32) || first_row < 0 ||
      first_row > INT64_MAX - INT32_MAX)
    return LOGP_ERR_VALUE;
  return LOGP_OK;
}

int32_t check_embedding(int64_t v, int64_t h, int32_t token_dtype, int64_t n, float scale) {
  if (token_dtype != LOGP_I64 && token_dtype != LOGP_I32) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || v < 1 || v > (int64_t{1} << 31) || h < 1 ||
      h > itl::kMaxEmbedWidth)
    return LOGP_ERR_SHAPE;
  return std::isfinite(scale) ? LOGP_OK : LOGP_ERR_VALUE;
}

itl::Targets tokens_of(const void* tokens, int32_t token_dtype) {
  return itl::Targets{tokens, token_dtype == LOGP_I32 ? 1 : 0};
}

}  // namespace

extern "C" {

int32_t embedding_fwd(const void* table, int64_t ld_t, int64_t v, int64_t h, int32_t dtype,
                      const void* tokens, int32_t token_dtype, int64_t n, int64_t ignore_index,
                      float scale, void* out, int64_t ld_o, void* hip_stream) {
  if (!known_dtype(dtype)) return LOGP_ERR_DTYPE;
  const int32_t st = check_embedding(v, h, token_dtype, n, scale);
  if (st != LOGP_OK) return st;
  if (ld_t < h || ld_o < h) return LOGP_ERR_SHAPE;
  if (n == 0) return LOGP_OK;
  if (!table || !tokens || !out) return LOGP_ERR_NULL;
  (void)hipGetLastError();
  itl::launch_embedding(dtype, table, ld_t, v, h, tokens_of(tokens, token_dtype), n, ignore_index,
                        scale, out, ld_o, static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t embedding_fp4_fwd(const void* data, int64_t ld_d, const void* scales, int64_t ld_s,
                          int64_t v, int64_t h, const void* tokens, int32_t token_dtype, int64_t n,
                          int64_t ignore_index, float scale, int32_t out_dtype, void* out,
                          int64_t ld_o, void* hip_stream) {
  if (!known_dtype(out_dtype)) return LOGP_ERR_DTYPE;
  const int32_t st = check_embedding(v, h, token_dtype, n, scale);
  if (st != LOGP_OK) return st;
  if (h % itl::kFp4Group || ld_d < h / 2 || ld_s < h / itl::kFp4Group || ld_o < h)
    return LOGP_ERR_SHAPE;
  if (n == 0) return LOGP_OK;
  if (!data || !scales || !tokens || !out) return LOGP_ERR_NULL;
  if (!rows_aligned16(data, ld_d, 1)) return LOGP_ERR_ALIGN;
  (void)hipGetLastError();
  itl::launch_embedding_fp4(static_cast<const uint8_t*>(data), ld_d,
                            static_cast<const uint8_t*>(scales), ld_s, v, h,
                            tokens_of(tokens, token_dtype), n, ignore_index, scale, out_dtype, out,
                            ld_o, static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

size_t embedding_bwd_workspace_bytes(int64_t n, int64_t v, int64_t h) {
  if (n < 1 || n > itl::kMaxEmbedTokens || check_embedding(v, h, LOGP_I64, n, 1.0f) != LOGP_OK)
    return 0;
  return static_cast<size_t>(itl::embedding_bwd_bytes(n, v, h));
}

int32_t embedding_bwd(const void* dy, int64_t ld_y, int32_t dtype, const void* tokens,
                      int32_t token_dtype, int64_t n, int64_t v, int64_t h, int64_t ignore_index,
                      float scale, int32_t out_dtype, int32_t accumulate, void* dtable,
                      int64_t ld_t, void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!known_dtype(dtype) || (out_dtype != dtype && out_dtype != LOGP_F32)) return LOGP_ERR_DTYPE;
  const int32_t st = check_embedding(v, h, token_dtype, n, scale);
  if (st != LOGP_OK) return st;
  if (n > itl::kMaxEmbedTokens || ld_y < h || ld_t < h) return LOGP_ERR_SHAPE;
  if (accumulate != 0 && accumulate != 1) return LOGP_ERR_VALUE;
  if (n == 0 && accumulate) return LOGP_OK;
  if (!dtable || (n > 0 && (!dy || !tokens))) return LOGP_ERR_NULL;
  if (!itl::ws_ok(workspace, workspace_bytes, embedding_bwd_workspace_bytes(n, v, h)))
    return LOGP_ERR_WORKSPACE;
  (void)hipGetLastError();
  itl::launch_embedding_bwd(dtype, dy, ld_y, tokens_of(tokens, token_dtype), n, v, h, ignore_index,
                            scale, out_dtype == LOGP_F32, accumulate != 0, dtable, ld_t,
                            static_cast<char*>(workspace), static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t dropout_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int32_t dtype,
                    int64_t n, int64_t h, double p, int64_t seed, const int64_t* seed_at,
                    int64_t draw, int64_t first_row, void* out, int64_t ld_o, void* hip_stream) {
  if (!known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < 1 || h > itl::kMaxEmbedWidth || ld_x < h || ld_o < h ||
      (residual && ld_r < h))
    return LOGP_ERR_SHAPE;
  const int32_t st = check_drop(p, draw, first_row);
  if (st != LOGP_OK) return st;
  if (n == 0) return LOGP_OK;
  if (!x || !out) return LOGP_ERR_NULL;
  (void)hipGetLastError();
  itl::launch_dropout(dtype, x, ld_x, residual, ld_r, n, h,
                      itl::make_drop(p, seed, seed_at, draw, first_row), out, ld_o,
                      static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t layer_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                       const void* weight, const void* bias, int32_t dtype, int64_t n, int64_t h,
                       float eps, double p, int64_t seed, const int64_t* seed_at, int64_t draw,
                       int64_t first_row, void* y, int64_t ld_y, void* sum_out, int64_t ld_s,
                       float* mean_out, float* rstd_out, void* hip_stream) {
  if (!known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < 1 || h > itl::kMaxNorm || ld_x < h || ld_y < h ||
      (residual && ld_r < h) || (sum_out && ld_s < h))
    return LOGP_ERR_SHAPE;
  if (!(std::isfinite(eps) && eps >= 0.0f)) return LOGP_ERR_VALUE;
  const int32_t st = check_drop(p, draw, first_row);
  if (st != LOGP_OK) return st;
  if (n == 0) return LOGP_OK;
  if (!x || !weight || !y || ((residual || p > 0.0) && !sum_out)) return LOGP_ERR_NULL;
  const itl::Drop drop = itl::make_drop(p, seed, seed_at, draw, first_row);
  (void)hipGetLastError();
  itl::launch_layer_norm(dtype, itl::NormRows{x, ld_x, residual, ld_r, sum_out, ld_s},
                         p > 0.0 ? &drop : nullptr, weight, bias, n, h, eps, y, ld_y, mean_out,
                         rstd_out, static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

size_t layer_norm_bwd_workspace_bytes(int64_t n, int64_t h) {
  if (n < 1 || h < 1 || h > itl::kMaxNorm) return 0;
  const int64_t wide = itl::layer_norm_bwd_blocks(itl::kF32, n, h);
  const int64_t half = itl::layer_norm_bwd_blocks(itl::kBF16, n, h);
  return itl::ws_round(static_cast<size_t>(wide > half ? wide : half) * static_cast<size_t>(h) * 8);
}

int32_t layer_norm_bwd(const void* s, int64_t ld_s, const void* weight, const float* mean,
                       const float* rstd, const void* dy, int64_t ld_dy, const void* ds,
                       int64_t ld_ds, int32_t dtype, int64_t n, int64_t h, double p, int64_t seed,
                       const int64_t* seed_at, int64_t draw, int64_t first_row, void* dx,
                       int64_t ld_dx, void* dresidual, int64_t ld_dr, void* dweight, void* dbias,
                       void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < 1 || h > itl::kMaxNorm || ld_s < h || ld_dy < h || ld_dx < h ||
      (ds && ld_ds < h) || (dresidual && ld_dr < h))
    return LOGP_ERR_SHAPE;
  const int32_t st = check_drop(p, draw, first_row);
  if (st != LOGP_OK) return st;
  if (dresidual && (p == 0.0 || dresidual == dx)) return LOGP_ERR_VALUE;
  if (n == 0 && !dweight && !dbias) return LOGP_OK;
  if (n > 0 && (!s || !weight || !mean || !rstd || !dy || !dx)) return LOGP_ERR_NULL;
  if ((dweight || dbias) &&
      !itl::ws_ok(workspace, workspace_bytes, layer_norm_bwd_workspace_bytes(n, h)))
    return LOGP_ERR_WORKSPACE;
  const itl::Drop drop = itl::make_drop(p, seed, seed_at, draw, first_row);
  const itl::LayerNormGrad g{s,  ld_s,  weight, mean, rstd, dy, ld_dy, ds, ld_ds,
                             p > 0.0 ? &drop : nullptr,
                             dx, ld_dx, dresidual, ld_dr, dweight, dbias};
  (void)hipGetLastError();
  itl::launch_layer_norm_bwd(dtype, g, n, h, static_cast<float*>(workspace),
                             static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t fp4_quantize(const void* x, int64_t ld_x, int32_t dtype, int64_t n, int64_t h, void* data,
                     int64_t ld_d, void* scales, int64_t ld_s, void* hip_stream) {
  if (!known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < itl::kFp4Group || h % itl::kFp4Group ||
      h > itl::kMaxEmbedWidth || ld_x < h || ld_d < h / 2 || ld_s < h / itl::kFp4Group)
    return LOGP_ERR_SHAPE;
  if (n == 0) return LOGP_OK;
  if (!x || !data || !scales) return LOGP_ERR_NULL;
  if (!rows_aligned16(data, ld_d, 1)) return LOGP_ERR_ALIGN;
  (void)hipGetLastError();
  itl::launch_fp4_quantize(dtype, x, ld_x, n, h, static_cast<uint8_t*>(data), ld_d,
                           static_cast<uint8_t*>(scales), ld_s,
                           static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

}  // extern "C"
