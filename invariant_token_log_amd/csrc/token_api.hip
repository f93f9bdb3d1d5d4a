// C ABI of the token operators (include/invariant_tokens.h): argument checks
// (all before any HIP call), workspace layouts and launch sequences.
#include "invariant_tokens.h"

#include "api_checks.h"
#include "fp4.h"
#include "linear_fp4.h"
#include "linear_q8.h"
#include "rms_norm.h"

namespace {

using itl::dtype_size;
using itl::rows_aligned16;
using itl::ws_round;

static_assert(itl::kMaxTokens == LOGP_MAX_TOKENS && itl::kMaxTop == LOGP_MAX_TOP, "limits");

constexpr int kMaxTiles = 4096;
// Rows of the head per chunk unless the caller asks for another number: with the
// chunk's logits in the workspace, and without (12 bytes of statistics a tile).
constexpr int64_t kDefaultRows = 4096;
constexpr int64_t kDefaultRowsNoLogits = 65536;

int32_t check_tokens(const void* tokens, int32_t token_dtype, int64_t m) {
  if (token_dtype != LOGP_I64 && token_dtype != LOGP_I32) return LOGP_ERR_DTYPE;
  if (m < 0 || m > itl::kMaxTokens) return LOGP_ERR_SHAPE;
  if (m > 0 && !tokens) return LOGP_ERR_NULL;
  return LOGP_OK;
}

int32_t check_top(int32_t top_k, int64_t v) {
  if (top_k < 0 || top_k > itl::kMaxTop || top_k > v) return LOGP_ERR_VALUE;
  if (top_k > 0 && v >= (int64_t{1} << 32) - 1) return LOGP_ERR_SHAPE;
  return LOGP_OK;
}

itl::TokenView view_of(const void* tokens, int32_t token_dtype, int64_t m, int64_t ignore) {
  return itl::TokenView{tokens, token_dtype == LOGP_I32 ? 1 : 0, m, ignore};
}

int32_t check_streamed(int32_t dtype, int64_t n, int64_t v, int64_t ld, int32_t w) {
  if (!itl::known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || v < 1 || ld < v) return LOGP_ERR_SHAPE;
  if (itl::tile_chunks(dtype, w) == 0) return LOGP_ERR_TILE;
  if ((v + w - 1) / w > kMaxTiles) return LOGP_ERR_SHAPE;
  return LOGP_OK;
}

// Tile statistics [n, T] (m, s, w), then the group maxima.
struct StreamLayout {
  size_t pm, ps, pw, gm, total;
};

StreamLayout stream_layout(int64_t n, int64_t v, int32_t dtype, int32_t w, int32_t top_k) {
  const int64_t ntiles = (v + w - 1) / w;
  const size_t rows = static_cast<size_t>(n);
  const size_t table = ws_round(rows * static_cast<size_t>(ntiles) * 4);
  StreamLayout l;
  l.pm = 0;
  l.ps = table;
  l.pw = 2 * table;
  l.gm = 3 * table;
  const int64_t groups = itl::token_groups(itl::tile_chunks(dtype, w), ntiles);
  l.total = l.gm + (top_k > 0 ? ws_round(rows * static_cast<size_t>(groups) * 4) : 0);
  return l;
}

// The head's forward, rc rows at a time: tile statistics [rc, T] (m, s, w),
// the one given token's logits, the rows' activity, the re-laid hidden rows
// and the chunk's logits.
struct HeadLayout {
  int64_t rc, ntiles, ld_z;
  int tile;  // vocabulary columns of a statistic tile
  bool single, own_z;
  size_t pm, ps, pw, pt, act, hb, z, total;
};

HeadLayout head_layout(int64_t n, int64_t h, int64_t v, int64_t m, int32_t top_k, int32_t flags,
                       int64_t row_chunk) {
  HeadLayout l;
  const bool keeps = flags & LOGP_TOKEN_KEEPS_LOGITS;
  const int zsize = flags & LOGP_TOKEN_ROUND_BF16 ? 2 : 4;
  l.single = m == 1 && top_k == 0 && !keeps;
  l.own_z = !l.single && !keeps && (m > 0 || top_k > 0);
  const int64_t want = row_chunk > 0 ? row_chunk : l.own_z ? kDefaultRows : kDefaultRowsNoLogits;
  l.rc = (want + 255) / 256 * 256;
  if (l.rc > n) l.rc = n;
  l.tile = flags & LOGP_TOKEN_Q8 ? itl::kQ8Tile : itl::kLinearTile;
  l.ntiles = (v + l.tile - 1) / l.tile;
  l.ld_z = (v + 7) / 8 * 8;
  const size_t rows = static_cast<size_t>(l.rc);
  const size_t table = ws_round(rows * static_cast<size_t>(l.ntiles) * 4);
  l.pm = 0;
  l.ps = table;
  l.pw = 2 * table;
  l.pt = 3 * table;
  l.act = l.pt + ws_round(rows * 4);
  l.hb = l.act + ws_round(rows * 4);
  const int64_t hb = flags & LOGP_TOKEN_Q8 ? itl::q8_fwd_scratch_bytes(l.rc, h)
                                           : itl::linear_fwd_blocked_bytes(l.rc, h);
  l.z = l.hb + ws_round(static_cast<size_t>(hb));
  l.total = l.z + (l.own_z ? ws_round(rows * static_cast<size_t>(l.ld_z) * zsize) : 0);
  return l;
}

int32_t check_head_sizes(int64_t n, int64_t h, int64_t v, int64_t m, int32_t top_k,
                         int64_t row_chunk) {
  if (n < 0 || v < 1 || h < 64 || h % 64 || m < 0 || m > itl::kMaxTokens || row_chunk < 0)
    return LOGP_ERR_SHAPE;
  if (h > (int64_t{1} << 24) || v > (int64_t{1} << 31) || n > (int64_t{1} << 31) ||
      row_chunk > (int64_t{1} << 31) ||
      (n + 127) / 128 * ((v + 255) / 256) > (int64_t{1} << 30))
    return LOGP_ERR_SHAPE;
  return check_top(top_k, v);
}

struct HeadArgs {
  const void* hidden;
  int64_t ld_h;
  const float* hidden_scale;  // 8-bit head only
  const void* weight;
  int64_t ld_w;
  const float* weight_scale;  // 8-bit head only
  int64_t n, h, v;
  itl::TokenView tok;
  float inv_t;
  int32_t round_bf16;
  int32_t top_k;
  itl::TokenOut out;
  void* z;  // caller's logits, or null
  int32_t z_bf16;
  int64_t ld_z;
  const uint16_t* wblk;
  bool q8;
  const itl::Fp4Weight* fp4;  // or null
};

// Rows r0 .. of every row operand.
itl::TokenView token_rows(const itl::TokenView& t, int64_t r0) {
  itl::TokenView o = t;
  if (t.p) o.p = static_cast<const char*>(t.p) + r0 * t.m * (t.is32 ? 4 : 8);
  return o;
}
itl::TokenOut out_rows(const itl::TokenOut& o, int64_t r0, int64_t m, int64_t k) {
  return itl::TokenOut{o.logp ? o.logp + r0 * m : nullptr, o.lse ? o.lse + r0 : nullptr,
                       o.ent ? o.ent + r0 : nullptr, o.top_logp ? o.top_logp + r0 * k : nullptr,
                       o.top_ids ? o.top_ids + r0 * k : nullptr};
}

void run_head(const HeadArgs& a, const HeadLayout& l, char* ws, hipStream_t s) {
  float* pm = reinterpret_cast<float*>(ws + l.pm);
  float* ps = reinterpret_cast<float*>(ws + l.ps);
  float* pw = a.out.ent ? reinterpret_cast<float*>(ws + l.pw) : nullptr;
  float* pt = reinterpret_cast<float*>(ws + l.pt);
  int32_t* act = reinterpret_cast<int32_t*>(ws + l.act);
  const int ntiles = static_cast<int>(l.ntiles);
  const int esize = a.q8 ? 1 : 2;
  for (int64_t r0 = 0; r0 < a.n; r0 += l.rc) {
    const int64_t rows = l.rc < a.n - r0 ? l.rc : a.n - r0;
    const itl::TokenView tok = token_rows(a.tok, r0);
    // One given token and nothing else: its logit comes out of the product's
    // epilogue, as in linear_logp_fwd.  Otherwise the rows' activity stands
    // in for the targets and the logits go to memory.
    itl::Targets tg{tok.p, tok.is32};
    int64_t ignore = tok.ignore;
    if (!l.single) {
      itl::launch_token_rows(rows, tok, itl::TopView{nullptr, 0}, nullptr, nullptr, act, nullptr,
                             s);
      tg = itl::Targets{act, 1};
      ignore = -2;
    }
    void* z = a.z ? static_cast<char*>(a.z) + r0 * a.ld_z * (a.z_bf16 ? 2 : 4)
                  : l.own_z ? static_cast<void*>(ws + l.z) : nullptr;
    const int64_t ld_z = a.z ? a.ld_z : l.ld_z;
    const int32_t z_bf16 = a.z ? a.z_bf16 : a.round_bf16;
    const char* hidden = static_cast<const char*>(a.hidden) + r0 * a.ld_h * esize;
    if (a.q8)
      itl::launch_q8_partials(reinterpret_cast<const uint8_t*>(hidden), a.ld_h,
                              a.hidden_scale + r0, static_cast<const uint8_t*>(a.weight), a.ld_w,
                              a.weight_scale, rows, a.h, a.v, tg, ignore, pm, ps, pt, a.inv_t, pw,
                              static_cast<float*>(z), ld_z, ws + l.hb, s);
    else if (a.fp4)
      itl::launch_fp4_partials(reinterpret_cast<const uint16_t*>(hidden), a.ld_h, *a.fp4, rows, a.h,
                               a.v, tg, ignore, pm, ps, pt, a.inv_t, a.round_bf16, pw, z, z_bf16,
                               ld_z, reinterpret_cast<uint16_t*>(ws + l.hb), s);
    else
      itl::launch_linear_partials(reinterpret_cast<const uint16_t*>(hidden), a.ld_h,
                                  static_cast<const uint16_t*>(a.weight), a.ld_w, rows, a.h, a.v,
                                  tg, ignore, pm, ps, pt, a.inv_t, a.round_bf16, pw, z, z_bf16,
                                  ld_z, a.wblk, reinterpret_cast<uint16_t*>(ws + l.hb), s);
    const bool read_z = !l.single && z;
    const int zdt = z_bf16 ? itl::kBF16 : itl::kF32;
    itl::launch_token_finish(zdt, read_z && rows_aligned16(z, ld_z, z_bf16 ? 2 : 4), l.tile,
                             read_z ? z : nullptr, ld_z, a.inv_t, pt, rows, a.v, tok, ntiles, pm,
                             ps, pw, pm, ntiles, a.top_k,
                             out_rows(a.out, r0, a.tok.m, a.top_k), s);
  }
}

int32_t check_outputs(int64_t m, int32_t top_k, const float* logp, const float* top_logp,
                      const int64_t* top_ids) {
  if (m > 0 && !logp) return LOGP_ERR_NULL;
  if (top_k > 0 && (!top_logp || !top_ids)) return LOGP_ERR_NULL;
  return LOGP_OK;
}

}  // namespace

extern "C" {

size_t token_logp_fwd_workspace_bytes(int64_t n, int64_t v, int32_t dtype, int32_t tile_width,
                                      int32_t top_k) {
  if (check_streamed(dtype, n, v, v, tile_width) != LOGP_OK || check_top(top_k, v) != LOGP_OK)
    return 0;
  return stream_layout(n, v, dtype, tile_width, top_k).total;
}

int32_t token_logp_fwd(const void* logits, int32_t dtype, int64_t n, int64_t v, int64_t ld,
                       const void* tokens, int32_t token_dtype, int64_t m, int64_t ignore_index,
                       int32_t tile_width, int32_t top_k, float* logp_out, float* lse_out,
                       float* entropy_out, float* top_logp_out, int64_t* top_ids_out,
                       void* workspace, size_t workspace_bytes, void* hip_stream) {
  int32_t st = check_streamed(dtype, n, v, ld, tile_width);
  if (st != LOGP_OK) return st;
  if ((st = check_top(top_k, v)) != LOGP_OK) return st;
  if (n == 0) return m < 0 || m > itl::kMaxTokens ? LOGP_ERR_SHAPE : LOGP_OK;
  if ((st = check_tokens(tokens, token_dtype, m)) != LOGP_OK) return st;
  if (!logits) return LOGP_ERR_NULL;
  if ((st = check_outputs(m, top_k, logp_out, top_logp_out, top_ids_out)) != LOGP_OK) return st;
  const StreamLayout l = stream_layout(n, v, dtype, tile_width, top_k);
  if (!itl::ws_ok(workspace, workspace_bytes, l.total)) return LOGP_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  float* pm = reinterpret_cast<float*>(ws + l.pm);
  float* ps = reinterpret_cast<float*>(ws + l.ps);
  float* pw = entropy_out ? reinterpret_cast<float*>(ws + l.pw) : nullptr;
  uint32_t* gm = top_k > 0 ? reinterpret_cast<uint32_t*>(ws + l.gm) : nullptr;
  const int chunks = itl::tile_chunks(dtype, tile_width);
  const int ntiles = static_cast<int>((v + tile_width - 1) / tile_width);
  const bool vec = rows_aligned16(logits, ld, dtype_size(dtype));
  const itl::TokenView tok = view_of(tokens, token_dtype, m, ignore_index);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  (void)hipGetLastError();
  itl::launch_token_partials(dtype, vec, chunks, logits, ld, n, v, tok, ntiles, pm, ps, pw, gm, s);
  itl::launch_token_finish(dtype, vec, false, logits, ld, 1.0f, nullptr, n, v, tok, ntiles, pm, ps,
                           pw, gm, itl::token_groups(chunks, ntiles), top_k,
                           itl::TokenOut{logp_out, lse_out, entropy_out, top_logp_out, top_ids_out},
                           s);
  return itl::launch_status();
}

int32_t token_logp_bwd(const void* logits, int32_t dtype, int64_t n, int64_t v, int64_t ld,
                       const void* tokens, int32_t token_dtype, int64_t m, int64_t ignore_index,
                       const int64_t* top_ids, int32_t top_k, const float* lse,
                       const float* grad_logp, const float* grad_top_logp, const float* entropy,
                       const float* grad_entropy, void* dlogits_out, int64_t ld_out,
                       void* hip_stream) {
  if (!itl::known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || v < 1 || ld < v || ld_out < v) return LOGP_ERR_SHAPE;
  if ((v + 1023) / 1024 > INT32_MAX) return LOGP_ERR_SHAPE;  // grid x
  int32_t st = check_top(top_k, v);
  if (st != LOGP_OK) return st;
  if (n == 0) return m < 0 || m > itl::kMaxTokens ? LOGP_ERR_SHAPE : LOGP_OK;
  if ((st = check_tokens(tokens, token_dtype, m)) != LOGP_OK) return st;
  if (!logits || !lse || !dlogits_out || (m > 0 && !grad_logp) ||
      (top_k > 0 && (!top_ids || !grad_top_logp)))
    return LOGP_ERR_NULL;
  if ((entropy == nullptr) != (grad_entropy == nullptr)) return LOGP_ERR_NULL;
  const int size = dtype_size(dtype);
  const bool vec = rows_aligned16(logits, ld, size) && rows_aligned16(dlogits_out, ld_out, size);
  (void)hipGetLastError();
  itl::launch_token_bwd(dtype, vec, logits, ld, n, v, view_of(tokens, token_dtype, m, ignore_index),
                        itl::TopView{top_ids, top_k}, lse, grad_logp, grad_top_logp, entropy,
                        grad_entropy, dlogits_out, ld_out, static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

size_t linear_token_logp_fwd_workspace_bytes(int64_t n, int64_t h, int64_t v, int64_t m,
                                             int32_t top_k, int32_t flags, int64_t row_chunk) {
  if (check_head_sizes(n, h, v, m, top_k, row_chunk) != LOGP_OK || flags < 0 || flags > 15 ||
      ((flags & LOGP_TOKEN_FP4) && (flags & (LOGP_TOKEN_Q8 | LOGP_TOKEN_KEEPS_LOGITS))))
    return 0;
  return head_layout(n, h, v, m, top_k, flags, row_chunk).total;
}

int32_t linear_token_logp_fwd(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                              int64_t n, int64_t h, int64_t v, const void* tokens,
                              int32_t token_dtype, int64_t m, int64_t ignore_index,
                              float temperature, int32_t logits_rounding, int32_t top_k,
                              float* logp_out, float* lse_out, float* entropy_out,
                              float* top_logp_out, int64_t* top_ids_out, void* logits_out,
                              int32_t logits_dtype, int64_t ld_logits, const void* prepared,
                              size_t prepared_bytes, int64_t row_chunk, void* workspace,
                              size_t workspace_bytes, void* hip_stream) {
  int32_t st = check_head_sizes(n, h, v, m, top_k, row_chunk);
  if (st != LOGP_OK) return st;
  if (ld_h < h || ld_w < h) return LOGP_ERR_SHAPE;
  if (!itl::usable_temperature(temperature) ||
      (logits_rounding != LOGP_ROUND_NONE && logits_rounding != LOGP_ROUND_BF16))
    return LOGP_ERR_VALUE;
  const bool rounded = logits_rounding == LOGP_ROUND_BF16;
  if (logits_out) {
    if (logits_dtype != LOGP_F32 && !(logits_dtype == LOGP_BF16 && rounded)) return LOGP_ERR_DTYPE;
    if (ld_logits < v) return LOGP_ERR_SHAPE;
  }
  if (n == 0) return LOGP_OK;
  if ((st = check_tokens(tokens, token_dtype, m)) != LOGP_OK) return st;
  if (!hidden || !weight) return LOGP_ERR_NULL;
  if ((st = check_outputs(m, top_k, logp_out, top_logp_out, top_ids_out)) != LOGP_OK) return st;
  if (!rows_aligned16(hidden, ld_h, 2) || !rows_aligned16(weight, ld_w, 2)) return LOGP_ERR_ALIGN;
  if (prepared) {
    if (prepared_bytes < linear_logp_prepared_bytes(v, h)) return LOGP_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(prepared) % 16) return LOGP_ERR_ALIGN;
  }
  const int32_t flags = (logits_out ? LOGP_TOKEN_KEEPS_LOGITS : 0) |
                        (rounded ? LOGP_TOKEN_ROUND_BF16 : 0);
  const HeadLayout l = head_layout(n, h, v, m, top_k, flags, row_chunk);
  if (!itl::ws_ok(workspace, workspace_bytes, l.total)) return LOGP_ERR_WORKSPACE;
  HeadArgs a{};
  a.hidden = hidden;
  a.ld_h = ld_h;
  a.weight = weight;
  a.ld_w = ld_w;
  a.n = n;
  a.h = h;
  a.v = v;
  a.tok = view_of(tokens, token_dtype, m, ignore_index);
  a.inv_t = itl::reciprocal_temperature(temperature);
  a.round_bf16 = rounded ? 1 : 0;
  a.top_k = top_k;
  a.out = itl::TokenOut{logp_out, lse_out, entropy_out, top_logp_out, top_ids_out};
  a.z = logits_out;
  a.z_bf16 = logits_dtype == LOGP_BF16 ? 1 : 0;
  a.ld_z = ld_logits;
  a.wblk = prepared ? itl::prepared_blocked_w(static_cast<const uint16_t*>(prepared)) : nullptr;
  (void)hipGetLastError();
  run_head(a, l, static_cast<char*>(workspace), static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t linear_token_logp_q8_fwd(const void* hidden, int64_t ld_h, const float* hidden_scale,
                                 const void* weight, int64_t ld_w, const float* weight_scale,
                                 int64_t n, int64_t h, int64_t v, const void* tokens,
                                 int32_t token_dtype, int64_t m, int64_t ignore_index,
                                 float temperature, int32_t top_k, float* logp_out,
                                 float* lse_out, float* entropy_out, float* top_logp_out,
                                 int64_t* top_ids_out, int64_t row_chunk, void* workspace,
                                 size_t workspace_bytes, void* hip_stream) {
  int32_t st = check_head_sizes(n, h, v, m, top_k, row_chunk);
  if (st != LOGP_OK) return st;
  if (ld_h < h || ld_w < h || ld_h > itl::kMaxQ8Stride || ld_w > itl::kMaxQ8Stride)
    return LOGP_ERR_SHAPE;
  if (!itl::usable_temperature(temperature)) return LOGP_ERR_VALUE;
  if (n == 0) return LOGP_OK;
  if ((st = check_tokens(tokens, token_dtype, m)) != LOGP_OK) return st;
  if (!hidden || !weight || !hidden_scale || !weight_scale) return LOGP_ERR_NULL;
  if ((st = check_outputs(m, top_k, logp_out, top_logp_out, top_ids_out)) != LOGP_OK) return st;
  if (!rows_aligned16(hidden, ld_h, 1) || !rows_aligned16(weight, ld_w, 1)) return LOGP_ERR_ALIGN;
  const HeadLayout l = head_layout(n, h, v, m, top_k, LOGP_TOKEN_Q8, row_chunk);
  if (!itl::ws_ok(workspace, workspace_bytes, l.total)) return LOGP_ERR_WORKSPACE;
  HeadArgs a{};
  a.hidden = hidden;
  a.ld_h = ld_h;
  a.hidden_scale = hidden_scale;
  a.weight = weight;
  a.ld_w = ld_w;
  a.weight_scale = weight_scale;
  a.n = n;
  a.h = h;
  a.v = v;
  a.tok = view_of(tokens, token_dtype, m, ignore_index);
  a.inv_t = itl::reciprocal_temperature(temperature);
  a.top_k = top_k;
  a.out = itl::TokenOut{logp_out, lse_out, entropy_out, top_logp_out, top_ids_out};
  a.q8 = true;
  (void)hipGetLastError();
  run_head(a, l, static_cast<char*>(workspace), static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t linear_token_logp_fp4_fwd(const void* hidden, int64_t ld_h, const void* data, int64_t ld_d,
                                  const void* scales, int64_t ld_s, int64_t n, int64_t h,
                                  int64_t v, const void* tokens, int32_t token_dtype, int64_t m,
                                  int64_t ignore_index, float temperature, int32_t logits_rounding,
                                  int32_t top_k, float* logp_out, float* lse_out,
                                  float* entropy_out, float* top_logp_out, int64_t* top_ids_out,
                                  int64_t row_chunk, void* workspace, size_t workspace_bytes,
                                  void* hip_stream) {
  int32_t st = check_head_sizes(n, h, v, m, top_k, row_chunk);
  if (st != LOGP_OK) return st;
  if (ld_h < h || ld_d < h / 2 || ld_s < h / itl::kFp4Group || ld_h > itl::kMaxHiddenStride ||
      ld_d > itl::kMaxFp4Stride || ld_s > itl::kMaxFp4Stride)
    return LOGP_ERR_SHAPE;
  if (!itl::usable_temperature(temperature) ||
      (logits_rounding != LOGP_ROUND_NONE && logits_rounding != LOGP_ROUND_BF16))
    return LOGP_ERR_VALUE;
  if (n == 0) return LOGP_OK;
  if ((st = check_tokens(tokens, token_dtype, m)) != LOGP_OK) return st;
  if (!hidden || !data || !scales) return LOGP_ERR_NULL;
  if ((st = check_outputs(m, top_k, logp_out, top_logp_out, top_ids_out)) != LOGP_OK) return st;
  if (!rows_aligned16(hidden, ld_h, 2) || !rows_aligned16(data, ld_d, 1)) return LOGP_ERR_ALIGN;
  const bool rounded = logits_rounding == LOGP_ROUND_BF16;
  const HeadLayout l = head_layout(n, h, v, m, top_k,
                                   LOGP_TOKEN_FP4 | (rounded ? LOGP_TOKEN_ROUND_BF16 : 0),
                                   row_chunk);
  if (!itl::ws_ok(workspace, workspace_bytes, l.total)) return LOGP_ERR_WORKSPACE;
  const itl::Fp4Weight w{static_cast<const uint8_t*>(data), ld_d,
                         static_cast<const uint8_t*>(scales), ld_s};
  HeadArgs a{};
  a.hidden = hidden;
  a.ld_h = ld_h;
  a.n = n;
  a.h = h;
  a.v = v;
  a.tok = view_of(tokens, token_dtype, m, ignore_index);
  a.inv_t = itl::reciprocal_temperature(temperature);
  a.round_bf16 = rounded ? 1 : 0;
  a.top_k = top_k;
  a.out = itl::TokenOut{logp_out, lse_out, entropy_out, top_logp_out, top_ids_out};
  a.fp4 = &w;
  (void)hipGetLastError();
  run_head(a, l, static_cast<char*>(workspace), static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

size_t linear_token_logp_bwd_workspace_bytes(int64_t n, int64_t h, int64_t v, int32_t flags,
                                             int64_t vocab_chunk) {
  if (linear_logp_bwd_workspace_bytes(n, h, v, itl::kLinearTile, flags, vocab_chunk) == 0) return 0;
  const int64_t base = itl::linear_bwd_layout(n, h, v, flags, vocab_chunk, true).total;
  return ws_round(static_cast<size_t>(base)) + 2 * ws_round(static_cast<size_t>(n) * 4);
}

int32_t linear_token_logp_bwd(const void* hidden, int64_t ld_h, const void* weight, int64_t ld_w,
                              int64_t n, int64_t h, int64_t v, const void* tokens,
                              int32_t token_dtype, int64_t m, int64_t ignore_index,
                              const int64_t* top_ids, int32_t top_k, float temperature,
                              int32_t logits_rounding, const void* saved_logits,
                              int32_t saved_dtype, int64_t ld_saved, const void* prepared,
                              size_t prepared_bytes, const float* lse, const float* logp,
                              const float* top_logp, const float* grad_logp,
                              const float* grad_top_logp, const float* entropy,
                              const float* grad_entropy, int32_t out_dtype, void* dhidden,
                              int64_t ld_dh, void* dweight, int64_t ld_dw, int64_t vocab_chunk,
                              void* workspace, size_t workspace_bytes, void* hip_stream) {
  int32_t st = check_head_sizes(n, h, v, m, top_k, 0);
  if (st != LOGP_OK) return st;
  if (ld_h < h || ld_w < h || vocab_chunk < 0 || vocab_chunk > (int64_t{1} << 40))
    return LOGP_ERR_SHAPE;
  if (((v + 255) / 256) * ((h + 255) / 256) > (int64_t{1} << 30)) return LOGP_ERR_SHAPE;
  if (out_dtype != LOGP_F32 && out_dtype != LOGP_BF16) return LOGP_ERR_DTYPE;
  if (!itl::usable_temperature(temperature) ||
      (logits_rounding != LOGP_ROUND_NONE && logits_rounding != LOGP_ROUND_BF16))
    return LOGP_ERR_VALUE;
  const bool rounded = logits_rounding == LOGP_ROUND_BF16;
  if (saved_logits) {
    if (saved_dtype != LOGP_F32 && !(saved_dtype == LOGP_BF16 && rounded)) return LOGP_ERR_DTYPE;
    if (ld_saved < v) return LOGP_ERR_SHAPE;
    if (!rows_aligned16(saved_logits, ld_saved, dtype_size(saved_dtype))) return LOGP_ERR_ALIGN;
  }
  if (prepared) {
    if (prepared_bytes < linear_logp_prepared_bytes(v, h)) return LOGP_ERR_SHAPE;
    if (reinterpret_cast<uintptr_t>(prepared) % 16) return LOGP_ERR_ALIGN;
  }
  if (!dhidden && !dweight) return LOGP_ERR_NULL;
  if ((dhidden && ld_dh < h) || (dweight && ld_dw < h)) return LOGP_ERR_SHAPE;
  if (n == 0 && !dweight) return LOGP_OK;
  if (!weight) return LOGP_ERR_NULL;
  if (!rows_aligned16(weight, ld_w, 2)) return LOGP_ERR_ALIGN;
  if ((entropy == nullptr) != (grad_entropy == nullptr)) return LOGP_ERR_NULL;
  if (n > 0) {
    if ((st = check_tokens(tokens, token_dtype, m)) != LOGP_OK) return st;
    if (!hidden || !lse || (m > 0 && (!logp || !grad_logp)) ||
        (top_k > 0 && (!top_ids || !top_logp || !grad_top_logp)))
      return LOGP_ERR_NULL;
    if (!rows_aligned16(hidden, ld_h, 2)) return LOGP_ERR_ALIGN;
  }
  const int32_t flags = (dhidden ? LOGP_BWD_DHIDDEN : 0) | (dweight ? LOGP_BWD_DWEIGHT : 0) |
                        (prepared ? LOGP_BWD_PREPARED : 0) |
                        (saved_logits ? LOGP_BWD_SAVED_LOGITS : 0) |
                        (out_dtype == LOGP_BF16 ? LOGP_BWD_BF16_OUT : 0);
  const size_t need = linear_token_logp_bwd_workspace_bytes(n, h, v, flags, vocab_chunk);
  if (!itl::ws_ok(workspace, workspace_bytes, need)) return LOGP_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  const size_t rows = ws_round(static_cast<size_t>(n) * 4);
  float* gsum = n ? reinterpret_cast<float*>(ws + need - rows) : nullptr;
  int32_t* act = n ? reinterpret_cast<int32_t*>(ws + need - 2 * rows) : nullptr;
  const itl::TokenDz t{view_of(tokens, token_dtype, m, ignore_index), itl::TopView{top_ids, top_k},
                       logp, top_logp, grad_logp, grad_top_logp, gsum};
  (void)hipGetLastError();
  if (n > 0) itl::launch_token_rows(n, t.tok, t.alt, grad_logp, grad_top_logp, act, gsum, s);
  itl::launch_linear_bwd(static_cast<const uint16_t*>(hidden), ld_h,
                         static_cast<const uint16_t*>(weight), ld_w, n, h, v,
                         itl::Targets{act, 1}, -2, saved_logits,
                         saved_dtype == LOGP_BF16 ? 1 : 0, ld_saved,
                         static_cast<const uint16_t*>(prepared), lse, gsum,
                         itl::reciprocal_temperature(temperature), rounded ? 1 : 0, entropy,
                         grad_entropy, out_dtype == LOGP_BF16, dhidden, ld_dh, dweight, ld_dw,
                         vocab_chunk, ws, s, &t);
  return itl::launch_status();
}

int32_t rms_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                     const void* weight, int32_t dtype, int64_t n, int64_t h, float eps, void* y,
                     int64_t ld_y, void* sum_out, int64_t ld_s, float* rstd_out,
                     void* hip_stream) {
  if (!itl::known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < 1 || h > itl::kMaxNorm || ld_x < h || ld_y < h ||
      (residual && ld_r < h) || (sum_out && ld_s < h))
    return LOGP_ERR_SHAPE;
  if (!(std::isfinite(eps) && eps >= 0.0f)) return LOGP_ERR_VALUE;
  if (n == 0) return LOGP_OK;
  if (!x || !weight || !y || (residual && !sum_out)) return LOGP_ERR_NULL;
  (void)hipGetLastError();
  itl::launch_rms_norm(dtype, itl::NormRows{x, ld_x, residual, ld_r, sum_out, ld_s}, weight, n, h,
                       eps, y, ld_y, nullptr, rstd_out, false, static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

int32_t rms_norm_q8_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                        const void* weight, int32_t dtype, int64_t n, int64_t h, float eps,
                        void* q_out, int64_t ld_q, float* scale_out, void* sum_out, int64_t ld_s,
                        void* hip_stream) {
  if (!itl::known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < 1 || h > itl::kMaxNorm || ld_x < h || ld_q < h ||
      (residual && ld_r < h) || (sum_out && ld_s < h))
    return LOGP_ERR_SHAPE;
  if (!(std::isfinite(eps) && eps >= 0.0f)) return LOGP_ERR_VALUE;
  if (n == 0) return LOGP_OK;
  if (!x || !q_out || !scale_out || (residual && !sum_out)) return LOGP_ERR_NULL;
  (void)hipGetLastError();
  itl::launch_rms_norm(dtype, itl::NormRows{x, ld_x, residual, ld_r, sum_out, ld_s}, weight, n, h,
                       eps, q_out, ld_q, scale_out, nullptr, true,
                       static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

size_t rms_norm_bwd_workspace_bytes(int64_t n, int64_t h) {
  if (n < 1 || h < 1 || h > itl::kMaxNorm) return 0;
  return ws_round(static_cast<size_t>(itl::norm_bwd_blocks(n, h)) * static_cast<size_t>(h) * 4);
}

int32_t rms_norm_bwd(const void* s, int64_t ld_s, const void* weight, const float* rstd,
                     const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds, int32_t dtype,
                     int64_t n, int64_t h, void* dx, int64_t ld_dx, void* dweight,
                     void* workspace, size_t workspace_bytes, void* hip_stream) {
  if (!itl::known_dtype(dtype)) return LOGP_ERR_DTYPE;
  if (n < 0 || n > INT32_MAX || h < 1 || h > itl::kMaxNorm || ld_s < h || ld_dy < h || ld_dx < h ||
      (ds && ld_ds < h))
    return LOGP_ERR_SHAPE;
  if (n == 0 && !dweight) return LOGP_OK;
  if (n > 0 && (!s || !weight || !rstd || !dy || !dx)) return LOGP_ERR_NULL;
  if (dweight && !itl::ws_ok(workspace, workspace_bytes, rms_norm_bwd_workspace_bytes(n, h)))
    return LOGP_ERR_WORKSPACE;
  (void)hipGetLastError();
  itl::launch_rms_norm_bwd(dtype, s, ld_s, weight, rstd, dy, ld_dy, ds, ld_ds, n, h, dx, ld_dx,
                           dweight, static_cast<float*>(workspace),
                           static_cast<hipStream_t>(hip_stream));
  return itl::launch_status();
}

}  // extern "C"
