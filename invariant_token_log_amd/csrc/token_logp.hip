// Log-probabilities of several given tokens a row, with the row's entropy and
// its k most probable tokens, on gfx950, and the gradient of all of them.
//
//   lse  = log sum_j e^x_j                     (the tile tree and merge of
//                                               logp_device.h: the bits of logp_fwd)
//   logp_m = x[t_m] - lse,   m < M             (+0 where t_m is ignore_index)
//   top  = the k greatest x_j, ordered by (x descending, column ascending)
//   dx_j = sum_{m: t_m = j} g_m - G e^(x_j - lse) [- gH p_j (x_j - lse + H)],
//          G = sum_m g_m (given tokens and alternatives alike).
//
// Selection.  Reading a row twice would double the bytes, and keeping k
// candidates a lane costs more vector instructions a value than the row has
// to spare, so the pass over the row only keeps what the tile maximum
// computes anyway: the maximum of every group of 16 lanes' chunks (128
// columns of 16-bit logits, 64 of fp32), one value for 256 bytes.  Order all
// values by (x, -column); a group's best value is its maximum at its first
// place, groups are disjoint column ranges in ascending order, so the k
// greatest groups by (maximum, -group) hold the k greatest values: whatever
// the ties, exactly k groups are read again, 256 bytes each, and of those the
// values that reach the k-th group's maximum are ranked.  At k = 20 and
// V = 151936 that is 5 KB of a 304 KB row.
#include "launch.h"
#include "logp_device.h"
#include "token_device.h"

namespace itl {

namespace {

constexpr int kPartBlock = 512;  // 8 waves, one tile each at a time
constexpr int kPartWaves = kPartBlock / kWave;
constexpr int kFinBlock = 256;   // 4 waves, one row each
constexpr int kFinWaves = kFinBlock / kWave;
constexpr int64_t kMaxBlocks = 1 << 20;  // grid-stride beyond this
constexpr int64_t kMaxRowsY = 65535;

// ---------------------------------------------------------------------------
// Row partials: tile statistics (row-major [n, T] tables) and, with TOP, the
// group maxima [n, T * C * 4].  Work item = (row, segment of the row's
// tiles): one segment a row when there are rows enough for the GPU, up to one
// tile a wave when there are few.  The statistics depend on the tile alone,
// so the split changes no bit.
// ---------------------------------------------------------------------------

// tile_stats of logp_device.h (same sum tree, same bits; rows of any
// alignment in 16-byte loads) that, with TOP, also leaves the maxima of the
// tile's C * 4 groups in gm: the maximum is exact in any order, so it is taken
// along the groups first (four lane moves a chunk), then over the chunks, then
// over the four rows of 16 lanes.
template <typename T, int C, bool VEC, bool ENT, bool TOP>
__device__ __forceinline__ void token_tile_stats(const T* row, int64_t col0, int64_t v, float* gm,
                                                  float& m_out, float& s_out, float& w_out) {
  constexpr int E = Elt<T>::kPerChunk;
  constexpr int W = C * kWave * E;
  const int lane = threadIdx.x & (kWave - 1);
  float x[C][E];
  if (col0 + W <= v) {
#pragma unroll
    for (int j = 0; j < C; ++j)
      load_row_chunk<T, VEC>(row, col0 + static_cast<int64_t>(j * kWave + lane) * E, INT64_MAX, x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < C; ++j)
      load_row_chunk<T, VEC>(row, col0 + static_cast<int64_t>(j * kWave + lane) * E, v, x[j]);
  }
  float m = -INFINITY, mine = -INFINITY;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    float g = x[j][0];
#pragma unroll
    for (int e = 1; e < E; ++e) g = fmaxf(g, x[j][e]);
    if constexpr (TOP) {
      g = fmaxf(g, dpp_mov<kDppXor1>(g));
      g = fmaxf(g, dpp_mov<kDppXor2>(g));
      g = fmaxf(g, dpp_mov<kDppRowHalfMirror>(g));
      g = fmaxf(g, dpp_mov<kDppRowMirror>(g));
      mine = (lane & 15) == j ? g : mine;
    }
    m = fmaxf(m, g);
  }
  constexpr bool kLds = C * E > 16;  // where the partners come from: as tile_stats
  if constexpr (TOP) {
    // lane (row r16, place j < C) stores group 4 j + r16 (ascending columns)
    if ((lane & 15) < C) gm[(lane & 15) * 4 + (lane >> 4)] = mine;
    m = swap_combine16(m, true);
    m = swap_combine32(m, true);
  } else {
    m = kLds ? wave_max_lds(m) : wave_max(m);
  }
  float s = 0.0f, w = 0.0f;
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (ENT) {
        const float d = x[j][e] - m;
        const float ex = __builtin_amdgcn_exp2f(d * kLog2e);
        s = s + ex;
        w = ent_term(ex, d, w);
      } else {
        s = s + exp_sub(x[j][e], m);
      }
    }
  m_out = m;
  s_out = kLds ? wave_sum_lds(s) : wave_sum(s);
  if constexpr (ENT) w_out = kLds ? wave_sum_lds(w) : wave_sum(w);
}

template <typename T, int C, bool VEC, bool ENT, bool TOP>
__global__ __launch_bounds__(kPartBlock) void token_partials_kernel(
    const T* __restrict__ logits, int64_t ld, int64_t n, int64_t v, TokenView tok, int ntiles,
    int segs, int tiles_per_seg, float* __restrict__ pm, float* __restrict__ ps,
    float* __restrict__ pw, float* __restrict__ gm) {
  constexpr int W = C * kWave * Elt<T>::kPerChunk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  for (int64_t i = blockIdx.x; i < n * segs; i += gridDim.x) {
    const int64_t r = i / segs;
    const int k0 = static_cast<int>(i - r * segs) * tiles_per_seg;
    if (!row_active(tok, r, lane)) continue;
    const T* row = logits + r * ld;
    const int k1 = min(k0 + tiles_per_seg, ntiles);
    for (int k = k0 + wave; k < k1; k += kPartWaves) {
      float mk, sk, wk = 0.0f;
      const int64_t col0 = static_cast<int64_t>(k) * W;
      const int64_t at = r * ntiles + k;
      token_tile_stats<T, C, VEC, ENT, TOP>(row, col0, v, TOP ? gm + at * (C * 4) : nullptr, mk,
                                            sk, wk);
      if (lane == 0) {
        pm[at] = mk;
        ps[at] = sk;
        if constexpr (ENT) pw[at] = wk;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Finish: one wave a row merges the tile statistics (merge_lse_t: the bits of
// logp_fwd), ranks the alternatives and writes every output of the row.
//   x          the row's logits ([n, ld], row r at x + r * ld), or null: then
//              M = 1, k = 0 and the token's logit is pt[r].
//   inv_t      factor on the logits read from x (the tables hold scaled ones).
//   gm         group maxima of row r at gm + r * groups, group g = columns
//              [g * LPG * E, + LPG * E).
// ---------------------------------------------------------------------------
template <typename T, int LPG, bool VEC, bool ENT>
__global__ __launch_bounds__(kFinBlock) void token_finish_kernel(
    const T* __restrict__ x, int64_t ld, float inv_t, const float* __restrict__ pt, int64_t n,
    int64_t v, TokenView tok, int ntiles, const float* __restrict__ pm,
    const float* __restrict__ ps, const float* __restrict__ pw, const float* __restrict__ gm,
    int64_t groups, int top_k, TokenOut out) {
  constexpr int E = Elt<T>::kPerChunk;
  constexpr int GW = LPG * E;            // columns per group
  constexpr int GPW = kWave / LPG;       // groups one wave load covers
  __shared__ MergeStage merge[kFinWaves];
  __shared__ TopStage top[kFinWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  TopStage& st = top[wave];
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kFinWaves + wave; r < n;
       r += static_cast<int64_t>(gridDim.x) * kFinWaves) {
    if (!row_active(tok, r, lane)) {
      for (int64_t i = lane; i < tok.m; i += kWave) out.logp[r * tok.m + i] = 0.0f;
      if (lane < top_k) {
        out.top_logp[r * top_k + lane] = 0.0f;
        out.top_ids[r * top_k + lane] = -1;
      }
      if (lane == 0) {
        if (out.lse) out.lse[r] = 0.0f;
        if constexpr (ENT) out.ent[r] = 0.0f;
      }
      continue;
    }
    float h = 0.0f;
    const int64_t at = r * ntiles;
    const float L = merge_lse_t<ENT, 4>(pm + at, ps + at, pw + at, ntiles, 1, merge[wave], &h);
    if (lane == 0) {
      if (out.lse) out.lse[r] = L;
      if constexpr (ENT) out.ent[r] = h;
    }
    const T* row = x + r * ld;
    for (int64_t i = lane; i < tok.m; i += kWave) {
      const int64_t t = tok.at(r, i);
      float lp = 0.0f;
      if (t != tok.ignore) {
        const bool valid = t >= 0 && t < v;
        const float xt = !valid ? 0.0f : x ? Elt<T>::load(row, t) * inv_t : pt[r];
        lp = combine(xt, L, valid);
      }
      out.logp[r * tok.m + i] = lp;
    }
    if (top_k == 0) continue;

    // 1. A bound: the k-th greatest of the 64 lanes' own greatest groups.  At
    // least k groups reach it.
    const float* g = gm + r * groups;
    uint32_t best = 0;
    for (int64_t c = lane; c < groups; c += kWave) best = max(best, order_key(g[c]));
    const uint32_t bound = wave_kth(best, top_k, lane);
    // 2. The k greatest groups (or all, when there are fewer).
    TopList list{0, 0};
    for (int64_t c0 = 0; c0 < groups; c0 += kWave) {
      const int64_t c = c0 + lane;
      const uint32_t key = c < groups ? order_key(g[c]) : 0u;
      top_push(st, list, top_k, c < groups && key >= bound, compose(key, static_cast<uint32_t>(c)));
    }
    top_rank(st, list, top_k);
    const int ng = list.n;
    const uint64_t mine = lane < ng ? st.e[lane] : 0;
    const uint32_t floor_key = ng == top_k ? static_cast<uint32_t>(st.e[ng - 1] >> 32) : 0u;
    wave_lds_fence();
    const int gid = static_cast<int>(compose_index(mine));
    // 3. Their values that reach the k-th group's maximum, four loads ahead.
    list = TopList{0, 0};
    constexpr int U = 4;
    for (int b0 = 0; b0 < ng; b0 += GPW * U) {
      float xv[U][E];
      int64_t col[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + u * GPW + lane / LPG;
        const int gi = __shfl(gid, b < ng ? b : 0, kWave);
        col[u] = b < ng ? static_cast<int64_t>(gi) * GW + (lane % LPG) * E : v;
        load_row_chunk<T, VEC>(row, col[u], v, xv[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t key = order_key(xv[u][e] * inv_t);
          top_push(st, list, top_k, col[u] + e < v && key >= floor_key,
                   compose(key, static_cast<uint32_t>(col[u] + e)));
        }
    }
    top_rank(st, list, top_k);
    if (lane < top_k) {
      const uint64_t c = st.e[lane];
      out.top_logp[r * top_k + lane] = order_value(static_cast<uint32_t>(c >> 32)) - L;
      out.top_ids[r * top_k + lane] = static_cast<int64_t>(compose_index(c));
    }
    wave_lds_fence();
  }
}

// ---------------------------------------------------------------------------
// Gradient of the logits.  Thread (x, tid) owns one 16-byte chunk of every
// row it visits, as logp_bwd_kernel does, so the launch streams the matrix in
// address order.  The row's entries (given tokens, then alternatives) come in
// 64 at a time, one a lane: every wave adds their gradients to G in one fixed
// tree, and a ballot picks the entries inside the wave's own 64 chunks, whose
// gradients go to their element in ascending entry order.  No LDS, no barrier,
// no atomics; an entry that occurs twice is added twice.
// ---------------------------------------------------------------------------
template <typename T, bool VEC, bool ENT>
__global__ __launch_bounds__(kFinBlock) void token_bwd_kernel(
    const T* logits, int64_t ld, int64_t n, int64_t v, TokenView tok, TopView alt,
    const float* __restrict__ lse, const float* __restrict__ grad,
    const float* __restrict__ grad_top, const float* __restrict__ ent,
    const float* __restrict__ gent, T* dlogits, int64_t ld_out) {
  constexpr int E = Elt<T>::kPerChunk;
  const int lane = threadIdx.x % kWave;
  const int64_t wave0 =
      (static_cast<int64_t>(blockIdx.x) * kFinBlock +
       __builtin_amdgcn_readfirstlane(threadIdx.x / kWave) * kWave) * E;  // the wave's first column
  if (wave0 >= v) return;
  const int64_t j0 = wave0 + lane * E;
  const int64_t entries = tok.m + alt.k;
  for (int64_t rr = blockIdx.y; rr < n; rr += gridDim.y) {
    const int64_t r = n - 1 - rr;  // last to first: what the forward read last may still be cached
    const bool active = row_active(tok, r, lane);
    float x[E], u[E];
#pragma unroll
    for (int e = 0; e < E; ++e) u[e] = 0.0f;
    float G = 0.0f;
    if (active) {
      load_row_chunk<T, VEC>(logits + r * ld, j0, v, x);
      for (int64_t i0 = 0; i0 < entries; i0 += kWave) {
        const int64_t i = i0 + lane;
        int64_t col = -1;
        float g = 0.0f;
        if (i < entries) entry_at(tok, alt, grad, grad_top, r, i, col, g);
        G = G + wave_sum(g);
        uint64_t hits = __builtin_amdgcn_ballot_w64(col >= wave0 && col < wave0 + kWave * E);
        const int off = static_cast<int>(col - wave0);
        while (hits) {
          const int b = __builtin_ctzll(hits);
          hits &= hits - 1;
          const int o = __builtin_amdgcn_readlane(off, b);
          const float gb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), b));
#pragma unroll
          for (int e = 0; e < E; ++e) u[e] = o == lane * E + e ? u[e] + gb : u[e];
        }
      }
      const float L = lse[r], ng = -G;
      const float H = ENT ? ent[r] : 0.0f, ngh = ENT ? -gent[r] : 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) u[e] = token_grad<ENT>(x[e] - L, u[e], ng, H, ngh);
    }
    store_row_chunk<T, VEC>(dlogits + r * ld_out, j0, v, u);
  }
}

// ---------------------------------------------------------------------------
// What the fused backward needs of every row: G, and the row's activity as an
// int32 target no column matches (-1), or -2 (its ignore_index) for a padding
// row.  One wave a row.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kFinBlock) void token_rows_kernel(
    int64_t n, TokenView tok, TopView alt, const float* __restrict__ grad,
    const float* __restrict__ grad_top, int32_t* __restrict__ act, float* __restrict__ gsum) {
  const int lane = threadIdx.x % kWave;
  const int64_t entries = tok.m + alt.k;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kFinWaves + threadIdx.x / kWave; r < n;
       r += static_cast<int64_t>(gridDim.x) * kFinWaves) {
    const bool active = row_active(tok, r, lane);
    if (gsum) {
      float G = 0.0f;
      for (int64_t i0 = 0; i0 < entries; i0 += kWave) {
        int64_t col = -1;
        float g = 0.0f;
        if (active && i0 + lane < entries)
          entry_at(tok, alt, grad, grad_top, r, i0 + lane, col, g);
        G = G + wave_sum(g);
      }
      if (lane == 0) gsum[r] = G;
    }
    if (lane == 0) act[r] = active ? -1 : -2;
  }
}

// ---------------------------------------------------------------------------
// The entries of one vocabulary chunk of the fused backward's dz.  The dz
// kernel has written -G p (and the entropy term) everywhere; every distinct
// (row, column) of the row's entries inside [c0, c0 + cols) is written again
// with its gradients added before the one bf16 rounding.  p comes from the
// forward's log-probability x - lse, the very difference the dz kernel takes.
// One wave a row; the entries' columns and gradients sit in LDS.
// ---------------------------------------------------------------------------
template <bool ENT>
__global__ __launch_bounds__(kWave) void token_dz_kernel(
    int64_t n, int64_t v, TokenView tok, TopView alt, const float* __restrict__ logp,
    const float* __restrict__ top_logp, const float* __restrict__ grad,
    const float* __restrict__ grad_top, const float* __restrict__ gsum,
    const float* __restrict__ ent, const float* __restrict__ gent, float inv_t, int64_t c0,
    int64_t cols, uint16_t* __restrict__ dz) {
  __shared__ int32_t scol[kMaxEntries];
  __shared__ float sg[kMaxEntries];
  const int lane = threadIdx.x;
  const int entries = static_cast<int>(tok.m + alt.k);
  for (int64_t r = blockIdx.x; r < n; r += gridDim.x) {
    if (!row_active(tok, r, lane)) continue;
    for (int i = lane; i < entries; i += kWave) {
      int64_t col = -1;
      float g = 0.0f;
      entry_at(tok, alt, grad, grad_top, r, i, col, g);
      const bool in = col >= c0 && col < c0 + cols && col < v;
      scol[i] = in ? static_cast<int32_t>(col - c0) : -1;
      sg[i] = g;
    }
    wave_lds_fence();
    for (int i = lane; i < entries; i += kWave) {
      const int32_t c = scol[i];
      if (c < 0) continue;
      float u = 0.0f;
      int first = i;
      for (int j = 0; j < entries; ++j)
        if (scol[j] == c) {
          u = u + sg[j];
          first = min(first, j);
        }
      if (first != i) continue;  // one writer a column
      const float dl = i < tok.m ? logp[r * tok.m + i] : top_logp[r * alt.k + (i - tok.m)];
      float d = token_grad<ENT>(dl, u, -gsum[r], ENT ? ent[r] : 0.0f, ENT ? -gent[r] : 0.0f);
      if (inv_t != 1.0f) d = d * inv_t;
      dz[kblocked_at(r, c, cols / 32)] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(d));
    }
    wave_lds_fence();
  }
}

unsigned clamp_grid(int64_t blocks) {
  return static_cast<unsigned>(blocks < 1 ? 1 : blocks < kMaxBlocks ? blocks : kMaxBlocks);
}

template <typename T, int C, bool VEC>
void partials_typed(const void* logits, int64_t ld, int64_t n, int64_t v, const TokenView& tok,
                    int ntiles, int segs, int tps, float* pm, float* ps, float* pw, float* gm,
                    hipStream_t s) {
  auto kern = gm ? (pw ? token_partials_kernel<T, C, VEC, true, true>
                       : token_partials_kernel<T, C, VEC, false, true>)
                 : (pw ? token_partials_kernel<T, C, VEC, true, false>
                       : token_partials_kernel<T, C, VEC, false, false>);
  hipLaunchKernelGGL(kern, dim3(clamp_grid(n * segs)), dim3(kPartBlock), 0, s,
                     static_cast<const T*>(logits), ld, n, v, tok, ntiles, segs, tps, pm, ps, pw,
                     gm);
}

template <typename T, bool VEC>
void partials_chunks(int chunks, const void* logits, int64_t ld, int64_t n, int64_t v,
                     const TokenView& tok, int ntiles, int segs, int tps, float* pm, float* ps,
                     float* pw, float* gm, hipStream_t s) {
  switch (chunks) {
    case 1: return partials_typed<T, 1, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 2: return partials_typed<T, 2, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 4: return partials_typed<T, 4, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 8: return partials_typed<T, 8, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 16: return partials_typed<T, 16, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
  }
}

template <typename T, int LPG, bool VEC>
void finish_typed(const void* x, int64_t ld, float inv_t, const float* pt, int64_t n, int64_t v,
                  const TokenView& tok, int ntiles, const float* pm, const float* ps,
                  const float* pw, const float* gm, int64_t groups, int top_k, const TokenOut& out,
                  hipStream_t s) {
  auto kern = out.ent ? token_finish_kernel<T, LPG, VEC, true>
                      : token_finish_kernel<T, LPG, VEC, false>;
  hipLaunchKernelGGL(kern, dim3(clamp_grid((n + kFinWaves - 1) / kFinWaves)), dim3(kFinBlock), 0,
                     s, static_cast<const T*>(x), ld, inv_t, pt, n, v, tok, ntiles, pm, ps,
                     pw ? pw : ps, gm, groups, top_k, out);
}

}  // namespace

int64_t token_groups(int chunks, int64_t ntiles) { return ntiles * chunks * 4; }

void launch_token_partials(int dtype, bool vec, int chunks, const void* logits, int64_t ld,
                           int64_t n, int64_t v, const TokenView& tok, int ntiles, float* pm,
                           float* ps, float* pw, float* gm, hipStream_t s) {
  // Segments: enough (row, segment) items for the GPU, each at least one
  // round of the workgroup's eight waves.
  const int most = (ntiles + kPartWaves - 1) / kPartWaves;
  const int64_t want = (4 * 8 * static_cast<int64_t>(xcd_cus()) + n - 1) / n;
  const int segs0 = static_cast<int>(want < most ? want : most);
  const int tps = (ntiles + segs0 - 1) / segs0;
  const int segs = (ntiles + tps - 1) / tps;
#define ITL_PARTS(T)                                                                             \
  vec ? partials_chunks<T, true>(chunks, logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw,   \
                                 gm, s)                                                          \
      : partials_chunks<T, false>(chunks, logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw,  \
                                  gm, s)
  if (dtype == kF32) ITL_PARTS(float);
  else if (dtype == kF16) ITL_PARTS(_Float16);
  else ITL_PARTS(uint16_t);
#undef ITL_PARTS
}

void launch_token_finish(int dtype, bool vec, bool vocab_tiles, const void* x, int64_t ld,
                         float inv_t, const float* pt, int64_t n, int64_t v, const TokenView& tok,
                         int ntiles, const float* pm, const float* ps, const float* pw,
                         const float* gm, int64_t groups, int top_k, const TokenOut& out,
                         hipStream_t s) {
#define ITL_FIN(T, LPG)                                                                          \
  vec ? finish_typed<T, LPG, true>(x, ld, inv_t, pt, n, v, tok, ntiles, pm, ps, pw, gm, groups,  \
                                   top_k, out, s)                                                \
      : finish_typed<T, LPG, false>(x, ld, inv_t, pt, n, v, tok, ntiles, pm, ps, pw, gm, groups, \
                                    top_k, out, s)
  // a group is 16 lanes' chunks of a streamed row, or a 256-column vocabulary
  // tile of the LM head (fp32: 64 lanes, bf16: 32)
  if (vocab_tiles) {
    if (dtype == kF32) ITL_FIN(float, 64);
    else ITL_FIN(uint16_t, 32);
  } else {
    if (dtype == kF32) ITL_FIN(float, 16);
    else if (dtype == kF16) ITL_FIN(_Float16, 16);
    else ITL_FIN(uint16_t, 16);
  }
#undef ITL_FIN
}

void launch_token_bwd(int dtype, bool vec, const void* logits, int64_t ld, int64_t n, int64_t v,
                      const TokenView& tok, const TopView& alt, const float* lse,
                      const float* grad, const float* grad_top, const float* ent,
                      const float* gent, void* dlogits, int64_t ld_out, hipStream_t s) {
  const int64_t per = dtype == kF32 ? 4 : 8;
  const int64_t chunks = (v + per - 1) / per;
  const dim3 grid(static_cast<unsigned>((chunks + kFinBlock - 1) / kFinBlock),
                  static_cast<unsigned>(n < kMaxRowsY ? n : kMaxRowsY));
#define ITL_BWD(T)                                                                              \
  do {                                                                                          \
    auto kern = vec ? (ent ? token_bwd_kernel<T, true, true> : token_bwd_kernel<T, true, false>) \
                    : (ent ? token_bwd_kernel<T, false, true>                                   \
                           : token_bwd_kernel<T, false, false>);                                \
    hipLaunchKernelGGL(kern, grid, dim3(kFinBlock), 0, s, static_cast<const T*>(logits), ld, n, \
                       v, tok, alt, lse, grad, grad_top, ent, gent, static_cast<T*>(dlogits),   \
                       ld_out);                                                                 \
  } while (0)
  if (dtype == kF32) ITL_BWD(float);
  else if (dtype == kF16) ITL_BWD(_Float16);
  else ITL_BWD(uint16_t);
#undef ITL_BWD
}

void launch_token_rows(int64_t n, const TokenView& tok, const TopView& alt, const float* grad,
                       const float* grad_top, int32_t* act, float* gsum, hipStream_t s) {
  hipLaunchKernelGGL(token_rows_kernel, dim3(clamp_grid((n + kFinWaves - 1) / kFinWaves)),
                     dim3(kFinBlock), 0, s, n, tok, alt, grad, grad_top, act, gsum);
}

void launch_token_dz(const TokenDz& t, int64_t n, int64_t v, float inv_t, const float* ent,
                     const float* gent, int64_t c0, int64_t cols, uint16_t* dz, hipStream_t s) {
  auto kern = ent ? token_dz_kernel<true> : token_dz_kernel<false>;
  hipLaunchKernelGGL(kern, dim3(clamp_grid(n)), dim3(kWave), 0, s, n, v, t.tok, t.alt, t.logp,
                     t.top_logp, t.grad, t.grad_top, t.gsum, ent, gent, inv_t, c0, cols, dz);
}

}  // namespace itl
