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
// 4096 such bf16 rows (5% padding) with the entropy take 215 us in the pass over
// the rows (5.5 TB/s) and 30 in the finishing one.  Without group maxima the
// pass runs at 6.4 TB/s; it is bound by the vector units, about 11 issue slots
// a value (the exponential alone four).  Loading the next tile ahead measured
// 7% slower (150 registers instead of 94).
#include "launch.h"
#include "logp_device.h"
#include "token_device.h"

namespace itl {

namespace {

constexpr int kPartBlock = 256;  // 4 waves, one tile each at a time
constexpr int kPartWaves = kPartBlock / kWave;
constexpr int kFinBlock = 256;   // 4 waves
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

// The maxima over each row of 16 lanes of C values, in every lane: xor 1, xor 2,
// half mirror, mirror, each one vector maximum that takes its partner through
// DPP (the compiler's own form is a move, a wait, a quieting and a maximum).
// The leading s_nop covers the wait that a DPP read needs after the write of
// its source; C values in turn cover the steps after it as well.
#define ITL_ROW_MAX_STEP(CTRL)                                                                 \
  if constexpr (C % 4 == 0) {                                                                  \
    _Pragma("unroll") for (int j = 0; j < C; j += 4) asm(                                      \
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 " CTRL " row_mask:0xf bank_mask:0xf\n\t"          \
        "v_max_f32_dpp %1, %1, %1 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                     \
        "v_max_f32_dpp %2, %2, %2 " CTRL " row_mask:0xf bank_mask:0xf\n\t"                     \
        "v_max_f32_dpp %3, %3, %3 " CTRL " row_mask:0xf bank_mask:0xf"                         \
        : "+v"(g[j]), "+v"(g[j + 1]), "+v"(g[j + 2]), "+v"(g[j + 3]));                         \
  } else {                                                                                     \
    _Pragma("unroll") for (int j = 0; j < C; ++j) asm(                                         \
        "s_nop 1\n\tv_max_f32_dpp %0, %0, %0 " CTRL " row_mask:0xf bank_mask:0xf"              \
        : "+v"(g[j]));                                                                         \
  }
template <int C>
__device__ __forceinline__ void row16_max(float (&g)[C]) {
  ITL_ROW_MAX_STEP("quad_perm:[1,0,3,2]")
  ITL_ROW_MAX_STEP("quad_perm:[2,3,0,1]")
  ITL_ROW_MAX_STEP("row_half_mirror")
  ITL_ROW_MAX_STEP("row_mirror")
}
#undef ITL_ROW_MAX_STEP

// tile_stats of logp_device.h (same sum tree, same bits; rows of any
// alignment in 16-byte loads) that, with TOP, also leaves the maxima of the
// tile's C * 4 groups in gm: the maximum is exact in any order, so it is taken
// along the groups first (four lane moves a chunk), then over the chunks, then
// over the four rows of 16 lanes.
template <typename T, int C, bool VEC, bool ENT, bool TOP>
__device__ __forceinline__ void token_tile_stats(const T* row, int64_t col0, int64_t v, uint32_t* gm,
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
  float g[C];
#pragma unroll
  for (int j = 0; j < C; ++j) {
    g[j] = x[j][0];
#pragma unroll
    for (int e = 1; e < E; ++e) g[j] = fmaxf(g[j], x[j][e]);
  }
  if constexpr (TOP) row16_max<C>(g);
  float m = g[0], mine = g[0];
#pragma unroll
  for (int j = 1; j < C; ++j) {
    m = fmaxf(m, g[j]);
    if constexpr (TOP) mine = (lane & 15) == j ? g[j] : mine;
  }
  constexpr bool kLds = C * E > 16;  // where the partners come from: as tile_stats
  if constexpr (TOP) {
    // lane (row r16, place j < C) stores group 4 j + r16 (ascending columns)
    if ((lane & 15) < C) gm[(lane & 15) * 4 + (lane >> 4)] = order_key(mine);
    m = swap_combine16(m, true);
    m = swap_combine32(m, true);
  } else {
    m = kLds ? wave_max_lds(m) : wave_max(m);
  }
  m = tile_max(x, m);
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
    float* __restrict__ pw, uint32_t* __restrict__ gm) {
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

// The 8-bit head's merge (its own arithmetic, so without merge_lse_t's one
// ascending chain, whose broadcast reads took 100 us for 4096 rows of 1187
// tiles): lane l folds tiles l, l + 64, ... in ascending order, the wave adds
// up in a butterfly.  All lanes return the lse (and H).
template <bool ENT>
__device__ __forceinline__ float merge_tree(const float* m, const float* s, const float* w,
                                            int ntiles, int lane, float* ent) {
  constexpr int U = 20;  // 1280 tiles in registers, about 164000 columns
  float mr[U], sr[U], wr[ENT ? U : 1];
  float mx = -INFINITY, acc = 0.0f, b = 0.0f;
  const bool one = ntiles <= U * kWave;
  auto load = [&](int k0, bool all) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * kWave + lane;
      mr[u] = m[k < ntiles ? k : 0];
      if (all) {
        sr[u] = s[k < ntiles ? k : 0];
        if constexpr (ENT) wr[u] = w[k < ntiles ? k : 0];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u * kWave + lane >= ntiles) mr[u] = -INFINITY;
  };
  for (int k0 = 0; k0 < ntiles; k0 += U * kWave) {
    load(k0, one);
#pragma unroll
    for (int u = 0; u < U; ++u) mx = max_exact(mx, mr[u]);
  }
#pragma unroll
  for (int o = 1; o < kWave; o <<= 1) mx = max_exact(mx, __shfl_xor(mx, o, kWave));
  for (int k0 = 0; k0 < ntiles; k0 += U * kWave) {
    if (!one) load(k0, true);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (mr[u] != -INFINITY) {  // a tile of masked columns only holds nothing
        const float e = exp_sub(mr[u], mx);
        acc = fmaf(sr[u], e, acc);
        if constexpr (ENT)  // e = 0: as in merge_lse_t
          b = fmaf(e > 0.0f ? fmaf(sr[u], mr[u] - mx, wr[u]) : 0.0f, e, b);
      }
  }
  const float la = log_nat(wave_sum(acc));
  if constexpr (ENT) *ent = la - wave_sum(b) / wave_sum(acc);
  return mx + la;
}

// ---------------------------------------------------------------------------
// Finish.  One wave a row merges the tile statistics (merge_lse_t: the bits of
// logp_fwd; merge_tree for the 8-bit head) and writes lse, entropy and the given
// tokens; with alternatives it then selects them, or, with few rows (per = 2),
// a second wave does so meanwhile and takes the lse at the end.
//   x          the row's logits ([n, ld], row r at x + r * ld), or null: then
//              M = 1, k = 0 and the token's logit is pt[r].
//   gm         what orders the groups of row r, at gm + r * groups: the order
//              keys of their maxima, or with HEAD the maxima themselves (the
//              LM head's tile table).  Group g = columns [g GW, g GW + GW).
//   inv_t      HEAD: factor on the logits read from x (the tables hold scaled
//              ones).
// Latency is what counts: a row is a chain of a few dependent loads, so all
// loads of a stage are in flight together, and what is executed is kept short
// (code that runs once is bound by its fetch): a lane marks its candidates among
// the values in a bit mask and reads the few marked ones again instead of
// carrying an append for each of up to 64.
// ---------------------------------------------------------------------------
// groups a lane holds at once: 640 of 256 columns or 1280 of 128, about 164000
// columns
template <int GW>
constexpr int kKeys = GW == 256 ? 10 : 20;

// Order keys of the groups b0 + 64 c + lane; 0 (below every key) past the last.
// The LM head's tile maximum is NaN as soon as one of the tile's logits is, while
// a NaN ranks as -inf beside the others: such a tile's key is kNanKey (above
// every key) until ordered_keys has taken it from the logits.
constexpr uint32_t kNanKey = 0xffffffffu;

template <bool HEAD>
__device__ __forceinline__ uint32_t group_key(uint32_t g) {
  if constexpr (!HEAD) return g;
  const float m = __uint_as_float(g);
  return m != m ? kNanKey : order_key(m);
}
template <int GW, bool HEAD>
__device__ __forceinline__ void load_keys(const uint32_t* g, int64_t b0, int64_t groups, int lane,
                                          uint32_t (&key)[kKeys<GW>]) {
#pragma unroll
  for (int c = 0; c < kKeys<GW>; ++c) {
    const int64_t i = b0 + c * kWave + lane;
    key[c] = g[i < groups ? i : 0];
  }
#pragma unroll
  for (int c = 0; c < kKeys<GW>; ++c) {
    const uint32_t k = group_key<HEAD>(key[c]);
    key[c] = b0 + c * kWave + lane < groups ? k : 0u;
  }
}

// Replaces the kNanKey of tiles b0 + 64 c + lane by the key of the greatest of
// the tile's logits that is no NaN (-inf when there is none), one tile after the
// other: a row with a NaN has no probabilities, so what counts is that its
// alternatives are right, and that rows without one only pay the test (no time
// in 249 us for 16 rows).  16 rows of nothing but NaN take 1.2 ms at V = 151936,
// 4096 such rows 2.5 ms more than others.
template <typename T, int GW, int N>
__device__ __forceinline__ void ordered_keys(const T* row, float inv_t, uint32_t v, int64_t b0,
                                             int lane, uint32_t (&key)[N]) {
  uint32_t top = key[0];
#pragma unroll
  for (int c = 1; c < N; ++c) top = max(top, key[c]);
  while (const uint64_t bad = __builtin_amdgcn_ballot_w64(top == kNanKey)) {
    const int b = __builtin_ctzll(bad);
    int mine = 0;  // this lane's last such tile
#pragma unroll
    for (int c = 0; c < N; ++c) mine = key[c] == kNanKey ? c : mine;
    const int at = __builtin_amdgcn_readlane(mine, b);
    const uint32_t c0 = static_cast<uint32_t>(b0 + at * kWave + b) * GW;
    float m = -INFINITY;
#pragma unroll
    for (int o = 0; o < GW; o += kWave) {
      const uint32_t c = c0 + o + lane;
      if (c < v) m = fmaxf(m, Elt<T>::load(row, c) * inv_t);  // drops a NaN
    }
    const uint32_t k = order_key(wave_max(m));
    top = 0;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      key[c] = lane == b && c == at ? k : key[c];
      top = max(top, key[c]);
    }
  }
}

// The select wave's part: the row's top_k greatest values, in order, as
// composites at st.e[0 ..).  Returns when they are in LDS.
template <typename T, int GW, bool VEC, bool HEAD>
__device__ __forceinline__ void select_top(TopStage& st, const T* row, float inv_t, uint32_t v,
                                           const uint32_t* g, int64_t groups, int top_k,
                                           uint32_t (&key)[kKeys<GW>], int lane) {
  constexpr int E = Elt<T>::kPerChunk;
  constexpr int LPG = GW / E;            // lanes per group
  constexpr int GPW = kWave / LPG;       // groups one wave load covers
  constexpr int U = 8;                   // such loads in flight: 32, 16 or 8 groups
  auto logit = [&](uint32_t c) {
    const float z = Elt<T>::load(row, c);
    return HEAD ? z * inv_t : z;
  };
  // 1. A bound: the k-th greatest of 256 maxima, four a lane, over disjoint
  // sets of groups.  At least k groups reach it.
  const bool one_block = groups <= kKeys<GW> * kWave;
  uint32_t best[4] = {0, 0, 0, 0};
  for (int64_t b0 = 0; b0 < groups; b0 += kKeys<GW> * kWave) {
    if (b0 > 0) load_keys<GW, HEAD>(g, b0, groups, lane, key);
    if constexpr (HEAD) ordered_keys<T, GW>(row, inv_t, v, b0, lane, key);
#pragma unroll
    for (int c = 0; c < kKeys<GW>; ++c) best[c % 4] = max(best[c % 4], key[c]);
  }
  const uint32_t bound = max(wave_bound(best, top_k), 1u);
  // 2. The k greatest groups (or all, when there are fewer).  Few groups
  // reach the bound; the list is only cut in between when more than it holds
  // do (plateaus), in a second walk.
  TopList list{0, 0};
  int reach = 0, place = 0;
  if (one_block) {
#pragma unroll
    for (int c = 0; c < kKeys<GW>; ++c) reach += key[c] >= bound;
  }
  if (one_block && top_reserve(st, list, reach, place)) {
#pragma unroll
    for (int c = 0; c < kKeys<GW>; ++c)
      if (key[c] >= bound)
        st.e[place++] = compose(key[c], static_cast<uint32_t>(c * kWave + lane));
  } else {
    for (int64_t c0 = 0; c0 < groups; c0 += kWave) {
      const int64_t c = c0 + lane;
      uint32_t one[1] = {c < groups ? group_key<HEAD>(g[c]) : 0u};
      if constexpr (HEAD) ordered_keys<T, GW>(row, inv_t, v, c0, lane, one);
      top_push(st, list, top_k, one[0] >= bound, compose(one[0], static_cast<uint32_t>(c)));
    }
  }
  top_rank(st, list, top_k);
  const int ng = list.n;
  // a value below the k-th group's maximum is none of the k greatest
  const uint64_t last = st.e[ng - 1];
  const float floor_x = ng == top_k ? order_value(static_cast<uint32_t>(last >> 32)) : -INFINITY;
  st.group[lane] = compose_index(st.e[lane < ng ? lane : 0]);
  wave_lds_fence();
  // 3. The values that are not below it: a register block of groups at a
  // time while the list holds them, else value by value.
  list = TopList{0, 0};
  bool fits = true;
  for (int b0 = 0; b0 < ng && fits; b0 += GPW * U) {
    uint64_t mark = 0;
    auto column = [&](int u) {
      const int b = b0 + u * GPW + lane / LPG;
      return b < ng ? min(st.group[b] * GW + (lane % LPG) * E, v) : v;
    };
    // Whole chunks (all but the row's last one) load without a branch, all
    // of them in flight together.
    bool part = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = column(u);
      part |= c < v && v - c < E;
    }
    if (__builtin_amdgcn_ballot_w64(part) == 0 && v >= E) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t c = column(u);
        q[u] = load_whole_chunk<T, VEC>(row + (c < v ? c : 0));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float xv[E];
        widen_chunk<T>(q[u], xv);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < E; ++e)
          m |= (HEAD ? xv[e] * inv_t : xv[e]) < floor_x ? 0u : 1u << e;
        if (column(u) >= v) m = 0;  // no such group, or past the row's end
        mark |= static_cast<uint64_t>(m) << (u * E);
      }
    } else {
#pragma unroll 1
      for (int u = 0; u < U; ++u)
#pragma unroll 1
        for (int e = 0; e < E; ++e) {
          const uint32_t c = column(u) + e;
          if (c < v && c >= column(u) && !(logit(c) < floor_x)) mark |= uint64_t{1} << (u * E + e);
        }
    }
    fits = top_reserve(st, list, __popcll(mark), place);
    while (fits && mark) {
      const int i = __builtin_ctzll(mark);
      mark &= mark - 1;
      const uint32_t c = column(i / E) + i % E;
      st.e[place++] = compose(order_key(logit(c)), c);
    }
  }
  if (!fits) {
    list = TopList{0, 0};
    for (int b = 0; b < ng; ++b) {
      const uint32_t c0 = st.group[b] * GW;
      for (int o = 0; o < GW; o += kWave) {
        const uint32_t c = c0 + o + lane;
        const float z = c < v ? logit(c) : 0.0f;
        top_push(st, list, top_k, c < v && !(z < floor_x),
                 compose(order_key(z), c));
      }
    }
  }
  top_rank(st, list, top_k);
}

template <typename T, int GW, bool VEC, bool ENT, bool HEAD>
__global__ __launch_bounds__(kFinBlock) void token_finish_kernel(
    const T* __restrict__ x, int64_t ld, float inv_t, const float* __restrict__ pt, int64_t n,
    int64_t v, TokenView tok, int ntiles, const float* __restrict__ pm,
    const float* __restrict__ ps, const float* __restrict__ pw, const uint32_t* __restrict__ gm,
    int64_t groups, int top_k, int per, TokenOut out) {
  __shared__ union {
    MergeStage merge;
    TopStage top;
  } stage[kFinWaves];
  __shared__ float row_lse[kFinWaves];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  const int rows = kFinWaves / per;        // rows a workgroup
  const int slot = wave / per;
  const bool merges = wave % per == 0, selects = top_k > 0 && wave % per == per - 1;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows; r0 < n;
       r0 += static_cast<int64_t>(gridDim.x) * rows) {
    const int64_t r = r0 + slot;
    bool live = r < n;
    // The group keys or the given tokens are on their way first.
    uint32_t key[kKeys<GW>];
    const uint32_t* g = gm + r * groups;
    if (live && selects) load_keys<GW, HEAD>(g, 0, groups, lane, key);
    int64_t t0 = live && lane < tok.m ? tok.at(r, lane) : tok.ignore;
    if (live && tok.m > 0 && __builtin_amdgcn_ballot_w64(t0 != tok.ignore) == 0)
      live = row_active(tok, r, lane);
    const T* row = x + r * ld;
    if (!live) {
      if (r < n && merges) {  // a padding row
        for (int64_t i = lane; i < tok.m; i += kWave) out.logp[r * tok.m + i] = 0.0f;
        if (lane == 0) {
          if (out.lse) out.lse[r] = 0.0f;
          if constexpr (ENT) out.ent[r] = 0.0f;
        }
      }
    }
    if (live && merges) {
      auto logit = [&](int64_t c) {
        const float z = Elt<T>::load(row, c);
        return HEAD ? z * inv_t : z;
      };
      float x0 = 0.0f;
      if (t0 != tok.ignore && t0 >= 0 && t0 < v) x0 = x ? logit(t0) : pt[r];
      float h = 0.0f;
      const int64_t at = r * ntiles;
      float L;
      if constexpr (HEAD && GW == 128)
        L = merge_tree<ENT>(pm + at, ps + at, pw + at, ntiles, lane, &h);
      else
        L = merge_lse_t<ENT, HEAD ? 10 : 1>(pm + at, ps + at, pw + at, ntiles, 1,
                                            stage[wave].merge, &h);
      if (lane == 0) {
        row_lse[slot] = L;
        if (out.lse) out.lse[r] = L;
        if constexpr (ENT) out.ent[r] = h;
      }
      for (int64_t i = lane; i < tok.m; i += kWave) {
        if (i >= kWave) {
          t0 = tok.at(r, i);
          x0 = t0 != tok.ignore && t0 >= 0 && t0 < v ? logit(t0) : 0.0f;
        }
        out.logp[r * tok.m + i] = t0 == tok.ignore ? 0.0f : combine(x0, L, t0 >= 0 && t0 < v);
      }
    }
    if (live && selects) {
      wave_lds_fence();
      select_top<T, GW, VEC, HEAD>(stage[wave].top, row, inv_t, static_cast<uint32_t>(v), g,
                                   groups, top_k, key, lane);
    }
    if (per == 2) __syncthreads();  // the row's lse
    if (selects && r < n && lane < top_k) {
      const uint64_t c = stage[wave].top.e[lane];
      out.top_logp[r * top_k + lane] =
          live ? order_value(static_cast<uint32_t>(c >> 32)) - row_lse[slot] : 0.0f;
      out.top_ids[r * top_k + lane] = live ? static_cast<int64_t>(compose_index(c)) : -1;
    }
    if (per == 2) __syncthreads();  // before the stages are taken again
    wave_lds_fence();
  }
}

// ---------------------------------------------------------------------------
// Gradient of the logits.  A wave owns kBwdChunks * 64 neighbouring 16-byte
// chunks of a row (lane l chunks l, l + 64, ...), so a launch streams the
// matrix in address order.  The row's entries (given tokens, then
// alternatives) come in 64 at a time, one a lane: every wave adds their
// gradients to G in one fixed tree, and a ballot picks the entries inside the
// wave's own columns, whose gradients go to their element in ascending entry
// order.  No LDS, no barrier, no atomics; an entry that occurs twice is added
// twice.
// Bound by memory, but a wave first has to know that its row is no padding:
// the entries' load, then the logits' (several chunks a lane, so that the wait
// for the entries is shared), and G is summed while the logits arrive.  4096 x
// 128256 bf16 with 16 entries a row and the entropy term takes 370 us (5.7 TB/s)
// with four chunks a lane; two 465, three 460, six 394, eight 606 (registers).
// ---------------------------------------------------------------------------
constexpr int kBwdChunks = 4;

template <typename T, bool VEC, bool ENT>
__global__ __launch_bounds__(kFinBlock) void token_bwd_kernel(
    const T* logits, int64_t ld, int64_t n, int64_t v, TokenView tok, TopView alt,
    const float* __restrict__ lse, const float* __restrict__ grad,
    const float* __restrict__ grad_top, const float* __restrict__ ent,
    const float* __restrict__ gent, T* dlogits, int64_t ld_out) {
  constexpr int E = Elt<T>::kPerChunk;
  constexpr int NC = kBwdChunks;
  constexpr int kSpan = NC * kWave * E;  // columns of a wave
  const int lane = threadIdx.x % kWave;
  const int64_t wave0 = (static_cast<int64_t>(blockIdx.x) * kFinWaves +
                         __builtin_amdgcn_readfirstlane(threadIdx.x / kWave)) * kSpan;
  if (wave0 >= v) return;
  const int entries = static_cast<int>(tok.m + alt.k);
  for (int64_t rr = blockIdx.y; rr < n; rr += gridDim.y) {
    const int64_t r = n - 1 - rr;  // last to first: what the forward read last may still be cached
    int64_t col = -1;
    float g = 0.0f;
    if (lane < entries) entry_at(tok, alt, grad, grad_top, r, lane, col, g);
    const float L = lse[r];
    const float H = ENT ? ent[r] : 0.0f, ngh = ENT ? -gent[r] : 0.0f;
    // an ignored entry has col = -1; so may an invalid token, hence the rest
    const bool active = __builtin_amdgcn_ballot_w64(lane < tok.m && col != -1) != 0 ||
                        row_active(tok, r, lane);
    const bool whole = wave0 + kSpan <= v;
    const T* row = logits + r * ld + wave0 + lane * E;
    T* drow = dlogits + r * ld_out + wave0 + lane * E;
    uint4 q[NC];
    float u[NC][E];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      q[c] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int e = 0; e < E; ++e) u[c][e] = 0.0f;
    }
    if (active) {
      if (whole) {
#pragma unroll
        for (int c = 0; c < NC; ++c) q[c] = load_whole_chunk<T, VEC>(row + c * kWave * E);
      } else {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          float x[E];
          load_row_chunk<T, VEC>(row, c * kWave * E, v - wave0 - lane * E, x);
          q[c] = round_chunk<T>(x);  // exact: the values are of type T
        }
      }
      float G = 0.0f;
      for (int i0 = 0; i0 < entries; i0 += kWave) {
        if (i0 > 0) {
          col = -1;
          g = 0.0f;
          if (i0 + lane < entries) entry_at(tok, alt, grad, grad_top, r, i0 + lane, col, g);
        }
        G = G + wave_sum(g);
        uint64_t hits = __builtin_amdgcn_ballot_w64(col >= wave0 && col < wave0 + kSpan);
        const int off = static_cast<int>(col - wave0);
        while (hits) {
          const int b = __builtin_ctzll(hits);
          hits &= hits - 1;
          const int o = __builtin_amdgcn_readlane(off, b);
          const float gb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), b));
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < E; ++e)
              u[c][e] = o == (c * kWave + lane) * E + e ? u[c][e] + gb : u[c][e];
        }
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float x[E];
        widen_chunk<T>(q[c], x);
#pragma unroll
        for (int e = 0; e < E; ++e) u[c][e] = token_grad<ENT>(x[e] - L, u[c][e], -G, H, ngh);
      }
    }
    if (whole) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        store_whole_chunk<T, VEC>(drow + c * kWave * E, round_chunk<T>(u[c]));
    } else {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        store_row_chunk<T, VEC>(drow, c * kWave * E, v - wave0 - lane * E, u[c]);
    }
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
                    int ntiles, int segs, int tps, float* pm, float* ps, float* pw, uint32_t* gm,
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
                     float* pw, uint32_t* gm, hipStream_t s) {
  switch (chunks) {
    case 1: return partials_typed<T, 1, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 2: return partials_typed<T, 2, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 4: return partials_typed<T, 4, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 8: return partials_typed<T, 8, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
    case 16: return partials_typed<T, 16, VEC>(logits, ld, n, v, tok, ntiles, segs, tps, pm, ps, pw, gm, s);
  }
}

template <typename T, int GW, bool VEC, bool HEAD>
void finish_typed(const void* x, int64_t ld, float inv_t, const float* pt, int64_t n, int64_t v,
                  const TokenView& tok, int ntiles, const float* pm, const float* ps,
                  const float* pw, const void* gm, int64_t groups, int top_k, const TokenOut& out,
                  hipStream_t s) {
  auto kern = out.ent ? token_finish_kernel<T, GW, VEC, true, HEAD>
                      : token_finish_kernel<T, GW, VEC, false, HEAD>;
  // Two waves a row while the GPU has waves to spare: a latency of 14 instead of
  // 20 us for 16 rows of the LM head, but 36 instead of 30 us for 4096 rows.
  const int per = top_k > 0 && n <= 8 * static_cast<int64_t>(xcd_cus()) * 2 ? 2 : 1;
  const int64_t rows = kFinWaves / per;
  hipLaunchKernelGGL(kern, dim3(clamp_grid((n + rows - 1) / rows)), dim3(kFinBlock), 0, s,
                     static_cast<const T*>(x), ld, inv_t, pt, n, v, tok, ntiles, pm, ps,
                     pw ? pw : ps, static_cast<const uint32_t*>(gm), groups, top_k, per, out);
}

}  // namespace

int64_t token_groups(int chunks, int64_t ntiles) { return ntiles * chunks * 4; }

void launch_token_partials(int dtype, bool vec, int chunks, const void* logits, int64_t ld,
                           int64_t n, int64_t v, const TokenView& tok, int ntiles, float* pm,
                           float* ps, float* pw, uint32_t* gm, hipStream_t s) {
  // Segments: enough (row, segment) items for the GPU, each at least one
  // round of the workgroup's four waves.
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

void launch_token_finish(int dtype, bool vec, int head_tile, const void* x, int64_t ld,
                         float inv_t, const float* pt, int64_t n, int64_t v, const TokenView& tok,
                         int ntiles, const float* pm, const float* ps, const float* pw,
                         const void* gm, int64_t groups, int top_k, const TokenOut& out,
                         hipStream_t s) {
#define ITL_FIN(T, GW, HEAD)                                                                     \
  vec ? finish_typed<T, GW, true, HEAD>(x, ld, inv_t, pt, n, v, tok, ntiles, pm, ps, pw, gm,     \
                                        groups, top_k, out, s)                                   \
      : finish_typed<T, GW, false, HEAD>(x, ld, inv_t, pt, n, v, tok, ntiles, pm, ps, pw, gm,    \
                                         groups, top_k, out, s)
  // a group is 16 lanes' chunks of a streamed row, or a vocabulary tile of the
  // LM head
  if (head_tile == 128) {
    ITL_FIN(float, 128, true);
  } else if (head_tile) {
    if (dtype == kF32) ITL_FIN(float, kLinearTile, true);
    else ITL_FIN(uint16_t, kLinearTile, true);
  } else {
    if (dtype == kF32) ITL_FIN(float, 64, false);
    else if (dtype == kF16) ITL_FIN(_Float16, 128, false);
    else ITL_FIN(uint16_t, 128, false);
  }
#undef ITL_FIN
}

void launch_token_bwd(int dtype, bool vec, const void* logits, int64_t ld, int64_t n, int64_t v,
                      const TokenView& tok, const TopView& alt, const float* lse,
                      const float* grad, const float* grad_top, const float* ent,
                      const float* gent, void* dlogits, int64_t ld_out, hipStream_t s) {
  const int64_t per = dtype == kF32 ? 4 : 8;
  const int64_t chunks = (v + per - 1) / per, block = kFinBlock * kBwdChunks;
  const dim3 grid(static_cast<unsigned>((chunks + block - 1) / block),
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
