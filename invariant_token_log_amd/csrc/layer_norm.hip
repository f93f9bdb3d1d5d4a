// Layer norm with dropout and the residual's addition before it, and its
// gradient, on gfx950.
//
//   s = rne(residual + drop(x));  m = mean(s),  rstd = 1 / sqrt(mean((s - m)^2) + eps)
//   y = rne((s - m) rstd w + b)
//   u = (s - m) rstd, g = dy w:  d = ds + rstd (g - mean(g) - u mean(g u))
//   dresidual = rne(d), dx = rne(drop's factor, or 0, times d)
//   dw = sum_r dy u,  db = sum_r dy
//
// Bound by memory: every element is read and written once, so a row stays in
// the registers of the team of threads that owns it: 64 threads for rows of up
// to 1024 elements, 256 up to 8192 and beyond that 1024 in the forward, 512 in
// the gradient, thread t holding the chunks of 8 elements t, t + TEAM, ...  The
// mean comes first and the squares are of differences from it, so a row far from
// zero loses nothing.  Rows too long for the registers (forward past 32768
// elements, 16384 in fp32; gradient past 12288, 8192 in fp32) are read again
// instead, from the caches.
// Each thread adds its elements in ascending order, the lanes of a wave follow
// in a butterfly and the waves in order: a row's results depend on h and the
// row alone.
// Measured, us (TB/s; a copy reaches 6.45).  Forward with a residual, calls in a
// row: 8192 x 4096 bf16 44, with dropout 42 (6.4), 4096 x 8192 bf16 44, 4096 x 4096
// fp32 44, 2048 x 16384 bf16 46, 8192 x 1024 bf16 15 (4.5); 2047 x 5117 fp16, rows off
// 16 bytes, 24 (3.5); behind a gradient, whose output the caches still write back,
// 50 to 55 for the first four.  (Mean and squares in one exchange a row, the squares
// from every wave's own mean: 44 with dropout, 78 for the longest.)
// Gradient, with the gradient of s, and with dropout and both gradients of it:
// 8192 x 4096 bf16 51 (5.2) and 71 (4.8), 4096 x 4096 fp32 51 (5.2) and 66 (5.1), 4096
// x 8192 bf16 61 (4.4) and 73 (4.6), 8192 x 1024 bf16 22 (3.1) and 26 (3.3): four waves
// a CU, each with its partial sums; 2048 x 16384 bf16 51 and 69, and 27 for the columns
// (3.5): read again; 2047 x 5117 fp16, rows off 16 bytes, 43 (1.9) and 51 (2.1): element
// by element in the chunks that are not whole.  The sum over the rows is 4 to 5
// more.  Rows two ahead, one exchange a row and the masks before it made no
// difference.
#include "layer_norm.h"

#include "launch.h"
#include "row_device.h"

namespace itl {

namespace {

// A row's chunk at element c, 0 past h.  VEC: 16-byte rows of whole chunks.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_chunk(const T* row, int64_t c, int64_t h) {
  if constexpr (VEC) {
    Raw<T> r;
#pragma unroll
    for (int p = 0; p < kRaw<T>; ++p) r.q[p] = make_uint4(0, 0, 0, 0);
    if (c < h) {
#pragma unroll
      for (int p = 0; p < kRaw<T>; ++p) r.q[p] = *(reinterpret_cast<const uint4*>(row + c) + p);
    }
    return r;
  } else {
    return load_raw<T, false>(row, c, h);
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int64_t c, int64_t h, const Raw<T>& r) {
  if constexpr (VEC) {
    if (c < h) {
#pragma unroll
      for (int p = 0; p < kRaw<T>; ++p) *(reinterpret_cast<uint4*>(row + c) + p) = r.q[p];
    }
  } else {
    store_raw<T, false>(row, c, h, r);
  }
}

// s of one chunk: x, dropped and added to the residual, rounded to its type.
template <typename T, bool DROP>
__device__ __forceinline__ Raw<T> stream_chunk(const Raw<T>& x, const Raw<T>& residual, bool add,
                                               const Drop& drop, uint64_t seed, int64_t r,
                                               int64_t chunk) {
  if (!DROP && !add) return x;
  float p[kE], q[kE];
  widen_raw<T>(x, p);
  if (add) widen_raw<T>(residual, q);
  if constexpr (DROP) {
    const uint4 u = drop_chunk(drop, seed, r, static_cast<uint32_t>(chunk));
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const bool keep = drop_keeps(drop, u, e);
      if (add)
        p[e] = keep ? fmaf(p[e], drop.factor, q[e]) : q[e];
      else
        p[e] = keep ? p[e] * drop.factor : 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) p[e] = p[e] + q[e];
  }
  return round_raw<T>(p);
}

// Adds a chunk's elements (0 past h), or the squares of their differences
// from m, in ascending order.
template <typename T>
__device__ __forceinline__ float add_chunk(const Raw<T>& s, float a) {
  float p[kE];
  widen_raw<T>(s, p);
#pragma unroll
  for (int e = 0; e < kE; ++e) a = a + p[e];
  return a;
}
template <typename T>
__device__ __forceinline__ float add_squares(const Raw<T>& s, int64_t c0, int64_t h, float m,
                                             float a) {
  float p[kE];
  widen_raw<T>(s, p);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float d = c0 + e < h ? p[e] - m : 0.0f;
    a = fmaf(d, d, a);
  }
  return a;
}

template <typename T>
__device__ __forceinline__ Raw<T> norm_chunk(const Raw<T>& s, const Raw<T>& w, const Raw<T>& b,
                                             bool biased, float m, float rstd) {
  float p[kE], g[kE], o[kE];
  widen_raw<T>(s, p);
  widen_raw<T>(w, g);
  if (biased) widen_raw<T>(b, o);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float u = (p[e] - m) * rstd;
    p[e] = biased ? fmaf(u, g[e], o[e]) : u * g[e];
  }
  return round_raw<T>(p);
}

// CH chunks a thread in registers.
template <typename T, int TEAM, int CH, bool VEC, bool DROP>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void layer_norm_kernel(
    const T* x, int64_t ld_x, const T* residual, int64_t ld_r, T* sum, int64_t ld_s, Drop drop,
    const T* weight, const T* bias, int64_t n, int64_t h, float eps, float inv_h, T* y,
    int64_t ld_y, float* mean_out, float* rstd_out) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM;
  constexpr int ROWS = BLOCK / TEAM;
  __shared__ float buf[2][ROWS][TEAM / kWave];
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + team;
  if (TEAM == kWave && r >= n) return;  // a wider team fills its workgroup: r < n
  Raw<T> s[CH], a[CH], w[CH], b[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) s[c] = load_chunk<T, VEC>(x + r * ld_x, (c * TEAM + t) * kE, h);
  if (residual) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      a[c] = load_chunk<T, VEC>(residual + r * ld_r, (c * TEAM + t) * kE, h);
  }
  const uint64_t seed = DROP ? drop_seed(drop) : 0;
  if (DROP || residual) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      s[c] = stream_chunk<T, DROP>(s[c], a[c], residual != nullptr, drop, seed, r, c * TEAM + t);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) w[c] = load_chunk<T, VEC>(weight, (c * TEAM + t) * kE, h);
  if (bias) {
#pragma unroll
    for (int c = 0; c < CH; ++c) b[c] = load_chunk<T, VEC>(bias, (c * TEAM + t) * kE, h);
  }
  if (sum) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      store_chunk<T, VEC>(sum + r * ld_s, (c * TEAM + t) * kE, h, s[c]);
  }
  float m = 0.0f, ss = 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c) m = add_chunk<T>(s[c], m);
  m = team_reduce<TEAM, false>(m, buf[0][team]) * inv_h;
#pragma unroll
  for (int c = 0; c < CH; ++c) ss = add_squares<T>(s[c], (c * TEAM + t) * kE, h, m, ss);
  ss = team_reduce<TEAM, false>(ss, buf[1][team]);
  const float rstd = 1.0f / sqrtf(ss * inv_h + eps);
  if (t == 0) {
    if (mean_out) mean_out[r] = m;
    if (rstd_out) rstd_out[r] = rstd;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
    store_chunk<T, VEC>(y + r * ld_y, (c * TEAM + t) * kE, h,
                      norm_chunk<T>(s[c], w[c], b[c], bias != nullptr, m, rstd));
}

// Longer rows: a team of 1024 that reads its row three times.  The later passes
// read s where the first stored it (a thread reads what it wrote itself), or x.
constexpr int kLongTeam = 1024;

template <typename T, bool VEC, bool DROP>
__global__ __launch_bounds__(kLongTeam) void layer_norm_long_kernel(
    const T* x, int64_t ld_x, const T* residual, int64_t ld_r, T* sum, int64_t ld_s, Drop drop,
    const T* weight, const T* bias, int64_t n, int64_t h, float eps, float inv_h, T* y,
    int64_t ld_y, float* mean_out, float* rstd_out) {
  __shared__ float buf[2][kLongTeam / kWave];
  const int64_t r = blockIdx.x;
  const T* xr = x + r * ld_x;
  const uint64_t seed = DROP ? drop_seed(drop) : 0;
  float m = 0.0f, ss = 0.0f;
  for (int64_t k = threadIdx.x; k * kE < h; k += kLongTeam) {
    Raw<T> s = load_chunk<T, VEC>(xr, k * kE, h), a;
    if (residual) a = load_chunk<T, VEC>(residual + r * ld_r, k * kE, h);
    s = stream_chunk<T, DROP>(s, a, residual != nullptr, drop, seed, r, k);
    if (sum) store_chunk<T, VEC>(sum + r * ld_s, k * kE, h, s);
    m = add_chunk<T>(s, m);
  }
  const T* sr = sum ? sum + r * ld_s : xr;
  m = team_reduce<kLongTeam, false>(m, buf[0]) * inv_h;
  for (int64_t k = threadIdx.x; k * kE < h; k += kLongTeam)
    ss = add_squares<T>(load_chunk<T, VEC>(sr, k * kE, h), k * kE, h, m, ss);
  ss = team_reduce<kLongTeam, false>(ss, buf[1]);
  const float rstd = 1.0f / sqrtf(ss * inv_h + eps);
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[r] = m;
    if (rstd_out) rstd_out[r] = rstd;
  }
  for (int64_t k = threadIdx.x; k * kE < h; k += kLongTeam) {
    const Raw<T> s = load_chunk<T, VEC>(sr, k * kE, h), w = load_chunk<T, VEC>(weight, k * kE, h);
    Raw<T> b;
    if (bias) b = load_chunk<T, VEC>(bias, k * kE, h);
    store_chunk<T, VEC>(y + r * ld_y, k * kE, h, norm_chunk<T>(s, w, b, bias != nullptr, m, rstd));
  }
}

// ---------------------------------------------------------------------------
// Gradient.
// ---------------------------------------------------------------------------
template <typename T>
struct GradRows {
  const T* s;
  int64_t ld_s;
  const T* weight;
  const float* mean;
  const float* rstd;
  const T* dy;
  int64_t ld_dy;
  const T* ds;
  int64_t ld_ds;
  T* dx;
  int64_t ld_dx;
  T* dres;
  int64_t ld_dres;
};

// Writes d of one chunk: as it is to dx, or with dropout to dres (unless null)
// and through the mask to dx.
template <typename T, bool VEC, bool DROP>
__device__ __forceinline__ void grad_store(const GradRows<T>& g, int64_t r, int64_t chunk,
                                           int64_t h, const Drop& drop, uint64_t seed,
                                           float (&d)[kE]) {
  if constexpr (DROP) {
    if (g.dres) store_chunk<T, VEC>(g.dres + r * g.ld_dres, chunk * kE, h, round_raw<T>(d));
    const uint4 u = drop_chunk(drop, seed, r, static_cast<uint32_t>(chunk));
#pragma unroll
    for (int e = 0; e < kE; ++e) d[e] = drop_keeps(drop, u, e) ? d[e] * drop.factor : 0.0f;
  }
  store_chunk<T, VEC>(g.dx + r * g.ld_dx, chunk * kE, h, round_raw<T>(d));
}

// d of one chunk, in place of dy.
template <typename T>
__device__ __forceinline__ void grad_chunk(const Raw<T>& s, const Raw<T>& dy, const Raw<T>& w,
                                           const Raw<T>& ds, bool add, float m, float rs,
                                           float mean_g, float mean_gu, float (&out)[kE]) {
  float sv[kE], wv[kE], dv[kE];
  widen_raw<T>(s, sv);
  widen_raw<T>(dy, out);
  widen_raw<T>(w, wv);
  if (add) widen_raw<T>(ds, dv);
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const float u = (sv[e] - m) * rs;
    const float v = fmaf(-u, mean_gu, fmaf(out[e], wv[e], -mean_g));
    out[e] = add ? fmaf(rs, v, dv[e]) : rs * v;
  }
}

// Team p of P takes rows p, p + P, ...; it keeps its shares of sum_r dy u and
// sum_r dy in registers and leaves them as row p of `partial` [P, 2 h].
// Elements past h hold dy = 0, and so add nothing to either sum.
template <typename T, int TEAM, int CH, bool VEC, bool DROP>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void layer_norm_bwd_kernel(
    GradRows<T> g, Drop drop, int64_t n, int64_t h, float inv_h, int64_t teams,
    float* __restrict__ partial) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM;
  constexpr int ROWS = BLOCK / TEAM;
  __shared__ float buf[2][2][ROWS][TEAM / kWave];
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * ROWS + team;
  if (TEAM == kWave && p >= teams) return;
  const uint64_t seed = DROP ? drop_seed(drop) : 0;
  float accw[CH][kE], accb[CH][kE];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < kE; ++e) accw[c][e] = accb[c][e] = 0.0f;
  Raw<T> w[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) w[c] = load_chunk<T, VEC>(g.weight, (c * TEAM + t) * kE, h);
  // The next row's loads are on their way while this one's sums go round.
  Raw<T> s[CH], dy[CH], ds[CH];
  float m = 0.0f, rs = 0.0f;
  auto load = [&](int64_t r, Raw<T> (&a)[CH], Raw<T> (&b)[CH], Raw<T> (&c)[CH]) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t c0 = (k * TEAM + t) * kE;
      a[k] = load_chunk<T, VEC>(g.s + r * g.ld_s, c0, h);
      b[k] = load_chunk<T, VEC>(g.dy + r * g.ld_dy, c0, h);
      if (g.ds) c[k] = load_chunk<T, VEC>(g.ds + r * g.ld_ds, c0, h);
    }
  };
  if (p < n) {
    load(p, s, dy, ds);
    m = g.mean[p];
    rs = g.rstd[p];
  }
  int turn = 0;
  for (int64_t r = p; r < n; r += teams, turn ^= 1) {
    Raw<T> s2[CH], dy2[CH], ds2[CH];
    const int64_t next = r + teams < n ? r + teams : r;
    load(next, s2, dy2, ds2);
    const float m2 = g.mean[next], rs2 = g.rstd[next];
    float sum_g = 0.0f, sum_gu = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float sv[kE], gv[kE], wv[kE];
      widen_raw<T>(s[c], sv);
      widen_raw<T>(dy[c], gv);
      widen_raw<T>(w[c], wv);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float u = (sv[e] - m) * rs;
        accw[c][e] = fmaf(gv[e], u, accw[c][e]);
        accb[c][e] = accb[c][e] + gv[e];
        const float gw = gv[e] * wv[e];
        sum_g = sum_g + gw;
        sum_gu = fmaf(gw, u, sum_gu);
      }
    }
    const float mean_g = team_reduce<TEAM, false>(sum_g, buf[turn][0][team]) * inv_h;
    const float mean_gu = team_reduce<TEAM, false>(sum_gu, buf[turn][1][team]) * inv_h;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float d[kE];
      grad_chunk<T>(s[c], dy[c], w[c], ds[c], g.ds != nullptr, m, rs, mean_g, mean_gu, d);
      grad_store<T, VEC, DROP>(g, r, c * TEAM + t, h, drop, seed, d);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      s[c] = s2[c];
      dy[c] = dy2[c];
      ds[c] = ds2[c];
    }
    m = m2;
    rs = rs2;
  }
  if (!partial) return;
  float* out = partial + p * 2 * h;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t c0 = (c * TEAM + t) * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (c0 + e < h) {
        out[c0 + e] = accw[c][e];
        out[h + c0 + e] = accb[c][e];
      }
  }
}

// Longer rows: the sums of a row, then its gradient from a second reading.
template <typename T, bool VEC, bool DROP>
__global__ __launch_bounds__(kLongTeam) void layer_norm_bwd_long_kernel(GradRows<T> g, Drop drop,
                                                                        int64_t h, float inv_h) {
  __shared__ float buf[2][kLongTeam / kWave];
  const int64_t r = blockIdx.x;
  const uint64_t seed = DROP ? drop_seed(drop) : 0;
  const float m = g.mean[r], rs = g.rstd[r];
  float sum_g = 0.0f, sum_gu = 0.0f;
  for (int64_t k = threadIdx.x; k * kE < h; k += kLongTeam) {
    float sv[kE], gv[kE], wv[kE];
    widen_raw<T>(load_chunk<T, VEC>(g.s + r * g.ld_s, k * kE, h), sv);
    widen_raw<T>(load_chunk<T, VEC>(g.dy + r * g.ld_dy, k * kE, h), gv);
    widen_raw<T>(load_chunk<T, VEC>(g.weight, k * kE, h), wv);
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const float gw = gv[e] * wv[e];
      sum_g = sum_g + gw;
      sum_gu = fmaf(gw, (sv[e] - m) * rs, sum_gu);
    }
  }
  const float mean_g = team_reduce<kLongTeam, false>(sum_g, buf[0]) * inv_h;
  const float mean_gu = team_reduce<kLongTeam, false>(sum_gu, buf[1]) * inv_h;
  for (int64_t k = threadIdx.x; k * kE < h; k += kLongTeam) {
    const Raw<T> s = load_chunk<T, VEC>(g.s + r * g.ld_s, k * kE, h);
    const Raw<T> dy = load_chunk<T, VEC>(g.dy + r * g.ld_dy, k * kE, h);
    const Raw<T> w = load_chunk<T, VEC>(g.weight, k * kE, h);
    Raw<T> ds;
    if (g.ds) ds = load_chunk<T, VEC>(g.ds + r * g.ld_ds, k * kE, h);
    float d[kE];
    grad_chunk<T>(s, dy, w, ds, g.ds != nullptr, m, rs, mean_g, mean_gu, d);
    grad_store<T, VEC, DROP>(g, r, k, h, drop, seed, d);
  }
}

// The weight's part for them, before dx may overwrite dy: 64 columns of chunks
// a wave, rows p, p + P, ...
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void layer_norm_columns_kernel(GradRows<T> g, int64_t n,
                                                                 int64_t h, int64_t teams,
                                                                 float* __restrict__ partial) {
  const int64_t c0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * kE;
  if (c0 >= h) return;
  float accw[kE] = {}, accb[kE] = {};
  for (int64_t r = blockIdx.y; r < n; r += teams) {
    float sv[kE], gv[kE];
    widen_raw<T>(load_chunk<T, VEC>(g.s + r * g.ld_s, c0, h), sv);
    widen_raw<T>(load_chunk<T, VEC>(g.dy + r * g.ld_dy, c0, h), gv);
    const float m = g.mean[r], rs = g.rstd[r];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      accw[e] = fmaf(gv[e], (sv[e] - m) * rs, accw[e]);
      accb[e] = accb[e] + gv[e];
    }
  }
  float* out = partial + static_cast<int64_t>(blockIdx.y) * 2 * h;
#pragma unroll
  for (int e = 0; e < kE; ++e)
    if (c0 + e < h) {
      out[c0 + e] = accw[e];
      out[h + c0 + e] = accb[e];
    }
}

// dweight and dbias = rne(sum over the P partial rows): 32 columns (whole lines
// where h is a multiple of 32; else every line is read twice) a workgroup, 32
// groups of rows, each in ascending order, then the groups in order.  512 rows of
// 2 x 4096: 4.9 us (16 columns: every line read twice, 7.8; 64: 5.2).
constexpr int kSumCols = 32, kSumGroups = 32;

template <typename T>
__global__ __launch_bounds__(kSumCols * kSumGroups) void layer_norm_sum_kernel(
    const float* __restrict__ partial, int64_t rows, int64_t h, T* __restrict__ dweight,
    T* __restrict__ dbias) {
  __shared__ float part[kSumGroups][kSumCols + 1];
  T* out = blockIdx.y ? dbias : dweight;
  if (!out) return;
  const float* in = partial + blockIdx.y * h;
  const int c = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kSumCols + c;
  float a = 0.0f;
  if (col < h)
#pragma unroll 8
    for (int64_t p = g; p < rows; p += kSumGroups) a = a + in[p * 2 * h + col];
  part[g][c] = a;
  __syncthreads();
  if (g == 0 && col < h) {
    for (int i = 1; i < kSumGroups; ++i) a = a + part[i][c];
    store_one<T>(out + col, a);
  }
}

// Team and chunks a thread for rows of h elements; ch 0: the kernels that read
// their rows again.  A team of 1024 has 128 registers a thread, one of 512 the
// 256 that the gradient's sums over the rows need.
struct Shape {
  int team, ch;
};
Shape layer_shape(int64_t h, int wide, int most) {
  const int64_t chunks = (h + kE - 1) / kE;
  const int team = chunks <= 128 ? 64 : chunks <= 1024 ? 256 : wide;
  const int ch = static_cast<int>((chunks + team - 1) / team);
  return Shape{team, ch <= most ? ch : 0};
}
template <typename T>
Shape fwd_shape(int64_t h) {
  return layer_shape(h, 1024, h > 8192 && sizeof(T) == 4 ? 2 : 4);
}
Shape bwd_shape(int size, int64_t h) {
  return layer_shape(h, 512, h <= 8192 ? 4 : size == 4 ? 0 : 3);
}

template <typename T>
void layer_norm_typed(const NormRows& rows, const Drop* drop, const void* weight, const void* bias,
                      int64_t n, int64_t h, float eps, void* y, int64_t ld_y, float* mean,
                      float* rstd, hipStream_t s) {
  const Shape sh = fwd_shape<T>(h);
  const int size = sizeof(T);
  const bool vec = fits16(rows.x, rows.ld_x, size) && fits16(rows.residual, rows.ld_r, size) &&
                   fits16(rows.sum, rows.ld_s, size) && fits16(weight, 8, size) &&
                   fits16(bias, 8, size) && fits16(y, ld_y, size) && h % kE == 0;
  const float inv_h = static_cast<float>(1.0 / static_cast<double>(h));
  const T* x = static_cast<const T*>(rows.x);
  const T* residual = static_cast<const T*>(rows.residual);
  T* sum = static_cast<T*>(rows.sum);
  auto launch = [&](auto kern, int block, int per) {
    for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups * per) {
      const int64_t m = n - r0 < kMaxGroups * per ? n - r0 : kMaxGroups * per;
      Drop d = drop ? *drop : Drop{};
      d.first_row += r0;
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((m + per - 1) / per)), dim3(block), 0, s,
                         row_at(x, r0, rows.ld_x), rows.ld_x, row_at(residual, r0, rows.ld_r),
                         rows.ld_r, row_at(sum, r0, rows.ld_s), rows.ld_s, d,
                         static_cast<const T*>(weight), static_cast<const T*>(bias), m, h, eps,
                         inv_h, row_at(static_cast<T*>(y), r0, ld_y), ld_y, row_at(mean, r0, 1),
                         row_at(rstd, r0, 1));
    }
  };
#define ITL_GO(TM, C)                                                                           \
  if (sh.team == TM && sh.ch == C)                                                              \
    return launch(drop ? (vec ? layer_norm_kernel<T, TM, C, true, true>                         \
                              : layer_norm_kernel<T, TM, C, false, true>)                       \
                       : (vec ? layer_norm_kernel<T, TM, C, true, false>                        \
                              : layer_norm_kernel<T, TM, C, false, false>),                     \
                  TM < 256 ? 256 : TM, TM < 256 ? 256 / TM : 1);
  ITL_GO(64, 1) ITL_GO(64, 2) ITL_GO(256, 1) ITL_GO(256, 2) ITL_GO(256, 3) ITL_GO(256, 4)
  ITL_GO(1024, 2)
  if constexpr (sizeof(T) == 2) {
    ITL_GO(1024, 3) ITL_GO(1024, 4)
  }
  launch(drop ? (vec ? layer_norm_long_kernel<T, true, true>
                     : layer_norm_long_kernel<T, false, true>)
              : (vec ? layer_norm_long_kernel<T, true, false>
                     : layer_norm_long_kernel<T, false, false>),
         kLongTeam, 1);
#undef ITL_GO
}

template <typename T>
void layer_norm_bwd_typed(const LayerNormGrad& a, int64_t n, int64_t h, float* partial,
                          hipStream_t s) {
  const int size = sizeof(T);
  const Shape sh = bwd_shape(size, h);
  const bool vec = fits16(a.s, a.ld_s, size) && fits16(a.dy, a.ld_dy, size) &&
                   fits16(a.ds, a.ld_ds, size) && fits16(a.dx, a.ld_dx, size) &&
                   fits16(a.dres, a.ld_dres, size) && fits16(a.weight, 8, size) && h % kE == 0;
  const float inv_h = static_cast<float>(1.0 / static_cast<double>(h));
  const GradRows<T> g{static_cast<const T*>(a.s), a.ld_s, static_cast<const T*>(a.weight), a.mean,
                      a.rstd, static_cast<const T*>(a.dy), a.ld_dy, static_cast<const T*>(a.ds),
                      a.ld_ds, static_cast<T*>(a.dx), a.ld_dx, static_cast<T*>(a.dres), a.ld_dres};
  const Drop drop = a.drop ? *a.drop : Drop{};
  const bool sums = a.dweight || a.dbias;
  const int64_t teams = n ? layer_norm_bwd_blocks(size == 4 ? kF32 : kBF16, n, h) : 0;
  if (n && sh.ch == 0) {
    if (sums)
      hipLaunchKernelGGL((vec ? layer_norm_columns_kernel<T, true>
                              : layer_norm_columns_kernel<T, false>),
                         dim3(static_cast<unsigned>((h + 2047) / 2048),
                              static_cast<unsigned>(teams)),
                         dim3(256), 0, s, g, n, h, teams, partial);
    auto kern = a.drop ? (vec ? layer_norm_bwd_long_kernel<T, true, true>
                              : layer_norm_bwd_long_kernel<T, false, true>)
                       : (vec ? layer_norm_bwd_long_kernel<T, true, false>
                              : layer_norm_bwd_long_kernel<T, false, false>);
    for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups) {
      const int64_t m = n - r0 < kMaxGroups ? n - r0 : kMaxGroups;
      Drop d = drop;
      d.first_row += r0;
      const GradRows<T> part{row_at(g.s, r0, g.ld_s), g.ld_s, g.weight, g.mean + r0, g.rstd + r0,
                             row_at(g.dy, r0, g.ld_dy), g.ld_dy, row_at(g.ds, r0, g.ld_ds),
                             g.ld_ds, row_at(g.dx, r0, g.ld_dx), g.ld_dx,
                             row_at(g.dres, r0, g.ld_dres), g.ld_dres};
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(m)), dim3(kLongTeam), 0, s, part, d, h,
                         inv_h);
    }
  } else if (n) {
#define ITL_GO(TM, C)                                                                           \
  case TM * 16 + C: {                                                                           \
    auto kern = a.drop ? (vec ? layer_norm_bwd_kernel<T, TM, C, true, true>                     \
                              : layer_norm_bwd_kernel<T, TM, C, false, true>)                   \
                       : (vec ? layer_norm_bwd_kernel<T, TM, C, true, false>                    \
                              : layer_norm_bwd_kernel<T, TM, C, false, false>);                 \
    constexpr int kBlock = TM < 256 ? 256 : TM;                                                 \
    hipLaunchKernelGGL(kern,                                                                    \
                       dim3(static_cast<unsigned>((teams + kBlock / TM - 1) / (kBlock / TM))),  \
                       dim3(kBlock), 0, s, g, drop, n, h, inv_h, teams,                         \
                       sums ? partial : nullptr);                                               \
  } break;
    switch (sh.team * 16 + sh.ch) {
      ITL_GO(64, 1) ITL_GO(64, 2) ITL_GO(256, 1) ITL_GO(256, 2) ITL_GO(256, 3) ITL_GO(256, 4)
      default:
        if constexpr (sizeof(T) == 2) {
          switch (sh.team * 16 + sh.ch) { ITL_GO(512, 3) }
        }
    }
#undef ITL_GO
  }
  if (sums)
    hipLaunchKernelGGL(layer_norm_sum_kernel<T>,
                       dim3(static_cast<unsigned>((h + kSumCols - 1) / kSumCols), 2),
                       dim3(kSumCols * kSumGroups), 0, s, partial, teams, h,
                       static_cast<T*>(a.dweight), static_cast<T*>(a.dbias));
}

}  // namespace

int64_t layer_norm_bwd_blocks(int dtype, int64_t n, int64_t h) {
  const Shape sh = bwd_shape(dtype == kF32 ? 4 : 2, h);
  // Eight waves a CU where the registers allow them (a team of 256 holding at
  // most 32 bytes a lane of each row), else four: fewer partial rows.  bf16, us
  // with the sum over the rows, eight against four: 8192 x 4096 72 (93), 4096 x
  // 8192 93 (64), 8192 x 1024 36 (30); fp32 4096 x 4096 73 (71).  For the column
  // kernel as many over its column blocks.
  const int size = dtype == kF32 ? 4 : 2;
  const int waves = sh.team == 512 || (sh.team == 256 && sh.ch * size <= 4) ? 8 : 4;
  const int64_t most = sh.ch ? 256 * waves / (sh.team / kWave)
                             : 512 * 2048 / ((h + 2047) / 2048 * 2048);
  return n < most ? n : most;
}

void launch_layer_norm(int dtype, const NormRows& rows, const Drop* drop, const void* weight,
                       const void* bias, int64_t n, int64_t h, float eps, void* y, int64_t ld_y,
                       float* mean, float* rstd, hipStream_t s) {
  auto run = dtype == kF32 ? layer_norm_typed<float>
             : dtype == kF16 ? layer_norm_typed<_Float16> : layer_norm_typed<uint16_t>;
  run(rows, drop, weight, bias, n, h, eps, y, ld_y, mean, rstd, s);
}

void launch_layer_norm_bwd(int dtype, const LayerNormGrad& g, int64_t n, int64_t h, float* partial,
                           hipStream_t s) {
  auto run = dtype == kF32 ? layer_norm_bwd_typed<float>
             : dtype == kF16 ? layer_norm_bwd_typed<_Float16> : layer_norm_bwd_typed<uint16_t>;
  run(g, n, h, partial, s);
}

}  // namespace itl
