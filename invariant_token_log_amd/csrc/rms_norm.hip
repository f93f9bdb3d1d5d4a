// Root-mean-square norm with the residual's addition, its 8-bit form and its
// gradient, on gfx950.
//
//   s = rne(x + residual);  rstd = 1 / sqrt(mean(s^2) + eps)
//   y = rne(s rstd w),  or  t = s rstd w,  a = max(max|t|, 448 * 2^-126),
//                           scale = a / 448,  q = rne_e4m3(t * (448 / a))
//   u = s rstd;  dx = rne(ds + rstd (dy w - u mean(dy w u)));  dw = sum_r dy u
//
// Bound by memory: every element is read and written once, so a row stays with
// the team of threads that owns it between its sum and its output.  A team is 64
// threads for rows of up to 1024 elements, 256 up to 8192 and 1024 beyond;
// thread t holds the chunks of 8 elements t, t + TEAM, ... of the row.
// The row is in registers up to 8192 elements in the gradient, 24576 in the
// 8-bit form and 32768 in the plain one.  Beyond, a thread of a team of 1024 has
// 128 registers and the compiler keeps the rest in scratch memory, more the
// longer the row.  bf16 in us, and its bytes at 6.45 TB/s: gradient with dweight
// 8192 x 4096 49 (42), 8192 x 8192 124 (83), 4096 x 8200 126 (42), 4096 x 16384
// 184 (83), 1024 x 65536 1322 (83); forward 8192 x 4096 41 (42), 4096 x 16384 100
// (83), 1024 x 65536 137 (83); 8 bits 4096 x 16384 103 (73), 1024 x 65536 348 (73).
// Each thread adds its squares in ascending order, the lanes of a wave follow in
// a butterfly and the waves in order, so the sum's tree depends on h alone: not
// on n, the row's place or its alignment.
// s is rounded to its type before it is normed, since the stored s is what
// the next layer and the backward read: the fused call then has the bits of
// an addition followed by a norm.
#include "rms_norm.h"

#include "launch.h"
#include "row_device.h"

namespace itl {

namespace {

constexpr float kE4m3Max = 448.0f;
// Below this magnitude a row's scale stays at 2^-126: its own would be
// subnormal and the factor 448 / max|t| pass fp32's range.
constexpr float kLeastMost = 0x1.cp-118f;

template <typename T, int TEAM, int CH, bool VEC, bool Q8>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_kernel(
    const T* x, int64_t ld_x, const T* residual, int64_t ld_r, T* sum, int64_t ld_s,
    const T* weight, int64_t n, int64_t h, float eps, float inv_h, void* y, int64_t ld_y,
    float* scale, float* rstd_out) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM;
  constexpr int ROWS = BLOCK / TEAM;
  __shared__ float buf[3][ROWS][TEAM / kWave];
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * ROWS + team;
  if (TEAM == kWave && r >= n) return;  // a wider team fills its workgroup: r < n
  const T* xr = x + r * ld_x;
  Raw<T> s[CH], w[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) s[c] = load_raw<T, VEC>(xr, (c * TEAM + t) * kE, h);
  if (residual) {
    const T* rr = residual + r * ld_r;
    Raw<T> a[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) a[c] = load_raw<T, VEC>(rr, (c * TEAM + t) * kE, h);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float p[kE], q[kE];
      widen_raw<T>(s[c], p);
      widen_raw<T>(a[c], q);
#pragma unroll
      for (int e = 0; e < kE; ++e) p[e] = p[e] + q[e];
      s[c] = round_raw<T>(p);
    }
  }
  if (weight) {
#pragma unroll
    for (int c = 0; c < CH; ++c) w[c] = load_raw<T, VEC>(weight, (c * TEAM + t) * kE, h);
  }
  if (sum) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      store_raw<T, VEC>(sum + r * ld_s, (c * TEAM + t) * kE, h, s[c]);
  }
  float rstd = 1.0f;
  if (weight) {
    float ss = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float p[kE];
      widen_raw<T>(s[c], p);
#pragma unroll
      for (int e = 0; e < kE; ++e) ss = fmaf(p[e], p[e], ss);
    }
    ss = team_reduce<TEAM, false>(ss, buf[0][team]);
    rstd = 1.0f / sqrtf(ss * inv_h + eps);
    if (rstd_out && t == 0) rstd_out[r] = rstd;
  }
  float inv = 0.0f;
  if constexpr (Q8) {
    float most = 0.0f, nan = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float p[kE], g[kE];
      widen_raw<T>(s[c], p);
      if (weight) widen_raw<T>(w[c], g);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float v = weight ? p[e] * rstd * g[e] : p[e];
        most = fmaxf(most, fabsf(v));
        nan = v != v ? 1.0f : nan;
      }
    }
    most = team_reduce<TEAM, true>(most, buf[1][team]);
    nan = team_reduce<TEAM, true>(nan, buf[2][team]);
    if (nan != 0.0f) most = __uint_as_float(0x7fc00000u);
    if (most > 0.0f && most < kLeastMost) most = kLeastMost;
    if (t == 0) scale[r] = most / kE4m3Max;
    inv = most == 0.0f ? 0.0f : kE4m3Max / most;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t c0 = (c * TEAM + t) * kE;
    float p[kE], g[kE];
    widen_raw<T>(s[c], p);
    if (weight) widen_raw<T>(w[c], g);
#pragma unroll
    for (int e = 0; e < kE; ++e) p[e] = weight ? p[e] * rstd * g[e] : p[e];
    if constexpr (Q8) {
      uint8_t* qr = static_cast<uint8_t*>(y) + r * ld_y;
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(p[0] * inv, p[1] * inv, lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(p[2] * inv, p[3] * inv, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(p[4] * inv, p[5] * inv, hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(p[6] * inv, p[7] * inv, hi, true);
      if (VEC && c0 + kE <= h) {
        *reinterpret_cast<int2*>(qr + c0) = make_int2(lo, hi);
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e)
          if (c0 + e < h)
            qr[c0 + e] = static_cast<uint8_t>((e < 4 ? lo : hi) >> (8 * (e & 3)));
      }
    } else {
      store_raw<T, VEC>(static_cast<T*>(y) + r * ld_y, c0, h, round_raw<T>(p));
    }
  }
}

// ---------------------------------------------------------------------------
// Gradient.  Team p of P takes rows p, p + P, ...; it keeps its share of
// sum_r dy u in registers and leaves it as row p of `partial` [P, h].
// ---------------------------------------------------------------------------
template <typename T, int TEAM, int CH, bool VEC>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rms_norm_bwd_kernel(
    const T* s, int64_t ld_s, const T* weight, const float* __restrict__ rstd, const T* dy,
    int64_t ld_dy, const T* ds, int64_t ld_ds, int64_t n, int64_t h, float inv_h, int64_t teams,
    T* dx, int64_t ld_dx, float* __restrict__ partial) {
  constexpr int BLOCK = TEAM < 256 ? 256 : TEAM;
  constexpr int ROWS = BLOCK / TEAM;
  __shared__ float buf[2][ROWS][TEAM / kWave];
  const int team = threadIdx.x / TEAM, t = threadIdx.x % TEAM;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * ROWS + team;
  if (TEAM == kWave && p >= teams) return;
  float acc[CH][kE];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[c][e] = 0.0f;
  Raw<T> w[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) w[c] = load_raw<T, VEC>(weight, (c * TEAM + t) * kE, h);
  int turn = 0;
  for (int64_t r = p; r < n; r += teams, turn ^= 1) {
    Raw<T> a[CH], g[CH], d[CH];
    const float rs = rstd[r];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t c0 = (c * TEAM + t) * kE;
      a[c] = load_raw<T, VEC>(s + r * ld_s, c0, h);
      g[c] = load_raw<T, VEC>(dy + r * ld_dy, c0, h);
      if (ds) d[c] = load_raw<T, VEC>(ds + r * ld_ds, c0, h);
    }
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float av[kE], gv[kE], wv[kE];
      widen_raw<T>(a[c], av);
      widen_raw<T>(g[c], gv);
      widen_raw<T>(w[c], wv);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float u = av[e] * rs;
        acc[c][e] = fmaf(gv[e], u, acc[c][e]);
        dot = fmaf(gv[e] * wv[e], u, dot);
      }
    }
    const float mean = team_reduce<TEAM, false>(dot, buf[turn][team]) * inv_h;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float av[kE], gv[kE], wv[kE], dv[kE];
      widen_raw<T>(a[c], av);
      widen_raw<T>(g[c], gv);
      widen_raw<T>(w[c], wv);
      if (ds) widen_raw<T>(d[c], dv);
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        const float u = av[e] * rs;
        const float v = fmaf(-u, mean, gv[e] * wv[e]);
        gv[e] = ds ? fmaf(rs, v, dv[e]) : rs * v;
      }
      store_raw<T, VEC>(dx + r * ld_dx, (c * TEAM + t) * kE, h, round_raw<T>(gv));
    }
  }
  if (!partial) return;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t c0 = (c * TEAM + t) * kE;
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (c0 + e < h) partial[p * h + c0 + e] = acc[c][e];
  }
}

// dweight = rne(sum over the P partial rows): 16 columns a workgroup, 64
// groups of rows, each in ascending order, then the groups in order.
constexpr int kSumCols = 16, kSumGroups = 64;

template <typename T>
__global__ __launch_bounds__(kSumCols * kSumGroups) void norm_weight_sum_kernel(
    const float* __restrict__ partial, int64_t rows, int64_t h, T* __restrict__ dweight) {
  __shared__ float part[kSumGroups][kSumCols + 1];
  const int c = threadIdx.x % kSumCols, g = threadIdx.x / kSumCols;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * kSumCols + c;
  float a = 0.0f;
  if (col < h)
#pragma unroll 8
    for (int64_t p = g; p < rows; p += kSumGroups) a = a + partial[p * h + col];
  part[g][c] = a;
  __syncthreads();
  if (g == 0 && col < h) {
    for (int i = 1; i < kSumGroups; ++i) a = a + part[i][c];
    store_one<T>(dweight + col, a);
  }
}

// Team and chunks a thread for rows of h elements.
struct Shape {
  int team, ch;
};
Shape norm_shape(int64_t h) {
  const int64_t chunks = (h + kE - 1) / kE;
  const int team = chunks <= 128 ? 64 : chunks <= 1024 ? 256 : 1024;
  const int ch = static_cast<int>((chunks + team - 1) / team);
  return Shape{team, ch <= 4 ? ch : 8};
}

#define ITL_NORM_SHAPES(GO)                                                                     \
  switch (sh.team * 16 + sh.ch) {                                                               \
    GO(64, 1) GO(64, 2) GO(256, 1) GO(256, 2) GO(256, 3) GO(256, 4) GO(1024, 2) GO(1024, 3)     \
    GO(1024, 4) GO(1024, 8)                                                                     \
  }

template <typename T>
void norm_typed(const NormRows& rows, const void* weight, int64_t n, int64_t h, float eps, void* y,
                int64_t ld_y, float* scale, float* rstd, bool q8, hipStream_t s) {
  const Shape sh = norm_shape(h);
  const int size = sizeof(T);
  const bool vec = fits16(rows.x, rows.ld_x, size) && fits16(rows.residual, rows.ld_r, size) &&
                   fits16(rows.sum, rows.ld_s, size) && fits16(weight, 8, size) &&
                   (q8 ? reinterpret_cast<uintptr_t>(y) % 8 == 0 && ld_y % 8 == 0
                       : fits16(y, ld_y, size));
  const float inv_h = static_cast<float>(1.0 / static_cast<double>(h));
  const T* x = static_cast<const T*>(rows.x);
  const T* residual = static_cast<const T*>(rows.residual);
  T* sum = static_cast<T*>(rows.sum);
  char* out = static_cast<char*>(y);
  const int64_t out_size = q8 ? 1 : size;
#define ITL_GO(TM, C)                                                                           \
  case TM * 16 + C: {                                                                           \
    auto kern = q8 ? (vec ? rms_norm_kernel<T, TM, C, true, true>                               \
                          : rms_norm_kernel<T, TM, C, false, true>)                             \
                   : (vec ? rms_norm_kernel<T, TM, C, true, false>                              \
                          : rms_norm_kernel<T, TM, C, false, false>);                           \
    constexpr int kBlock = TM < 256 ? 256 : TM, kRows = kBlock / TM;                            \
    for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups * kRows) {                                    \
      const int64_t m = n - r0 < kMaxGroups * kRows ? n - r0 : kMaxGroups * kRows;              \
      hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((m + kRows - 1) / kRows)),            \
                         dim3(kBlock), 0, s, row_at(x, r0, rows.ld_x), rows.ld_x,               \
                         row_at(residual, r0, rows.ld_r), rows.ld_r,                            \
                         row_at(sum, r0, rows.ld_s), rows.ld_s, static_cast<const T*>(weight),  \
                         m, h, eps, inv_h, static_cast<void*>(out + r0 * ld_y * out_size), ld_y, \
                         row_at(scale, r0, 1), row_at(rstd, r0, 1));                            \
    }                                                                                           \
  } break;
  ITL_NORM_SHAPES(ITL_GO)
#undef ITL_GO
}

template <typename T>
void norm_bwd_typed(const void* sm, int64_t ld_s, const void* weight, const float* rstd,
                    const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds, int64_t n,
                    int64_t h, void* dx, int64_t ld_dx, void* dweight, float* partial,
                    hipStream_t s) {
  const Shape sh = norm_shape(h);
  const int size = sizeof(T);
  const bool vec = fits16(sm, ld_s, size) && fits16(dy, ld_dy, size) && fits16(ds, ld_ds, size) &&
                   fits16(dx, ld_dx, size) && fits16(weight, 8, size);
  const float inv_h = static_cast<float>(1.0 / static_cast<double>(h));
  const int64_t teams = n ? norm_bwd_blocks(n, h) : 0;
#define ITL_GO(TM, C)                                                                           \
  case TM * 16 + C: {                                                                           \
    auto kern = vec ? rms_norm_bwd_kernel<T, TM, C, true> : rms_norm_bwd_kernel<T, TM, C, false>; \
    constexpr int kBlock = TM < 256 ? 256 : TM;                                                 \
    hipLaunchKernelGGL(kern,                                                                    \
                       dim3(static_cast<unsigned>((teams + kBlock / TM - 1) / (kBlock / TM))),  \
                       dim3(kBlock), 0, s, static_cast<const T*>(sm), ld_s,                     \
                       static_cast<const T*>(weight), rstd, static_cast<const T*>(dy), ld_dy,   \
                       static_cast<const T*>(ds), ld_ds, n, h, inv_h, teams,                    \
                       static_cast<T*>(dx), ld_dx, dweight ? partial : nullptr);                \
  } break;
  if (n) ITL_NORM_SHAPES(ITL_GO)
#undef ITL_GO
  if (dweight)
    hipLaunchKernelGGL(norm_weight_sum_kernel<T>,
                       dim3(static_cast<unsigned>((h + kSumCols - 1) / kSumCols)),
                       dim3(kSumCols * kSumGroups), 0, s, partial, teams, h,
                       static_cast<T*>(dweight));
}

}  // namespace

int64_t norm_bwd_blocks(int64_t n, int64_t h) {
  // Eight waves a CU: 8192 x 4096 bf16 takes 46 us and the weight's sum 4; with
  // sixteen 55 and 7 (twice the partial rows), with six 48 and 4.
  const int64_t most = 256 * 8 / (norm_shape(h).team / kWave);
  return n < most ? n : most;
}

void launch_rms_norm(int dtype, const NormRows& rows, const void* weight, int64_t n, int64_t h,
                     float eps, void* y, int64_t ld_y, float* scale, float* rstd, bool q8,
                     hipStream_t s) {
  if (dtype == kF32) norm_typed<float>(rows, weight, n, h, eps, y, ld_y, scale, rstd, q8, s);
  else if (dtype == kF16) norm_typed<_Float16>(rows, weight, n, h, eps, y, ld_y, scale, rstd, q8, s);
  else norm_typed<uint16_t>(rows, weight, n, h, eps, y, ld_y, scale, rstd, q8, s);
}

void launch_rms_norm_bwd(int dtype, const void* s, int64_t ld_s, const void* weight,
                         const float* rstd, const void* dy, int64_t ld_dy, const void* ds,
                         int64_t ld_ds, int64_t n, int64_t h, void* dx, int64_t ld_dx,
                         void* dweight, float* partial, hipStream_t stream) {
  if (dtype == kF32)
    norm_bwd_typed<float>(s, ld_s, weight, rstd, dy, ld_dy, ds, ld_ds, n, h, dx, ld_dx, dweight,
                          partial, stream);
  else if (dtype == kF16)
    norm_bwd_typed<_Float16>(s, ld_s, weight, rstd, dy, ld_dy, ds, ld_ds, n, h, dx, ld_dx,
                             dweight, partial, stream);
  else
    norm_bwd_typed<uint16_t>(s, ld_s, weight, rstd, dy, ld_dy, ds, ld_ds, n, h, dx, ld_dx,
                             dweight, partial, stream);
}

}  // namespace itl
