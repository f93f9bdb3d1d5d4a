// The LM head on 8-bit rows (e4m3) with one scale a row, and the tile
// statistics of its logits, on gfx950.
//
//   z[r, j] = (sum_k hidden[r, k] weight[j, k]) hs[r] ws[j]
//
// Arithmetic: every sum is one fp32 accumulator fed by
// v_mfma_f32_32x32x64_f8f6f4 over K in ascending steps of 64, no split;
// z = (acc hs) ws, x = z * fl32(1 / T).  The statistic tile is 256 vocabulary
// columns in eight groups of 32.  Maximum: exact.  Sum (and entropy moment):
// in a group, the 16 columns 8a + b (b < 4) and the 16 columns 8a + 4 + b are
// folded in ascending order from +0 and added; the groups follow as ((g0 + g1)
// + (g2 + g3)) + ((g4 + g5) + (g6 + g7)).  Every kernel below evaluates exactly
// this, so a row's outputs do not depend on n or on its place.
//
// The weight rows are the matrix product's first operand, so that an
// accumulator register holds a vocabulary column and a lane a hidden row: the
// statistics are folds over registers and one exchange between the two halves
// of the wave, where the other order needs a five-level butterfly a value.
//
// Two kernels:
//   q8_stats_wide (n > 128): 256 x 256 tiles, eight waves of 128 vocabulary
//     columns x 64 hidden rows; bound by the matrix cores and their power.
//   q8_stats_narrow<NB> (n <= 32 NB, NB = 1, 2, 4): 256 vocabulary columns x
//     32 NB hidden rows, eight waves of 32 columns; bound by the weight's
//     bytes, so it keeps two to three 128-byte steps of 256 rows in flight.
#include "linear_q8.h"

#include "logp_device.h"
#include "mfma_gemm.h"

namespace itl {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kV = kLinearTile;    // vocabulary columns per tile
constexpr int kStep = 64;          // K bytes per matrix instruction
constexpr int kQThreads = 512;     // 8 waves
constexpr int kUnitScale = 0x7f7f7f7f;  // block scales of 2^0

__device__ __forceinline__ f32x16 mfma_q8(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, kUnitScale, 0,
                                                         kUnitScale);
}

// Two 16-byte chunks as one operand.  Which K index a byte of a lane stands
// for does not matter as long as both operands agree: lane (row l % 32, half
// hf = l / 32) holds chunks 2 hf and 2 hf + 1 of its row's 64 bytes.
__device__ __forceinline__ i32x8 join(const uint8_t* lo, const uint8_t* hi) {
  const i32x4 a = *reinterpret_cast<const i32x4*>(lo);
  const i32x4 b = *reinterpret_cast<const i32x4*>(hi);
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// What the epilogue needs of the tile's hidden rows and vocabulary columns.
template <int ROWS>
struct Q8Reduce {
  float red[8][ROWS];   // per vocabulary group maxima (wide: per wave pair)
  float sum[8][ROWS];   // group sums
  float wsum[8][ROWS];  // group entropy moments
  float tval[ROWS];
  float hs[ROWS];
  float ws[kV];
  int code[ROWS];       // -2: no statistics; -1: target elsewhere; else column
};

template <int ROWS>
__device__ __forceinline__ void q8_fill(Q8Reduce<ROWS>& rd, int tid, const float* hs,
                                        const float* ws, int64_t n, int64_t v, int64_t m0,
                                        int64_t v0, Targets targets, int64_t ignore) {
  if (tid < ROWS) {
    const int64_t r = m0 + tid;
    int code = -2;
    float s = 0.0f;
    if (r < n) {
      const int64_t t = targets[r];
      if (t != ignore)
        code = (t >= v0 && t < v0 + kV && t < v) ? static_cast<int>(t - v0) : -1;
      s = hs[r];
    }
    rd.code[tid] = code;
    rd.hs[tid] = s;
  }
  if (tid >= kQThreads - kV) {
    const int c = tid - (kQThreads - kV);
    rd.ws[c] = v0 + c < v ? ws[v0 + c] : 0.0f;
  }
}

// Statistics of a wave's NI groups (32 vocabulary columns each, from group
// g0 on) for its NJ blocks of 32 hidden rows from row0 on:
//   acc[i][j][q] = z[m0 + row0 + 32 j + l % 32][v0 + 32 (g0 + i) + 8 (q / 4) + 4 hf + q % 4].
// rd's rows and columns are filled; all threads of the workgroup call.
template <int NI, int NJ, int ROWS, bool ENT>
__device__ __forceinline__ void q8_epilogue(f32x16 (&acc)[NI][NJ], Q8Reduce<ROWS>& rd, int g0,
                                            int row0, int tid, int64_t m0, int64_t v0, int vb,
                                            int vblocks, int64_t n, int64_t v, float inv_t,
                                            float* pm, float* ps, float* pw, float* pt, float* z,
                                            int64_t ld_z) {
  const int lane = tid % kWave;
  const int col = lane % 32, hf = lane / 32;
  // z, its output, x and the masked columns of the last tile
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int lr = row0 + 32 * j + col;
    const float h = rd.hs[lr];
    const int64_t r = m0 + lr;
    float* zr = z && r < n ? z + r * ld_z + v0 : nullptr;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int c = 32 * (g0 + i) + 8 * a + 4 * hf;
        const float4 w = *reinterpret_cast<const float4*>(&rd.ws[c]);
        float x[4] = {acc[i][j][4 * a] * h * w.x, acc[i][j][4 * a + 1] * h * w.y,
                      acc[i][j][4 * a + 2] * h * w.z, acc[i][j][4 * a + 3] * h * w.w};
        if (zr) {
          if (v0 + c + 4 <= v && (ld_z & 3) == 0) {
            *reinterpret_cast<float4*>(zr + c) = make_float4(x[0], x[1], x[2], x[3]);
          } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (v0 + c + b < v) zr[c + b] = x[b];
          }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[i][j][4 * a + b] = v0 + c + b < v ? x[b] * inv_t : -INFINITY;
      }
  }
  // maxima: registers, the other half of the wave, the other waves
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    float m = acc[0][j][0];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int q = 0; q < 16; ++q) m = max_exact(m, acc[i][j][q]);
    m = max_exact(m, __shfl_xor(m, 32, kWave));
    if (hf == 0) rd.red[g0 / NI][row0 + 32 * j + col] = m;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int lr = row0 + 32 * j + col;
    float m = rd.red[0][lr];
#pragma unroll
    for (int w = 1; w < 8 / NI; ++w) m = max_exact(m, rd.red[w][lr]);
    const int code = rd.code[lr];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int off = code - 32 * (g0 + i);  // the target's place in this group
      if (off >= 0 && off < 32 && ((off >> 2) & 1) == hf) {
        const int q = (off >> 3) * 4 + (off & 3);
        float t = acc[i][j][0];
#pragma unroll
        for (int k = 1; k < 16; ++k) t = q == k ? acc[i][j][k] : t;
        rd.tval[lr] = t;
      }
      float s = 0.0f, w = 0.0f;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const float d = acc[i][j][q] - m;
        const float e = __builtin_amdgcn_exp2f(d * kLog2e);
        s = s + e;
        if constexpr (ENT) w = ent_term(e, d, w);
      }
      s = s + __shfl_xor(s, 32, kWave);
      if constexpr (ENT) w = w + __shfl_xor(w, 32, kWave);
      if (hf == 0) {
        rd.sum[g0 + i][lr] = s;
        if constexpr (ENT) rd.wsum[g0 + i][lr] = w;
      }
    }
  }
  __syncthreads();
  for (int lr = tid; lr < ROWS; lr += kQThreads) {
    const int code = rd.code[lr];
    if (code == -2) continue;
    const int64_t r = m0 + lr;
    float m = rd.red[0][lr];
#pragma unroll
    for (int w = 1; w < 8 / NI; ++w) m = max_exact(m, rd.red[w][lr]);
    auto fold = [&](const float (&g)[8][ROWS]) {
      return ((g[0][lr] + g[1][lr]) + (g[2][lr] + g[3][lr])) +
             ((g[4][lr] + g[5][lr]) + (g[6][lr] + g[7][lr]));
    };
    pm[r * vblocks + vb] = m;
    ps[r * vblocks + vb] = fold(rd.sum);
    if constexpr (ENT) pw[r * vblocks + vb] = fold(rd.wsum);
    if (code >= 0) pt[r] = rd.tval[lr];
  }
}

// ---------------------------------------------------------------------------
// Wide: the staging of mfma_gemm.h's mainloop_pairs in bytes.  Hidden rows
// come K32-blocked in its sense (16 rows x 64 bytes contiguous) into four
// slots of 256 x 64 bytes, weight rows row-major into two slots of 256 x 128
// bytes (whole lines), three steps in flight; waves 0-3 issue the loads, each
// wave's fragments of the next step are read while the matrix instructions of
// this one run.
// ---------------------------------------------------------------------------
constexpr int kHSlot = 256 * kStep;      // bytes
constexpr int kWSlot = 256 * 2 * kStep;

struct SmemWide {
  uint8_t h[4][kHSlot];
  uint8_t w[2][kWSlot];
  Q8Reduce<256> rd;
  int slot;
};

using gemm::swz;
using gemm::swzp;
using gemm::wait_vm;
using gemm::wait_vm_lgkm0;

template <bool LOADER>
__device__ __forceinline__ void q8_mainloop(SmemWide& sm, const uint8_t* __restrict__ H,
                                            int64_t m0, const uint8_t* __restrict__ W,
                                            int64_t ld_w, int64_t v0, int64_t v, int ksteps,
                                            f32x16 (&acc)[4][2]) {
  const int tid = threadIdx.x;
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / 4, wn = wave % 4;
  const int row = lane % 32, hf = lane / 32;
  const int npairs = (ksteps + 1) / 2;
  // loader sources: hidden blocks wave + 4u (1 KiB, 16 rows), weight rows
  // (wave + 4u) * 8 + lane / 8
  const uint8_t* hp[4];
  const uint8_t* wp[8];
  int wback = 0;  // an odd last pair has no second half: those lanes read the first
  if constexpr (LOADER) {
    const int lrow = lane / 4;
    const int lofs = lrow * kStep + ((lane % 4) ^ swz(lrow)) * 16;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      hp[u] = H + (m0 / 16 + wave + 4 * u) * (static_cast<int64_t>(ksteps) * 1024) + lofs;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int r = (wave + 4 * u) * 8 + lane / 8;
      wp[u] = W + min(v0 + r, v - 1) * ld_w + ((lane % 8) ^ swzp(r)) * 16;
    }
    // swzp depends on u only through multiples of 32 rows, which it ignores
    if (((lane % 8) ^ swzp(wave * 8 + lane / 8)) >= 4 && (ksteps & 1)) wback = kStep;
  }
#define ITL_ISSUE_H(SLOT, STEP)                                                                 \
  if constexpr (LOADER) {                                                                       \
    const int64_t k_ = static_cast<int64_t>(STEP) * 1024;                                       \
    _Pragma("unroll") for (int u = 0; u < 4; ++u) __builtin_amdgcn_global_load_lds(             \
        hp[u] + k_, sm.h[SLOT] + (wave + 4 * u) * 1024, 16, 0, 0);                              \
  }
#define ITL_ISSUE_W(SLOT, PAIR)                                                                 \
  if constexpr (LOADER) {                                                                       \
    const int p_ = (PAIR);                                                                      \
    const int64_t k_ = static_cast<int64_t>(p_) * (2 * kStep) - (p_ == npairs - 1 ? wback : 0); \
    _Pragma("unroll") for (int u = 0; u < 8; ++u) __builtin_amdgcn_global_load_lds(             \
        wp[u] + k_, sm.w[SLOT] + (wave + 4 * u) * 1024, 16, 0, 0);                              \
  }
  const int wrow = wm * 128 + row, hrow = wn * 64 + row;
  const int wsw = swzp(wrow), hsw = swz(hrow);  // both repeat every 32 rows
  constexpr int NH = LOADER ? 4 : 0, NW = LOADER ? 8 : 0;
  ITL_ISSUE_H(0, 0);
  ITL_ISSUE_H(1, 1 < ksteps ? 1 : ksteps - 1);
  ITL_ISSUE_W(0, 0);
  ITL_ISSUE_H(2, 2 < ksteps ? 2 : ksteps - 1);
  ITL_ISSUE_H(3, 3 < ksteps ? 3 : ksteps - 1);
  ITL_ISSUE_W(1, 1 < npairs ? 1 : npairs - 1);
  wait_vm<2 * NH + NW>();
  __builtin_amdgcn_s_barrier();
  i32x8 xw[4], xh[2], yw[4], yh[2];
#define ITL_READ(FW, FH, STEP)                                                                  \
  {                                                                                             \
    const uint8_t* h_ = sm.h[(STEP) % 4];                                                       \
    const uint8_t* w_ = sm.w[((STEP) / 2) % 2];                                                 \
    const int c_ = 4 * ((STEP) % 2) + 2 * hf;                                                   \
    _Pragma("unroll") for (int j = 0; j < 2; ++j)                                               \
      FH[j] = join(h_ + (hrow + 32 * j) * kStep + ((2 * hf) ^ hsw) * 16,                        \
                   h_ + (hrow + 32 * j) * kStep + ((2 * hf + 1) ^ hsw) * 16);                   \
    _Pragma("unroll") for (int i = 0; i < 4; ++i)                                               \
      FW[i] = join(w_ + (wrow + 32 * i) * 2 * kStep + (c_ ^ wsw) * 16,                          \
                   w_ + (wrow + 32 * i) * 2 * kStep + ((c_ + 1) ^ wsw) * 16);                   \
  }
#define ITL_MFMA(CW, CH)                                                                        \
  _Pragma("unroll") for (int i = 0; i < 4; ++i)                                                 \
    _Pragma("unroll") for (int j = 0; j < 2; ++j) acc[i][j] = mfma_q8(CW[i], CH[j], acc[i][j]);
  ITL_READ(xw, xh, 0)
  // Waits as in mainloop_pairs: before an even step KT the hidden block of
  // KT + 1 (issued at KT - 3) has landed once only the loads issued after it
  // are in flight, before an odd one the weight pair of KT + 1 too.
#define ITL_QSTEP(CW, CH, NXW, NXH, KT, ODD)                                                    \
  {                                                                                             \
    if constexpr (ODD)                                                                          \
      wait_vm_lgkm0<NH>();                                                                      \
    else                                                                                        \
      wait_vm_lgkm0<2 * NH + NW>();                                                             \
    __builtin_amdgcn_s_barrier();                                                               \
    ITL_ISSUE_H((KT) % 4, (KT) + 4 < ksteps ? (KT) + 4 : ksteps - 1);                           \
    if constexpr (ODD) {                                                                        \
      const int q_ = ((KT) + 3) / 2;                                                            \
      ITL_ISSUE_W(q_ % 2, q_ < npairs ? q_ : npairs - 1);                                       \
    }                                                                                           \
    ITL_READ(NXW, NXH, (KT) + 1)                                                                \
    ITL_MFMA(CW, CH)                                                                            \
    if constexpr (LOADER) __builtin_amdgcn_sched_group_barrier(0x020, ODD ? NH + NW : NH, 0);   \
    _Pragma("unroll") for (int u = 0; u < 6; ++u) {                                             \
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                                        \
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);                                        \
    }                                                                                           \
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);                                          \
  }
  int kt = 0;
  for (; kt + 1 < ksteps; kt += 2) {
    ITL_QSTEP(xw, xh, yw, yh, kt, false)
    ITL_QSTEP(yw, yh, xw, xh, kt + 1, true)
  }
  if (kt < ksteps) {
    ITL_MFMA(xw, xh)
  }
#undef ITL_QSTEP
#undef ITL_MFMA
#undef ITL_READ
#undef ITL_ISSUE_W
#undef ITL_ISSUE_H
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <bool ENT>
__global__ __launch_bounds__(kQThreads) void q8_stats_wide(
    const uint8_t* __restrict__ hidden, const float* __restrict__ hs,
    const uint8_t* __restrict__ weight, int64_t ld_w, const float* __restrict__ ws, int64_t n,
    int64_t v, int ksteps, int mblocks, int vblocks, const void* __restrict__ tgt, int32_t tgt32,
    int64_t ignore, float inv_t, float* __restrict__ pm, float* __restrict__ ps,
    float* __restrict__ pw, float* __restrict__ pt, float* __restrict__ z, int64_t ld_z,
    int* queue, int queued) {
  const Targets targets{tgt, tgt32};
  __shared__ __align__(16) SmemWide sm;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int logical = gemm::queue_tile(queue, mblocks * vblocks, queued, &sm.slot);
  if (logical < 0) return;
  int mb, vb;
  gemm::tile_coords(logical, mblocks, vblocks, mb, vb);
  const int64_t m0 = static_cast<int64_t>(mb) * 256, v0 = static_cast<int64_t>(vb) * kV;
  q8_fill(sm.rd, tid, hs, ws, n, v, m0, v0, targets, ignore);
  f32x16 acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  if (gemm::loader_wave())
    q8_mainloop<true>(sm, hidden, m0, weight, ld_w, v0, v, ksteps, acc);
  else
    q8_mainloop<false>(sm, hidden, m0, weight, ld_w, v0, v, ksteps, acc);
  __syncthreads();
  q8_epilogue<4, 2, 256, ENT>(acc, sm.rd, (wave / 4) * 4, (wave % 4) * 64, tid, m0, v0, vb,
                              vblocks, n, v, inv_t, pm, ps, pw, pt, z, ld_z);
}

// ---------------------------------------------------------------------------
// Narrow: S slots of [256 weight rows | 32 NB hidden rows] x 128 bytes, both
// row-major, every wave loading; wave w computes vocabulary group w for all
// 32 NB rows.
// ---------------------------------------------------------------------------
// One direct 16-byte load a lane, global -> LDS at dst + 16 * lane; NT: past the caches.
template <bool NT>
__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 16, 0, NT ? 2 : 0);
}

template <int NB>
constexpr int kNarrowSlots = NB == 1 ? 4 : 3;

template <int NB>
struct SmemNarrowQ8 {
  uint8_t s[kNarrowSlots<NB>][(kV + 32 * NB) * 2 * kStep];
  Q8Reduce<32 * NB> rd;
};

template <int NB>
__device__ __forceinline__ void q8_mainloop_narrow(SmemNarrowQ8<NB>& sm,
                                                   const uint8_t* __restrict__ hidden,
                                                   int64_t ld_h, int64_t n,
                                                   const uint8_t* __restrict__ weight,
                                                   int64_t ld_w, int64_t v0, int64_t v, int ksteps,
                                                   f32x16 (&acc)[1][NB]) {
  constexpr int S = kNarrowSlots<NB>;
  const int tid = threadIdx.x;
  const int lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int npairs = (ksteps + 1) / 2;
  // A load fills 8 rows x 128 bytes; weight loads wave + 8 u (u < 4), and a
  // hidden load for the waves below 4 NB.  Chunk c of row r sits in slot c ^
  // swzp(r).
  const bool has_h = wave < 4 * NB;
  const uint8_t* wp[4];
  int back_w = 0, back_h = 0;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = (wave + 8 * u) * 8 + lane / 8;
    wp[u] = weight + min(v0 + r, v - 1) * ld_w + ((lane % 8) ^ swzp(r)) * 16;
  }
  constexpr int kHLoads = 4 * NB;  // hidden loads per pair: one or two a wave
  constexpr int NH = kHLoads > 8 ? 2 : 1;
  const uint8_t* hp[NH];
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    const int r = (wave % kHLoads + 8 * u) * 8 + lane / 8;
    hp[u] = hidden + min(static_cast<int64_t>(r), n - 1) * ld_h + ((lane % 8) ^ swzp(r)) * 16;
  }
  if (ksteps & 1) {  // no second half in the last pair: its lanes read the first
    if (((lane % 8) ^ swzp(wave * 8 + lane / 8)) >= 4) back_w = kStep;
    if (((lane % 8) ^ swzp((wave % kHLoads) * 8 + lane / 8)) >= 4) back_h = kStep;
  }
#define ITL_ISSUE_PAIR(SLOT, PAIR)                                                              \
  {                                                                                             \
    const int s_ = (SLOT);                                                                      \
    const int p_ = (PAIR) < npairs ? (PAIR) : npairs - 1;                                       \
    const int64_t k_ = static_cast<int64_t>(p_) * 2 * kStep;                                    \
    const bool end_ = p_ == npairs - 1;                                                         \
    _Pragma("unroll") for (int u = 0; u < 4; ++u) load_lds16<true>(                             \
        wp[u] + k_ - (end_ ? back_w : 0), sm.s[s_] + (wave + 8 * u) * 1024);          \
    if (has_h) {                                                                                \
      _Pragma("unroll") for (int u = 0; u < NH; ++u) load_lds16<false>(                         \
          hp[u] + k_ - (end_ ? back_h : 0),                                                     \
          sm.s[s_] + kV * 2 * kStep + (wave + 8 * u) * 1024);                         \
    }                                                                                           \
  }
  const int row = lane % 32, hf = lane / 32;
  const int sw = swzp(row);
  for (int p = 0; p < S - 1; ++p) ITL_ISSUE_PAIR(p, p)
  // Before pair p is read its loads have landed once only those of the S - 2
  // pairs issued after it are in flight; after the barrier that holds for
  // every wave, and nobody reads slot (p - 1) % S any more, which the pair
  // S - 1 ahead then takes.
  for (int p = 0; p < npairs; ++p) {
    if (has_h)
      wait_vm_lgkm0<(S - 2) * (4 + NH)>();
    else
      wait_vm_lgkm0<(S - 2) * 4>();
    __builtin_amdgcn_s_barrier();
    ITL_ISSUE_PAIR((p + S - 1) % S, p + S - 1)
    const uint8_t* w_ = sm.s[p % S] + (wave * 32 + row) * 2 * kStep;
    const uint8_t* h_ = sm.s[p % S] + (kV + row) * 2 * kStep;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half == 1 && 2 * p + 1 >= ksteps) break;
      const int c0 = ((4 * half + 2 * hf) ^ sw) * 16, c1 = ((4 * half + 2 * hf + 1) ^ sw) * 16;
      const i32x8 a = join(w_ + c0, w_ + c1);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const uint8_t* hj = h_ + 32 * j * 2 * kStep;
        acc[0][j] = mfma_q8(a, join(hj + c0, hj + c1), acc[0][j]);
      }
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#undef ITL_ISSUE_PAIR
}

template <int NB, bool ENT>
__global__ __launch_bounds__(kQThreads) void q8_stats_narrow(
    const uint8_t* __restrict__ hidden, int64_t ld_h, const float* __restrict__ hs,
    const uint8_t* __restrict__ weight, int64_t ld_w, const float* __restrict__ ws, int64_t n,
    int64_t v, int ksteps, int vblocks, const void* __restrict__ tgt, int32_t tgt32,
    int64_t ignore, float inv_t, float* __restrict__ pm, float* __restrict__ ps,
    float* __restrict__ pw, float* __restrict__ pt, float* __restrict__ z, int64_t ld_z) {
  const Targets targets{tgt, tgt32};
  __shared__ __align__(16) SmemNarrowQ8<NB> sm;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int vb = gemm::xcd_logical(blockIdx.x, vblocks);
  const int64_t v0 = static_cast<int64_t>(vb) * kV;
  q8_fill(sm.rd, tid, hs, ws, n, v, 0, v0, targets, ignore);
  f32x16 acc[1][NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[0][j][q] = 0.0f;
  q8_mainloop_narrow<NB>(sm, hidden, ld_h, n, weight, ld_w, v0, v, ksteps, acc);
  __syncthreads();
  q8_epilogue<1, NB, 32 * NB, ENT>(acc, sm.rd, wave, 0, tid, 0, v0, vb, vblocks, n, v, inv_t, pm,
                                    ps, pw, pt, z, ld_z);
}

}  // namespace

int64_t q8_fwd_scratch_bytes(int64_t n, int64_t h) {
  return n > 128 ? (n + 255) / 256 * 256 * h + gemm::kQueueBytes : 0;
}

void launch_q8_partials(const uint8_t* hidden, int64_t ld_h, const float* hs,
                        const uint8_t* weight, int64_t ld_w, const float* ws, int64_t n, int64_t h,
                        int64_t v, Targets targets, int64_t ignore, float* pm, float* ps,
                        float* pt, float inv_t, float* pw, float* z, int64_t ld_z, char* scratch,
                        hipStream_t s) {
  const int vblocks = static_cast<int>((v + kV - 1) / kV);
  const int ksteps = static_cast<int>(h / kStep);
  if (n <= 128) {
    auto kern = n <= 32   ? (pw ? q8_stats_narrow<1, true> : q8_stats_narrow<1, false>)
                : n <= 64 ? (pw ? q8_stats_narrow<2, true> : q8_stats_narrow<2, false>)
                          : (pw ? q8_stats_narrow<4, true> : q8_stats_narrow<4, false>);
    hipLaunchKernelGGL(kern, dim3(vblocks), dim3(kQThreads), 0, s, hidden, ld_h, hs, weight, ld_w,
                       ws, n, v, ksteps, vblocks, targets.p, targets.is32, ignore, inv_t, pm, ps,
                       pw, pt, z, ld_z);
    return;
  }
  const int mblocks = static_cast<int>((n + 255) / 256);
  const int64_t np = static_cast<int64_t>(mblocks) * 256;
  // The re-laid hidden rows: pieces of 16 rows x 64 bytes, which is the bf16
  // blocking of rows of h / 2 two-byte elements.
  int* queue = reinterpret_cast<int*>(scratch + np * h);
  launch_block_rows(reinterpret_cast<const uint16_t*>(hidden), ld_h / 2, n, np, h / 2,
                    reinterpret_cast<uint16_t*>(scratch), s, queue, gemm::kQueueBytes / 4);
  const gemm::QueuePlan qp = gemm::queue_plan(mblocks * vblocks, xcd_cus());
  auto kern = pw ? q8_stats_wide<true> : q8_stats_wide<false>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(qp.grid)), dim3(kQThreads), 0, s,
                     reinterpret_cast<const uint8_t*>(scratch), hs, weight, ld_w, ws, n, v, ksteps,
                     mblocks, vblocks, targets.p, targets.is32, ignore, inv_t, pm, ps, pw, pt, z,
                     ld_z, queue, qp.queued);
}

}  // namespace itl
