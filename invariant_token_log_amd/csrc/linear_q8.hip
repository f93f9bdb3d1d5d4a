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
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kV = kLinearTile;    // vocabulary columns per tile
constexpr int kStep = 64;          // K bytes per matrix instruction
constexpr int kQThreads = 512;     // 8 waves

// Eight e4m3 values (two dwords of a chunk) as bf16, exactly.
__device__ __forceinline__ bf16x8 widen_q8(int lo, int hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// acc[i][j] += the 32 products of the 16-byte chunks w[i] and h[j] that the two
// halves of the wave hold, 16 at a time.  Which K index a byte stands for does
// not matter as long as both operands agree.
template <int NI, int NJ>
__device__ __forceinline__ void mfma_q8(const i32x4 (&w)[NI], const i32x4 (&h)[NJ],
                                        f32x16 (&acc)[NI][NJ]) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    bf16x8 b[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = widen_q8(h[j][2 * t], h[j][2 * t + 1]);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bf16x8 a = widen_q8(w[i][2 * t], w[i][2 * t + 1]);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b[j], acc[i][j], 0, 0, 0);
    }
  }
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
// Staging, for both kernels: slots of [256 weight rows | R hidden rows] x 128
// bytes, a "pair" of K steps, whole lines of row-major operands; chunk c (16
// bytes) of row r sits in place c ^ swzp(r), which puts the 16 rows of a read
// on different banks.  A load fills 8 rows; rows past the data read the last
// row, and the missing second half of an odd last pair the first half: every
// load stays in bounds, and what it brings is masked or not read.
// ---------------------------------------------------------------------------
using gemm::swzp;
using gemm::wait_vm;
using gemm::wait_vm_lgkm0;

constexpr int kPair = 2 * kStep;  // bytes of a row per pair

// One direct 16-byte load a lane, global -> LDS at dst + 16 * lane; NT: past
// the caches.
template <bool NT>
__device__ __forceinline__ void load_lds16(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds(src, dst, 16, 0, NT ? 2 : 0);
}

// Offset from row row0 of this lane's chunk of row block `blk` (8 rows) at
// pair 0; at most 256 rows of at most kMaxQ8Stride bytes, so 32 bits hold it.
__device__ __forceinline__ uint32_t pair_source(int64_t ld, int64_t row0, int64_t rows, int blk,
                                                int lane) {
  const int r = blk * 8 + lane / 8;
  const int64_t last = rows - 1 - row0;
  return static_cast<uint32_t>((r < last ? r : last) * ld) + ((lane % 8) ^ swzp(r)) * 16;
}
// How far the lane steps back in an odd last pair (blocks 4 apart agree).
__device__ __forceinline__ int pair_back(int ksteps, int blk, int lane) {
  return (ksteps & 1) && ((lane % 8) ^ swzp(blk * 8 + lane / 8)) >= 4 ? kStep : 0;
}

// ---------------------------------------------------------------------------
// Wide: two slots of 64 KiB; while a pair is multiplied the next one loads,
// issued by waves 0-3 right after the barrier.
// ---------------------------------------------------------------------------
struct SmemWide {
  uint8_t s[2][(kV + 256) * kPair];
  Q8Reduce<256> rd;
  int slot;
};

template <bool LOADER>
__device__ __forceinline__ void q8_mainloop(SmemWide& sm, const uint8_t* __restrict__ H,
                                            int64_t ld_h, int64_t m0, int64_t n,
                                            const uint8_t* __restrict__ W, int64_t ld_w,
                                            int64_t v0, int64_t v, int ksteps,
                                            f32x16 (&acc)[4][2]) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int row = lane % 32, hf = lane / 32;
  const int npairs = (ksteps + 1) / 2;
  uint32_t wp[8], hp[8];
  int back = 0;
  if constexpr (LOADER) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      wp[u] = pair_source(ld_w, v0, v, wave + 4 * u, lane);
      hp[u] = pair_source(ld_h, m0, n, wave + 4 * u, lane);
    }
    back = pair_back(ksteps, wave, lane);
  }
  auto issue = [&](int p) {
    if constexpr (LOADER) {
      const uint8_t* w0 = W + v0 * ld_w + static_cast<int64_t>(p) * kPair;
      const uint8_t* h0 = H + m0 * ld_h + static_cast<int64_t>(p) * kPair;
      const int b = p == npairs - 1 ? back : 0;
      uint8_t* d = sm.s[p % 2] + wave * 1024;
#pragma unroll
      for (int u = 0; u < 8; ++u) load_lds16<false>(w0 + (wp[u] - b), d + u * 4096);
#pragma unroll
      for (int u = 0; u < 8; ++u) load_lds16<false>(h0 + (hp[u] - b), d + kV * kPair + u * 4096);
    }
  };
  const int sw = swzp(row);  // repeats every 16 rows
  const int wofs = ((wave / 4) * 128 + row) * kPair;
  const int hofs = (kV + (wave % 4) * 64 + row) * kPair;
  issue(0);
  for (int p = 0; p < npairs; ++p) {
    // pair p has landed (it is all that was in flight), and nobody reads the
    // other slot any more
    wait_vm_lgkm0<0>();
    __builtin_amdgcn_s_barrier();
    if (p + 1 < npairs) issue(p + 1);
    const uint8_t* w_ = sm.s[p % 2] + wofs;
    const uint8_t* h_ = sm.s[p % 2] + hofs;
    i32x4 cw[2][4], ch[2][2];
    auto read = [&](int u, i32x4 (&fw)[4], i32x4 (&fh)[2]) {
      const int c = ((2 * u + hf) ^ sw) * 16;
#pragma unroll
      for (int j = 0; j < 2; ++j) fh[j] = *reinterpret_cast<const i32x4*>(h_ + 32 * j * kPair + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) fw[i] = *reinterpret_cast<const i32x4*>(w_ + 32 * i * kPair + c);
    };
    read(0, cw[0], ch[0]);
    read(1, cw[1], ch[1]);
    mfma_q8<4, 2>(cw[0], ch[0], acc);
    if (2 * p + 1 < ksteps) {
      read(2, cw[0], ch[0]);
      mfma_q8<4, 2>(cw[1], ch[1], acc);
      read(3, cw[1], ch[1]);
      mfma_q8<4, 2>(cw[0], ch[0], acc);
    }
    mfma_q8<4, 2>(cw[1], ch[1], acc);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <bool ENT>
__global__ __launch_bounds__(kQThreads) void q8_stats_wide(
    const uint8_t* __restrict__ hidden, int64_t ld_h, const float* __restrict__ hs,
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
    q8_mainloop<true>(sm, hidden, ld_h, m0, n, weight, ld_w, v0, v, ksteps, acc);
  else
    q8_mainloop<false>(sm, hidden, ld_h, m0, n, weight, ld_w, v0, v, ksteps, acc);
  __syncthreads();
  q8_epilogue<4, 2, 256, ENT>(acc, sm.rd, (wave / 4) * 4, (wave % 4) * 64, tid, m0, v0, vb,
                              vblocks, n, v, inv_t, pm, ps, pw, pt, z, ld_z);
}

// ---------------------------------------------------------------------------
// Narrow: three or four slots with 32 NB hidden rows, every wave loading; wave
// w computes vocabulary group w for all hidden rows.
// ---------------------------------------------------------------------------
template <int NB>
constexpr int kNarrowSlots = NB == 1 ? 4 : 3;

template <int NB>
struct SmemNarrowQ8 {
  uint8_t s[kNarrowSlots<NB>][(kV + 32 * NB) * kPair];
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
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int npairs = (ksteps + 1) / 2;
  constexpr int kHBlocks = 4 * NB;              // hidden blocks of 8 rows
  constexpr int NH = kHBlocks > 8 ? 2 : 1;      // loads of them a wave
  const bool has_h = wave < kHBlocks;
  const uint8_t* wp[4];
  const uint8_t* hp[NH];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    wp[u] = weight + v0 * ld_w + pair_source(ld_w, v0, v, wave + 8 * u, lane);
#pragma unroll
  for (int u = 0; u < NH; ++u)
    hp[u] = hidden + pair_source(ld_h, 0, n, wave % kHBlocks + 8 * u, lane);
  const int back_w = pair_back(ksteps, wave, lane);
  const int back_h = pair_back(ksteps, wave % kHBlocks, lane);
  auto issue = [&](int slot, int pair) {
    const int p = pair < npairs ? pair : npairs - 1;
    const int64_t k = static_cast<int64_t>(p) * kPair;
    const bool end = p == npairs - 1;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      load_lds16<true>(wp[u] + k - (end ? back_w : 0), sm.s[slot] + (wave + 8 * u) * 1024);
    if (has_h) {
#pragma unroll
      for (int u = 0; u < NH; ++u)
        load_lds16<false>(hp[u] + k - (end ? back_h : 0),
                          sm.s[slot] + kV * kPair + (wave + 8 * u) * 1024);
    }
  };
  const int row = lane % 32, hf = lane / 32;
  const int sw = swzp(row);
  for (int p = 0; p < S - 1; ++p) issue(p, p);
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
    issue((p + S - 1) % S, p + S - 1);
    const uint8_t* w_ = sm.s[p % S] + (wave * 32 + row) * kPair;
    const uint8_t* h_ = sm.s[p % S] + (kV + row) * kPair;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u == 2 && 2 * p + 1 >= ksteps) break;
      const int c = ((2 * u + hf) ^ sw) * 16;
      const i32x4 a[1] = {*reinterpret_cast<const i32x4*>(w_ + c)};
      i32x4 b[NB];
#pragma unroll
      for (int j = 0; j < NB; ++j) b[j] = *reinterpret_cast<const i32x4*>(h_ + 32 * j * kPair + c);
      mfma_q8<1, NB>(a, b, acc);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
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

// The tile queue's counters, before the wide kernel.
__global__ void clear_queue(int* queue) { queue[threadIdx.x] = 0; }

}  // namespace

int64_t q8_fwd_scratch_bytes(int64_t n, int64_t h) {
  (void)h;
  return n > 128 ? gemm::kQueueBytes : 0;
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
  int* queue = reinterpret_cast<int*>(scratch);
  hipLaunchKernelGGL(clear_queue, dim3(1), dim3(gemm::kQueueBytes / 4), 0, s, queue);
  const gemm::QueuePlan qp = gemm::queue_plan(mblocks * vblocks, xcd_cus());
  auto kern = pw ? q8_stats_wide<true> : q8_stats_wide<false>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(qp.grid)), dim3(kQThreads), 0, s,
                     hidden, ld_h, hs, weight, ld_w, ws, n, v, ksteps,
                     mblocks, vblocks, targets.p, targets.is32, ignore, inv_t, pm, ps, pw, pt, z,
                     ld_z, queue, qp.queued);
}

}  // namespace itl
