// The statistic epilogue of the LM-head kernels: from a workgroup's accumulators
// of 256 vocabulary columns to the tile statistics, the target logits and the
// unscaled logits.  The arithmetic is that of linear_logp.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "logp_device.h"
#include "mfma_gemm.h"

namespace itl {
namespace linear_stats {

using gemm::f32x4;

constexpr int BN = kLinearTile;  // vocabulary columns per workgroup (= statistic tile)
constexpr int BK = gemm::kK;     // K per MFMA step

template <int BM>
struct Reduce {
  float red[BM][4];  // per-row quarter maxima
  float sum[BM][4];  // per-row quarter sums
  float wsum[BM][4]; // per-row quarter entropy moments (when requested)
  float tmax[BM];    // per-row tile maximum
  float tval[BM];    // target logit, when the target column is in this block
  int code[BM];      // row_code() of each row
};

// Per-row code for the epilogue: -2 = no statistics (row past n, or its
// target is ignore_index), -1 = target column outside this vocabulary block,
// else the target column minus v0.
__device__ __forceinline__ int row_code(int64_t r, int64_t n, Targets targets,
                                        int64_t ignore_index, int64_t v0, int64_t v) {
  if (r >= n) return -2;
  const int64_t t = targets[r];
  if (t == ignore_index) return -2;
  return (t >= v0 && t < v0 + BN && t < v) ? static_cast<int>(t - v0) : -1;
}

// Workgroup barrier for LDS traffic only: waits for this wave's LDS
// operations, not for its outstanding global loads or stores.
__device__ __forceinline__ void block_sync_lds() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Statistic epilogue.  The wave holds acc[i][j][q] =
//   z[m0 + row0 + i*16 + 4g + q][v0 + col0 + j*16 + li],  j < NJ,
// where its NJ column groups form NJ / 4 whole quarters starting at quarter
// col0 / 64.  NT = threads of the workgroup.  rd.code must be filled, and
// accumulators of columns >= v must already hold -inf.
template <int MI, int NJ, int BM, int NT, bool ENT>
__device__ __forceinline__ void stats_epilogue_body(const f32x4 (&acc)[MI][NJ], Reduce<BM>& rd,
                                                    int row0, int col0, int li, int g, int tid,
                                                    int64_t m0, int64_t v0, int vb, int vblocks,
                                                    int64_t v, float* pm, float* ps, float* pw,
                                                    float* pt) {
  constexpr int NQ = NJ / 4;  // quarters held by this wave
  const int q0 = col0 / 64;
  auto z = [&](int i, int j, int q) { return acc[i][j][q]; };

  // Pass 1: quarter maxima (exact, order-free).
  float part[MI][4][NQ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        float m = z(i, 4 * h, q);
#pragma unroll
        for (int j = 4 * h + 1; j < 4 * h + 4; ++j) m = max_exact(m, z(i, j, q));
        part[i][q][h] = row16_max_first(m);
      }
  if (li == 0) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < NQ; ++h) rd.red[row0 + i * 16 + 4 * g + q][q0 + h] = part[i][q][h];
  }
  block_sync_lds();
  for (int lr = tid; lr < BM; lr += NT) {
    const float4 r4 = *reinterpret_cast<const float4*>(rd.red[lr]);
    rd.tmax[lr] = max_exact(max_exact(r4.x, r4.y), max_exact(r4.z, r4.w));
  }
  block_sync_lds();

  // Pass 2.  The lane's rows are 4 consecutive rows per row group i, so their
  // codes and tile maxima come in as one 16-byte LDS read per group, all
  // issued before any use.  First the target copies: the one lane holding
  // the target column of a row parks z[r, t] in LDS.  A wave's 64 columns
  // hold a target only now and then, so the hit tests run branch-free and
  // one wave-uniform branch enters the copy only when some lane has a hit.
  // Then the quarter sums against the tile maximum (and, with ENT, the
  // entropy moments sum e (z - m), same tree) as one branch-free block, so
  // that the exponentials of all row groups interleave.
  int4 code4[MI];
  float4 m4[MI];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const int lr = row0 + i * 16 + 4 * g;
    code4[i] = *reinterpret_cast<const int4*>(&rd.code[lr]);
    m4[i] = *reinterpret_cast<const float4*>(&rd.tmax[lr]);
  }
  // 1 when this lane holds the target column of a row with this code (the
  // code is -1 or -2 for rows whose target is elsewhere or absent)
  auto holds_target = [&](int code) {
    const unsigned off = static_cast<unsigned>(code - col0);
    return static_cast<int>(off < static_cast<unsigned>(NJ * 16)) &
           static_cast<int>((off & 15u) == static_cast<unsigned>(li));
  };
  int any_hit = 0;
#pragma unroll
  for (int i = 0; i < MI; ++i)
    any_hit |= holds_target(code4[i].x) | holds_target(code4[i].y) | holds_target(code4[i].z) |
               holds_target(code4[i].w);
  if (__builtin_amdgcn_ballot_w64(any_hit != 0)) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int c4[4] = {code4[i].x, code4[i].y, code4[i].z, code4[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (holds_target(c4[q])) {
          const int off = c4[q] - col0;
          float zt = acc[i][0][q];
#pragma unroll
          for (int j = 1; j < NJ; ++j)
            if ((off >> 4) == j) zt = acc[i][j][q];
          rd.tval[row0 + i * 16 + 4 * g + q] = zt;
        }
      }
    }
  }
  float wpart[ENT ? MI : 1][4][NQ];
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const float mq[4] = {m4[i].x, m4[i].y, m4[i].z, m4[i].w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float m = mq[q];
#pragma unroll
      for (int h = 0; h < NQ; ++h) {
        if constexpr (ENT) {
          float s = 0.0f, w = 0.0f;
#pragma unroll
          for (int j = 4 * h; j < 4 * h + 4; ++j) {
            const float d = z(i, j, q) - m;  // exp_sub(z, m) in two steps
            const float e = __builtin_amdgcn_exp2f(d * kLog2e);
            s = j == 4 * h ? e : s + e;
            w = ent_term(e, d, w);
          }
          part[i][q][h] = row16_sum_first(s);
          wpart[i][q][h] = row16_sum_first(w);
        } else {
          float s = exp_sub(z(i, 4 * h, q), m);
#pragma unroll
          for (int j = 4 * h + 1; j < 4 * h + 4; ++j) s = s + exp_sub(z(i, j, q), m);
          part[i][q][h] = row16_sum_first(s);
        }
      }
    }
  }
  if (li == 0) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < NQ; ++h) {
          rd.sum[row0 + i * 16 + 4 * g + q][q0 + h] = part[i][q][h];
          if constexpr (ENT) rd.wsum[row0 + i * 16 + 4 * g + q][q0 + h] = wpart[i][q][h];
        }
  }
  block_sync_lds();

  for (int lr = tid; lr < BM; lr += NT) {
    const int code = rd.code[lr];
    if (code != -2) {
      const int64_t r = m0 + lr;
      const float4 s4 = *reinterpret_cast<const float4*>(rd.sum[lr]);
      pm[r * vblocks + vb] = rd.tmax[lr];
      ps[r * vblocks + vb] = (s4.x + s4.y) + (s4.z + s4.w);
      if constexpr (ENT) {
        const float4 w4 = *reinterpret_cast<const float4*>(rd.wsum[lr]);
        pw[r * vblocks + vb] = (w4.x + w4.y) + (w4.z + w4.w);
      }
      if (code >= 0) pt[r] = rd.tval[lr];
    }
  }
}

// Options of the forward statistic kernels: the logits' rounding point, the
// temperature's reciprocal (logits are multiplied by it before any
// statistic), the entropy moment table and the unscaled logits.
struct LinearExtras {
  float inv_t;      // 1 = no temperature
  int32_t round_bf16;  // 1 = z is RNE_bf16 of the accumulator
  float* pw;        // [n, T] entropy moments, or null
  void* z;          // [n, ld_z] unscaled logits (fp32 or bf16), or null
  int32_t z_bf16;
  int64_t ld_z;
  int32_t z_vec;    // z and its rows are 16-byte aligned: staged 16-byte stores
};

// Logits output through LDS: the tile's accumulators go to `scratch` (the
// main loop's stages, free by now) a row chunk at a time, then leave as
// whole 16-byte pieces along the rows (the accumulator layout would store
// 4 or 2 bytes per lane).  RPC rows per chunk: the largest power-of-two part
// of the tile that fits.
template <typename E, int MI, int NJ, int BM, int NT, int SCRATCH>
__device__ __forceinline__ void store_logits_staged(const f32x4 (&acc)[MI][NJ], void* scratch,
                                                    int row0, int col0, int li, int g, int tid,
                                                    int64_t m0, int64_t v0, int64_t n,
                                                    int64_t v, E* z, int64_t ld_z) {
  constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements per 16-byte piece
  constexpr int kStride = BN + kPer;                       // padded LDS row
  constexpr int kRowBytes = kStride * static_cast<int>(sizeof(E));
  constexpr int RPC = BM * kRowBytes <= SCRATCH       ? BM
                      : BM / 2 * kRowBytes <= SCRATCH ? BM / 2
                      : BM / 4 * kRowBytes <= SCRATCH ? BM / 4
                                                      : BM / 8;
  static_assert(RPC * kRowBytes <= SCRATCH && RPC % 16 == 0, "logits chunk does not fit");
  E* tile = static_cast<E*>(scratch);
  for (int c = 0; c < BM / RPC; ++c) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int lr0 = row0 + i * 16 - c * RPC;  // uniform
      if (lr0 < 0 || lr0 >= RPC) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float x = acc[i][j][q];
          E e;
          if constexpr (sizeof(E) == 2)
            e = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
          else
            e = x;
          tile[(lr0 + 4 * g + q) * kStride + col0 + j * 16 + li] = e;
        }
    }
    __syncthreads();
    constexpr int kCpr = BN / kPer;  // pieces per row
    for (int idx = tid; idx < RPC * kCpr; idx += NT) {
      const int lr = idx / kCpr, pc = (idx % kCpr) * kPer;
      const int64_t r = m0 + c * RPC + lr, col = v0 + pc;
      if (r >= n) continue;
      E* dst = z + r * ld_z + col;
      const E* src = tile + lr * kStride + pc;
      if (col + kPer <= v) {
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
      } else {
        for (int u = 0; u < kPer; ++u)
          if (col + u < v) dst[u] = src[u];
      }
    }
    __syncthreads();
  }
}

// (ex by value: taken by reference it was kept in memory, which the compiler puts
// into 16 bytes of LDS a thread and finds by reading the dispatch packet: up to
// 13 us a launch.)
template <int MI, int NJ, int BM, int NT, int SCRATCH>
__device__ __forceinline__ void stats_epilogue(f32x4 (&acc)[MI][NJ], Reduce<BM>& rd, void* scratch,
                                               int row0, int col0, int li, int g, int tid,
                                               int64_t m0, int64_t v0, int vb, int vblocks,
                                               int64_t n, int64_t v, float* pm, float* ps,
                                               float* pt, LinearExtras ex) {
  // The bf16-rounded variant: z becomes RNE_bf16(accumulator), widened
  // exactly, before anything reads it (logits output, temperature, every
  // statistic and the target copy).
  if (ex.round_bf16) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i][j][q] = static_cast<float>(static_cast<__bf16>(acc[i][j][q]));
  }
  // The unscaled logits, when asked for: they are the accumulators as they
  // are (the statistics below do not change them).
  if (ex.z && ex.z_vec) {
    if (ex.z_bf16)
      store_logits_staged<uint16_t, MI, NJ, BM, NT, SCRATCH>(acc, scratch, row0, col0, li, g, tid,
                                                             m0, v0, n, v,
                                                             static_cast<uint16_t*>(ex.z), ex.ld_z);
    else
      store_logits_staged<float, MI, NJ, BM, NT, SCRATCH>(acc, scratch, row0, col0, li, g, tid, m0,
                                                          v0, n, v, static_cast<float*>(ex.z),
                                                          ex.ld_z);
  } else if (ex.z) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t r = m0 + row0 + i * 16 + 4 * g + q;
        if (r >= n) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const int64_t c = v0 + col0 + j * 16 + li;
          if (c >= v) continue;
          if (ex.z_bf16)
            static_cast<uint16_t*>(ex.z)[r * ex.ld_z + c] =
                __builtin_bit_cast(uint16_t, static_cast<__bf16>(acc[i][j][q]));
          else
            static_cast<float*>(ex.z)[r * ex.ld_z + c] = acc[i][j][q];
        }
      }
  }
  // Temperature: x = z * (1 / T) on every accumulator before any statistic.
  if (ex.inv_t != 1.0f) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = acc[i][j] * ex.inv_t;
  }
  // Columns >= v exist only in the last vocabulary block.  Their -inf takes
  // no part in a maximum and adds an exact 0 to a sum; no target lies there.
  if (v0 + BN > v) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      if (v0 + col0 + j * 16 + li >= v)
#pragma unroll
        for (int i = 0; i < MI; ++i) acc[i][j] = f32x4{-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  }
  if (ex.pw)
    stats_epilogue_body<MI, NJ, BM, NT, true>(acc, rd, row0, col0, li, g, tid, m0, v0, vb,
                                              vblocks, v, pm, ps, ex.pw, pt);
  else
    stats_epilogue_body<MI, NJ, BM, NT, false>(acc, rd, row0, col0, li, g, tid, m0, v0, vb,
                                               vblocks, v, pm, ps, ex.pw, pt);
}

}  // namespace linear_stats
}  // namespace itl
