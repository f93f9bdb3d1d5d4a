// The LM head on 8-bit rows (e4m3) with one scale a row, and the tile
// statistics of its logits, on gfx950.
//
//   z[r, j] = (sum_k hidden[r, k] weight[j, k]) hs[r] ws[j]
//
// Arithmetic: e4m3 values widen exactly to bf16, every sum is one fp32
// accumulator fed by v_mfma_f32_32x32x16_bf16, no split; z = (acc hs) ws,
// x = z * fl32(1 / T).  (The 8-bit matrix instruction runs at twice the rate,
// but it aligns a group's products to about 17 bits before it adds them: logits
// off by 1.4e-5 of their spread, a hundred times what fp32 sums cost, and
// nothing in the inputs bounds it.  4096 rows took 2.1 ms with it.)
// The statistic tile is 128 vocabulary columns in four groups of 32.  Maximum:
// exact.  Sum (and entropy moment): in a group, the 16 columns 8a + b (b < 4)
// and the 16 columns 8a + 4 + b are folded in ascending order from +0 and
// added; the groups follow as (g0 + g1) + (g2 + g3).  Every kernel below
// evaluates exactly this, so a row's outputs do not depend on n or its place.
//
// The weight rows are the matrix product's first operand, so that an
// accumulator register holds a vocabulary column and a lane a hidden row: the
// statistics are folds over registers and one exchange between the two halves
// of the wave, where the other order needs a five-level butterfly a value.
//
// Two kernels:
//   q8_stats_wide (n > 128): 256 x 256 blocks, eight waves of 128 vocabulary
//     columns (one tile) x 64 hidden rows; bound by the matrix cores.
//   q8_stats_narrow<NB> (n <= 32 NB, NB = 1, 2, 4): 128 vocabulary columns x
//     32 NB hidden rows, four waves of 32 columns, two workgroups a CU; bound
//     by the weight's bytes.  Tiles of 128 columns leave less of the GPU idle
//     at the end than 256 would (V = 151936: 1187 tiles instead of 594).
#include "linear_q8.h"

#include "logp_device.h"
#include "mfma_gemm.h"

namespace itl {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kV = 256;            // vocabulary columns of a wide block
constexpr int kVT = kQ8Tile;       // vocabulary columns per statistic tile
constexpr int kStep = 64;          // K bytes per matrix instruction
constexpr int kQThreads = 512;     // 8 waves (wide)
constexpr int kNThreads = 256;     // 4 waves (narrow)

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

// What the epilogue needs of a block's R hidden rows and C vocabulary columns.
template <int R, int C>
struct Q8Rows {
  float hs[R];
  float ws[C];
  int code[R];  // -2: no statistics; -1: target elsewhere; else its column
};

template <int R, int C, int THREADS>
__device__ __forceinline__ void q8_fill(Q8Rows<R, C>& rd, const float* hs, const float* ws,
                                        int64_t n, int64_t v, int64_t m0, int64_t v0,
                                        Targets targets, int64_t ignore) {
  for (int i = threadIdx.x; i < R; i += THREADS) {
    const int64_t r = m0 + i;
    int code = -2;
    float s = 0.0f;
    if (r < n) {
      const int64_t t = targets[r];
      if (t != ignore) code = (t >= v0 && t < v0 + C && t < v) ? static_cast<int>(t - v0) : -1;
      s = hs[r];
    }
    rd.code[i] = code;
    rd.hs[i] = s;
  }
  for (int i = threadIdx.x; i < C; i += THREADS) rd.ws[i] = v0 + i < v ? ws[v0 + i] : 0.0f;
}

// From accumulators to scaled logits: acc[i][j][q] of the wave's groups (32
// columns each, from block column c0 on) and hidden rows (32 each, from row0
// on) is column c0 + 32 i + 8 (q / 4) + 4 hf + q % 4 of row row0 + 32 j + l %
// 32.  Writes z when asked and leaves x, -inf past the vocabulary.
template <int NI, int NJ, int R, int C>
__device__ __forceinline__ void q8_logits(f32x16 (&acc)[NI][NJ], const Q8Rows<R, C>& rd, int c0,
                                          int row0, int64_t m0, int64_t v0, int64_t n, int64_t v,
                                          float inv_t, float* z, int64_t ld_z) {
  const int col = threadIdx.x % 32, hf = (threadIdx.x % kWave) / 32;
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
        const int c = c0 + 32 * i + 8 * a + 4 * hf;
        const float4 w = *reinterpret_cast<const float4*>(&rd.ws[c]);
        float x[4] = {acc[i][j][4 * a] * h * w.x, acc[i][j][4 * a + 1] * h * w.y,
                      acc[i][j][4 * a + 2] * h * w.z, acc[i][j][4 * a + 3] * h * w.w};
        if (zr) {
          if (v0 + c + 4 <= v) {  // the workspace's rows are 16-byte aligned
            *reinterpret_cast<float4*>(zr + c) = make_float4(x[0], x[1], x[2], x[3]);
          } else {
#pragma unroll
            for (int b = 0; b < 4; ++b)
              if (v0 + c + b < v) zr[c + b] = x[b];
          }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) acc[i][j][4 * a + b] = x[b] * inv_t;
      }
  }
  if (v0 + C > v) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          if (v0 + c0 + 32 * i + 8 * (q / 4) + 4 * hf + q % 4 >= v) acc[i][j][q] = -INFINITY;
  }
}

// A group's sum (and entropy moment) against m: both halves of the wave get it.
template <bool ENT>
__device__ __forceinline__ void q8_group_sum(const f32x16& x, float m, float& s, float& w) {
  s = 0.0f;
  w = 0.0f;
#pragma unroll
  for (int q = 0; q < 16; ++q) {
    const float d = x[q] - m;
    const float e = __builtin_amdgcn_exp2f(d * kLog2e);
    s = s + e;
    if constexpr (ENT) w = ent_term(e, d, w);
  }
  s = s + __shfl_xor(s, 32, kWave);
  if constexpr (ENT) w = w + __shfl_xor(w, 32, kWave);
}

__device__ __forceinline__ float q8_group_max(const f32x16& x) {
  float m = x[0];
#pragma unroll
  for (int q = 1; q < 16; ++q) m = max_exact(m, x[q]);
  return m;
}

// The target's logit, if column `off` of the group is one of this lane's.
__device__ __forceinline__ bool q8_target(const f32x16& x, int off, float& t) {
  const int hf = (threadIdx.x % kWave) / 32;
  if (off < 0 || off >= 32 || ((off >> 2) & 1) != hf) return false;
  const int q = (off >> 3) * 4 + (off & 3);
  t = x[0];
#pragma unroll
  for (int k = 1; k < 16; ++k) t = q == k ? x[k] : t;
  return true;
}

// ---------------------------------------------------------------------------
// Staging, for both kernels: slots of [weight rows | hidden rows] x 128
// bytes, a "pair" of K steps, whole lines of row-major operands; chunk c (16
// bytes) of row r sits in place c ^ swzp(r), which puts the 16 rows of a read
// on different banks.  A load fills 8 rows; rows past the data read the last
// row, and the missing second half of an odd last pair the first half: every
// load stays in bounds, and what it brings is masked or not read.
// ---------------------------------------------------------------------------
using gemm::swzp;
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
// Wide: two slots of 64 KiB.  The one barrier of a pair sits before its last
// chunk's products: by then every wave has read the whole slot, which the pair
// after next takes (loads issued by waves 0-3), and the next pair, issued a
// pair's time ago, has landed, so its first chunk is read while the last
// products run and the matrix cores do not pause at the barrier.
// ---------------------------------------------------------------------------
struct SmemWide {
  uint8_t s[2][(kV + 256) * kPair];
  Q8Rows<256, kV> rd;
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
  // Blocks of 8 rows: wave + 4 u of either operand, u < 8.  The offsets are
  // taken anew for every pair (registers are short here, a pair is long).
  const int lrow = wave * 8 + lane / 8;
  const int lchunk = ((lane % 8) ^ swzp(lrow)) * 16;  // swzp ignores multiples of 32 rows
  const int back = (ksteps & 1) && lchunk >= kStep ? kStep : 0;
  const int wlast = static_cast<int>(min(v - 1 - v0, int64_t{255}));
  const int hlast = static_cast<int>(min(n - 1 - m0, int64_t{255}));
  auto issue = [&](int slot, int p) {  // into slot % 2
    if constexpr (LOADER) {
      const int64_t k = static_cast<int64_t>(p) * kPair;
      const uint8_t* w0 = W + v0 * ld_w + k;
      const uint8_t* h0 = H + m0 * ld_h + k;
      const uint32_t c = lchunk - (p == npairs - 1 ? back : 0);
      const uint32_t lw = static_cast<uint32_t>(ld_w), lh = static_cast<uint32_t>(ld_h);
      uint8_t* d = sm.s[slot % 2] + wave * 1024;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        load_lds16<false>(w0 + (min(lrow + 32 * u, wlast) * lw + c), d + u * 4096);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        load_lds16<false>(h0 + (min(lrow + 32 * u, hlast) * lh + c), d + kV * kPair + u * 4096);
    }
  };
  const int sw = swzp(row);  // repeats every 16 rows
  const int wofs = ((wave / 4) * 128 + row) * kPair;
  const int hofs = (kV + (wave % 4) * 64 + row) * kPair;
  i32x4 xw[4], xh[2], yw[4], yh[2];
  auto read = [&](int p, int u, i32x4 (&fw)[4], i32x4 (&fh)[2]) {
    const uint8_t* base = sm.s[p % 2] + ((2 * u + hf) ^ sw) * 16;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      fh[j] = *reinterpret_cast<const i32x4*>(base + hofs + 32 * j * kPair);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      fw[i] = *reinterpret_cast<const i32x4*>(base + wofs + 32 * i * kPair);
  };
  // Past the end the last pair is loaded again into the slot that is no longer
  // read, so that every pair of the loop is alike.
  issue(0, 0);
  issue(1, npairs > 1 ? 1 : 0);
  // Also the LDS writes of q8_fill: with one pair this is the only barrier
  // between them and the epilogue's reads.
  wait_vm_lgkm0<LOADER ? 16 : 0>();
  __builtin_amdgcn_s_barrier();
  read(0, 0, xw, xh);
  // Order inside a block: the next chunk's six reads, then the conversions of
  // one operand pair ahead of its products (left alone, the compiler reads a
  // chunk right before its use and the matrix cores wait for LDS).
#define ITL_Q8_ORDER                                                                            \
  __builtin_amdgcn_sched_group_barrier(0x100, 6, 0);                                            \
  __builtin_amdgcn_sched_group_barrier(0x002, 12, 0);                                           \
  _Pragma("unroll") for (int o = 0; o < 7; ++o) {                                               \
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);                                          \
    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);                                          \
  }                                                                                             \
  __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
  for (int p = 0; p + 1 < npairs; ++p) {
    read(p, 1, yw, yh);
    mfma_q8<4, 2>(xw, xh, acc);
    ITL_Q8_ORDER
    read(p, 2, xw, xh);
    mfma_q8<4, 2>(yw, yh, acc);
    ITL_Q8_ORDER
    read(p, 3, yw, yh);
    mfma_q8<4, 2>(xw, xh, acc);
    ITL_Q8_ORDER
    wait_vm_lgkm0<0>();  // this wave's reads of pair p, its loads of pair p + 1
    __builtin_amdgcn_s_barrier();
    issue(p, p + 2 < npairs ? p + 2 : npairs - 1);
    read(p + 1, 0, xw, xh);
    mfma_q8<4, 2>(yw, yh, acc);
    ITL_Q8_ORDER
  }
  {
    const int p = npairs - 1;
    read(p, 1, yw, yh);
    mfma_q8<4, 2>(xw, xh, acc);
    if (2 * p + 1 < ksteps) {
      read(p, 2, xw, xh);
      mfma_q8<4, 2>(yw, yh, acc);
      read(p, 3, yw, yh);
      mfma_q8<4, 2>(xw, xh, acc);
    }
    mfma_q8<4, 2>(yw, yh, acc);
  }
#undef ITL_Q8_ORDER
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <bool ENT>
__global__ __launch_bounds__(kQThreads) void q8_stats_wide(
    const uint8_t* __restrict__ hidden, int64_t ld_h, const float* __restrict__ hs,
    const uint8_t* __restrict__ weight, int64_t ld_w, const float* __restrict__ ws, int64_t n,
    int64_t v, int ksteps, int mblocks, int vblocks, int ntiles, const void* __restrict__ tgt,
    int32_t tgt32, int64_t ignore, float inv_t, float* __restrict__ pm, float* __restrict__ ps,
    float* __restrict__ pw, float* __restrict__ pt, float* __restrict__ z, int64_t ld_z,
    int* queue, int queued) {
  const Targets targets{tgt, tgt32};
  __shared__ __align__(16) SmemWide sm;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int logical = gemm::queue_tile(queue, mblocks * vblocks, queued, &sm.slot);
  if (logical < 0) return;
  int mb, vb;
  gemm::tile_coords(logical, mblocks, vblocks, mb, vb);
  const int64_t m0 = static_cast<int64_t>(mb) * 256, v0 = static_cast<int64_t>(vb) * kV;
  q8_fill<256, kV, kQThreads>(sm.rd, hs, ws, n, v, m0, v0, targets, ignore);
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
  // A wave holds its 64 rows' whole tile: no exchange between waves.
  const int c0 = (wave / 4) * kVT, row0 = (wave % 4) * 64;
  q8_logits<4, 2, 256, kV>(acc, sm.rd, c0, row0, m0, v0, n, v, inv_t, z, ld_z);
  const int tile = vb * (kV / kVT) + wave / 4;
  if (tile >= ntiles) return;  // the second half of the last block may be empty
  const int col = threadIdx.x % 32, hf = (threadIdx.x % kWave) / 32;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int lr = row0 + 32 * j + col;
    const int64_t r = m0 + lr;
    const int code = sm.rd.code[lr];
    float m = q8_group_max(acc[0][j]);
#pragma unroll
    for (int i = 1; i < 4; ++i) m = max_exact(m, q8_group_max(acc[i][j]));
    m = max_exact(m, __shfl_xor(m, 32, kWave));
    float s[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float t;
      if (q8_target(acc[i][j], code - c0 - 32 * i, t)) pt[r] = t;
      q8_group_sum<ENT>(acc[i][j], m, s[i], w[i]);
    }
    if (hf == 0 && code != -2) {
      pm[r * ntiles + tile] = m;
      ps[r * ntiles + tile] = (s[0] + s[1]) + (s[2] + s[3]);
      if constexpr (ENT) pw[r * ntiles + tile] = (w[0] + w[1]) + (w[2] + w[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// Narrow: two or three slots with 32 NB hidden rows, every wave loading; wave
// w computes vocabulary group w for all hidden rows.
// ---------------------------------------------------------------------------
template <int NB>
constexpr int kNarrowSlots = NB == 4 ? 2 : 3;

template <int NB>
struct SmemNarrowQ8 {
  uint8_t s[kNarrowSlots<NB>][(kVT + 32 * NB) * kPair];
  Q8Rows<32 * NB, kVT> rd;
  float max[4][32 * NB];
  float sum[4][32 * NB];
  float wsum[4][32 * NB];
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
  // blocks of 8 rows: wave + 4 u of the weight's 16 and the hidden rows' 4 NB
  const uint8_t* wp[4];
  const uint8_t* hp[NB];
#pragma unroll
  for (int u = 0; u < 4; ++u)
    wp[u] = weight + v0 * ld_w + pair_source(ld_w, v0, v, wave + 4 * u, lane);
#pragma unroll
  for (int u = 0; u < NB; ++u) hp[u] = hidden + pair_source(ld_h, 0, n, wave + 4 * u, lane);
  const int back = pair_back(ksteps, wave, lane);
  auto issue = [&](int slot, int pair) {
    const int p = pair < npairs ? pair : npairs - 1;
    const int64_t k = static_cast<int64_t>(p) * kPair - (p == npairs - 1 ? back : 0);
    uint8_t* d = sm.s[slot] + wave * 1024;
#pragma unroll
    for (int u = 0; u < 4; ++u) load_lds16<true>(wp[u] + k, d + u * 4096);
#pragma unroll
    for (int u = 0; u < NB; ++u) load_lds16<false>(hp[u] + k, d + kVT * kPair + u * 4096);
  };
  const int row = lane % 32, hf = lane / 32;
  const int sw = swzp(row);
  for (int p = 0; p < S - 1; ++p) issue(p, p);
  // Before pair p is read its loads have landed once only those of the S - 2
  // pairs issued after it are in flight; after the barrier that holds for
  // every wave, and nobody reads slot (p - 1) % S any more, which the pair
  // S - 1 ahead then takes.
  for (int p = 0; p < npairs; ++p) {
    wait_vm_lgkm0<(S - 2) * (4 + NB)>();
    __builtin_amdgcn_s_barrier();
    issue((p + S - 1) % S, p + S - 1);
    const uint8_t* w_ = sm.s[p % S] + (wave * 32 + row) * kPair;
    const uint8_t* h_ = sm.s[p % S] + (kVT + row) * kPair;
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
__global__ __launch_bounds__(kNThreads) void q8_stats_narrow(
    const uint8_t* __restrict__ hidden, int64_t ld_h, const float* __restrict__ hs,
    const uint8_t* __restrict__ weight, int64_t ld_w, const float* __restrict__ ws, int64_t n,
    int64_t v, int ksteps, int ntiles, const void* __restrict__ tgt, int32_t tgt32,
    int64_t ignore, float inv_t, float* __restrict__ pm, float* __restrict__ ps,
    float* __restrict__ pw, float* __restrict__ pt, float* __restrict__ z, int64_t ld_z) {
  constexpr int R = 32 * NB;
  const Targets targets{tgt, tgt32};
  __shared__ __align__(16) SmemNarrowQ8<NB> sm;
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int col = tid % 32, hf = (tid % kWave) / 32;
  const int tile = gemm::xcd_logical(blockIdx.x, ntiles);
  const int64_t v0 = static_cast<int64_t>(tile) * kVT;
  q8_fill<R, kVT, kNThreads>(sm.rd, hs, ws, n, v, 0, v0, targets, ignore);
  f32x16 acc[1][NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int q = 0; q < 16; ++q) acc[0][j][q] = 0.0f;
  q8_mainloop_narrow<NB>(sm, hidden, ld_h, n, weight, ld_w, v0, v, ksteps, acc);
  __syncthreads();
  q8_logits<1, NB, R, kVT>(acc, sm.rd, wave * 32, 0, 0, v0, n, v, inv_t, z, ld_z);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    float m = q8_group_max(acc[0][j]);
    m = max_exact(m, __shfl_xor(m, 32, kWave));
    if (hf == 0) sm.max[wave][32 * j + col] = m;
  }
  __syncthreads();
  auto tile_max = [&](int lr) {
    return max_exact(max_exact(sm.max[0][lr], sm.max[1][lr]),
                     max_exact(sm.max[2][lr], sm.max[3][lr]));
  };
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int lr = 32 * j + col;
    float t, s, w;
    if (q8_target(acc[0][j], sm.rd.code[lr] - wave * 32, t)) pt[lr] = t;
    q8_group_sum<ENT>(acc[0][j], tile_max(lr), s, w);
    if (hf == 0) {
      sm.sum[wave][lr] = s;
      if constexpr (ENT) sm.wsum[wave][lr] = w;
    }
  }
  __syncthreads();
  for (int lr = tid; lr < R; lr += kNThreads) {
    if (sm.rd.code[lr] == -2) continue;
    const int64_t at = static_cast<int64_t>(lr) * ntiles + tile;
    pm[at] = tile_max(lr);
    ps[at] = (sm.sum[0][lr] + sm.sum[1][lr]) + (sm.sum[2][lr] + sm.sum[3][lr]);
    if constexpr (ENT)
      pw[at] = (sm.wsum[0][lr] + sm.wsum[1][lr]) + (sm.wsum[2][lr] + sm.wsum[3][lr]);
  }
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
  const int ntiles = static_cast<int>((v + kVT - 1) / kVT);
  const int ksteps = static_cast<int>(h / kStep);
  if (n <= 128) {
    auto kern = n <= 32   ? (pw ? q8_stats_narrow<1, true> : q8_stats_narrow<1, false>)
                : n <= 64 ? (pw ? q8_stats_narrow<2, true> : q8_stats_narrow<2, false>)
                          : (pw ? q8_stats_narrow<4, true> : q8_stats_narrow<4, false>);
    hipLaunchKernelGGL(kern, dim3(ntiles), dim3(kNThreads), 0, s, hidden, ld_h, hs, weight, ld_w,
                       ws, n, v, ksteps, ntiles, targets.p, targets.is32, ignore, inv_t, pm, ps,
                       pw, pt, z, ld_z);
    return;
  }
  const int vblocks = static_cast<int>((v + kV - 1) / kV);
  const int mblocks = static_cast<int>((n + 255) / 256);
  int* queue = reinterpret_cast<int*>(scratch);
  hipLaunchKernelGGL(clear_queue, dim3(1), dim3(gemm::kQueueBytes / 4), 0, s, queue);
  const gemm::QueuePlan qp = gemm::queue_plan(mblocks * vblocks, xcd_cus());
  auto kern = pw ? q8_stats_wide<true> : q8_stats_wide<false>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(qp.grid)), dim3(kQThreads), 0, s, hidden,
                     ld_h, hs, weight, ld_w, ws, n, v, ksteps, mblocks, vblocks, ntiles, targets.p,
                     targets.is32, ignore, inv_t, pm, ps, pw, pt, z, ld_z, queue, qp.queued);
}

}  // namespace itl
