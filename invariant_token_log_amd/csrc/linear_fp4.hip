// The LM head on 4-bit rows (fp4.h) and bf16 hidden rows, and the tile
// statistics of its logits, on gfx950.
//
//   z[r, j] = sum_k hidden[r, k] e2m1[j, k] 2^(b[j, k / 32] - 127)
//
// Arithmetic: a decoded weight is exact in bf16 (v_cvt_scalef32_pk_bf16_fp4
// decodes two values and applies their group's scale, a group of 32 columns
// being one K step of the matrix instruction), so every product is one of bf16
// values, and the sums and statistics are exactly those of linear_logp.hip: a
// row has the bits of the bf16 head on the decoded weight.
//
// Few rows: bound by the weight's bytes, 17 / 32 of a byte a value.  A workgroup
// takes 256 columns and ROWS hidden rows, eight waves of 64 columns x ROWS / 2
// rows.  Slots of 256 K values hold whole 128-byte lines of the weight's rows,
// brought by direct loads, their scales, which pass through registers (their
// rows have any alignment), and the hidden rows' pieces.
#include "linear_fp4.h"

#include "fp4.h"
#include "linear_stats.h"
#include "logp_device.h"
#include "mfma_gemm.h"

namespace itl {

namespace {

using gemm::bf16x8;
using gemm::f32x4;
using gemm::wait_vm_lgkm0;
using namespace linear_stats;

constexpr int kThreads4 = 512;
constexpr int kSlotSteps = 8;                   // K steps (of 32) a slot
constexpr int kSlotK = kSlotSteps * BK;         // 256
constexpr int kSlotBytes = kSlotK / 2;          // of a weight row: one line

template <int ROWS>
constexpr int kSlots = ROWS == 32 ? 3 : 2;

template <int ROWS>
struct Fp4Stages {
  uint8_t w[kSlots<ROWS>][BN * kSlotBytes];
  uint16_t h[kSlots<ROWS>][ROWS * kSlotK];
  uint16_t scale[kSlots<ROWS>][BN * kSlotSteps / 2];
};

template <int ROWS>
struct SmemFp4 {
  Fp4Stages<ROWS> st;
  Reduce<ROWS> rd;
};

// Two scale bytes at any address.
struct __attribute__((packed)) ScalePair {
  uint16_t w;
};

// Eight weights (a dword of codes) under the scale 2^(b - 127) given as the fp32
// with exponent b.
__device__ __forceinline__ bf16x8 decode8(uint32_t q, float scale) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// The places of a row's 16-byte pieces in a slot, so that the 16 rows of a read
// lie on different banks: weight piece c (a K step) of row r at c ^ (r / 2) % 8,
// hidden piece c at c ^ r % 16.
__device__ __forceinline__ int weight_swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int hidden_swz(int r) { return r & 15; }

template <int ROWS>
__device__ __forceinline__ void mainloop_fp4(Fp4Stages<ROWS>& sm,
                                             const uint16_t* __restrict__ hidden, int64_t ld_h,
                                             int64_t m0, int64_t n,
                                             const uint8_t* __restrict__ data, int64_t ld_d,
                                             const uint8_t* __restrict__ scales, int64_t ld_s,
                                             int64_t v0, int64_t v, int ksteps,
                                             f32x4 (&acc)[ROWS / 32][4]) {
  constexpr int S = kSlots<ROWS>, MI = ROWS / 32;
  constexpr int NH = ROWS / 16;      // hidden loads a wave and slot (1 KiB each: two rows)
  constexpr int kLoads = 4 + NH;  // a slot's direct loads, beside those of its scales
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / 4, wn = wave % 4, li = lane % 16, g = lane / 16;
  const int nslots = (ksteps + kSlotSteps - 1) / kSlotSteps;
  const int last = ksteps - (nslots - 1) * kSlotSteps;  // steps of the last slot

  // Rows past the data read the last one, pieces past K the last one of the
  // row: every load stays in bounds, and what it brings is masked or not read.
  const uint8_t* wp[4];
  int wc[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = (wave + 8 * u) * 8 + lane / 8;
    wp[u] = data + min(v0 + r, v - 1) * ld_d;
    wc[u] = (lane % 8) ^ weight_swz(r);
  }
  const uint16_t* hp[NH];
  int hc[NH];
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    const int r = (wave + 8 * u) * 2 + lane / 32;
    hp[u] = hidden + min(m0 + r, n - 1) * ld_h;
    hc[u] = (lane % 32) ^ hidden_swz(r);
  }
  // Scales: thread t takes four of column t / 2, two at a time (K is a multiple
  // of 64), past the end the last two.
  const uint8_t* sp = scales + min(v0 + tid / 2, v - 1) * ld_s;
  auto load_scales = [&](int p, uint16_t (&x)[2]) {
    const int at = p * kSlotSteps + 4 * (tid % 2);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x[i] = reinterpret_cast<const ScalePair*>(sp + min(at + 2 * i, ksteps - 2))->w;
  };
  auto issue = [&](int slot, int q, uint16_t (&sc)[2]) {
    const int p = q < nslots ? q : nslots - 1;
    const int most = p == nslots - 1 ? last : kSlotSteps;
    load_scales(p, sc);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      __builtin_amdgcn_global_load_lds(
          wp[u] + static_cast<int64_t>(p) * kSlotBytes + min(wc[u], most - 1) * 16,
          sm.w[slot] + (wave + 8 * u) * 1024, 16, 0, 0);
#pragma unroll
    for (int u = 0; u < NH; ++u)
      __builtin_amdgcn_global_load_lds(
          hp[u] + static_cast<int64_t>(p) * kSlotK + min(hc[u], 4 * most - 1) * 8,
          sm.h[slot] + (wave + 8 * u) * 512, 16, 0, 0);
  };

  const int sw = weight_swz(li);  // the same for rows 16 apart
  auto steps = [&](int slot, int count) {
    uint2 sc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sc[j] = *reinterpret_cast<const uint2*>(&sm.scale[slot][(wn * 64 + 16 * j + li) * 4]);
#pragma unroll
    for (int s = 0; s < kSlotSteps; ++s) {
      if (s % 2 == 0 && s >= count) break;  // uniform; K is a multiple of 64
      bf16x8 a[MI], b[4];
#pragma unroll
      for (int i = 0; i < MI; ++i)
        a[i] = *reinterpret_cast<const bf16x8*>(
            sm.h[slot] + (wm * (ROWS / 2) + 16 * i + li) * kSlotK + ((4 * s + g) ^ li) * 8);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t q = *reinterpret_cast<const uint32_t*>(
            sm.w[slot] + (wn * 64 + 16 * j + li) * kSlotBytes + (s ^ sw) * 16 + g * 4);
        const uint32_t e = s < 4 ? sc[j].x >> (8 * s) : sc[j].y >> (8 * (s - 4));
        b[j] = decode8(q, __uint_as_float((e & 255u) << 23));
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[j], acc[i][j], 0, 0, 0);
    }
  };

  uint16_t sc[S - 1][2];
#pragma unroll
  for (int p = 0; p < S - 1; ++p) issue(p, p, sc[p]);
  // Slot p's loads have landed once only those of the S - 2 slots issued after
  // it are in flight; after the barrier that holds for every wave, the scales
  // are in LDS, and nobody reads slot p - 1 any more, whose place the loads for
  // slot p + S - 1 take.
  for (int p0 = 0; p0 < nslots; p0 += S - 1) {
#pragma unroll
    for (int u = 0; u < S - 1; ++u) {
      const int p = p0 + u;  // past the end: nothing is added
      wait_vm_lgkm0<(S - 2) * kLoads>();
      sm.scale[p % S][2 * tid] = sc[u][0];
      sm.scale[p % S][2 * tid + 1] = sc[u][1];
      wait_vm_lgkm0<(S - 2) * kLoads>();
      __builtin_amdgcn_s_barrier();
      issue((p + S - 1) % S, p + S - 1, sc[u]);
      steps(p % S, p < nslots - 1 ? kSlotSteps : p == nslots - 1 ? last : 0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int ROWS>
__global__ __launch_bounds__(kThreads4) void linear_fp4_narrow(
    const uint16_t* __restrict__ hidden, int64_t ld_h, const uint8_t* __restrict__ data,
    int64_t ld_d, const uint8_t* __restrict__ scales, int64_t ld_s, int64_t n, int64_t v,
    int ksteps, int mblocks, int vblocks, const void* __restrict__ tgt, int32_t tgt32,
    int64_t ignore, float* __restrict__ pm, float* __restrict__ ps, float* __restrict__ pt,
    LinearExtras ex) {
  constexpr int MI = ROWS / 32;
  const Targets targets{tgt, tgt32};
  __shared__ __align__(16) SmemFp4<ROWS> sm;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int logical = gemm::xcd_logical(blockIdx.x, mblocks * vblocks);
  const int mb = logical % mblocks, vb = logical / mblocks;
  const int64_t m0 = static_cast<int64_t>(mb) * ROWS, v0 = static_cast<int64_t>(vb) * BN;
  if (tid < ROWS) sm.rd.code[tid] = row_code(m0 + tid, n, targets, ignore, v0, v);
  f32x4 acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  mainloop_fp4<ROWS>(sm.st, hidden, ld_h, m0, n, data, ld_d, scales, ld_s, v0, v, ksteps, acc);
  __syncthreads();
  stats_epilogue<MI, 4, ROWS, kThreads4, sizeof(sm.st)>(
      acc, sm.rd, &sm.st, (wave / 4) * (ROWS / 2), (wave % 4) * 64, lane % 16, lane / 16, tid, m0,
      v0, vb, vblocks, n, v, pm, ps, pt, ex);
}

// The decoded copy: a wave takes 16 rows x 4 K steps, a lane one row's step (16
// bytes of codes, 64 bytes of values: whole blocks of 1 KiB).
__global__ __launch_bounds__(256) void fp4_decode_kernel(const uint8_t* __restrict__ data,
                                                         int64_t ld_d,
                                                         const uint8_t* __restrict__ scales,
                                                         int64_t ld_s, int64_t v, int64_t ksteps,
                                                         uint16_t* __restrict__ out) {
  const int lane = threadIdx.x % kWave;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 16 + lane % 16;
  for (int64_t k = (static_cast<int64_t>(blockIdx.y) * 4 + threadIdx.x / kWave) * 4 + lane / 16;
       k < ksteps; k += static_cast<int64_t>(gridDim.y) * 16) {
    uint4 q = make_uint4(0, 0, 0, 0);
    float scale = 1.0f;
    if (row < v) {
      q = *reinterpret_cast<const uint4*>(data + row * ld_d + k * 16);
      scale = __uint_as_float(static_cast<uint32_t>(scales[row * ld_s + k]) << 23);
    }
    bf16x8* to = reinterpret_cast<bf16x8*>(
        out + (static_cast<int64_t>(blockIdx.x) * ksteps + k) * 512 + (lane % 16) * 32);
    to[0] = decode8(q.x, scale);
    to[1] = decode8(q.y, scale);
    to[2] = decode8(q.z, scale);
    to[3] = decode8(q.w, scale);
  }
}

}  // namespace

int64_t fp4_decoded_bytes(int64_t v, int64_t h) { return (v + 255) / 256 * 256 * h * 2; }

void launch_fp4_decode(const Fp4Weight& w, int64_t v, int64_t h, uint16_t* out, hipStream_t s) {
  const int64_t ksteps = h / BK, blocks = (v + 255) / 256 * 16, ky = (ksteps + 15) / 16;
  hipLaunchKernelGGL(fp4_decode_kernel,
                     dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(ky < 64 ? ky : 64)),
                     dim3(256), 0, s, w.data, w.ld_d, w.scales, w.ld_s, v, ksteps, out);
}

void launch_fp4_partials(const uint16_t* hidden, int64_t ld_h, const Fp4Weight& w, int64_t n,
                         int64_t h, int64_t v, Targets targets, int64_t ignore, float* pm,
                         float* ps, float* pt, float inv_t, int32_t round_bf16, float* pw, void* z,
                         int32_t z_bf16, int64_t ld_z, hipStream_t s) {
  const int vblocks = static_cast<int>((v + BN - 1) / BN);
  const int rows = n <= 32 ? 32 : 64;
  const int mblocks = static_cast<int>((n + rows - 1) / rows);
  const int32_t z_vec = z && reinterpret_cast<uintptr_t>(z) % 16 == 0 &&
                        (ld_z * (z_bf16 ? 2 : 4)) % 16 == 0;
  const LinearExtras ex{inv_t, round_bf16, pw, z, z_bf16, ld_z, z_vec};
  auto kern = rows == 32 ? linear_fp4_narrow<32> : linear_fp4_narrow<64>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(mblocks * vblocks)), dim3(kThreads4), 0, s,
                     hidden, ld_h, w.data, w.ld_d, w.scales, w.ld_s, n, v,
                     static_cast<int>(h / BK), mblocks, vblocks, targets.p, targets.is32, ignore,
                     pm, ps, pt, ex);
}

}  // namespace itl
