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
// Few rows (linear_fp4_narrow): bound by the weight's bytes, 17 / 32 of a byte a
// value.  A workgroup takes tiles of 256 columns x ROWS hidden rows, eight waves
// of 32 columns x ROWS rows, so that every weight is decoded once.  Slots of 256
// K values hold whole 128-byte lines of the weight's rows and the hidden rows'
// pieces, panels of two slots the scales (16 bytes a row: taken slot by slot
// their requests were as many as the weight's, 16 us of 92), all brought by
// direct loads.  The slots of a workgroup's tiles follow one another, so that the
// next tile's first ones are on their way during a tile's epilogue.
// V = 151936, H = 4096 (330 MB, 51 us at 6.45 TB/s): 76 us at 16 rows, 95 at 32,
// 133 at 64; without the products and decoding 65, 71 and 93 (594 tiles on 256
// CUs, the last 82 nearly alone), without the loads 52, 62 and 86.  Two to four
// slots, whole or half lines, four waves a workgroup and three workgroups a CU
// (81, 96, 153) made no difference or a worse one.
//
// Many rows (linear_fp4_wide): bound by the matrix cores.  Blocks of 256 (128)
// hidden rows x 256 columns like those of the bf16 head, the weight's codes in LDS in
// place of its values (a quarter of the bytes to bring and to read) and decoded
// beside the products of the step, 20 vector instructions to 32 products.  A wave
// holds a step's hidden rows in two halves, one read while the other's products
// run: whole steps ahead, as the bf16 head holds them, do not fit its registers
// beside the decoding.  1000 rows: 850 to 890 us (1.4 to 1.46 PFLOP/s), what the
// bf16 head takes on a decoded copy of the weight, whose making took 256 more.
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
constexpr int kSlots = ROWS == 64 ? 2 : 3;
constexpr int kPanels = 3;  // those of slots p .. p + 2, each of which may begin one
// Rows of the epilogue, whose waves take 64 columns x half of them.
template <int ROWS>
constexpr int kEpiRows = ROWS < 32 ? 32 : ROWS;

template <int ROWS>
struct Fp4Slot {
  uint8_t w[BN * kSlotBytes];
  uint16_t h[ROWS * kSlotK];
};

template <int ROWS>
struct SmemFp4 {
  Fp4Slot<ROWS> slot[kSlots<ROWS>];
  uint8_t scale[kPanels][BN * 2 * kSlotSteps];
  Reduce<kEpiRows<ROWS>> rd;
  int64_t target[ROWS];
};

// Two scale bytes at any address.
struct __attribute__((packed)) ScalePair {
  uint16_t w;
};

// Eight weights (a dword of codes) under the scale 2^(b - 127) given as an fp32
// with exponent bits b, whatever its other bits.
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

// Where a workgroup's loads are: the next slot to issue, in its tiles.  An
// address is a scalar base and a lane's 32-bit offset from it, which changes
// with the tile alone (strides: kMaxFp4Stride and kMaxHiddenStride).
template <int ROWS, bool ALIGNED>
struct Fp4Loader {
  static constexpr int NH = ROWS / 16;  // hidden loads a wave and slot (1 KiB each: two rows)
  // A wave's direct loads of a slot, and those of a slot that begins a panel.
  static constexpr int kOdd = 4 + NH, kEven = kOdd + (ALIGNED ? 2 : 0);
  int64_t ld_h, n, ld_d, ld_s, v;
  int ksteps, nslots, last;  // last: steps of a tile's last slot
  int tile, step, end;
  int p, ring, panel;  // the next slot: of its tile, its place, its panel's
  int64_t w0, s0;      // where the tile's rows begin
  uint32_t wofs[4], hofs[NH], sofs[2];

  // Rows past the data read the last one: every load stays in bounds, and what
  // it brings is masked or not read.
  __device__ __forceinline__ void rows(int tid, int wave, int lane) {
    const int64_t v0 = static_cast<int64_t>(tile) * BN;
    const int vmax = static_cast<int>(min(v - 1 - v0, int64_t{BN - 1}));
    const int hmax = static_cast<int>(n) - 1;
    w0 = v0 * ld_d;
    s0 = v0 * ld_s;
    const uint32_t lw = static_cast<uint32_t>(ld_d), lh = static_cast<uint32_t>(ld_h) * 2;
    const uint32_t ls = static_cast<uint32_t>(ld_s);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (wave + 8 * u) * 8 + lane / 8;
      wofs[u] = min(r, vmax) * lw + ((lane % 8) ^ weight_swz(r)) * 16;
    }
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      const int r = (wave + 8 * u) * 2 + lane / 32;
      hofs[u] = min(r, hmax) * lh + ((lane % 32) ^ hidden_swz(r)) * 16;
    }
    if constexpr (ALIGNED) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        sofs[u] = min((wave + 8 * u) * 16 + lane / 4, vmax) * ls + 4 * (lane % 4);
    } else {
      sofs[0] = min(tid / 2, vmax) * ls;
    }
  }

  // Issues the next slot's loads; past the last tile the last slot's again, so
  // that every slot has its loads in flight behind it.  Pieces past K are the
  // row's last.  sc: scale bytes that pass through registers, four of column
  // tid / 2, two and two.
  __device__ __forceinline__ void issue(SmemFp4<ROWS>& sm, const uint16_t* hidden,
                                        const uint8_t* data, const uint8_t* scales, int tid,
                                        int wave, int lane, uint16_t (&sc)[2]) {
    if (p % 2 == 0) panel = panel == kPanels - 1 ? 0 : panel + 1;
    const uint8_t* sb = scales + s0 + p * kSlotSteps;
    if constexpr (ALIGNED) {
      if (p % 2 == 0) {
        const int past = max(p * kSlotSteps + 4 * (lane % 4) - (ksteps - 4), 0);
#pragma unroll
        for (int u = 0; u < 2; ++u)
          __builtin_amdgcn_global_load_lds(sb + (sofs[u] - past),
                                           sm.scale[panel] + (wave + 8 * u) * 256, 4, 0, 0);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sc[i] = reinterpret_cast<const ScalePair*>(
                    scales + (s0 + sofs[0] +
                              min(p * kSlotSteps + 4 * (tid % 2) + 2 * i, ksteps - 2)))
                    ->w;
    }
    Fp4Slot<ROWS>& to = sm.slot[ring];
    const uint8_t* wb = data + w0 + static_cast<int64_t>(p) * kSlotBytes;
    const uint8_t* hb =
        reinterpret_cast<const uint8_t*>(hidden + static_cast<int64_t>(p) * kSlotK);
    const bool whole = p < nslots - 1 || last == kSlotSteps;
    if (whole) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        __builtin_amdgcn_global_load_lds(wb + wofs[u], to.w + (wave + 8 * u) * 1024, 16, 0, 0);
#pragma unroll
      for (int u = 0; u < NH; ++u)
        __builtin_amdgcn_global_load_lds(hb + hofs[u], to.h + (wave + 8 * u) * 512, 16, 0, 0);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = (lane % 8) ^ weight_swz((wave + 8 * u) * 8 + lane / 8);
        __builtin_amdgcn_global_load_lds(wb + (wofs[u] - max(c - last + 1, 0) * 16),
                                         to.w + (wave + 8 * u) * 1024, 16, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        const int c = (lane % 32) ^ hidden_swz((wave + 8 * u) * 2 + lane / 32);
        __builtin_amdgcn_global_load_lds(hb + (hofs[u] - max(c - 4 * last + 1, 0) * 16),
                                         to.h + (wave + 8 * u) * 512, 16, 0, 0);
      }
    }
    ring = ring == kSlots<ROWS> - 1 ? 0 : ring + 1;
    if (p < nslots - 1) {
      ++p;
    } else if (tile + step < end) {
      tile += step;
      p = 0;
      rows(tid, wave, lane);
    }
  }
};

// The first `count` of a slot's eight steps: acc += hidden rows x the wave's 32
// columns.  Steps are read from LDS NR at a time, one such part ahead of the
// decoding and the products.
template <int ROWS, bool WHOLE>
__device__ __forceinline__ void slot_steps(const Fp4Slot<ROWS>& slot, const uint8_t* scale,
                                           int count, int wave, int li, int g,
                                           f32x4 (&acc)[ROWS / 16][2]) {
  constexpr int MI = ROWS / 16, NR = MI == 4 ? 1 : 2, NP = kSlotSteps / NR;
  const int col = wave * 32 + li;
  const int sw = weight_swz(li);  // the same for rows 16 apart
  uint2 sc[2];
#pragma unroll
  for (int j = 0; j < 2; ++j)
    sc[j] = *reinterpret_cast<const uint2*>(scale + (col + 16 * j) * 2 * kSlotSteps);
  uint32_t q[2][NR][2];
  bf16x8 a[2][NR][MI];
  auto read = [&](int part) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int s = part * NR + r;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        q[part % 2][r][j] = *reinterpret_cast<const uint32_t*>(
            slot.w + (col + 16 * j) * kSlotBytes + (s ^ sw) * 16 + g * 4);
#pragma unroll
      for (int i = 0; i < MI; ++i)
        a[part % 2][r][i] = *reinterpret_cast<const bf16x8*>(
            slot.h + (16 * i + li) * kSlotK + ((4 * s + g) ^ li) * 8);
    }
  };
  read(0);
#pragma unroll
  for (int part = 0; part < NP; ++part) {
    if (part + 1 < NP) read(part + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int s = part * NR + r;
      if (!WHOLE && s % 2 == 0 && s >= count) return;  // uniform; K is a multiple of 64
      bf16x8 b[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        // the scale byte to the exponent's place: the conversion takes no other bit
        const uint32_t x = s < 4 ? sc[j].x : sc[j].y;
        const uint32_t e = s % 4 == 3 ? x >> 1 : x << (23 - 8 * (s % 4));
        b[j] = decode8(q[part % 2][r][j], __uint_as_float(e));
      }
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[part % 2][r][i], b[j], acc[i][j],
                                                              0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// From 32 columns x ROWS rows a wave to the epilogue's 64 x EPI / 2 through z, a
// slot's place; columns are turned by 16 every 4 rows, which puts a wave's
// stores on different banks.
template <int ROWS, int MI>
__device__ __forceinline__ void regroup(const f32x4 (&part)[ROWS / 16][2], float* z, int wave,
                                        int row0, int col0, int li, int g, f32x4 (&acc)[MI][4]) {
  static_assert(ROWS * BN * 4 <= sizeof(Fp4Slot<ROWS>), "z in a slot");
  auto at = [&](int row, int col) { return row * BN + (col ^ ((row >> 2 & 3) << 4)); };
  block_sync_lds();
#pragma unroll
  for (int i = 0; i < ROWS / 16; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        z[at(16 * i + 4 * g + q, wave * 32 + 16 * j + li)] = part[i][j][q];
  block_sync_lds();
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        acc[i][j][q] = row0 + 16 * i < ROWS  // the others are past n
                           ? z[at(row0 + 16 * i + 4 * g + q, col0 + 16 * j + li)]
                           : 0.0f;
  block_sync_lds();
}

// A workgroup's tiles.  (A function of its own for its __restrict__ operands:
// inlined, they tell the compiler that the direct loads read nothing that LDS
// holds; otherwise it waits for all of them before every read of LDS.)
template <int ROWS, bool ALIGNED>
__device__ __forceinline__ void fp4_tiles(
    SmemFp4<ROWS>& sm, const uint16_t* __restrict__ hidden, int64_t ld_h,
    const uint8_t* __restrict__ data, int64_t ld_d, const uint8_t* __restrict__ scales,
    int64_t ld_s, int64_t n, int64_t v, int ksteps, int vblocks, Targets targets, int64_t ignore,
    float* __restrict__ pm, float* __restrict__ ps, float* __restrict__ pt,
    float inv_t, int32_t round_bf16, float* pw, void* z, int32_t z_bf16, int64_t ld_z,
    int32_t z_vec) {
  const LinearExtras ex{inv_t, round_bf16, pw, z, z_bf16, ld_z, z_vec};
  constexpr int S = kSlots<ROWS>, EPI = kEpiRows<ROWS>, MI = EPI / 32;
  using Loader = Fp4Loader<ROWS, ALIGNED>;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int li = lane % 16, g = lane / 16;
  // Workgroup b takes tiles of XCD b % 8's range.
  int first, end;
  gemm::xcd_range(vblocks, blockIdx.x % 8, first, end);
  const int step = gridDim.x / 8;
  const int begin = first + blockIdx.x / 8;
  if (begin >= end) return;
  if (tid < n) sm.target[tid] = targets[tid];

  Loader load;
  load.ld_h = ld_h;
  load.n = n;
  load.ld_d = ld_d;
  load.ld_s = ld_s;
  load.v = v;
  load.ksteps = ksteps;
  load.nslots = (ksteps + kSlotSteps - 1) / kSlotSteps;
  load.last = ksteps - (load.nslots - 1) * kSlotSteps;
  load.tile = begin;
  load.step = step;
  load.end = end;
  load.p = load.ring = 0;
  load.panel = kPanels - 1;
  load.rows(tid, wave, lane);
  // Scales that pass through registers go to their panel once their loads are
  // back, in the iteration that issued them.
  auto issue = [&](auto between) {
    uint16_t sc[2];
    const int p = load.p;
    load.issue(sm, hidden, data, scales, tid, wave, lane, sc);
    uint8_t* to = sm.scale[load.panel] + (tid / 2) * 2 * kSlotSteps + (p % 2) * kSlotSteps +
                  4 * (tid % 2);
    between();
    if constexpr (!ALIGNED)
      *reinterpret_cast<uint32_t*>(to) = sc[0] | static_cast<uint32_t>(sc[1]) << 16;
  };
  for (int i = 0; i < S - 1; ++i) issue([] {});

  int ring = 0, panel = kPanels - 1;
  for (int tile = begin; tile < end; tile += step) {
    const int64_t v0 = static_cast<int64_t>(tile) * BN;
    f32x4 part[ROWS / 16][2];
#pragma unroll
    for (int i = 0; i < ROWS / 16; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) part[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < load.nslots; ++p) {
      // This slot's loads have landed once only those of the S - 2 slots issued
      // after it are in flight; after the barrier that holds for every wave, and
      // nobody reads the slot before it any more, whose place the next loads
      // take.  (Past the tile's end the next slot may be the last one again: no
      // more than kOdd can be counted on.)
      if constexpr (S == 2) {
        wait_vm_lgkm0<0>();
      } else {
        if (p % 2 == 1 && p + 1 < load.nslots) wait_vm_lgkm0<Loader::kEven>();
        else wait_vm_lgkm0<Loader::kOdd>();
      }
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (p % 2 == 0) panel = panel == kPanels - 1 ? 0 : panel + 1;
      const Fp4Slot<ROWS>& slot = sm.slot[ring];
      const uint8_t* scale = sm.scale[panel] + (p % 2) * kSlotSteps;
      issue([&] {
        if (p < load.nslots - 1 || load.last == kSlotSteps) {
          slot_steps<ROWS, true>(slot, scale, kSlotSteps, wave, li, g, part);
        } else {
          slot_steps<ROWS, false>(slot, scale, load.last, wave, li, g, part);
        }
      });
      if (p < load.nslots - 1) ring = ring == S - 1 ? 0 : ring + 1;
    }
    // The last slot's place is free until the next tile's first slot is waited
    // for: the epilogue's.
    if (tid < EPI) {
      int code = -2;
      if (tid < n) {
        const int64_t t = sm.target[tid];
        if (t != ignore) code = t >= v0 && t < v0 + BN && t < v ? static_cast<int>(t - v0) : -1;
      }
      sm.rd.code[tid] = code;
    }
    const int row0 = (wave / 4) * (EPI / 2), col0 = (wave % 4) * 64;
    f32x4 acc[MI][4];
    regroup<ROWS, MI>(part, reinterpret_cast<float*>(&sm.slot[ring]), wave, row0, col0, li, g, acc);
    stats_epilogue<MI, 4, EPI, kThreads4, sizeof(Fp4Slot<ROWS>)>(
        acc, sm.rd, &sm.slot[ring], row0, col0, li, g, tid, 0, v0, tile, vblocks, n, v, pm, ps,
        pt, ex);
    ring = ring == S - 1 ? 0 : ring + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int ROWS, bool ALIGNED>
__global__ __launch_bounds__(kThreads4) void linear_fp4_narrow(
    const uint16_t* __restrict__ hidden, int64_t ld_h, const uint8_t* __restrict__ data,
    int64_t ld_d, const uint8_t* __restrict__ scales, int64_t ld_s, int64_t n, int64_t v,
    int ksteps, int vblocks, const void* __restrict__ tgt, int32_t tgt32,
    int64_t ignore, float* __restrict__ pm, float* __restrict__ ps, float* __restrict__ pt,
    LinearExtras ex) {
  __shared__ __align__(16) SmemFp4<ROWS> sm;
  fp4_tiles<ROWS, ALIGNED>(sm, hidden, ld_h, data, ld_d, scales, ld_s, n, v, ksteps, vblocks,
                           Targets{tgt, tgt32}, ignore, pm, ps, pt, ex.inv_t,
                           ex.round_bf16, ex.pw, ex.z, ex.z_bf16, ex.ld_z, ex.z_vec);
}

// ---------------------------------------------------------------------------
// Many rows: blocks of ROWS hidden rows x 256 columns, eight waves of ROWS / 2 x 64.
// 256 rows: the hidden rows K32-blocked, tiles from the queue of mfma_gemm.h;
// 128: one block of rows as they are.
// ---------------------------------------------------------------------------
constexpr int kWideSteps = 4;                       // K steps a slot
constexpr int kWideBytes = kWideSteps * BK / 2;     // of a weight row: 64
constexpr int kWideSlots = 3;

template <int ROWS>
struct SmemFp4Wide {
  uint16_t a[kWideSteps][ROWS * BK];        // a K step's hidden rows each
  uint8_t w[kWideSlots][BN * kWideBytes];
  uint32_t scale[kWideSlots][BN];
  Reduce<ROWS> rd;
  int slot;  // tile-queue broadcast
};

// The main loop of one role.  LOADER, waves 0 to 3: all direct loads, in step
// kt those of the hidden rows of step kt + 4 (NA a wave) and a quarter of the
// weight slot after next; waves 4 to 7 the scales of that slot, a thread a column,
// through registers.  (Of the loads in flight before step kt, those of the hidden
// rows of step kt + 1 were issued in step kt - 3 and the last of a slot that
// begins with step kt + 1 in step kt - 4: those of kt - 1 and kt - 2 may be left.)
// Weight piece s of row r lies at s ^ (r / 4) % 4 of its 64 bytes, which puts the 64
// reads of a wave on different banks.
template <int ROWS, bool LOADER>
__device__ __forceinline__ void fp4_wide_loop(SmemFp4Wide<ROWS>& sm,
                                              const uint16_t* __restrict__ hidden, int64_t ld_h,
                                              int64_t m0, int64_t rows,
                                              const uint8_t* __restrict__ data, int64_t ld_d,
                                              const uint8_t* __restrict__ scales, int64_t ld_s,
                                              int64_t v0, int64_t v, int ksteps,
                                              f32x4 (&acc)[ROWS / 32][4]) {
  constexpr bool kBlocked = ROWS == 256;
  constexpr int MH = ROWS / 64, NA = ROWS / 64;  // of a half; hidden loads a wave and step
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wm = wave / 4, wn = wave % 4, li = lane % 16, g = lane / 16;
  const int nslots = (ksteps + kWideSteps - 1) / kWideSteps;
  const int last = ksteps - (nslots - 1) * kWideSteps;  // 2 or 4: K is a multiple of 64
  const int vmax = static_cast<int>(min(v - 1 - v0, int64_t{BN - 1}));
  const uint16_t* ha[NA];
  uint32_t wofs[4];
  uint32_t back = 0;  // of a piece past the last slot's end
  const uint8_t* wb = data + v0 * ld_d;
  const uint8_t* sb = scales;
  if constexpr (LOADER) {
    const int lrow = lane / 4, c = (lane % 4) ^ (lrow >> 2 & 3);
#pragma unroll
    for (int u = 0; u < NA; ++u)
      ha[u] = gemm::lane_chunk<kBlocked>(hidden, ld_h, m0, rows, wave + 4 * u, lrow,
                                         ((lane % 4) ^ gemm::swz(lrow)) * 8);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      wofs[j] = min((wave + 4 * j) * 16 + lrow, vmax) * static_cast<uint32_t>(ld_d) + c * 16;
    back = max(c - last + 1, 0) * 16;
  } else {
    sb = scales + (v0 + min(tid - 256, vmax)) * ld_s;
  }
  auto issue_a = [&](int stage, int step) {
    if constexpr (LOADER) {
      const int64_t k = static_cast<int64_t>(min(step, ksteps - 1)) * (kBlocked ? 512 : BK);
#pragma unroll
      for (int u = 0; u < NA; ++u)
        __builtin_amdgcn_global_load_lds(ha[u] + k, sm.a[stage] + (wave + 4 * u) * 512, 16, 0, 0);
    }
  };
  auto issue_w = [&](int place, int slot, int j) {
    if constexpr (LOADER) {
      const int p = min(slot, nslots - 1);
      __builtin_amdgcn_global_load_lds(
          wb + static_cast<int64_t>(p) * kWideBytes + (wofs[j] - (p == nslots - 1 ? back : 0)),
          sm.w[place] + (wave + 4 * j) * 1024, 16, 0, 0);
    }
  };
  uint16_t sc[2];
  auto load_scale = [&](int slot) {
    if constexpr (!LOADER) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        sc[i] = reinterpret_cast<const ScalePair*>(
                    sb + min(slot * kWideSteps + 2 * i, ksteps - 2))
                    ->w;
    }
  };
  auto store_scale = [&](int place) {
    if constexpr (!LOADER)
      sm.scale[place][tid - 256] = sc[0] | static_cast<uint32_t>(sc[1]) << 16;
  };
  const int aoff = (wm * (ROWS / 2) + li) * BK + ((g ^ gemm::swz(li)) * 8);
  const int col = wn * 64 + li, sw = li >> 2 & 3;
  bf16x8 a[2][MH], b[4];  // a step's hidden rows in two halves; its weights
  uint32_t q[4], e[4];   // their codes, the slot's scales
  auto read_a = [&](int stage, int half) {
#pragma unroll
    for (int i = 0; i < MH; ++i)
      a[half][i] =
          *reinterpret_cast<const bf16x8*>(sm.a[stage] + aoff + (MH * half + i) * 16 * BK);
  };
  auto read_q = [&](int stage, int place) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] = *reinterpret_cast<const uint32_t*>(sm.w[place] + (col + 16 * j) * kWideBytes +
                                                ((stage ^ sw) * 16) + g * 4);
  };
  auto read_e = [&](int place) {
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = sm.scale[place][col + 16 * j];
  };
  // Steps -4 to -1.
#pragma unroll
  for (int j = 0; j < 4; ++j) issue_w(0, 0, j);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    issue_a(j, j);
    issue_w(1, 1, j);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    load_scale(i);
    store_scale(i);
  }
  wait_vm_lgkm0<LOADER ? 3 * (NA + 1) + 1 : 0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  read_a(0, 0);
  read_q(0, 0);
  read_e(0);
  int p0 = 0, p1 = 1, p2 = 2;  // places of this slot and the next two
  // A step: the products of one half of its hidden rows while the other half is
  // read; then, everything of it being read and step kt + 1 there, the barrier,
  // and those of the other half while the next step's first half is read.
  for (int p = 0; p < nslots; ++p) {
#pragma unroll
    for (int t = 0; t < kWideSteps; ++t) {
      read_a(t, 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        b[j] = decode8(q[j], __uint_as_float(t == 3 ? e[j] >> 1 : e[j] << (23 - 8 * (t % 3))));
#pragma unroll
        for (int i = 0; i < MH; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[0][i], b[j], acc[i][j], 0, 0, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, MH, 0);
#pragma unroll
      for (int o = 0; o < 2 * MH; ++o) {
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 8 / MH, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      wait_vm_lgkm0<LOADER ? 2 * (NA + 1) : 63>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      issue_a(t, 4 * p + t + 4);
      issue_w(p2, p + 2, t);
      if (t == 0) load_scale(p + 2);
      if (t == 3) store_scale(p2);
      read_a((t + 1) % 4, 0);
      read_q((t + 1) % 4, t == 3 ? p1 : p0);
      if (t == 3) read_e(p1);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < MH; ++i)
          acc[MH + i][j] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[1][i], b[j], acc[MH + i][j], 0, 0, 0);
      if constexpr (LOADER) __builtin_amdgcn_sched_group_barrier(0x020, NA + 1, 0);
#pragma unroll
      for (int o = 0; o < 2 * MH + 4; ++o) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x008, 2 * MH - 4, 0);
      __builtin_amdgcn_sched_barrier(0);
      if (t == 1 && p == nslots - 1 && last == 2) break;
    }
    const int x = p0;
    p0 = p1;
    p1 = p2;
    p2 = x;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <int ROWS>
__global__ __launch_bounds__(kThreads4) void linear_fp4_wide(
    const uint16_t* __restrict__ hidden, int64_t ld_h, const uint8_t* __restrict__ data,
    int64_t ld_d, const uint8_t* __restrict__ scales, int64_t ld_s, int64_t n, int64_t v,
    int ksteps, int mblocks, int vblocks, const void* __restrict__ tgt, int32_t tgt32,
    int64_t ignore, float* __restrict__ pm, float* __restrict__ ps, float* __restrict__ pt,
    LinearExtras ex, int* queue, int queued) {
  __shared__ __align__(16) SmemFp4Wide<ROWS> sm;
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int logical = ROWS == 256 ? gemm::queue_tile(queue, mblocks * vblocks, queued, &sm.slot)
                                  : gemm::xcd_logical(blockIdx.x, mblocks * vblocks);
  if (logical < 0) return;
  int mb, vb;
  gemm::tile_coords(logical, mblocks, vblocks, mb, vb);
  const int64_t m0 = static_cast<int64_t>(mb) * ROWS, v0 = static_cast<int64_t>(vb) * BN;
  if (tid < ROWS) sm.rd.code[tid] = row_code(m0 + tid, n, Targets{tgt, tgt32}, ignore, v0, v);
  constexpr int MI = ROWS / 32;
  f32x4 acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t rows = ROWS == 256 ? static_cast<int64_t>(mblocks) * 256 : n;
  if (gemm::loader_wave())
    fp4_wide_loop<ROWS, true>(sm, hidden, ld_h, m0, rows, data, ld_d, scales, ld_s, v0, v, ksteps,
                              acc);
  else
    fp4_wide_loop<ROWS, false>(sm, hidden, ld_h, m0, rows, data, ld_d, scales, ld_s, v0, v, ksteps,
                               acc);
  __syncthreads();
  stats_epilogue<MI, 4, ROWS, kThreads4, sizeof(sm.a) + sizeof(sm.w)>(
      acc, sm.rd, &sm.a, (wave / 4) * (ROWS / 2), (wave % 4) * 64, lane % 16, lane / 16, tid, m0,
      v0, vb, vblocks, n, v, pm, ps, pt, ex);
}

}  // namespace

void launch_fp4_partials(const uint16_t* hidden, int64_t ld_h, const Fp4Weight& w, int64_t n,
                         int64_t h, int64_t v, Targets targets, int64_t ignore, float* pm,
                         float* ps, float* pt, float inv_t, int32_t round_bf16, float* pw, void* z,
                         int32_t z_bf16, int64_t ld_z, uint16_t* hb, hipStream_t s) {
  const int vblocks = static_cast<int>((v + BN - 1) / BN);
  // The weight streams for up to 64 rows; then its decoding, which a block of 128
  // rows does no more often, takes longer than the stream (V = 151936, H = 4096:
  // 64 rows 144 us against 166 in such a block, 128 rows 224 in two streams against
  // 177; 129 to 256 rows 256 to 277 in a block of 256).
  const int rows = n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
  const int mblocks = static_cast<int>((n + rows - 1) / rows);
  const int32_t z_vec = z && reinterpret_cast<uintptr_t>(z) % 16 == 0 &&
                        (ld_z * (z_bf16 ? 2 : 4)) % 16 == 0;
  const LinearExtras ex{inv_t, round_bf16, pw, z, z_bf16, ld_z, z_vec};
  if (rows == 128) {
    hipLaunchKernelGGL(linear_fp4_wide<128>, dim3(static_cast<unsigned>(mblocks * vblocks)),
                       dim3(kThreads4), 0, s, hidden, ld_h, w.data, w.ld_d, w.scales, w.ld_s, n, v,
                       static_cast<int>(h / BK), mblocks, vblocks, targets.p, targets.is32, ignore,
                       pm, ps, pt, ex, static_cast<int*>(nullptr), 0);
    return;
  }
  if (rows == 256) {
    const int64_t np = static_cast<int64_t>(mblocks) * 256;
    int* queue = reinterpret_cast<int*>(hb + np * h);  // cleared by launch_block_rows
    launch_block_rows(hidden, ld_h, n, np, h, hb, s, queue, gemm::kQueueBytes / 4);
    const gemm::QueuePlan qp = gemm::queue_plan(mblocks * vblocks, xcd_cus());
    hipLaunchKernelGGL(linear_fp4_wide<256>, dim3(static_cast<unsigned>(qp.grid)), dim3(kThreads4),
                       0, s, hb, h * 16, w.data, w.ld_d, w.scales, w.ld_s, n, v,
                       static_cast<int>(h / BK), mblocks, vblocks, targets.p, targets.is32, ignore,
                       pm, ps, pt, ex, queue, qp.queued);
    return;
  }
  // a workgroup a CU, as many on every XCD
  const int per = (vblocks + 7) / 8, cus = xcd_cus();
  const int grid = 8 * (per < cus ? per : cus);
  const bool aligned = h % 128 == 0 && w.ld_s % 4 == 0 &&
                       reinterpret_cast<uintptr_t>(w.scales) % 4 == 0;
  auto kern = rows == 16   ? (aligned ? linear_fp4_narrow<16, true> : linear_fp4_narrow<16, false>)
              : rows == 32 ? (aligned ? linear_fp4_narrow<32, true> : linear_fp4_narrow<32, false>)
                           : (aligned ? linear_fp4_narrow<64, true> : linear_fp4_narrow<64, false>);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(grid)), dim3(kThreads4), 0, s,
                     hidden, ld_h, w.data, w.ld_d, w.scales, w.ld_s, n, v,
                     static_cast<int>(h / BK), vblocks, targets.p, targets.is32, ignore, pm, ps,
                     pt, ex);
}

}  // namespace itl
