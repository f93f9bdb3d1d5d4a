// Device pieces of the token operators (several given tokens a row, the most
// probable tokens, their gradients): row views, 16-byte row access at any
// alignment, the order of the alternatives and their ranking in one wave.
#pragma once

#include <hip/hip_runtime.h>
#include <float.h>
#include <stdint.h>

#include "logp_device.h"
#include "token_launch.h"

namespace itl {

// ---------------------------------------------------------------------------
// Row access.  VEC: row starts are 16-byte aligned and chunks stream past the
// caches (load_stream / store_stream).  Otherwise a whole chunk is still one
// 16-byte access: global memory takes any alignment on gfx950, and a row that
// starts at an odd element costs an extra line here and there instead of one
// access an element.  Columns at or past v are -inf on reading and not
// touched in memory.
// ---------------------------------------------------------------------------
struct __attribute__((packed, aligned(2))) AnyChunk {
  uint32_t w[4];
};

// A whole chunk as it is in memory: unlike load_row_chunk it has no branch, so
// that several of them wait together.
template <typename T, bool VEC>
__device__ __forceinline__ uint4 load_whole_chunk(const T* p) {
  if constexpr (VEC) {
    return load_stream(p);
  } else {
    const AnyChunk q = *reinterpret_cast<const AnyChunk*>(p);
    return make_uint4(q.w[0], q.w[1], q.w[2], q.w[3]);
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_whole_chunk(T* p, const uint4 q) {
  if constexpr (VEC) {
    store_stream(p, q);
  } else {
    AnyChunk a;
    a.w[0] = q.x; a.w[1] = q.y; a.w[2] = q.z; a.w[3] = q.w;
    *reinterpret_cast<AnyChunk*>(p) = a;
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void load_row_chunk(const T* row, int64_t c, int64_t v,
                                               float (&x)[Elt<T>::kPerChunk]) {
  constexpr int E = Elt<T>::kPerChunk;
  if (c + E <= v) {
    widen_chunk<T>(load_whole_chunk<T, VEC>(row + c), x);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = (c + e < v) ? Elt<T>::load(row, c + e) : -INFINITY;
  }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (__is_same(T, _Float16))
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(lo))) |
           (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<_Float16>(hi))) << 16);
  else
    return static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(lo))) |
           (static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(hi))) << 16);
}

// E values rounded once (RNE) to T.
template <typename T>
__device__ __forceinline__ uint4 round_chunk(const float (&x)[Elt<T>::kPerChunk]) {
  if constexpr (Elt<T>::kPerChunk == 4)
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  else
    return make_uint4(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]), pack2<T>(x[4], x[5]),
                      pack2<T>(x[6], x[7]));
}

template <typename T>
__device__ __forceinline__ void store_one(T* p, float x) {
  if constexpr (sizeof(T) == 4)
    *p = x;
  else if constexpr (__is_same(T, _Float16))
    *p = static_cast<_Float16>(x);
  else
    *p = __builtin_bit_cast(uint16_t, static_cast<__bf16>(x));
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_row_chunk(T* row, int64_t c, int64_t v,
                                                const float (&x)[Elt<T>::kPerChunk]) {
  constexpr int E = Elt<T>::kPerChunk;
  if (c + E <= v) {
    store_whole_chunk<T, VEC>(row + c, round_chunk<T>(x));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c + e < v) store_one<T>(row + c + e, x[e]);
  }
}

// ---------------------------------------------------------------------------
// Rows.  A row is active unless it has given tokens and every one of them is
// ignore_index; an inactive row is not read.  All lanes of a wave call.
// ---------------------------------------------------------------------------
__device__ __forceinline__ bool row_active(const TokenView& tok, int64_t r, int lane) {
  if (tok.m == 0) return true;
  for (int64_t i0 = 0; i0 < tok.m; i0 += kWave) {
    const int64_t i = i0 + lane;
    if (__builtin_amdgcn_ballot_w64(i < tok.m && tok.at(r, i) != tok.ignore)) return true;
  }
  return false;
}

// Entry i of an active row: given token i, then alternative i - M.  col = -1
// and g = 0 for an entry that is left out.  A given token outside [0, v)
// keeps its g (it lowers every probability) and matches no column the caller
// owns.
__device__ __forceinline__ void entry_at(const TokenView& tok, const TopView& alt,
                                         const float* grad, const float* grad_top, int64_t r,
                                         int64_t i, int64_t& col, float& g) {
  if (i < tok.m) {
    const int64_t t = tok.at(r, i);
    if (t != tok.ignore) {
      col = t;
      g = grad ? grad[r * tok.m + i] : 0.0f;
    }
  } else {
    const int64_t j = r * alt.k + (i - tok.m);
    const int64_t t = alt.ids[j];
    if (t >= 0) {
      col = t;
      g = grad_top[j];
    }
  }
}

// d = u - G p [- gH p (log p + H)], log p = dl = x - lse.  p of a masked
// (-inf) logit is 0 and its entropy term an exact -0.  -G p alone is the
// product the fused backward's dz takes.
template <bool ENT>
__device__ __forceinline__ float token_grad(float dl, float u, float ng, float H, float ngh) {
  const float p = __builtin_amdgcn_exp2f(dl * kLog2e);
  float d = fmaf(ng, p, u);
  if constexpr (ENT) d = fmaf(ngh, p * fmaxf(dl + H, -FLT_MAX), d);
  return d;
}

// Element (r, c) of the K32-blocked layout (kblocked_index of mfma_gemm.h).
__device__ __forceinline__ int64_t kblocked_at(int64_t r, int64_t c, int64_t ksteps) {
  return ((r >> 4) * ksteps + (c >> 5)) * 512 + (r & 15) * 32 + (c & 31);
}

// ---------------------------------------------------------------------------
// The order of the alternatives: greater value first, then smaller index.
// order_key maps floats to unsigned integers in ascending order, with -0 as
// +0 and NaN as -inf (a row with a NaN has a NaN lse anyway); no key is 0.
// compose puts the index, counted down, below the key, so that composites
// are distinct and one comparison orders two candidates.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t order_key(float x) {
  x = x + 0.0f;
  const uint32_t b = __float_as_uint(x != x ? -INFINITY : x);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}
__device__ __forceinline__ uint64_t compose(uint32_t key, uint32_t index) {
  return (static_cast<uint64_t>(key) << 32) | (0xffffffffu - index);
}
__device__ __forceinline__ uint32_t compose_index(uint64_t c) {
  return 0xffffffffu - static_cast<uint32_t>(c);
}

// Orders this wave's LDS accesses around a point (one wave's LDS operations
// execute in order; this keeps the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ uint32_t lane_u32(uint32_t x, int lane) {
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(x), lane));
}

// A key that at least k of the wave's 256 keys (four a lane) reach: the k-th
// greatest, or a smaller one that exactly k reach; 0 when fewer than k are not
// 0.  Bit by bit from the top.
__device__ __forceinline__ uint32_t wave_bound(const uint32_t (&key)[4], int k) {
  uint32_t bound = 0;
#pragma unroll 1
  for (uint32_t bit = 0x80000000u; bit; bit >>= 1) {
    const uint32_t t = bound | bit;
    int reach = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) reach += __popcll(__builtin_amdgcn_ballot_w64(key[i] >= t));
    if (reach >= k) bound = t;
    if (reach == k) break;
  }
  return bound;
}

// A wave's candidate list in LDS.  top_push appends the composites of the
// lanes that want to; when they would not fit, the list is first cut to its
// k greatest, after which only composites above the k-th may enter.  k <= 64,
// so a push of 64 always fits after a cut.
constexpr int kTopCap = 256;
struct TopStage {
  uint64_t e[kTopCap];
  uint32_t group[kWave];  // the greatest groups, best first
  int used;
};
struct TopList {
  int n;           // entries (uniform)
  uint64_t floor;  // composites at or below it are out (uniform)
};

// Adds to rank[c] the entries of `from` (one a lane, n of them) that are
// greater than mine[c]: a broadcast an entry, no LDS latency.
template <int N>
__device__ __forceinline__ void count_greater(uint64_t from, int n, const uint64_t (&mine)[N],
                                              int (&rank)[N]) {
  const uint32_t lo = static_cast<uint32_t>(from), hi = static_cast<uint32_t>(from >> 32);
  for (int j0 = 0; j0 < n; j0 += 8) {  // past the end: zeros, greater than nothing
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t o = (static_cast<uint64_t>(lane_u32(hi, j0 + j)) << 32) | lane_u32(lo, j0 + j);
#pragma unroll
      for (int c = 0; c < N; ++c) rank[c] += o > mine[c];
    }
  }
}

// Cut to the min(n, k) greatest, in descending order at e[0 ..).  The rank of
// an entry is the number of greater ones; composites are distinct.
__device__ __forceinline__ void top_rank(TopStage& st, TopList& list, int k) {
  const int lane = threadIdx.x & (kWave - 1);
  wave_lds_fence();
  if (list.n <= kWave) {
    const uint64_t mine[1] = {lane < list.n ? st.e[lane] : 0};
    int rank[1] = {0};
    count_greater<1>(mine[0], list.n, mine, rank);
    wave_lds_fence();
    if (lane < list.n && rank[0] < k) st.e[rank[0]] = mine[0];
  } else {
    uint64_t mine[kTopCap / kWave];
    int rank[kTopCap / kWave];
#pragma unroll
    for (int c = 0; c < kTopCap / kWave; ++c) {
      const int i = c * kWave + lane;
      mine[c] = i < list.n ? st.e[i] : 0;
      rank[c] = 0;
    }
    if (list.n <= 2 * kWave) {
      const uint64_t two[2] = {mine[0], mine[1]};
      int r2[2] = {0, 0};
      count_greater<2>(mine[0], kWave, two, r2);
      count_greater<2>(mine[1], list.n - kWave, two, r2);
      rank[0] = r2[0];
      rank[1] = r2[1];
    } else {
      for (int j = 0; j < list.n; ++j) {
        const uint64_t o = st.e[j];
#pragma unroll
        for (int c = 0; c < kTopCap / kWave; ++c) rank[c] += o > mine[c];
      }
    }
    wave_lds_fence();
#pragma unroll
    for (int c = 0; c < kTopCap / kWave; ++c)
      if (c * kWave + lane < list.n && rank[c] < k) st.e[rank[c]] = mine[c];
  }
  wave_lds_fence();
  if (list.n > k) list.n = k;
}

// Append count (>= 0) composites of this lane, which the caller then writes at
// the returned place on; false, with nothing appended, when those of all lanes
// do not fit.  The places the lanes get are in no fixed order; ranking the list
// gives it one.
__device__ __forceinline__ bool top_reserve(TopStage& st, TopList& list, int count, int& place) {
  const int lane = threadIdx.x & (kWave - 1);
  if (lane == 0) st.used = list.n;
  wave_lds_fence();
  place = 0;
  if (count > 0) place = atomicAdd(&st.used, count);
  wave_lds_fence();
  const int n = __builtin_amdgcn_readfirstlane(st.used);
  wave_lds_fence();
  if (n > kTopCap) return false;
  list.n = n;
  return true;
}

__device__ __forceinline__ void top_push(TopStage& st, TopList& list, int k, bool want,
                                         uint64_t composite) {
  uint64_t mask = __builtin_amdgcn_ballot_w64(want && composite > list.floor);
  if (mask == 0) return;
  if (list.n + __popcll(mask) > kTopCap) {
    top_rank(st, list, k);
    list.floor = st.e[list.n - 1];
    mask = __builtin_amdgcn_ballot_w64(want && composite > list.floor);
  }
  const int lane = threadIdx.x & (kWave - 1);
  if ((mask >> lane) & 1)
    st.e[list.n + __popcll(mask & ((uint64_t{1} << lane) - 1))] = composite;
  list.n += __popcll(mask);
}

}  // namespace itl
