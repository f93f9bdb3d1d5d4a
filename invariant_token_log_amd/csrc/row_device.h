// Rows of elements in chunks of 8, for the kernels that own whole rows (the
// norms, dropout, the embedding): access at any alignment, widening and
// rounding, reductions over the team of threads that shares a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "logp_device.h"
#include "token_device.h"

namespace itl {

constexpr int kE = 8;  // elements per chunk, every type

template <typename T>
constexpr int kRaw = sizeof(T) == 4 ? 2 : 1;  // 16-byte pieces per chunk

// One chunk of 8 elements as stored.
template <typename T>
struct Raw {
  uint4 q[kRaw<T>];
};

template <typename T>
__device__ __forceinline__ void widen_raw(const Raw<T>& r, float (&x)[kE]) {
  if constexpr (sizeof(T) == 4) {
    float lo[4], hi[4];
    widen_chunk<T>(r.q[0], lo);
    widen_chunk<T>(r.q[1], hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = lo[e];
      x[4 + e] = hi[e];
    }
  } else {
    widen_chunk<T>(r.q[0], x);
  }
}

template <typename T>
__device__ __forceinline__ Raw<T> round_raw(const float (&x)[kE]) {
  Raw<T> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      r.q[p] = make_uint4(__float_as_uint(x[4 * p]), __float_as_uint(x[4 * p + 1]),
                          __float_as_uint(x[4 * p + 2]), __float_as_uint(x[4 * p + 3]));
  } else {
    r.q[0] = round_chunk<T>(x);
  }
  return r;
}

// The chunk at element c of a row of h; elements past h are 0.
template <typename T, bool VEC>
__device__ __forceinline__ Raw<T> load_raw(const T* row, int64_t c, int64_t h) {
  Raw<T> r;
  if (c + kE <= h) {
#pragma unroll
    for (int p = 0; p < kRaw<T>; ++p) {
      if constexpr (VEC) {
        r.q[p] = *(reinterpret_cast<const uint4*>(row + c) + p);
      } else {
        const AnyChunk a = *(reinterpret_cast<const AnyChunk*>(row + c) + p);
        r.q[p] = make_uint4(a.w[0], a.w[1], a.w[2], a.w[3]);
      }
    }
    return r;
  }
  float x[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) x[e] = c + e < h ? Elt<T>::load(row, c + e) : 0.0f;
  return round_raw<T>(x);  // exact: the values are of type T
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_raw(T* row, int64_t c, int64_t h, const Raw<T>& r) {
  if (c + kE <= h) {
#pragma unroll
    for (int p = 0; p < kRaw<T>; ++p) {
      if constexpr (VEC) {
        *(reinterpret_cast<uint4*>(row + c) + p) = r.q[p];
      } else {
        AnyChunk a;
        a.w[0] = r.q[p].x; a.w[1] = r.q[p].y; a.w[2] = r.q[p].z; a.w[3] = r.q[p].w;
        *(reinterpret_cast<AnyChunk*>(row + c) + p) = a;
      }
    }
    return;
  }
  float x[kE];
  widen_raw<T>(r, x);
#pragma unroll
  for (int e = 0; e < kE; ++e)
    if (c + e < h) store_one<T>(row + c + e, x[e]);
}

// Sum (or maximum) over the team; every thread gets it.  buf: TEAM / 64
// floats of the team; two calls in a row take different buffers, so one
// barrier a call is enough.
template <int TEAM, bool MAX>
__device__ __forceinline__ float team_reduce(float x, float* buf) {
  x = MAX ? wave_max(x) : wave_sum(x);
  if constexpr (TEAM > kWave) {
    const int wave = (threadIdx.x % TEAM) / kWave;
    if (threadIdx.x % kWave == 0) buf[wave] = x;
    __syncthreads();
    x = buf[0];
#pragma unroll
    for (int w = 1; w < TEAM / kWave; ++w) x = MAX ? fmaxf(x, buf[w]) : x + buf[w];
  }
  return x;
}

// Workgroups of a launch: a grid holds fewer than 2^32 threads, so more rows
// take several launches.
constexpr int64_t kMaxGroups = int64_t{1} << 20;

template <typename T>
T* row_at(T* p, int64_t r, int64_t ld) {
  return p ? p + r * ld : nullptr;
}

// Threads of a workgroup of 256 along a row of `chunks` chunks (a power of two);
// the others take further rows.
inline int row_threads(int64_t chunks) {
  int tx = 1;
  while (tx < chunks && tx < 256) tx *= 2;
  return tx;
}

inline bool fits16(const void* p, int64_t ld, int size) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (ld * size) % 16 == 0);
}

}  // namespace itl
