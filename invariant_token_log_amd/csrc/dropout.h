// Dropout from a counter-based generator: its arguments, its device form (for
// the kernels that drop elements of rows they hold) and the launcher of the
// operator itself.  Arguments are checked by the callers in layer_api.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace itl {

// Which elements are kept: those whose 16-bit number reaches `least`, scaled
// by `factor`.  The seed comes from memory when seed_at is set.
struct Drop {
  const int64_t* seed_at;
  uint64_t seed;
  int64_t first_row;
  uint32_t draw;
  uint32_t least;
  float factor;
};

// p in [0, 1] to the 2^-16 that it is realised in; the factor is the
// reciprocal of what is kept, so that the expectation is exact.
inline Drop make_drop(double p, int64_t seed, const int64_t* seed_at, int64_t draw,
                      int64_t first_row) {
  const uint32_t least = static_cast<uint32_t>(p * 65536.0 + 0.5);
  return Drop{seed_at, static_cast<uint64_t>(seed), first_row, static_cast<uint32_t>(draw), least,
              least < 65536u ? static_cast<float>(65536.0 / (65536.0 - least)) : 0.0f};
}

// Philox-4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers: as easy
// as 1, 2, 3, 2011): ten rounds of two 32 x 32 -> 64 bit products.
__device__ __forceinline__ uint4 philox(uint4 c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c.x;
    const uint64_t b = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return c;
}

__device__ __forceinline__ uint64_t drop_seed(const Drop& d) {
  return d.seed_at ? static_cast<uint64_t>(*d.seed_at) : d.seed;
}

// The eight numbers of chunk `chunk` (columns 8 chunk ..) of row `row` (of the
// tensor), and whether element e of it is kept.
__device__ __forceinline__ uint4 drop_chunk(const Drop& d, uint64_t seed, int64_t row,
                                            uint32_t chunk) {
  const uint64_t r = static_cast<uint64_t>(d.first_row + row);
  return philox(make_uint4(chunk, static_cast<uint32_t>(r), static_cast<uint32_t>(r >> 32), d.draw),
                static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
}
__device__ __forceinline__ bool drop_keeps(const Drop& d, const uint4& u, int e) {
  const uint32_t w = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
  return ((e & 1) ? w >> 16 : w & 0xffffu) >= d.least;
}

// out = rne(residual + kept(x) factor), or without a residual rne(kept(x)
// factor); [n, h] rows.  out may be exactly x or residual.
void launch_dropout(int dtype, const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                    int64_t n, int64_t h, const Drop& drop, void* out, int64_t ld_o,
                    hipStream_t s);

}  // namespace itl
