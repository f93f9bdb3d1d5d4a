// 4-bit rows of a matrix (fp4.h), on gfx950.  A thread takes 8 columns, four
// lanes a group of 32.  Made once per weight version.  151936 x 4096 bf16: 341 us
// (1.58 GB, 4.6 TB/s, of the 6.45 that a copy reaches: a thread has one chunk's load
// in flight); with comparisons in place of the conversion instruction 510, bound
// by them.
#include "fp4.h"

#include "launch.h"
#include "row_device.h"

namespace itl {

namespace {

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void fp4_quantize_kernel(const T* __restrict__ x, int64_t ld_x,
                                                           int64_t n, int64_t h, int tx,
                                                           uint8_t* __restrict__ data,
                                                           int64_t ld_d,
                                                           uint8_t* __restrict__ scales,
                                                           int64_t ld_s) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / tx) + threadIdx.x / tx;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * tx + threadIdx.x % tx) * kE;
  // tx is at least 4 and h a multiple of 32: a group's four lanes stay together
  if (r >= n || c >= h) return;
  float v[kE];
  widen_raw<T>(load_raw<T, VEC>(x + r * ld_x, c, h), v);
  // the greatest magnitude as bits, which order like the magnitudes with
  // infinities and NaN on top
  uint32_t most = 0;
#pragma unroll
  for (int e = 0; e < kE; ++e) most = max(most, __float_as_uint(v[e]) & 0x7fffffffu);
  most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 1, 4)));
  most = max(most, static_cast<uint32_t>(__shfl_xor(static_cast<int>(most), 2, 4)));
  // 6 2^k reaches m 2^e (1 <= m < 2) with k = e - 2 up to m = 3 / 2, else with
  // k = e - 1.  Past 252 the code 6 would be infinite: values saturate there.
  uint32_t b = 255, q = 0;
  if (most < 0x7f800000u) {
    const int e = static_cast<int>(most >> 23) + ((most & 0x7fffffu) > 0x400000u);
    b = e <= 3 ? 1 : e < 254 ? e - 2 : 252;
    const float inv = __uint_as_float((254u - b) << 23);  // 1 / scale, a normal number
#pragma unroll
    for (int k = 0; k < kE; ++k) v[k] = v[k] * inv;  // exact, or far below the least code
    // ties to an even code, past 6 the code 6
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0], v[1], 1.0f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2], v[3], 1.0f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4], v[5], 1.0f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6], v[7], 1.0f, 3);
  }
  *reinterpret_cast<uint32_t*>(data + r * ld_d + c / 2) = q;
  if ((c & (kFp4Group - 1)) == 0) scales[r * ld_s + c / kFp4Group] = static_cast<uint8_t>(b);
}

template <typename T>
void quantize_typed(const void* x, int64_t ld_x, int64_t n, int64_t h, uint8_t* data, int64_t ld_d,
                    uint8_t* scales, int64_t ld_s, hipStream_t s) {
  auto kern = fits16(x, ld_x, sizeof(T)) ? fp4_quantize_kernel<T, true>
                                         : fp4_quantize_kernel<T, false>;
  const int64_t chunks = h / kE;
  const int tx = row_threads(chunks);
  const int64_t rows = 256 / tx;
  for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups * rows) {
    const int64_t m = n - r0 < kMaxGroups * rows ? n - r0 : kMaxGroups * rows;
    hipLaunchKernelGGL(kern,
                       dim3(static_cast<unsigned>((m + rows - 1) / rows),
                            static_cast<unsigned>((chunks + tx - 1) / tx)),
                       dim3(256), 0, s, static_cast<const T*>(x) + r0 * ld_x, ld_x, m, h, tx,
                       data + r0 * ld_d, ld_d, scales + r0 * ld_s, ld_s);
  }
}

}  // namespace

void launch_fp4_quantize(int dtype, const void* x, int64_t ld_x, int64_t n, int64_t h,
                         uint8_t* data, int64_t ld_d, uint8_t* scales, int64_t ld_s,
                         hipStream_t s) {
  auto run = dtype == kF32 ? quantize_typed<float>
             : dtype == kF16 ? quantize_typed<_Float16> : quantize_typed<uint16_t>;
  run(x, ld_x, n, h, data, ld_d, scales, ld_s, s);
}

}  // namespace itl
