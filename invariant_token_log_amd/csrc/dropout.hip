// Dropout with the residual's addition, on gfx950.
//
//   out[r, j] = rne(residual[r, j] + (u[r, j] >= T ? x[r, j] c : 0))
//
// u: eight 16-bit numbers a call of the generator, a chunk of 8 columns, so the
// mask is a function of (seed, draw, row, column) and is never stored: the
// backward pass is the same kernel on the gradient.  A dropped element is not
// multiplied, so an infinity or a NaN there is dropped too.
// Bound by memory: every element is read and written once.  The generator takes
// twenty 32 x 32 bit products for 8 elements, which run beside the loads.  8192 x
// 4096 bf16: 29 to 31 us with a residual (201 MB, 6.5 to 6.9 TB/s), 21 to 23 without,
// what a copy of as many bytes takes and no more than with p = 0.
#include "dropout.h"

#include "launch.h"
#include "row_device.h"

namespace itl {

namespace {

// Threads along a row: TX chunks of 8 columns at a time, 256 / TX rows a
// workgroup.
template <typename T, bool VEC>
__global__ __launch_bounds__(256) void dropout_kernel(const T* x, int64_t ld_x, const T* residual,
                                                      int64_t ld_r, int64_t n, int64_t h, int tx,
                                                      Drop drop, T* out, int64_t ld_o) {
  const int rows = 256 / tx;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * rows + threadIdx.x / tx;
  const int64_t chunk = static_cast<int64_t>(blockIdx.y) * tx + threadIdx.x % tx;
  if (r >= n || chunk * kE >= h) return;
  const Raw<T> a = load_raw<T, VEC>(x + r * ld_x, chunk * kE, h);
  Raw<T> b;
  if (residual) b = load_raw<T, VEC>(residual + r * ld_r, chunk * kE, h);
  const uint4 u = drop_chunk(drop, drop_seed(drop), r, static_cast<uint32_t>(chunk));
  float p[kE], q[kE];
  widen_raw<T>(a, p);
  if (residual) {
    widen_raw<T>(b, q);
#pragma unroll
    for (int e = 0; e < kE; ++e)
      p[e] = drop_keeps(drop, u, e) ? fmaf(p[e], drop.factor, q[e]) : q[e];
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) p[e] = drop_keeps(drop, u, e) ? p[e] * drop.factor : 0.0f;
  }
  store_raw<T, VEC>(out + r * ld_o, chunk * kE, h, round_raw<T>(p));
}

template <typename T>
void dropout_typed(const void* x, int64_t ld_x, const void* residual, int64_t ld_r, int64_t n,
                   int64_t h, const Drop& drop, void* out, int64_t ld_o, hipStream_t s) {
  const int size = sizeof(T);
  const bool vec = fits16(x, ld_x, size) && fits16(residual, ld_r, size) && fits16(out, ld_o, size);
  const int64_t chunks = (h + kE - 1) / kE;
  const int tx = row_threads(chunks);
  const int rows = 256 / tx;
  auto kern = vec ? dropout_kernel<T, true> : dropout_kernel<T, false>;
  for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups * rows) {
    const int64_t m = n - r0 < kMaxGroups * rows ? n - r0 : kMaxGroups * rows;
    Drop d = drop;
    d.first_row += r0;
    hipLaunchKernelGGL(kern,
                       dim3(static_cast<unsigned>((m + rows - 1) / rows),
                            static_cast<unsigned>((chunks + tx - 1) / tx)),
                       dim3(256), 0, s, row_at(static_cast<const T*>(x), r0, ld_x), ld_x,
                       row_at(static_cast<const T*>(residual), r0, ld_r), ld_r, m, h, tx, d,
                       row_at(static_cast<T*>(out), r0, ld_o), ld_o);
  }
}

}  // namespace

void launch_dropout(int dtype, const void* x, int64_t ld_x, const void* residual, int64_t ld_r,
                    int64_t n, int64_t h, const Drop& drop, void* out, int64_t ld_o,
                    hipStream_t s) {
  auto run = dtype == kF32 ? dropout_typed<float>
             : dtype == kF16 ? dropout_typed<_Float16> : dropout_typed<uint16_t>;
  run(x, ld_x, residual, ld_r, n, h, drop, out, ld_o, s);
}

}  // namespace itl
