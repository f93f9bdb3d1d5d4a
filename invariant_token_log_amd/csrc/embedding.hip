// Embedding lookup with scaling, from rows of any type or in 4 bits, and the
// table's gradient by sorted tokens, on gfx950.
//
//   y[i] = rne(scale E[t_i])
//   dE[t] = rne([dE[t] +] scale sum over i ascending with t_i = t of dy[i])
//
// The lookup is bound by memory: one 16-byte access a thread, a row's column
// chunks side by side.
//
// The gradient sorts the tokens with their positions, so that the occurrences of
// a token form a run in ascending position, and sums every run in fp32:
//   1. embed_sort_kernel: tiles of 4096 tokens, a workgroup each, a bitonic
//      network in registers, lane moves and LDS (no order-dependent atomics, so
//      the same bits every time).  More than one tile: embed_rank_kernel places
//      every token by binary searches in the other tiles.
//   2. embed_sum_kernel: a wave for every piece of 32 occurrences; a run of one
//      piece goes straight to the table, a longer one leaves a partial row a
//      piece.
//   3. embed_join_kernel: adds the partial rows of the longer runs: eight
//      chains of every eighth piece, then the chains in order.
// A row of the gradient depends on its token's own occurrences and their
// order, not on the batch around them.
// Without accumulation the rows of absent tokens are written with zeros by
// embed_zero_kernel; with a large vocabulary that is what takes the time.
#include "embedding.h"

#include <type_traits>

#include "fp4.h"
#include "row_device.h"

namespace itl {

namespace {

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void embedding_kernel(const T* __restrict__ table, int64_t ld_t,
                                                        int64_t v, int64_t h,
                                                        const void* __restrict__ tok,
                                                        int32_t tok32, int64_t n, int64_t ignore,
                                                        float scale, int tx, T* __restrict__ out,
                                                        int64_t ld_o) {
  const Targets tokens{tok, tok32};
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / tx) + threadIdx.x / tx;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * tx + threadIdx.x % tx) * kE;
  if (r >= n || c >= h) return;
  const int64_t t = tokens[r];
  float x[kE];
  if (t >= 0 && t < v && t != ignore) {
    widen_raw<T>(load_raw<T, VEC>(table + t * ld_t, c, h), x);
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = x[e] * scale;
  } else {
    const float fill = t == ignore ? 0.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = fill;
  }
  store_raw<T, VEC>(out + r * ld_o, c, h, round_raw<T>(x));
}

template <typename T, bool VEC>
__global__ __launch_bounds__(256) void embedding_fp4_kernel(
    const uint8_t* __restrict__ data, int64_t ld_d, const uint8_t* __restrict__ scales,
    int64_t ld_s, int64_t v, int64_t h, const void* __restrict__ tok, int32_t tok32, int64_t n,
    int64_t ignore, float scale, int tx, T* __restrict__ out, int64_t ld_o) {
  const Targets tokens{tok, tok32};
  const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / tx) + threadIdx.x / tx;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * tx + threadIdx.x % tx) * kE;
  if (r >= n || c >= h) return;
  const int64_t t = tokens[r];
  float x[kE];
  if (t >= 0 && t < v && t != ignore) {
    const uint32_t q = *reinterpret_cast<const uint32_t*>(data + t * ld_d + c / 2);
    const float s = fp4_scale(scales[t * ld_s + c / kFp4Group]);
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = fp4_value(q >> (4 * e)) * s * scale;
  } else {
    const float fill = t == ignore ? 0.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int e = 0; e < kE; ++e) x[e] = fill;
  }
  store_raw<T, VEC>(out + r * ld_o, c, h, round_raw<T>(x));
}

// ---------------------------------------------------------------------------
// Sort.
// ---------------------------------------------------------------------------
constexpr int kTile = 4096;      // tokens a workgroup sorts
constexpr int kSortThreads = 1024;
constexpr int kPer = kTile / kSortThreads;  // tokens a thread: 4 in a row
constexpr int kPiece = 32;       // occurrences a wave adds

// The run of slot i's token: where it starts, and the token itself (v: left
// out, at the end).
struct Sorted {
  uint32_t* id;
  uint32_t* pos;
  uint32_t* start;
};

__device__ __forceinline__ uint32_t shfl_xor_key(uint32_t x, int o) {
  return static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), o, kWave));
}
__device__ __forceinline__ uint64_t shfl_xor_key(uint64_t x, int o) {
  return static_cast<uint64_t>(shfl_xor_key(static_cast<uint32_t>(x >> 32), o)) << 32 |
         shfl_xor_key(static_cast<uint32_t>(x), o);
}

// Ascending bitonic sort of the workgroup's 4096 keys, thread t holding keys 4 t
// ..; only the stages that `count` keys need (the others are the greatest).
// buf: 4096 keys of LDS.
template <typename K>
__device__ __forceinline__ void sort_tile(K (&key)[kPer], K* buf, int count) {
  const int t = threadIdx.x;
  for (int size = 2; size < 2 * count && size <= kTile; size *= 2) {
    for (int s = size / 2; s > 0; s /= 2) {
      if (s >= kPer * kWave) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j) buf[j * kSortThreads + t] = key[j];
        __syncthreads();
        const int o = t ^ (s / kPer);
        const bool low = ((kPer * t & s) == 0) == ((kPer * t & size) == 0);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const K other = buf[j * kSortThreads + o];
          key[j] = (key[j] < other) == low ? key[j] : other;
        }
      } else if (s >= kPer) {
        const bool low = ((kPer * t & s) == 0) == ((kPer * t & size) == 0);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const K other = shfl_xor_key(key[j], s / kPer);
          key[j] = (key[j] < other) == low ? key[j] : other;
        }
      } else {
        auto order = [&](int a, int b) {
          const bool up = ((kPer * t + a) & size) == 0;
          const K x = key[a], y = key[b];
          const bool swap = (x > y) == up;
          key[a] = swap ? y : x;
          key[b] = swap ? x : y;
        };
        if (s == 2) {
          order(0, 2);
          order(1, 3);
        } else {
          order(0, 1);
          order(2, 3);
        }
      }
    }
  }
}

// Tile blockIdx.x of the tokens.  Keys are (token, position in the tile), the
// token of an entry that is left out being v.  One tile: the sorted arrays; more:
// the tile's sorted keys (token << 32 | position) for embed_rank_kernel.
// SMALL: v < 2^20 - 1, so that a key fits 32 bits.
template <bool SMALL>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(
    const void* __restrict__ tok, int32_t tok32, int64_t n, int64_t v, int64_t ignore, Sorted out,
    uint64_t* __restrict__ tiles) {
  using K = typename std::conditional<SMALL, uint32_t, uint64_t>::type;
  constexpr int kShift = SMALL ? 12 : 32;
  __shared__ K buf[kTile];
  const Targets tokens{tok, tok32};
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kTile;
  const int count = static_cast<int>(n - base < kTile ? n - base : kTile);
  K key[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    key[j] = ~K{0};
    if (i < count) {
      const int64_t t = tokens[base + i];
      const bool live = t >= 0 && t < v && t != ignore;
      key[j] = static_cast<K>(live ? t : v) << kShift | static_cast<K>(i);
    }
  }
  sort_tile<K>(key, buf, count);
  auto token = [](K k) { return static_cast<uint32_t>(k >> kShift); };
  if (tiles) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)  // i < count holds the tile's own keys: the rest sort behind
      if (kPer * static_cast<int>(threadIdx.x) + j < count)
        tiles[base + kPer * threadIdx.x + j] =
            static_cast<uint64_t>(token(key[j])) << 32 |
            static_cast<uint64_t>(base + static_cast<int64_t>(key[j] & (kTile - 1)));
    return;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j) buf[kPer * threadIdx.x + j] = key[j];
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = kPer * threadIdx.x + j;
    if (i >= count) break;
    const K first = static_cast<K>(token(key[j])) << kShift;
    int lo = 0, hi = i;  // the first key of this token: at most i
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (buf[mid] < first) lo = mid + 1; else hi = mid;
    }
    out.id[i] = token(key[j]);
    out.pos[i] = static_cast<uint32_t>(key[j] & (kTile - 1));
    out.start[i] = static_cast<uint32_t>(lo);
  }
}

// Where key k would stand among the `count` ascending keys.
__device__ __forceinline__ int lower_bound(const uint64_t* keys, int count, uint64_t k) {
  int lo = 0;
  while (count > 0) {
    const int half = count / 2;
    if (keys[lo + half] < k) {
      lo += half + 1;
      count -= half + 1;
    } else {
      count = half;
    }
  }
  return lo;
}

__global__ __launch_bounds__(256) void embed_rank_kernel(const uint64_t* __restrict__ tiles,
                                                         int64_t n, Sorted out) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= n) return;
  const uint64_t key = tiles[i], first = key >> 32 << 32;
  const int64_t own = i / kTile * kTile;
  int64_t rank = 0, start = 0;
  for (int64_t b = 0; b < n; b += kTile) {
    const int count = static_cast<int>(n - b < kTile ? n - b : kTile);
    const int lo = lower_bound(tiles + b, count, first);
    start += lo;
    if (b == own) {
      rank += i - own;
    } else {
      rank += lo;
      // the same token in an earlier tile stands before this one
      if (b < own && lo < count && tiles[b + lo] >> 32 == key >> 32)
        rank += lower_bound(tiles + b + lo, count - lo, key);
    }
  }
  out.id[rank] = static_cast<uint32_t>(key >> 32);
  out.pos[rank] = static_cast<uint32_t>(key);
  out.start[rank] = static_cast<uint32_t>(start);
}

// ---------------------------------------------------------------------------
// Sums.
// ---------------------------------------------------------------------------
// The partial row of the piece at slot s of a run of several pieces.  In a
// window of kPiece slots at most one such run goes on and one begins.
__device__ __forceinline__ int64_t partial_row(int64_t s, int64_t start) {
  return 2 * (s / kPiece) + (s != start);
}

// Writes scale a[], added to what is there with accumulate.
template <typename U, bool VEC>
__device__ __forceinline__ void table_store(U* row, int64_t c, int64_t h, float scale,
                                            bool accumulate, float (&a)[kE]) {
  if (accumulate) {
    float old[kE];
    widen_raw<U>(load_raw<U, VEC>(row, c, h), old);
#pragma unroll
    for (int e = 0; e < kE; ++e) a[e] = fmaf(a[e], scale, old[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) a[e] = a[e] * scale;
  }
  store_raw<U, VEC>(row, c, h, round_raw<U>(a));
}

// A wave a slot; those that begin a piece add its rows, CH chunks a lane.
template <typename T, typename U, int CH, bool VEC>
__global__ __launch_bounds__(256) void embed_sum_kernel(const T* __restrict__ dy, int64_t ld_y,
                                                        Sorted sorted, int64_t n, int64_t v,
                                                        int64_t h, float scale, bool accumulate,
                                                        U* __restrict__ dtable, int64_t ld_t,
                                                        float* __restrict__ partial, int64_t ld_p) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t s = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  if (s >= n) return;
  const uint32_t id = sorted.id[s], start = sorted.start[s];
  if (id >= v || (s - start) % kPiece) return;
  // lane l looks at slot s + l: the piece's rows, and whether the run goes on
  const int64_t at = s + lane;
  const bool same = at < n && sorted.id[at] == id;
  const uint32_t pos = lane < kPiece && same ? sorted.pos[at] : 0;
  const uint64_t run = __builtin_amdgcn_ballot_w64(same);
  const int reach = ~run ? __builtin_ctzll(~run) : kWave;
  const int count = reach < kPiece ? reach : kPiece;
  const bool pieces = s != start || reach > kPiece;
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * (CH * kWave * kE) + lane * kE;
  float acc[CH][kE];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[c][e] = 0.0f;
  constexpr int kRows = 4;  // rows whose loads are in flight together
  for (int i0 = 0; i0 < count; i0 += kRows) {
    Raw<T> x[kRows][CH];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i0 + i < count) {
        const T* row = dy + static_cast<int64_t>(__builtin_amdgcn_readlane(pos, i0 + i)) * ld_y;
#pragma unroll
        for (int c = 0; c < CH; ++c) x[i][c] = load_raw<T, VEC>(row, c0 + c * kWave * kE, h);
      }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (i0 + i < count) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          float p[kE];
          widen_raw<T>(x[i][c], p);
#pragma unroll
          for (int e = 0; e < kE; ++e) acc[c][e] = acc[c][e] + p[e];
        }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int64_t col = c0 + c * kWave * kE;
    if (col >= h) break;
    if (pieces) {
      float4* to = reinterpret_cast<float4*>(partial + partial_row(s, start) * ld_p + col);
      to[0] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
      to[1] = make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]);
    } else {
      table_store<U, VEC>(dtable + static_cast<int64_t>(id) * ld_t, col, h, scale, accumulate,
                          acc[c]);
    }
  }
}

// The runs of several pieces: at most one begins in window blockIdx.x of kPiece
// slots.  256 columns a workgroup, eight groups of 32 lanes.
constexpr int kJoinCols = 256, kJoinGroups = 8;

template <typename U, bool VEC>
__global__ __launch_bounds__(256) void embed_join_kernel(const float* __restrict__ partial,
                                                         int64_t ld_p, Sorted sorted, int64_t n,
                                                         int64_t v, int64_t h, float scale,
                                                         bool accumulate, U* __restrict__ dtable,
                                                         int64_t ld_t) {
  __shared__ float part[kJoinGroups][kJoinCols];
  const int lane = threadIdx.x % kWave;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * kPiece + lane;
  const bool head = lane < kPiece && s + kPiece < n && sorted.start[s] == s && sorted.id[s] < v &&
                    sorted.id[s + kPiece] == sorted.id[s];
  const uint64_t heads = __builtin_amdgcn_ballot_w64(head);
  if (!heads) return;  // the same in every wave
  const int64_t start = static_cast<int64_t>(blockIdx.x) * kPiece + __builtin_ctzll(heads);
  const uint32_t id = sorted.id[start];
  int64_t lo = start + kPiece + 1, hi = n;  // the run's end
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (sorted.id[mid] == id) lo = mid + 1; else hi = mid;
  }
  const int64_t pieces = (lo - start + kPiece - 1) / kPiece;
  const int group = threadIdx.x / 32, t = threadIdx.x % 32;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * kJoinCols + t * kE;
  float a[kE] = {};
  if (col < h)
#pragma unroll 4
    for (int64_t k = group; k < pieces; k += kJoinGroups) {
      const float4* from = reinterpret_cast<const float4*>(
          partial + partial_row(start + k * kPiece, start) * ld_p + col);
      const float4 x = from[0], y = from[1];
      a[0] = a[0] + x.x; a[1] = a[1] + x.y; a[2] = a[2] + x.z; a[3] = a[3] + x.w;
      a[4] = a[4] + y.x; a[5] = a[5] + y.y; a[6] = a[6] + y.z; a[7] = a[7] + y.w;
    }
#pragma unroll
  for (int e = 0; e < kE; ++e) part[group][e * 32 + t] = a[e];
  __syncthreads();
  if (group || col >= h) return;
  for (int g = 1; g < kJoinGroups; ++g)
#pragma unroll
    for (int e = 0; e < kE; ++e) a[e] = a[e] + part[g][e * 32 + t];
  table_store<U, VEC>(dtable + static_cast<int64_t>(id) * ld_t, col, h, scale, accumulate, a);
}

// Zeros in the rows of absent tokens, 64 rows a workgroup and step.
template <typename U, bool VEC>
__global__ __launch_bounds__(256) void embed_zero_kernel(const uint32_t* __restrict__ id, int64_t n,
                                                         int64_t v, int64_t h,
                                                         U* __restrict__ dtable, int64_t ld_t) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int64_t v0 = static_cast<int64_t>(blockIdx.x) * kWave; v0 < v;
       v0 += static_cast<int64_t>(gridDim.x) * kWave) {
    const int64_t row = v0 + lane;
    int64_t lo = 0, hi = n;
    while (lo < hi) {
      const int64_t mid = (lo + hi) / 2;
      if (id[mid] < row) lo = mid + 1; else hi = mid;
    }
    const uint64_t absent =
        __builtin_amdgcn_ballot_w64(row < v && !(lo < n && id[lo] == row));
    Raw<U> zero;
#pragma unroll
    for (int p = 0; p < kRaw<U>; ++p) zero.q[p] = make_uint4(0, 0, 0, 0);
    for (int i = wave; i < kWave; i += 4) {
      if (!((absent >> i) & 1)) continue;
      for (int64_t c = lane * kE; c < h; c += kWave * kE)
        store_raw<U, VEC>(dtable + (v0 + i) * ld_t, c, h, zero);
    }
  }
}

// Workspace: id, pos, start [n]; the tiles' keys when there are several; the
// partial rows.
struct BwdLayout {
  int64_t id, pos, start, tiles, partial, ld_p, total;
};
BwdLayout bwd_layout(int64_t n, int64_t h) {
  auto round = [](int64_t x) { return (x + 255) / 256 * 256; };
  BwdLayout l;
  l.ld_p = (h + 7) / 8 * 8;
  l.id = 0;
  l.pos = round(4 * n);
  l.start = 2 * l.pos;
  l.tiles = 3 * l.pos;
  l.partial = l.tiles + (n > kTile ? round(8 * n) : 0);
  // runs of several pieces need more than kPiece tokens
  const int64_t rows = n > kPiece ? 2 * ((n + kPiece - 1) / kPiece) : 0;
  l.total = l.partial + round(rows * l.ld_p * 4);
  return l;
}

template <typename T, typename U>
void bwd_typed(const void* dy, int64_t ld_y, Targets tokens, int64_t n, int64_t v, int64_t h,
               int64_t ignore, float scale, bool accumulate, void* dtable, int64_t ld_t, char* ws,
               hipStream_t s) {
  const BwdLayout l = bwd_layout(n, h);
  const Sorted sorted{reinterpret_cast<uint32_t*>(ws + l.id),
                      reinterpret_cast<uint32_t*>(ws + l.pos),
                      reinterpret_cast<uint32_t*>(ws + l.start)};
  uint64_t* tiles = n > kTile ? reinterpret_cast<uint64_t*>(ws + l.tiles) : nullptr;
  float* partial = reinterpret_cast<float*>(ws + l.partial);
  U* out = static_cast<U*>(dtable);
  const bool vec_out = fits16(dtable, ld_t, sizeof(U));
  if (n) {
    auto sort = v < (1 << 20) - 1 ? embed_sort_kernel<true> : embed_sort_kernel<false>;
    hipLaunchKernelGGL(sort, dim3(static_cast<unsigned>((n + kTile - 1) / kTile)),
                       dim3(kSortThreads), 0, s, tokens.p, tokens.is32, n, v, ignore, sorted,
                       tiles);
    if (tiles)
      hipLaunchKernelGGL(embed_rank_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256),
                         0, s, tiles, n, sorted);
  }
  if (!accumulate) {
    const int64_t groups = (v + kWave - 1) / kWave;
    hipLaunchKernelGGL((vec_out ? embed_zero_kernel<U, true> : embed_zero_kernel<U, false>),
                       dim3(static_cast<unsigned>(groups < kMaxGroups ? groups : kMaxGroups)),
                       dim3(256), 0, s, sorted.id, n, v, h, out, ld_t);
  }
  if (!n) return;
  const bool vec = vec_out && fits16(dy, ld_y, sizeof(T));
  constexpr int CH = sizeof(T) == 4 ? 2 : 4;  // four rows of 64 bytes a lane in flight
  const bool narrow = h <= kWave * kE;
  auto sum = narrow ? (vec ? embed_sum_kernel<T, U, 1, true> : embed_sum_kernel<T, U, 1, false>)
                    : (vec ? embed_sum_kernel<T, U, CH, true> : embed_sum_kernel<T, U, CH, false>);
  const int64_t cols = (narrow ? 1 : CH) * kWave * kE;
  hipLaunchKernelGGL(sum,
                     dim3(static_cast<unsigned>((n + 3) / 4),
                          static_cast<unsigned>((h + cols - 1) / cols)),
                     dim3(256), 0, s, static_cast<const T*>(dy), ld_y, sorted, n, v, h, scale,
                     accumulate, out, ld_t, partial, l.ld_p);
  if (n > kPiece)
    hipLaunchKernelGGL((vec_out ? embed_join_kernel<U, true> : embed_join_kernel<U, false>),
                       dim3(static_cast<unsigned>((n + kPiece - 1) / kPiece),
                            static_cast<unsigned>((h + kJoinCols - 1) / kJoinCols)),
                       dim3(256), 0, s, partial, l.ld_p, sorted, n, v, h, scale, accumulate, out,
                       ld_t);
}

// Rows a launch, with tx threads along a row.
template <typename F>
void over_rows(int64_t n, int64_t chunks, F launch) {
  const int tx = row_threads(chunks);
  const int64_t rows = 256 / tx;
  for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups * rows) {
    const int64_t m = n - r0 < kMaxGroups * rows ? n - r0 : kMaxGroups * rows;
    launch(dim3(static_cast<unsigned>((m + rows - 1) / rows),
                static_cast<unsigned>((chunks + tx - 1) / tx)),
           tx, r0, m);
  }
}

const void* tokens_at(Targets t, int64_t r0) {
  return static_cast<const char*>(t.p) + r0 * (t.is32 ? 4 : 8);
}

template <typename T>
void embedding_typed(const void* table, int64_t ld_t, int64_t v, int64_t h, Targets tokens,
                     int64_t n, int64_t ignore, float scale, void* out, int64_t ld_o,
                     hipStream_t s) {
  const bool vec = fits16(table, ld_t, sizeof(T)) && fits16(out, ld_o, sizeof(T));
  auto kern = vec ? embedding_kernel<T, true> : embedding_kernel<T, false>;
  over_rows(n, (h + kE - 1) / kE, [&](dim3 grid, int tx, int64_t r0, int64_t m) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, static_cast<const T*>(table), ld_t, v, h,
                       tokens_at(tokens, r0), tokens.is32, m, ignore, scale, tx,
                       static_cast<T*>(out) + r0 * ld_o, ld_o);
  });
}

template <typename T>
void embedding_fp4_typed(const uint8_t* data, int64_t ld_d, const uint8_t* scales, int64_t ld_s,
                         int64_t v, int64_t h, Targets tokens, int64_t n, int64_t ignore,
                         float scale, void* out, int64_t ld_o, hipStream_t s) {
  const bool vec = fits16(out, ld_o, sizeof(T));
  auto kern = vec ? embedding_fp4_kernel<T, true> : embedding_fp4_kernel<T, false>;
  over_rows(n, h / kE, [&](dim3 grid, int tx, int64_t r0, int64_t m) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, data, ld_d, scales, ld_s, v, h,
                       tokens_at(tokens, r0), tokens.is32, m, ignore, scale, tx,
                       static_cast<T*>(out) + r0 * ld_o, ld_o);
  });
}

}  // namespace

void launch_embedding(int dtype, const void* table, int64_t ld_t, int64_t v, int64_t h,
                      Targets tokens, int64_t n, int64_t ignore, float scale, void* out,
                      int64_t ld_o, hipStream_t s) {
  auto run = dtype == kF32 ? embedding_typed<float>
             : dtype == kF16 ? embedding_typed<_Float16> : embedding_typed<uint16_t>;
  run(table, ld_t, v, h, tokens, n, ignore, scale, out, ld_o, s);
}

void launch_embedding_fp4(const uint8_t* data, int64_t ld_d, const uint8_t* scales, int64_t ld_s,
                          int64_t v, int64_t h, Targets tokens, int64_t n, int64_t ignore,
                          float scale, int out_dtype, void* out, int64_t ld_o, hipStream_t s) {
  auto run = out_dtype == kF32 ? embedding_fp4_typed<float>
             : out_dtype == kF16 ? embedding_fp4_typed<_Float16> : embedding_fp4_typed<uint16_t>;
  run(data, ld_d, scales, ld_s, v, h, tokens, n, ignore, scale, out, ld_o, s);
}

int64_t embedding_bwd_bytes(int64_t n, int64_t v, int64_t h) {
  (void)v;
  return bwd_layout(n, h).total;
}

void launch_embedding_bwd(int dtype, const void* dy, int64_t ld_y, Targets tokens, int64_t n,
                          int64_t v, int64_t h, int64_t ignore, float scale, bool f32_out,
                          bool accumulate, void* dtable, int64_t ld_t, char* ws, hipStream_t s) {
  auto run = dtype == kF32   ? bwd_typed<float, float>
             : dtype == kF16 ? (f32_out ? bwd_typed<_Float16, float> : bwd_typed<_Float16, _Float16>)
                             : (f32_out ? bwd_typed<uint16_t, float> : bwd_typed<uint16_t, uint16_t>);
  run(dy, ld_y, tokens, n, v, h, ignore, scale, accumulate, dtable, ld_t, ws, s);
}

}  // namespace itl
