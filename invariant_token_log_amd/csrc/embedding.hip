// Embedding lookup with scaling, from rows of any type or in 4 bits, and the
// table's gradient by sorted tokens, on gfx950.
//
//   y[i] = rne(scale E[t_i])
//   dE[t] = rne([dE[t] +] scale sum over i ascending with t_i = t of dy[i])
//
// The lookup is bound by memory: 16-byte accesses, a row's column chunks side by
// side, several rows a thread.
//
// The gradient sorts the tokens with their positions, so that the occurrences of
// a token form a run in ascending position, and sums every run in fp32:
//   1. embed_sort_kernel: tiles of 2048 tokens, a workgroup each, a bitonic
//      network in registers, lane moves and LDS (no order-dependent atomics, so
//      the same bits every time).  More than one tile: embed_merge_kernel merges
//      eight at a time, placing every token by binary searches in the others.
//   2. embed_sum_kernel: a wave for every piece of 32 occurrences; a run of one
//      piece goes straight to the table, a longer one leaves a partial row a
//      piece.
//   3. embed_join_kernel: adds the partial rows of the longer runs: eight
//      chains of every eighth piece, then the chains in order.
// A row of the gradient depends on its token's own occurrences and their
// order, not on the batch around them.
// Without accumulation the rows of absent tokens are written with zeros, which
// with a large vocabulary is most of the work: beside the sort and the last merge
// workgroups clear the table's first rows whole, beside the sums the absent
// rows of the rest.
#include "embedding.h"

#include <type_traits>

#include "fp4.h"
#include "row_device.h"

namespace itl {

namespace {

// Rows a thread takes when whole 16-byte accesses of one row a thread would make
// more than kLookupGroups workgroups, their loads in flight together.  V = 151936, H = 4096, one,
// two, four, eight rows, us: 16384 bf16 rows 44.5, 40.1, 41.3, 43.0, from 4 bits 49.5,
// 45.8, 42.9, 44.7; 4096 from 4 bits 14.6, 13.9, 13.6, 14.3 (the floors are 41.6, 26.4
// and 6.6 at 6.45 TB/s; the tokens' most frequent rows come from the caches).  16 rows
// take 2.6 us with one and 3.0 with two, unaligned rows 5 to 10% longer with two.
constexpr int kLookupRows = 2, kLookupRowsFp4 = 4, kLookupGroups = 4096;

template <typename T, bool VEC, int R>
__global__ __launch_bounds__(256) void embedding_kernel(const T* __restrict__ table, int64_t ld_t,
                                                        int64_t v, int64_t h,
                                                        const void* __restrict__ tok,
                                                        int32_t tok32, int64_t n, int64_t ignore,
                                                        float scale, int tx, T* __restrict__ out,
                                                        int64_t ld_o) {
  const Targets tokens{tok, tok32};
  const int64_t rows = 256 / tx;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * R * rows + threadIdx.x / tx;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * tx + threadIdx.x % tx) * kE;
  if (r0 >= n || c >= h) return;
  int64_t t[R];
  Raw<T> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) t[i] = tokens[min(r0 + i * rows, n - 1)];
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (t[i] >= 0 && t[i] < v && t[i] != ignore)
      raw[i] = load_raw<T, VEC>(table + t[i] * ld_t, c, h);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * rows;
    float x[kE];
    if (t[i] >= 0 && t[i] < v && t[i] != ignore) {
      widen_raw<T>(raw[i], x);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] = x[e] * scale;
    } else {
      const float fill = t[i] == ignore ? 0.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] = fill;
    }
    if (r < n) store_raw<T, VEC>(out + r * ld_o, c, h, round_raw<T>(x));
  }
}

template <typename T, bool VEC, int R>
__global__ __launch_bounds__(256) void embedding_fp4_kernel(
    const uint8_t* __restrict__ data, int64_t ld_d, const uint8_t* __restrict__ scales,
    int64_t ld_s, int64_t v, int64_t h, const void* __restrict__ tok, int32_t tok32, int64_t n,
    int64_t ignore, float scale, int tx, T* __restrict__ out, int64_t ld_o) {
  const Targets tokens{tok, tok32};
  const int64_t rows = 256 / tx;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * R * rows + threadIdx.x / tx;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * tx + threadIdx.x % tx) * kE;
  if (r0 >= n || c >= h) return;
  int64_t t[R];
  uint32_t q[R];
  uint8_t sb[R];
#pragma unroll
  for (int i = 0; i < R; ++i) t[i] = tokens[min(r0 + i * rows, n - 1)];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    q[i] = sb[i] = 0;
    if (t[i] >= 0 && t[i] < v && t[i] != ignore) {
      q[i] = *reinterpret_cast<const uint32_t*>(data + t[i] * ld_d + c / 2);
      sb[i] = scales[t[i] * ld_s + c / kFp4Group];
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t r = r0 + i * rows;
    float x[kE];
    if (t[i] >= 0 && t[i] < v && t[i] != ignore) {
      const float s = fp4_scale(sb[i]);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] = fp4_value(q[i] >> (4 * e)) * s * scale;
    } else {
      const float fill = t[i] == ignore ? 0.0f : __uint_as_float(0x7fc00000u);
#pragma unroll
      for (int e = 0; e < kE; ++e) x[e] = fill;
    }
    if (r < n) store_raw<T, VEC>(out + r * ld_o, c, h, round_raw<T>(x));
  }
}

// ---------------------------------------------------------------------------
// Sort.
// ---------------------------------------------------------------------------
constexpr int kTile = 2048;      // tokens a workgroup sorts
constexpr int kSortThreads = 512;
constexpr int kPer = kTile / kSortThreads;  // tokens a thread: 4 in a row
constexpr int kPiece = 32;       // occurrences a wave adds

// The run of slot i's token: where it starts, and the token itself (v: left
// out, at the end).
struct Sorted {
  uint32_t* id;
  uint32_t* pos;
  uint32_t* start;
};

// The value of lane ^ O, by lane moves within rows of 16 and swaps of rows.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xF, 0xF, true));
}
template <int O>
__device__ __forceinline__ uint32_t lane_xor(uint32_t x) {
  if constexpr (O == 1) return dpp_u32<kDppXor1>(x);
  if constexpr (O == 2) return dpp_u32<kDppXor2>(x);
  if constexpr (O == 4) return dpp_u32<0x1B>(dpp_u32<kDppRowHalfMirror>(x));  // i ^ 7 ^ 3
  if constexpr (O == 8) return dpp_u32<kDppRowRor8>(x);
  if constexpr (O == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return threadIdx.x & 16 ? r[0] : r[1];
  }
  if constexpr (O == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return threadIdx.x & 32 ? r[0] : r[1];
  }
}
template <int O>
__device__ __forceinline__ uint64_t lane_xor(uint64_t x) {
  return static_cast<uint64_t>(lane_xor<O>(static_cast<uint32_t>(x >> 32))) << 32 |
         lane_xor<O>(static_cast<uint32_t>(x));
}

// Ascending bitonic sort of the workgroup's keys, thread t holding keys 4 t ..;
// only the stages that `count` keys need (the others are the greatest).  buf:
// kTile keys of LDS.
template <typename K>
__device__ __forceinline__ void sort_tile(K (&key)[kPer], K* buf, int count) {
  const int t = threadIdx.x;
  auto keep = [&](K& mine, K other, bool low) { mine = (mine < other) == low ? mine : other; };
  for (int size = 2; size < 2 * count && size <= kTile; size *= 2) {
    const bool up = ((kPer * t) & size) == 0;
    for (int s = size / 2; s >= kPer * kWave; s /= 2) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kPer; ++j) buf[j * kSortThreads + t] = key[j];
      __syncthreads();
      const int o = t ^ (s / kPer);
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        keep(key[j], buf[j * kSortThreads + o], ((kPer * t & s) == 0) == up);
    }
#define ITL_LANES(O)                                                                            \
  if (size >= 2 * kPer * O) {                                                                   \
    const bool low = ((t & O) == 0) == up;                                                      \
    _Pragma("unroll") for (int j = 0; j < kPer; ++j) keep(key[j], lane_xor<O>(key[j]), low);    \
  }
    ITL_LANES(32) ITL_LANES(16) ITL_LANES(8) ITL_LANES(4) ITL_LANES(2) ITL_LANES(1)
#undef ITL_LANES
    auto order = [&](int a, int b) {
      const K x = key[a], y = key[b];
      const bool swap = (x > y) == (((kPer * t + a) & size) == 0);
      key[a] = swap ? y : x;
      key[b] = swap ? x : y;
    };
    if (size >= 4) {
      order(0, 2);
      order(1, 3);
    }
    order(0, 1);
    order(2, 3);
  }
}

// Zeros in `bytes` bytes (even) from p on, by `count` threads.
__device__ __forceinline__ void zero_bytes(char* p, int64_t bytes, int t, int count) {
  const int64_t head = min((16 - static_cast<int64_t>(reinterpret_cast<uintptr_t>(p) % 16)) % 16,
                           bytes);
  const int64_t body = (bytes - head) / 16;
  for (int64_t i = 2 * t; i < head; i += 2 * count) *reinterpret_cast<uint16_t*>(p + i) = 0;
  uint4* q = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = t; i < body; i += count) q[i] = make_uint4(0, 0, 0, 0);
  for (int64_t i = head + 16 * body + 2 * t; i < bytes; i += 2 * count)
    *reinterpret_cast<uint16_t*>(p + i) = 0;
}

// Rows [begin, end) of the table, which workgroups beside another kernel's clear:
// `step` rows each, from workgroup `first` on.  (A launch that waits for one
// workgroup's sort would leave the memory idle.)
struct Clear {
  char* table;
  int64_t ld, row_bytes;  // bytes
  int64_t begin, end;
  int first, step;
};
__device__ __forceinline__ void clear_rows(const Clear& c, int threads) {
  const int64_t block = static_cast<int>(blockIdx.x) - c.first;
  const int64_t r0 = c.begin + block * c.step;
  const int64_t r1 = min(r0 + c.step, c.end);
  if (c.ld == c.row_bytes) {
    zero_bytes(c.table + r0 * c.ld, (r1 - r0) * c.ld, threadIdx.x, threads);
    return;
  }
  for (int64_t r = r0 + threadIdx.x / kWave; r < r1; r += threads / kWave)
    zero_bytes(c.table + r * c.ld, c.row_bytes, threadIdx.x % kWave, kWave);
}

// Tile blockIdx.x of the tokens.  Keys are (token, position in the tile), the
// token of an entry that is left out being v.  One tile: the sorted arrays; more:
// the tile's sorted keys (token << 32 | position) for embed_merge_kernel.
// SMALL: v < 2^20 - 1, so that a key fits 32 bits.
template <bool SMALL>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(
    const void* __restrict__ tok, int32_t tok32, int64_t n, int64_t v, int64_t ignore, Sorted out,
    uint64_t* __restrict__ tiles, Clear clear) {
  using K = typename std::conditional<SMALL, uint32_t, uint64_t>::type;
  constexpr int kShift = SMALL ? 12 : 32;
  __shared__ K buf[kTile];
  if (static_cast<int>(blockIdx.x) >= clear.first) return clear_rows(clear, kSortThreads);
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

// Merges groups of eight sorted runs of `width` keys: eight lanes a key, each
// searching one run of the group for it.  (Keys are distinct, so the number of
// smaller ones is the place.)  LAST, one group: the sorted arrays, a token's
// first key searched for too.
constexpr int kFan = 8, kRankKeys = 256 / kFan;

template <bool LAST>
__global__ __launch_bounds__(256) void embed_merge_kernel(const uint64_t* __restrict__ runs,
                                                          int64_t n, int64_t width,
                                                          uint64_t* __restrict__ to, Sorted out,
                                                          Clear clear) {
  if (static_cast<int>(blockIdx.x) >= clear.first) return clear_rows(clear, 256);
  const int sub = threadIdx.x % kFan;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kRankKeys + threadIdx.x / kFan;
  const uint64_t key = runs[i < n ? i : n - 1], first = key >> 32 << 32;
  const int64_t base = (i < n ? i : n - 1) / (kFan * width) * (kFan * width);
  const int64_t b = base + sub * width;
  uint32_t rank = 0, start = 0;
  if (b < n) {
    const uint32_t count = static_cast<uint32_t>(n - b < width ? n - b : width);
    const uint64_t* t = runs + b;
    for (uint32_t step = static_cast<uint32_t>(width) / 2; step; step /= 2) {  // width - 1 at most
      const uint32_t x = rank + step - 1, y = start + step - 1;
      const uint64_t kx = t[min(x, count - 1)], ky = LAST ? t[min(y, count - 1)] : 0;
      if (x < count && kx < key) rank += step;
      if (LAST && y < count && ky < first) start += step;
    }
    if (count == width) {  // all of a whole run
      const uint64_t k = t[width - 1];
      if (rank == width - 1 && k < key) ++rank;
      if (LAST && start == width - 1 && k < first) ++start;
    }
  }
#define ITL_ADD(O)                  \
  rank += lane_xor<O>(rank);        \
  start += lane_xor<O>(start);
  ITL_ADD(1) ITL_ADD(2) ITL_ADD(4)
#undef ITL_ADD
  if (sub || i >= n) return;
  if constexpr (LAST) {
    out.id[rank] = static_cast<uint32_t>(key >> 32);
    out.pos[rank] = static_cast<uint32_t>(key);
    out.start[rank] = start;
  } else {
    to[base + rank] = key;
  }
}

// ---------------------------------------------------------------------------
// Sums.
// ---------------------------------------------------------------------------
// The partial row of the piece at slot s of a run of several pieces.  In a
// window of kPiece slots at most one such run goes on and one begins.
__device__ __forceinline__ int64_t partial_row(int64_t s, int64_t start) {
  return 2 * (s / kPiece) + (s != start);
}

// The table's element c: scale a, added to what is there with accumulate.
template <typename U>
__device__ __forceinline__ void table_store_one(U* row, int64_t c, float scale, bool accumulate,
                                                float a) {
  store_one<U>(row + c, accumulate ? fmaf(a, scale, Elt<U>::load(row, c)) : a * scale);
}
// Its whole chunk from element c on.
template <typename U, bool VEC>
__device__ __forceinline__ void table_store(U* row, int64_t c, float scale, bool accumulate,
                                            float (&a)[kE]) {
  if (accumulate) {
    float old[kE];
    widen_raw<U>(load_raw<U, VEC>(row, c, c + kE), old);
#pragma unroll
    for (int e = 0; e < kE; ++e) a[e] = fmaf(a[e], scale, old[e]);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e) a[e] = a[e] * scale;
  }
  store_raw<U, VEC>(row, c, c + kE, round_raw<U>(a));
}

// acc += R rows of the wave's piece, from its row i0 on; cl: where the lane's
// chunks are read.
template <typename T, int R, int CH, bool VEC, bool TINY>
__device__ __forceinline__ void add_rows(const T* __restrict__ dy, int64_t ld_y, uint32_t pos,
                                         int i0, const int64_t (&cl)[CH], int64_t h,
                                         float (&acc)[CH][kE]) {
  Raw<T> x[R][CH];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const T* row = dy + static_cast<int64_t>(__builtin_amdgcn_readlane(pos, i0 + i)) * ld_y;
#pragma unroll
    for (int c = 0; c < CH; ++c)
      x[i][c] = load_raw<T, VEC>(row, cl[c], TINY ? h : cl[c] + kE);
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float p[kE];
      widen_raw<T>(x[i][c], p);
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[c][e] = acc[c][e] + p[e];
    }
}

// A wave a slot; those that begin a piece add its rows, `span` columns of them,
// CH chunks of 8 a lane at a time.  A chunk that would pass the row's end is
// read from its last 8 elements and stores its own; rows of fewer than 8 are
// TINY.
template <typename T, typename U, int CH, bool VEC, bool TINY>
__device__ __forceinline__ void sum_slot(const T* __restrict__ dy, int64_t ld_y,
                                         const Sorted& sorted, int64_t s, int64_t n, int64_t v,
                                         int64_t h, int64_t c_begin, int64_t c_end, float scale,
                                         bool accumulate, U* dtable, int64_t ld_t, float* partial,
                                         int64_t ld_p) {
  const int lane = threadIdx.x % kWave;
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
  for (int64_t c0 = c_begin; c0 < c_end; c0 += CH * kWave * kE) {
    int64_t cl[CH];
    float acc[CH][kE];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = c0 + (c * kWave + lane) * kE;
      cl[c] = TINY ? col : col + kE <= h ? col : h - kE;
#pragma unroll
      for (int e = 0; e < kE; ++e) acc[c][e] = 0.0f;
    }
    int i = 0;
    for (; i + 8 <= count; i += 8) add_rows<T, 8, CH, VEC, TINY>(dy, ld_y, pos, i, cl, h, acc);
    if (count & 4) {
      add_rows<T, 4, CH, VEC, TINY>(dy, ld_y, pos, i, cl, h, acc);
      i += 4;
    }
    if (count & 2) {
      add_rows<T, 2, CH, VEC, TINY>(dy, ld_y, pos, i, cl, h, acc);
      i += 2;
    }
    if (count & 1) add_rows<T, 1, CH, VEC, TINY>(dy, ld_y, pos, i, cl, h, acc);
    U* row = dtable + static_cast<int64_t>(id) * ld_t;
    float* part = partial + partial_row(s, start) * ld_p;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int64_t col = c0 + (c * kWave + lane) * kE;
      if (col >= h) break;
      if (!TINY && col + kE <= h) {
        if (pieces) {
          float4* to = reinterpret_cast<float4*>(part + col);
          to[0] = make_float4(acc[c][0], acc[c][1], acc[c][2], acc[c][3]);
          to[1] = make_float4(acc[c][4], acc[c][5], acc[c][6], acc[c][7]);
        } else {
          table_store<U, VEC>(row, col, scale, accumulate, acc[c]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kE; ++e) {
          const int64_t k = cl[c] + e;
          if (k < col || k >= h) continue;
          if (pieces)
            part[k] = acc[c][e];
          else
            table_store_one<U>(row, k, scale, accumulate, acc[c][e]);
        }
      }
    }
  }
}

// Zeros in the rows of absent tokens, 64 rows from v0 on.
template <typename U>
__device__ __forceinline__ void zero_absent(const uint32_t* __restrict__ id, int64_t n, int64_t v0,
                                            int64_t v, int64_t h, U* dtable, int64_t ld_t) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t row = v0 + lane;
  int64_t lo = 0, hi = n;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (id[mid] < row) lo = mid + 1; else hi = mid;
  }
  const uint64_t absent = __builtin_amdgcn_ballot_w64(row < v && !(lo < n && id[lo] == row));
  const int64_t row_bytes = h * static_cast<int64_t>(sizeof(U));
  // Rows without gaps: a run of absent ones at once (512 tokens, 151936 x 256 bf16: 9
  // us for the kernel, 14 row by row; no difference for rows of 4096).
  if (ld_t == h) {
    for (uint64_t left = absent; left;) {
      const int first = __builtin_ctzll(left);
      const uint64_t ends = ~(left >> first);
      const int count = ends ? __builtin_ctzll(ends) : kWave;
      zero_bytes(reinterpret_cast<char*>(dtable + (v0 + first) * ld_t), count * row_bytes,
                 threadIdx.x, 256);
      left = first + count < kWave ? left >> (first + count) << (first + count) : 0;
    }
    return;
  }
  for (int i = wave; i < kWave; i += 4)
    if ((absent >> i) & 1)
      zero_bytes(reinterpret_cast<char*>(dtable + (v0 + i) * ld_t), row_bytes, lane, kWave);
}

// Workgroups below sum_groups: four slots each, `splits` column spans; the others
// clear the absent rows from row z0 on.  In one launch the sums, which wait for
// a chain of loads, run beside the zeros, which fill the memory's time.
template <typename T, typename U, int CH, bool VEC, bool TINY>
__global__ __launch_bounds__(256) void embed_sum_kernel(const T* __restrict__ dy, int64_t ld_y,
                                                        Sorted sorted, int64_t n, int64_t v,
                                                        int64_t h, int splits, int64_t span,
                                                        int64_t sum_groups, float scale,
                                                        bool accumulate, U* __restrict__ dtable,
                                                        int64_t ld_t, float* __restrict__ partial,
                                                        int64_t ld_p, int64_t z0) {
  const int64_t g = blockIdx.x;
  if (g < sum_groups) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t s = g / splits * 4 + wave, c0 = g % splits * span;
    if (s < n)
      sum_slot<T, U, CH, VEC, TINY>(dy, ld_y, sorted, s, n, v, h, c0,
                                    c0 + span < h ? c0 + span : h, scale, accumulate, dtable, ld_t,
                                    partial, ld_p);
    return;
  }
  const int64_t step = (gridDim.x - sum_groups) * kWave;
  for (int64_t v0 = z0 + (g - sum_groups) * kWave; v0 < v; v0 += step)
    zero_absent<U>(sorted.id, n, v0, v, h, dtable, ld_t);
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
  U* row = dtable + static_cast<int64_t>(id) * ld_t;
  if (col + kE <= h) {
    table_store<U, VEC>(row, col, scale, accumulate, a);
  } else {
#pragma unroll
    for (int e = 0; e < kE; ++e)
      if (col + e < h) table_store_one<U>(row, col + e, scale, accumulate, a[e]);
  }
}

// Workspace: id, pos, start [n]; the tiles' keys when there are several, twice
// when they are merged more than once; the partial rows.
struct BwdLayout {
  int64_t id, pos, start, tiles, tiles2, partial, ld_p, total;
};
BwdLayout bwd_layout(int64_t n, int64_t h) {
  auto round = [](int64_t x) { return (x + 255) / 256 * 256; };
  BwdLayout l;
  l.ld_p = (h + 7) / 8 * 8;
  l.id = 0;
  l.pos = round(4 * n);
  l.start = 2 * l.pos;
  l.tiles = 3 * l.pos;
  l.tiles2 = l.tiles + (n > kTile ? round(8 * n) : 0);
  l.partial = l.tiles2 + (n > kFan * kTile ? round(8 * n) : 0);
  // runs of several pieces need more than kPiece tokens
  const int64_t rows = n > kPiece ? 2 * ((n + kPiece - 1) / kPiece) : 0;
  l.total = l.partial + round(rows * l.ld_p * 4);
  return l;
}

// Bytes that workgroups beside the sort, and beside the last merge, clear: about
// what the memory takes in their time (16384 tokens: 11.5 us each with them).
constexpr int64_t kSortClears = int64_t{40} << 20, kRankClears = int64_t{32} << 20;

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
  const int size = sizeof(U);
  const bool vec_out = fits16(dtable, ld_t, size);
  // Rows below `clear.end` are cleared whole before the sums are written.
  Clear clear{static_cast<char*>(dtable), ld_t * size, h * size, 0, 0, 0, 0};
  // Workgroups for the next `bytes` bytes, about 256 KiB each.
  auto clears = [&](int64_t bytes, int first) -> unsigned {
    clear.first = first;
    if (accumulate) return 0;
    const int64_t rows = bytes / clear.row_bytes, left = v - clear.end;
    clear.begin = clear.end;
    clear.end += rows < left ? rows : left;
    const int64_t step = (int64_t{256} << 10) / clear.row_bytes;
    clear.step = step > 1 ? static_cast<int>(step) : 1;
    return static_cast<unsigned>((clear.end - clear.begin + clear.step - 1) / clear.step);
  };
  if (n) {
    const unsigned groups = static_cast<unsigned>((n + kTile - 1) / kTile);
    const unsigned more = clears(kSortClears, static_cast<int>(groups));
    auto sort = v < (1 << 20) - 1 ? embed_sort_kernel<true> : embed_sort_kernel<false>;
    hipLaunchKernelGGL(sort, dim3(groups + more), dim3(kSortThreads), 0, s, tokens.p, tokens.is32,
                       n, v, ignore, sorted, tiles, clear);
  }
  if (tiles) {
    const unsigned groups = static_cast<unsigned>((n + kRankKeys - 1) / kRankKeys);
    uint64_t* other = reinterpret_cast<uint64_t*>(ws + l.tiles2);
    int64_t width = kTile;
    for (; kFan * width < n; width *= kFan) {
      clear.first = static_cast<int>(groups);
      hipLaunchKernelGGL(embed_merge_kernel<false>, dim3(groups), dim3(256), 0, s, tiles, n, width,
                         other, sorted, clear);
      uint64_t* t = tiles;
      tiles = other;
      other = t;
    }
    const unsigned more = clears(kRankClears, static_cast<int>(groups));
    hipLaunchKernelGGL(embed_merge_kernel<true>, dim3(groups + more), dim3(256), 0, s, tiles, n,
                       width, other, sorted, clear);
  }
  const bool vec = vec_out && fits16(dy, ld_y, sizeof(T)) && h % kE == 0;
  constexpr int CH = sizeof(T) == 4 ? 1 : 2;  // 32 bytes a lane and row
  auto kern = h < kE ? embed_sum_kernel<T, U, CH, false, true>
              : vec  ? embed_sum_kernel<T, U, CH, true, false>
                     : embed_sum_kernel<T, U, CH, false, false>;
  // A slot's columns are split while there are fewer waves than the GPU holds.
  const int64_t unit = CH * kWave * kE, units = (h + unit - 1) / unit;
  int64_t splits = n ? 8192 / n : 1;
  splits = splits < 1 ? 1 : splits > units ? units : splits;
  const int64_t span = (units + splits - 1) / splits * unit;
  const int64_t sum_groups = (n + 3) / 4 * splits;
  const int64_t z0 = accumulate ? v : clear.end;
  const int64_t absent = (v - z0 + kWave - 1) / kWave;
  const int64_t total = sum_groups + (absent < kMaxGroups ? absent : kMaxGroups);
  if (total)
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(total)), dim3(256), 0, s,
                       static_cast<const T*>(dy), ld_y, sorted, n, v, h, static_cast<int>(splits),
                       span, sum_groups, scale, accumulate, out, ld_t, partial, l.ld_p, z0);
  if (n > kPiece)
    hipLaunchKernelGGL((vec_out ? embed_join_kernel<U, true> : embed_join_kernel<U, false>),
                       dim3(static_cast<unsigned>((n + kPiece - 1) / kPiece),
                            static_cast<unsigned>((h + kJoinCols - 1) / kJoinCols)),
                       dim3(256), 0, s, partial, l.ld_p, sorted, n, v, h, scale, accumulate, out,
                       ld_t);
}

// Rows a launch, with tx threads along a row and one or `several` rows a thread.
template <typename F>
void over_rows(int64_t n, int64_t chunks, int several, bool vec, F launch) {
  const int tx = row_threads(chunks);
  const int64_t across = (chunks + tx - 1) / tx;
  const bool more = vec && n * tx / 256 * across > kLookupGroups;
  const int64_t rows = 256 / tx * (more ? several : 1);
  for (int64_t r0 = 0; r0 < n; r0 += kMaxGroups * rows) {
    const int64_t m = n - r0 < kMaxGroups * rows ? n - r0 : kMaxGroups * rows;
    launch(more, dim3(static_cast<unsigned>((m + rows - 1) / rows), static_cast<unsigned>(across)),
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
  over_rows(n, (h + kE - 1) / kE, kLookupRows, vec,
            [&](bool more, dim3 grid, int tx, int64_t r0, int64_t m) {
    auto kern = more ? embedding_kernel<T, true, kLookupRows>
                     : vec ? embedding_kernel<T, true, 1> : embedding_kernel<T, false, 1>;
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
  over_rows(n, h / kE, kLookupRowsFp4, vec,
            [&](bool more, dim3 grid, int tx, int64_t r0, int64_t m) {
    auto kern = more ? embedding_fp4_kernel<T, true, kLookupRowsFp4>
                     : vec ? embedding_fp4_kernel<T, true, 1> : embedding_fp4_kernel<T, false, 1>;
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
             : dtype == kF16 ? f32_out ? bwd_typed<_Float16, float> : bwd_typed<_Float16, _Float16>
             : f32_out       ? bwd_typed<uint16_t, float>
                             : bwd_typed<uint16_t, uint16_t>;
  run(dy, ld_y, tokens, n, v, h, ignore, scale, accumulate, dtable, ld_t, ws, s);
}

}  // namespace itl
