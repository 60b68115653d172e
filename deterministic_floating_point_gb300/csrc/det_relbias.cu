// det_relative_bias and det_relative_bias_backward (include/det_model.h).
//
// The bias of a (query i, key j) pair depends on the diagonal j - i alone.
// Forward: every output is one table entry.  Backward: the sum over a bucket
// is taken by diagonals (within a tile of queries and keys), then over the
// bucket's diagonals, which are neighbours (a bucket is one interval of
// distances), then over the tiles.  The order of the additions is fixed by
// indices, so neither strides nor alignment nor the launch change the bits.
#include "det_model.cuh"

#include <algorithm>
#include <type_traits>

namespace det {
namespace {

// The distances, as key position - query position, of the pairs of a problem.
struct Distances {
  const int32_t* bounds;
  int num_bounds;
  int bidirectional;
  int first;   // the distance of diagonal 0: key 0, last query

  __device__ __forceinline__ int bounds_at_most(int n) const {
    int lo = 0, hi = num_bounds;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (bounds[mid] <= n) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ int bucket(int r) const {
    if (!bidirectional) return bounds_at_most(r < 0 ? -r : 0);
    return bounds_at_most(r < 0 ? -r : r) + (r > 0 ? num_bounds + 1 : 0);
  }
  // Distances [lo, hi) of bucket k, clipped to [from, to).
  __device__ __forceinline__ void interval(int k, int from, int to, int& lo, int& hi) const {
    const bool after = k > num_bounds;   // keys after the query (bidirectional)
    const int b = after ? k - num_bounds - 1 : k;
    const int near = b > 0 ? max(bounds[b - 1], 0) : 0;                  // least |distance|
    const int far = b < num_bounds ? bounds[b] : 0x7fffffff;   // first |distance| beyond
    if (far <= near) {
      lo = hi = from;
      return;
    }
    if (after) {
      lo = max(near, 1);
      hi = far;
    } else {
      lo = 1 - far;
      hi = near == 0 && !bidirectional ? 0x7fffffff : 1 - near;
    }
    lo = max(lo, from);
    hi = max(min(hi, to), lo);
  }
};

// Few rows (at most kDirectRows): a thread per pair, its bucket searched.
constexpr int kDirectRows = 8;
template <typename T>
__global__ void __launch_bounds__(256)
bias_direct_kernel(const void* table, int table_dtype, int heads, Distances dist, int q_len, int k_len,
                   T* __restrict__ out) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x, q = blockIdx.y, h = blockIdx.z;
  dep_wait();   // launched early: all loads come after, and none is a read-only one, which need not
  dep_launch();
  if (j >= k_len) return;
  const int k = dist.bucket(j - q + (q_len - 1) + dist.first);
  out[((long long)h * q_len + q) * k_len + j] = from_f32<T>(load_as_f32(table, (long long)k * heads + h, table_dtype));
}

// Otherwise a CTA writes 32 rows by 128 units of 16 bytes (aligned rows in 32
// bits: 16 by 256) from the strip of diagonals that they cross, kept
// in shared memory (in 16-bit types as the pairs of diagonals d, d + 1 that make
// up a word of the output).  A row's
// units start where its memory is 16-byte aligned, so every store but those
// at a row's ends is a whole unit, whatever the row length.  Word u of the strip
// lies at u + u / U, U elements to a unit: threads are U diagonals apart, which
// then is an odd number of banks.
//
// Bound by the writes.  What matters is how much of the output is being
// written at a time (16 x 4,096 x 4,096 bf16, threads x rows of a CTA: 128 x 128 117 us,
// 256 x 64 98, 256 x 32 93, 128 x 32 86, and launched early 83 to 85, 93 to 95% of
// the measured copy bandwidth; 8 x 4,096 x 4,096 f32: 256 x 16 81 us, 98%; torch's
// fill of the same bytes takes 136 us).  Rows of 4,097: 96 us.
template <typename T, bool ALIGNED> struct BiasTile {
  static constexpr int kThreads = sizeof(T) == 4 && ALIGNED ? 256 : 128, kRows = sizeof(T) == 4 && ALIGNED ? 16 : 32;
};

template <typename T> struct Out16;
template <> struct Out16<float> {
  static __device__ __forceinline__ unsigned word(float a, float) { return __float_as_uint(a); }
};
template <> struct Out16<__nv_bfloat16> {
  static __device__ __forceinline__ unsigned word(float a, float b) {
    return (unsigned)__bfloat16_as_ushort(__float2bfloat16_rn(a)) | ((unsigned)__bfloat16_as_ushort(__float2bfloat16_rn(b)) << 16);
  }
};
template <> struct Out16<__half> {
  static __device__ __forceinline__ unsigned word(float a, float b) {
    return (unsigned)__half_as_ushort(__float2half_rn(a)) | ((unsigned)__half_as_ushort(__float2half_rn(b)) << 16);
  }
};

template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(BiasTile<T, ALIGNED>::kThreads)
bias_strip_kernel(const void* table, int table_dtype, int heads, Distances dist, int q_len, int k_len,
                  T* __restrict__ out) {
  constexpr int E = 4 / sizeof(T);    // elements of a word
  constexpr int U = 16 / sizeof(T);   // elements of a unit
  constexpr int kBiasThreads = BiasTile<T, ALIGNED>::kThreads, kBiasRows = BiasTile<T, ALIGNED>::kRows;
  constexpr int kStrip = U * kBiasThreads + kBiasRows + 2 * U;
  __shared__ unsigned strip[kStrip + kStrip / U + 1];
  __shared__ float value[kStrip + 1];
  dep_wait();
  dep_launch();
  const int h = blockIdx.z, i0 = blockIdx.y * kBiasRows, c0 = blockIdx.x * kBiasThreads;
  const int rows = min(kBiasRows, q_len - i0);
  // strip[u] holds diagonal u + d0: key - query from U (c0 - 1) - (i0 + kBiasRows - 1) up
  const int d0 = U * (c0 - 1) - (i0 + kBiasRows - 1);
  const int base = d0 + (q_len - 1) + dist.first;   // distance of strip[0]
  for (int u = threadIdx.x; u <= kStrip; u += kBiasThreads)
    value[u] = load_as_f32(table, (long long)dist.bucket(base + u) * heads + h, table_dtype);
  __syncthreads();
  for (int u = threadIdx.x; u < kStrip; u += kBiasThreads) strip[u + u / U] = Out16<T>::word(value[u], value[u + 1]);
  __syncthreads();
  if constexpr (ALIGNED) {
    // Every row's units start at the same keys.  U rows of a thread's unit
    // cross 2 U - 1 diagonals: two runs of U words of the strip, of which the
    // next U rows need one more.
    const int j = U * (c0 - 1 + (int)threadIdx.x);
    if (j < 0 || j + U > k_len) return;   // a row holds whole units
    unsigned lo[U], hi[U];
    const unsigned* at = strip + (U + 1) * (threadIdx.x + kBiasRows / U);
#pragma unroll
    for (int x = 0; x < U; ++x) hi[x] = at[x];
    T* p = out + ((long long)h * q_len + i0) * k_len + j;
    for (int y0 = 0; y0 < rows; y0 += U) {
      at -= U + 1;
#pragma unroll
      for (int x = 0; x < U; ++x) lo[x] = at[x];
#pragma unroll
      for (int y = 0; y < U; ++y) {
        if (y0 + y < rows) {
          unsigned w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int k = U - 1 - y + x * E;
            w[x] = k < U ? lo[k] : hi[k - U];
          }
          *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
          p += k_len;
        }
      }
#pragma unroll
      for (int x = 0; x < U; ++x) hi[x] = lo[x];
    }
  } else {
#pragma unroll 4
    for (int y = 0; y < rows; ++y) {
      const int i = i0 + y;
      T* row = out + ((long long)h * q_len + i) * k_len;
      // keys before the row's first 16-byte boundary
      const int head = (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T);
      const int j = head + U * (c0 - 1 + (int)threadIdx.x);
      if (j >= k_len || j + U <= 0) continue;
      const int u = j - i - d0;
      unsigned w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) w[x] = strip[u + x * E + (u + x * E) / U];
      if (j >= 0 && j + U <= k_len) {
        *reinterpret_cast<uint4*>(row + j) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int x = 0; x < U; ++x) {
          if (j + x < 0 || j + x >= k_len) continue;
          if constexpr (E == 1) row[j + x] = __uint_as_float(w[x]);
          else reinterpret_cast<unsigned short*>(row)[j + x] = (unsigned short)(w[x / 2] >> (16 * (x & 1)));
        }
      }
    }
  }
}

struct GradView {
  long long stride_b, stride_h, stride_q;
  int batch, q_len, k_len;
  uintptr_t lo, hi;   // the bytes from the first element to the end of the last
};

// The gradient is cut into tiles of 64 queries by 248 diagonals, a warp each:
// lane l < 31 takes 8 neighbouring keys of 8 queries at a time and moves 8 keys
// on with every 8 queries, so its 64 pairs always lie on the same 15 diagonals
// (the key within the eight less the query within the eight), whose sums
// stay in registers.  Lane 31 takes no pairs: where eights are not 16-byte
// aligned it reads what lane 30 lacks.
//
// Bound by the reads: one addition and one unpacking an element, 16 bytes a
// load, 4 KB a warp in flight (8 x 16 x 2,048 x 2,048 bf16 with the join 163 us, 97% of
// the measured copy bandwidth).  Unaligned rows shift their eights across
// lanes, 9 instructions an element instead of 4 (2,047 keys: 237 us;
// 3 x 12 x 509 x 1,531 f32: 28 us, of which the launches are a third).
constexpr int kTileRows = 64;
constexpr int kTileGroups = kTileRows / 8;
constexpr int kTileLanes = 31;
constexpr int kStripDiags = 8 * kTileLanes;
constexpr int kTileDiags = kStripDiags + 8;   // diagonals of a tile: the lanes' eights, and the 8 below
constexpr int kTileWarps = 4;                 // warps of a CTA

struct TileGrid {
  int row_blocks, strips;   // tiles along the queries and along the keys
  __host__ __device__ TileGrid(int q_len, int k_len)
      : row_blocks((q_len + kTileRows - 1) / kTileRows),
        strips(((k_len + 7) / 8 + kTileGroups + kTileLanes - 1) / kTileLanes) {}
  __host__ __device__ int per_matrix() const { return row_blocks * strips; }
  // First key eight of lane 0 in the tile's first group.
  __device__ __forceinline__ int first_eight(int strip) const { return strip * kTileLanes - kTileGroups; }
  // Key - query of the tile's diagonal 0.
  __device__ __forceinline__ int first_diagonal(int row_block, int strip) const {
    return 8 * first_eight(strip) - row_block * kTileRows - 8;
  }
};

template <typename T> struct Eight {   // 8 neighbouring elements as 32-bit words
  static constexpr int W = 8 * sizeof(T) / 4;
  unsigned w[W];
  __device__ __forceinline__ float get(int x) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[x]);
    const unsigned v = w[x >> 1];
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float((x & 1) ? (v & 0xffff0000u) : (v << 16));
    return __half2float(__ushort_as_half((unsigned short)((x & 1) ? (v >> 16) : v)));
  }
};

__device__ __forceinline__ uint4 load_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The 16-byte blocks from `at` up that make an eight when they are aligned.
template <typename T, bool ALIGNED> __device__ __forceinline__ Eight<T> load_blocks(uintptr_t at) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < Eight<T>::W; i += 4) {
    // (unaligned in 32 bits a sector is often halved between two of the loads:
    // kept in L1; 3 x 12 x 509 x 1531: 40 -> 29 us)
    const uint4 v = sizeof(T) == 4 && !ALIGNED ? reinterpret_cast<const uint4*>(at)[i / 4]
                                               : load_16(reinterpret_cast<const void*>(at + 4 * i));
    e.w[i] = v.x, e.w[i + 1] = v.y, e.w[i + 2] = v.z, e.w[i + 3] = v.w;
  }
  return e;
}
// The eight that starts `off` bytes (the same of every lane) into the lane's
// blocks and ends in the next lane's first.
template <typename T, int WORDS> __device__ __forceinline__ Eight<T> shift_eight_by(const Eight<T>& mine, bool half) {
  constexpr int W = Eight<T>::W;
  unsigned v[W + WORDS + 1];
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] = mine.w[i];
#pragma unroll
  for (int i = 0; i < WORDS; ++i) v[W + i] = __shfl_down_sync(0xffffffffu, mine.w[i], 1);
  Eight<T> e;
  if (sizeof(T) == 2 && half) {
    v[W + WORDS] = __shfl_down_sync(0xffffffffu, mine.w[WORDS], 1);
#pragma unroll
    for (int i = 0; i < W; ++i) e.w[i] = __funnelshift_r(v[WORDS + i], v[WORDS + i + 1], 16);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) e.w[i] = v[WORDS + i];
  }
  return e;
}
template <typename T> __device__ __forceinline__ Eight<T> shift_eight(const Eight<T>& mine, unsigned off) {
  const bool half = off & 2;
  switch (off >> 2) {
    case 0: return shift_eight_by<T, 0>(mine, half);
    case 1: return shift_eight_by<T, 1>(mine, half);
    case 2: return shift_eight_by<T, 2>(mine, half);
    default: return shift_eight_by<T, 3>(mine, half);
  }
}
// Elements j .. j + 7 of a row one by one, 0 outside [0, k_len).
template <typename T>
__device__ __forceinline__ Eight<T> load_singly(const T* row, int j, int k_len) {
  Eight<T> e;
#pragma unroll
  for (int i = 0; i < Eight<T>::W; ++i) e.w[i] = 0u;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    if (j + x < 0 || j + x >= k_len) continue;
    if constexpr (sizeof(T) == 4) e.w[x] = __float_as_uint(row[j + x]);
    else e.w[x >> 1] |= (unsigned)reinterpret_cast<const unsigned short*>(row)[j + x] << (16 * (x & 1));
  }
  return e;
}

// part[h][bucket][tile] = the tile's sum over the bucket, for the buckets
// that the tile's diagonals reach.
template <typename T, bool ALIGNED>
__global__ void __launch_bounds__(32 * kTileWarps, ALIGNED ? 4 : sizeof(T) == 4 ? 3 : 5)
bias_tiles_kernel(const T* grad, GradView g, Distances dist, int q_offset, int buckets, float* part) {
  __shared__ float sh[kTileWarps][kTileDiags];
  dep_wait();
  dep_launch();
  const TileGrid tiles(g.q_len, g.k_len);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int per_matrix = tiles.per_matrix(), per_head = per_matrix * g.batch;   // below 2^31: the launch checks
  const int tile = blockIdx.x * kTileWarps + warp, h = blockIdx.y;
  if (tile >= per_head) return;
  const int b = tile / per_matrix, in_matrix = tile - b * per_matrix;
  const int row_block = in_matrix / tiles.strips, strip = in_matrix - row_block * tiles.strips;

  const T* matrix = grad + b * g.stride_b + h * g.stride_h;
  const int i0 = row_block * kTileRows;
  int j = 8 * (tiles.first_eight(strip) + lane);
  float acc[15];
#pragma unroll
  for (int i = 0; i < 15; ++i) acc[i] = 0.0f;
  for (int i = i0; i < min(i0 + kTileRows, g.q_len); i += 8, j += 8) {
    const T* p = matrix + (long long)i * g.stride_q + j;
    const int count = min(8, g.q_len - i);
    const bool whole = j >= 0 && j + 8 <= g.k_len && lane < kTileLanes;
    const bool some = j + 8 > 0 && j < g.k_len && lane < kTileLanes;
    if constexpr (ALIGNED) {
      if (whole && count == 8) {
        Eight<T> e[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) e[y] = load_blocks<T, true>(reinterpret_cast<uintptr_t>(p + y * g.stride_q));
#pragma unroll
        for (int y = 0; y < 8; ++y)
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[x - y + 7] += e[y].get(x);
        continue;
      }
    } else if (count == 8) {
      // the blocks of all rows, where they hold some of the rows' keys and lie
      // in the matrices' memory
      const uintptr_t at = reinterpret_cast<uintptr_t>(p), step = sizeof(T) * g.stride_q;
      const uintptr_t top = at & ~(uintptr_t)15, bottom = (at + 7 * step) & ~(uintptr_t)15;
      Eight<T> e[8] = {};
      if (j > -16 && j < g.k_len + 8 && top >= g.lo && bottom + 4 * Eight<T>::W <= g.hi) {
#pragma unroll
        for (int y = 0; y < 8; ++y) e[y] = load_blocks<T, false>((at + y * step) & ~(uintptr_t)15);
      }
      // whether the next lane's do too
      const bool shifted = whole && top >= g.lo && bottom + 8 * Eight<T>::W <= g.hi;
      const unsigned off = __shfl_sync(0xffffffffu, (unsigned)at, 0);
      const unsigned off_step = (unsigned)step;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const Eight<T> f = shift_eight(e[y], (off + y * off_step) & 15);
        if (shifted) {
#pragma unroll
          for (int x = 0; x < 8; ++x) acc[x - y + 7] += f.get(x);
        }
      }
      if (shifted) continue;
    }
    if (!some) continue;
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      if (y >= count) break;
      const Eight<T> e = load_singly(p + y * g.stride_q - j, j, g.k_len);
#pragma unroll
      for (int x = 0; x < 8; ++x) acc[x - y + 7] += e.get(x);
    }
  }
  // the tile's diagonals: one's own 0 .. 7, then the 7 below on top of the
  // neighbour's
  float* diag = sh[warp];
  if (lane < 8) diag[lane] = 0.0f;
  if (lane < kTileLanes) {
#pragma unroll
    for (int s = 0; s < 8; ++s) diag[8 * (lane + 1) + s] = acc[s + 7];
  }
  __syncwarp();
  if (lane < kTileLanes) {
#pragma unroll
    for (int s = 1; s < 8; ++s) diag[8 * lane + s] += acc[s - 1];
  }
  __syncwarp();
  // The buckets of both signs, a lane each; a bucket of 32 diagonals or more
  // is added by the whole warp.
  const int from = tiles.first_diagonal(row_block, strip) - q_offset, to = from + kTileDiags;
  float* out = part + (long long)h * buckets * per_head + tile;
  for (int side = 0; side < 2; ++side) {
    // the least and the largest |distance| on this side of the query
    int k0, k1;
    if (side == 0) {
      if (from > 0 && dist.bidirectional) continue;
      k0 = dist.bounds_at_most(to - 1 < 0 ? 1 - to : 0);
      k1 = dist.bounds_at_most(from < 0 ? -from : 0);
    } else {
      if (to <= 1 || !dist.bidirectional) continue;
      k0 = dist.bounds_at_most(from > 1 ? from : 1) + dist.num_bounds + 1;
      k1 = dist.bounds_at_most(to - 1) + dist.num_bounds + 1;
    }
    for (int kb = k0; kb <= k1; kb += 32) {
      const int k = kb + lane;
      int lo = 0, hi = 0;
      if (k <= k1) {
        dist.interval(k, from, to, lo, hi);
        lo -= from;
        hi -= from;
      }
      unsigned wide = __ballot_sync(0xffffffffu, hi - lo >= 32);
      if (hi - lo < 32 && hi > lo) {
        float sum = 0.0f;
        for (int d = lo; d < hi; ++d) sum += diag[d];
        out[(long long)k * per_head] = sum;
      }
      while (wide) {
        const int owner = __ffs(wide) - 1;
        wide &= wide - 1;
        const int l = __shfl_sync(0xffffffffu, lo, owner), u = __shfl_sync(0xffffffffu, hi, owner);
        float sum = 0.0f;
        for (int d = l + lane; d < u; d += 32) sum += diag[d];
        sum = warp_pt(sum);
        if (lane == 0) out[(long long)(kb + owner) * per_head] = sum;
      }
    }
  }
}

// One CTA per (bucket, head): thread t adds the tiles of the rows of tiles t,
// t + 128, ... that reach the bucket (neighbours in the row), then the
// threads are added by a tree.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads)
bias_join_kernel(const float* part, int batch, int q_len, int k_len, Distances dist, int q_offset, int heads,
                 int buckets, void* __restrict__ grad_table, int table_dtype) {
  __shared__ float sh[kJoinThreads / 32];
  dep_wait();
  dep_launch();
  const TileGrid tiles(q_len, k_len);
  const int k = blockIdx.x, h = blockIdx.y, rows = tiles.row_blocks * batch;
  const float* p = part + ((long long)h * buckets + k) * rows * tiles.strips;
  float sum = 0.0f;
  for (int t = threadIdx.x; t < rows; t += kJoinThreads) {
    // strip s holds the distances from + kStripDiags s up to kTileDiags more
    const int from = tiles.first_diagonal(t % tiles.row_blocks, 0) - q_offset;
    int lo, hi;
    dist.interval(k, from, from + kStripDiags * (tiles.strips - 1) + kTileDiags, lo, hi);
    if (lo >= hi) continue;
    lo -= from;
    hi -= from;
    const int s0 = lo < kTileDiags ? 0 : (lo - kTileDiags) / kStripDiags + 1;
    const int s1 = min((hi - 1) / kStripDiags, tiles.strips - 1);
    for (int s = s0; s <= s1; ++s) sum += p[(long long)t * tiles.strips + s];
  }
  sum = warp_pt(sum);
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0f;
    for (int w = 0; w < kJoinThreads / 32; ++w) sum += sh[w];
    store_from_f32(grad_table, (long long)k * heads + h, sum, table_dtype);
  }
}

int check_shape(int64_t heads, int64_t num_bounds, int64_t q_len, int64_t k_len, int64_t q_offset) {
  if (heads < 0 || num_bounds < 0 || q_len < 0 || k_len < 0) return DET_ERR_INVALID_ARG;
  const int64_t most = (1LL << 30);   // so that no distance, nor one of a tile past the edge, leaves 32 bits
  if (heads > 65535 || num_bounds > DET_MAX_BOUNDS || q_len > most || k_len > most || q_offset > most ||
      q_offset < -most || q_len + k_len + (q_offset < 0 ? -q_offset : q_offset) > most)
    return DET_ERR_TOO_LARGE;
  return DET_OK;
}

// Tiles of a head's gradient, or 2^31 when there are that many or more.
inline int64_t tiles_of_head(int64_t batch, int64_t q_len, int64_t k_len) {
  const int64_t rows = (q_len + kTileRows - 1) / kTileRows;
  const int64_t strips = ((k_len + 7) / 8 + kTileGroups + kTileLanes - 1) / kTileLanes;
  if (rows * strips >= (1LL << 31) || (rows * strips > 0 && batch > (1LL << 31) / (rows * strips))) return 1LL << 31;
  return rows * strips * batch;
}

template <typename T>
int launch_bias(const void* table, int table_dtype, int heads, const Distances& dist, int q_len, int k_len, void* out,
                cudaStream_t s) {
  cudaError_t e;
  if (q_len <= kDirectRows) {
    const dim3 grid((unsigned)((k_len + 255) / 256), (unsigned)q_len, (unsigned)heads);
    launch_begin("det_relative_bias", s);
    e = launch_dep(bias_direct_kernel<T>, grid, dim3(256), 0, s, table, table_dtype, heads, dist, q_len, k_len,
                   static_cast<T*>(out));
  } else {
    // a row has units from the one before its first boundary up
    const int unit = 16 / sizeof(T), units = (k_len + unit - 1) / unit + 1;
    // (the tile of aligned rows in 32 bits has 16 rows, with which a grid ends a few
    // queries before 2^20: from there on rows go 32 at a time as if unaligned)
    const bool aligned = (reinterpret_cast<uintptr_t>(out) | (uintptr_t)k_len * sizeof(T)) % 16 == 0 &&
                         q_len <= 65535LL * BiasTile<T, true>::kRows;
    const int threads = aligned ? BiasTile<T, true>::kThreads : BiasTile<T, false>::kThreads;
    const int rows = aligned ? BiasTile<T, true>::kRows : BiasTile<T, false>::kRows;
    const dim3 grid((unsigned)((units + threads - 1) / threads), (unsigned)((q_len + rows - 1) / rows), (unsigned)heads);
    if (grid.y > 65535) return DET_ERR_TOO_LARGE;
    launch_begin("det_relative_bias", s);
    e = launch_dep(aligned ? bias_strip_kernel<T, true> : bias_strip_kernel<T, false>, grid, dim3(threads), 0, s, table,
                   table_dtype, heads, dist, q_len, k_len, static_cast<T*>(out));
  }
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_relative_bias");
}

template <typename T, bool ALIGNED>
int launch_tiles(const void* grad, const GradView& g, const Distances& dist, int q_offset, int buckets,
                 float* part, dim3 grid, cudaStream_t s) {
  launch_begin("det_relative_bias_tiles", s);
  const cudaError_t e = launch_dep(bias_tiles_kernel<T, ALIGNED>, grid, dim3(32 * kTileWarps), 0, s,
                                   static_cast<const T*>(grad), g, dist, q_offset, buckets, part);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_relative_bias_tiles");
}

template <typename T>
int launch_bias_grad(const void* grad, GradView g, const Distances& dist, int q_offset, int heads, int buckets,
                     float* part, void* grad_table, int table_dtype, cudaStream_t s) {
  const long long tiles = (long long)TileGrid(g.q_len, g.k_len).per_matrix() * g.batch;   // of a head
  if (tiles > 0) {
    const dim3 grid((unsigned)((tiles + kTileWarps - 1) / kTileWarps), (unsigned)heads);
    g.lo = reinterpret_cast<uintptr_t>(grad);
    g.hi = g.lo + sizeof(T) * (size_t)((g.batch - 1) * g.stride_b + (heads - 1) * g.stride_h +
                                       (g.q_len - 1) * g.stride_q + g.k_len);
    // an eight of keys starts on 16 bytes if every row does
    const bool aligned = (g.lo | (uintptr_t)(sizeof(T) * (g.stride_b | g.stride_h | g.stride_q))) % 16 == 0;
    const int rc = aligned ? launch_tiles<T, true>(grad, g, dist, q_offset, buckets, part, grid, s)
                           : launch_tiles<T, false>(grad, g, dist, q_offset, buckets, part, grid, s);
    if (rc) return rc;
  }
  launch_begin("det_relative_bias_join", s);
  const cudaError_t e = launch_dep(bias_join_kernel, dim3((unsigned)buckets, (unsigned)heads), dim3(kJoinThreads), 0, s,
                                   (const float*)part, tiles > 0 ? g.batch : 0, g.q_len, g.k_len, dist, q_offset, heads,
                                   buckets, grad_table, table_dtype);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_relative_bias_join");
}

}  // namespace
}  // namespace det

using namespace det;

extern "C" int det_relative_bias(const void* table, int table_dtype, int64_t heads, const int32_t* bounds,
                                 int64_t num_bounds, int bidirectional, int64_t q_len, int64_t k_len, int64_t q_offset,
                                 void* out, int dtype, void* stream) {
  if (!valid_model_dtype(dtype) || !valid_model_dtype(table_dtype)) return DET_ERR_DTYPE;
  if (const int rc = check_shape(heads, num_bounds, q_len, k_len, q_offset)) return rc;
  if (heads == 0 || q_len == 0 || k_len == 0) return DET_OK;
  if (!table || !out || (num_bounds > 0 && !bounds)) return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(table) % model_elem_size(table_dtype) ||
      reinterpret_cast<uintptr_t>(out) % model_elem_size(dtype))
    return DET_ERR_INVALID_ARG;
  const Distances dist = {bounds, (int)num_bounds, bidirectional ? 1 : 0, (int)(1 - q_len - q_offset)};
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32)
    return launch_bias<float>(table, table_dtype, (int)heads, dist, (int)q_len, (int)k_len, out, s);
  if (dtype == DET_BF16)
    return launch_bias<__nv_bfloat16>(table, table_dtype, (int)heads, dist, (int)q_len, (int)k_len, out, s);
  return launch_bias<__half>(table, table_dtype, (int)heads, dist, (int)q_len, (int)k_len, out, s);
}

extern "C" size_t det_relative_bias_backward_workspace_bytes(int64_t batch, int64_t heads, int64_t q_len,
                                                             int64_t k_len, int64_t num_bounds, int bidirectional) {
  if (batch < 0 || check_shape(heads, num_bounds, q_len, k_len, 0) != DET_OK) return 0;
  const size_t buckets = (size_t)(num_bounds + 1) * (bidirectional ? 2 : 1);
  return 256 + align_up((size_t)heads * buckets * (size_t)tiles_of_head(batch, q_len, k_len) * sizeof(float), 256);
}

extern "C" int det_relative_bias_backward(const void* grad, int dtype, int64_t batch, int64_t heads, int64_t q_len,
                                          int64_t k_len, int64_t stride_b, int64_t stride_h, int64_t stride_q,
                                          const int32_t* bounds, int64_t num_bounds, int bidirectional,
                                          int64_t q_offset, void* grad_table, int table_dtype, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  if (!valid_model_dtype(dtype) || !valid_model_dtype(table_dtype)) return DET_ERR_DTYPE;
  if (batch < 0) return DET_ERR_INVALID_ARG;
  if (const int rc = check_shape(heads, num_bounds, q_len, k_len, q_offset)) return rc;
  if (batch >= (1LL << 31) || tiles_of_head(batch, q_len, k_len) >= (1LL << 31)) return DET_ERR_TOO_LARGE;
  if (heads == 0) return DET_OK;
  const bool none = batch == 0 || q_len == 0 || k_len == 0;
  if (!grad_table || (!none && !grad) || (num_bounds > 0 && !bounds)) return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(grad) % model_elem_size(dtype) ||
      reinterpret_cast<uintptr_t>(grad_table) % model_elem_size(table_dtype))
    return DET_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      workspace_bytes < det_relative_bias_backward_workspace_bytes(batch, heads, q_len, k_len, num_bounds, bidirectional))
    return DET_ERR_WORKSPACE;
  if (stride_b < 0 || stride_h < 0 || stride_q < 0) return DET_ERR_INVALID_ARG;
  const GradView g = {stride_b, stride_h, stride_q, none ? 0 : (int)batch, (int)q_len, (int)k_len, 0, 0};
  const Distances dist = {bounds, (int)num_bounds, bidirectional ? 1 : 0, (int)(1 - q_len - q_offset)};
  const int buckets = (int)(num_bounds + 1) * (bidirectional ? 2 : 1);
  float* part = static_cast<float*>(workspace);
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32)
    return launch_bias_grad<float>(grad, g, dist, (int)q_offset, (int)heads, buckets, part, grad_table, table_dtype, s);
  if (dtype == DET_BF16)
    return launch_bias_grad<__nv_bfloat16>(grad, g, dist, (int)q_offset, (int)heads, buckets, part, grad_table, table_dtype, s);
  return launch_bias_grad<__half>(grad, g, dist, (int)q_offset, (int)heads, buckets, part, grad_table, table_dtype, s);
}
