// det_layer_norm and its gradients.
//
// A row lies in the registers of a group of threads: whole warps, 1 to 32, eight to
// 32 columns each (eights, the group's threads apart), so it is read once.
// The mean is the rows' sum, the variance the sum of squares of what the mean
// leaves -- two trees over the same columns, across lanes by shuffles and across
// warps through shared memory -- and never a difference of two large sums.
// CTAs stay and take one row (or, of narrow ones, several) after the other with
// weight and bias in registers and the next row on its way.
//
// The gradient adds a row's share of the weight's and bias' gradients into 32-bit
// registers of the column's thread; CTAs leave these as rows of partial sums, which
// a second launch joins.  Row r belongs to partial sum r mod parts, and parts is a
// function of rows and cols, so the order of every sum is too.
//
// Bytes bound it: 16,384 x 4,096 in bf16 take 42 us (a copy of as many bytes 45), 56% of the issue slots,
// the gradients 73 (5.5 TB/s); 65,536 x 4,096 in bf16 169 and 262 us, 6.4 and 6.1 TB/s.  (Figures
// below that compare two ways were taken side by side when the choice was made.)  A few rows: the launch and
// one row's chain of a copy, two sums across the group (one in the gradient) and a store, about 6 us.
#include "det_model.cuh"

#include <algorithm>

namespace det {
namespace {

// (A Two holds two adjacent columns.)

// The lanes' sums of a group, in every thread: a tree over lanes, then over warps
// through `slot`, where a group has LEAVES places (those of no warp are 0).  A group of
// one warp needs no barrier.
template <int LEAVES>
__device__ __forceinline__ float over_warps(const float* slot, int lane) {
  if constexpr (LEAVES == 8) {         // the same tree as below, without shuffles
    const float4 a = *reinterpret_cast<const float4*>(slot), b = *reinterpret_cast<const float4*>(slot + 4);
    return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
  } else {
    float v = slot[lane & (LEAVES - 1)];
#pragma unroll
    for (int s = 1; s < LEAVES; s <<= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
    return v;
  }
}
__device__ __forceinline__ float lanes(Two v) {
  return __fadd_rn(v.x, v.y);
}

// 1 / sqrt(v) from the hardware's approximation by a step of Newton's method.  NaN for an infinite v, a sum of squares that
// has left 32 bits: 0 would make the row's results its bias.
__device__ __forceinline__ float inverse_root(float v) {
  const float r = rsqrtf(v), e = fmaf(-0.5f * v * r, r, 0.5f);
  return v > 0.0f && r < 1e18f ? fmaf(r, e, r) : r;       // 0 and NaN as they are
}

// sum / n to nearest, for a whole number n below 2^15 and of = 1 / n to nearest (the product alone is a step off where n * of
// rounds to less than 1: 1,000 in each of 41 columns had a mean of 999.99994).  The product q is off by less than 2 steps of
// its last place; sum and n q are multiples of such a step, so what is left, n q from sum, is exact; and a quotient by n
// lies no nearer than 1 / (2 n) steps to the middle between two values, where the last sum's error of 2^-22 of a step would
// matter.  (Means below 2^-126 may be a step off.  A division instead: 87,381 x 768 in bf16 56.9 us against 54.1; the product
// alone 53.7.)  NaN where the sum is infinite.
__device__ __forceinline__ float mean_of(float sum, float n, float of) {
  const float q = __fmul_rn(sum, of);
  return fmaf(fmaf(-q, n, sum), of, q);
}

// A group's place: `threads` of them, whole warps, take a row, of a CTA of MOST threads and less.
template <int MOST>
struct Group {
  static constexpr int LEAVES = MOST / 32;       // of the tree over its warps (`leaves` of them are enough)
  int me, threads, warps, warp, lane, index, count;
  int leaves, first_leaf, leaf;
  __device__ __forceinline__ explicit Group(int threads_of_a_row) {
    threads = threads_of_a_row;
    warps = threads >> 5;
    warp = threadIdx.x >> 5;
    index = warp / warps;
    me = threadIdx.x - index * threads;
    lane = threadIdx.x & 31;
    count = (blockDim.x >> 5) / warps;
    leaves = 1 << (32 - __clz(warps - 1));
    first_leaf = index * (MOST > 256 ? leaves : LEAVES);       // (four groups of two warps and more have 32)
    leaf = first_leaf + (me >> 5);
  }
};

// ---------------------------------------------------------------------------
// Rows.  A thread's columns are eights, `threads` eights apart.  Rows are copied into
// shared memory up to two rounds ahead of their turn, each warp the 256 columns of
// its eights, as 16-byte vectors.  (Rows ahead in registers instead left an SM with two CTAs.)
// Where rows or outputs do not all start on 16 bytes (VEC is false), the vectors that hold a
// row's columns are copied and shifted as they are taken (what else such a first vector holds
// is not the row's, but lies beside it in 16 bytes); outputs go through the warp's part of
// shared memory to words in the order of memory.  (Gradient of 16,384 x 4,095 in bf16: 125 us; rows copied
// word by word 133, read and written element by element 176.  16,384 x 4,096: 80.)

// Where a thread reads and writes in a row: its first column, and how many of each
// of its eights there are.
template <typename T, bool VEC, int K> struct Columns {
  int first, step;       // step: from one eight to the next
  int read;              // the first column that the thread copies: in 32 bits vectors lie lane after lane
  int n[K];              // VEC: columns of the thread's eights; else columns of the row from the first one on
  int span[K];           // columns of the row from the first one that it copies on
  template <typename G>
  __device__ __forceinline__ Columns(const G& g, int cols) {
    const int warp = (g.me & ~31) * 8;                   // the warp's first
    first = VEC ? g.me * 8 : warp;
    read = VEC && sizeof(T) == 4 ? warp + 4 * g.lane : first;
    step = g.threads * 8;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      n[k] = cols - first - k * step;
      if (VEC) n[k] = max(0, min(8, n[k]));
      span[k] = cols - read - k * step;
    }
  }
};

__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the last `ahead` (0 or 1) groups have arrived.
__device__ __forceinline__ void copies_wait(int ahead) {
  if (ahead) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
}

// A warp's rows of one operand: asked for, and taken in the same order.
template <typename T, bool VEC, int K>
struct Feed {
  enum : int {
    kHalves = sizeof(T) / 2,             // 16-byte vectors of an eight
    kSpan = 256 * (int)sizeof(T) + (VEC ? 0 : 16),       // from the vector that holds the first column on
    kStage = K * kSpan                   // bytes of a warp's columns
  };
  char* s;               // the warp's stages
  __device__ __forceinline__ explicit Feed(char* stages) : s(stages) {}
  // at: the row, from the first column that the thread copies on; `any` is aligned to what is copied at a time
  __device__ __forceinline__ void ask(int stage, const T* at, const void* any, const Columns<T, VEC, K>& c, bool valid, int lane) {
    char* to = s + stage * kStage;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (VEC) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {              // (a warp's copies go to one place after the other, or take longer)
          const bool ok = valid && c.span[k] > 128 * h;
          copy_async(to + ((k * kHalves + h) * 32 + lane) * 16, ok ? at + k * c.step + 128 * h : any, ok ? 16 : 0);
        }
      } else {
        const uintptr_t p = reinterpret_cast<uintptr_t>(at + k * c.step);
        const int off = (int)(p & 15);
        const char* vectors = reinterpret_cast<const char*>(p & ~(uintptr_t)15);
        const int left = valid && c.n[k] > 0 ? c.n[k] * (int)sizeof(T) + off : 0;       // bytes from the first vector on
        if (left >= kSpan) {
#pragma unroll
          for (int h = 0; h < kHalves; ++h) copy_async(to + k * kSpan + 16 * (32 * h + lane), vectors + 16 * (32 * h + lane), 16);
          if (off && lane == 0) copy_async(to + k * kSpan + kSpan - 16, vectors + kSpan - 16, 16);
        } else {
#pragma unroll
          for (int h = 0; h <= kHalves; ++h) {
            const int i = 32 * h + lane, bytes = max(0, min(16, left - 16 * i));
            if (h < kHalves || lane == 0) copy_async(to + k * kSpan + 16 * i, bytes ? vectors + 16 * i : any, bytes);
          }
        }
      }
    }
  }
  // An eight of the row in a stage.  off: bytes from the vector that holds the row's first column to that
  __device__ __forceinline__ Eight<T> eight(int stage, int k, int off, int lane) const {
    Eight<T> e;
    if constexpr (VEC) {
      const uint4* q = reinterpret_cast<const uint4*>(s + stage * kStage) + kHalves * (k * 32 + lane);
      e.q = q[0];
      if constexpr (kHalves == 2) e.r = q[1];
    } else {
      const uint4* q = reinterpret_cast<const uint4*>(s + stage * kStage + k * kSpan) + kHalves * lane;
      unsigned w[4 * kHalves + 4];
#pragma unroll
      for (int h = 0; h <= kHalves; ++h) {
        const uint4 v = h < kHalves || off ? q[h] : make_uint4(0, 0, 0, 0);
        w[4 * h] = v.x, w[4 * h + 1] = v.y, w[4 * h + 2] = v.z, w[4 * h + 3] = v.w;
      }
      // (off is the same for the whole warp)
      if (off & 8) {
#pragma unroll
        for (int i = 0; i < 4 * kHalves + 2; ++i) w[i] = w[i + 2];
      }
      if (off & 4) {
#pragma unroll
        for (int i = 0; i < 4 * kHalves + 1; ++i) w[i] = w[i + 1];
      }
      if (sizeof(T) == 2 && (off & 2)) {
#pragma unroll
        for (int i = 0; i < 4 * kHalves; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
      }
      e.q = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (kHalves == 2) e.r = make_uint4(w[4], w[5], w[6], w[7]);
    }
    return e;
  }
  __device__ __forceinline__ void take(int stage, Eight<T> (&e)[K], int off, int lane) const {
#pragma unroll
    for (int k = 0; k < K; ++k) e[k] = eight(stage, k, off, lane);
    __syncwarp();                                        // the stage may be written again
  }
  // Where row r of rows at p, stride elements apart, starts in 16 bytes.
  static __device__ __forceinline__ int offset(const T* p, unsigned r, long long stride) {
    return VEC ? 0 : ((unsigned)reinterpret_cast<uintptr_t>(p) + r * (unsigned)stride * (unsigned)sizeof(T)) & 15;
  }
  static __device__ __forceinline__ const void* aligned(const T* p) {
    return reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15);
  }
};
// Bytes of a warp's stages, and of the place where its outputs turn into rows.
template <typename T, bool VEC, int K>
__host__ __device__ constexpr int feed_bytes(int stages) { return stages * Feed<T, VEC, K>::kStage; }
template <typename T, bool VEC>
__host__ __device__ constexpr int turn_bytes() { return VEC ? 0 : sizeof(T) == 2 ? 528 : 1024; }

template <typename T, bool VEC, int K>
__device__ __forceinline__ void store_columns(T* at, const float (&v)[8], const Columns<T, VEC, K>& c, int k, bool valid,
                                              char* turn, int lane) {
  // a warp's lanes are of one row and start at one column.  (With four eights the branch costs registers that are
  // not there: 4,096 x 12,001 in 32 bits 235 us against 209.)
  if (!VEC && K < 4 && (!valid || c.n[k] <= 0)) return;
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 4) {
      if (valid && c.n[k] == 8 && reinterpret_cast<uintptr_t>(at) % 32 == 0) {
        st_256(at + k * c.step, v);                      // whole sectors
        return;
      }
    }
    if (valid) store_eight(at + k * c.step, v, c.n[k]);
  } else if constexpr (sizeof(T) == 4) {
    float* s = reinterpret_cast<float*>(turn);
    store_eight(s + 8 * lane, v, 8);
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (valid && 32 * j + lane < c.n[k]) at[k * c.step + 32 * j + lane] = s[32 * j + lane];
    __syncwarp();
  } else {
    // the span's words: at an odd element each holds the element before its own first
    unsigned* s = reinterpret_cast<unsigned*>(turn);
    const uintptr_t p = reinterpret_cast<uintptr_t>(at + k * c.step);
    const int odd = (int)(p >> 1 & 1);
    uint4 q = make_uint4(pack_two<T>(v[0], v[1]), pack_two<T>(v[2], v[3]), pack_two<T>(v[4], v[5]), pack_two<T>(v[6], v[7]));
    if (odd) {
      const unsigned before = __shfl_up_sync(0xffffffffu, q.w, 1);
      if (lane == 31) s[128] = q.w >> 16;
      q = make_uint4(__funnelshift_r(before, q.x, 16), __funnelshift_r(q.x, q.y, 16), __funnelshift_r(q.y, q.z, 16),
                     __funnelshift_r(q.z, q.w, 16));
    }
    *reinterpret_cast<uint4*>(s + 4 * lane) = q;
    __syncwarp();
    char* words = reinterpret_cast<char*>(p & ~(uintptr_t)3);
    const int end = valid ? min(256, c.n[k]) + odd : 0;   // halves of words from `odd` on
    if (end >= 256 + odd) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 32 * j + lane;
        if (j > 0 || lane >= odd) *reinterpret_cast<unsigned*>(words + 4 * i) = s[i];
      }
      if (odd && lane == 0) {
        *reinterpret_cast<unsigned short*>(words + 2) = (unsigned short)(s[0] >> 16);
        *reinterpret_cast<unsigned short*>(words + 512) = (unsigned short)s[128];
      }
      __syncwarp();
      return;
    }
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int i = 32 * j + lane;
      if (j == 4 && lane > 0) break;
      const bool low = 2 * i < end && 2 * i >= odd, high = 2 * i + 1 < end;
      unsigned short* h = reinterpret_cast<unsigned short*>(words + 4 * i);
      if (low && high) *reinterpret_cast<unsigned*>(h) = s[i];
      else if (low) h[0] = (unsigned short)s[i];
      else if (high) h[1] = (unsigned short)(s[i] >> 16);
    }
    __syncwarp();
  }
}

template <typename T>
__device__ __forceinline__ void pairs_of(const Eight<T>& e, Two (&v)[4]) {
  float f[8];
  unpack_eight(e, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = two(f[2 * i], f[2 * i + 1]);
}
// The first n of eight values, the others 0.
__device__ __forceinline__ void keep_first(Two (&v)[4], int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = two(2 * i < n ? v[i].x : 0.0f, 2 * i + 1 < n ? v[i].y : 0.0f);
  }
}
// Columns c .. c + 7 of a weight or bias, `other` without one.
template <typename P>
__device__ __forceinline__ void load_param(Two (&v)[4], const P* p, int c, int cols) {
  const int n = max(0, min(8, cols - c));
  pairs_of(n == 8 && reinterpret_cast<uintptr_t>(p) % 16 == 0 ? load_eight<true>(p + c, 8) : load_eight<false>(p + c, n), v);
}
__device__ __forceinline__ void load_param(Two (&v)[4], const void* p, int c, int cols, int dtype, float other) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = twice(other);
  } else if (dtype == DET_F32) {
    load_param(v, static_cast<const float*>(p), c, cols);
  } else if (dtype == DET_BF16) {
    load_param(v, static_cast<const __nv_bfloat16*>(p), c, cols);
  } else {
    load_param(v, static_cast<const __half*>(p), c, cols);
  }
}

constexpr int kThreads = 256;       // a CTA's, unless a row takes more
// Of a row of partial sums, so that eights lie on 16 bytes.
__host__ __device__ constexpr int whole_eights(int cols) { return (cols + 7) / 8 * 8; }

// A weight or bias in shared memory, where they leave registers for rows: halves of
// eights, so that a warp reads 512 bytes in a row.
template <typename G>
__device__ __forceinline__ void keep_param(float4* s, const void* p, const G& g, int k, int cols, int dtype, float other) {
  Two v[4];
  load_param(v, p, (g.me + k * g.threads) * 8, cols, dtype, other);
  s[(2 * k) * g.threads + g.me] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  s[(2 * k + 1) * g.threads + g.me] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}
template <typename G>
__device__ __forceinline__ void param(Two (&v)[4], const float4* s, const G& g, int k) {
  const float4 a = s[(2 * k) * g.threads + g.me], b = s[(2 * k + 1) * g.threads + g.me];
  v[0] = two(a.x, a.y), v[1] = two(a.z, a.w), v[2] = two(b.x, b.y), v[3] = two(b.z, b.w);
}

template <typename T, int K, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST, MOST > 256 ? 1024 / MOST : K == 1 ? 4 : 3)
layer_norm_kernel(const T* x, unsigned rows, int cols, long long x_stride, const void* weight, const void* bias,
                  int param_dtype, float eps, T* out, float* mean_out, float* rstd_out, int threads, int stages) {
  __shared__ __align__(16) float s_sum[32], s_sq[32];
  extern __shared__ __align__(16) char s_dynamic[];
  dep_wait();
  dep_launch();
  const Group<MOST> g(threads);
  // weight and bias are in registers where CTAs of 256 threads leave enough of them (48 us for 16,384 x 4,096 in bf16 against
  // 52 with shared memory), else in shared memory
  constexpr bool HELD = MOST == 256;
  Two held_w[HELD ? K : 1][4], held_b[HELD ? K : 1][4];
  float4* s_w = reinterpret_cast<float4*>(s_dynamic);
  float4* s_b = s_w + (HELD ? 0 : 2 * K * g.threads);
  char* mine = reinterpret_cast<char*>(s_b + (HELD ? 0 : 2 * K * g.threads)) +
               g.warp * (feed_bytes<T, VEC, K>(stages) + turn_bytes<T, VEC>());
  char* turn = mine + feed_bytes<T, VEC, K>(stages);
  const bool whole = (g.me + (K - 1) * g.threads) * 8 + 8 <= cols;   // all of the thread's columns are there
  const unsigned step = gridDim.x * g.count;
  const float of = 1.0f / (float)cols;
  const Columns<T, VEC, K> c(g, cols);
  unsigned r = blockIdx.x * g.count + g.index, asked = r;
  const T* from = x + r * x_stride + c.read;
  T* to = out + (long long)r * cols + c.first;
  Feed<T, VEC, K> feed(mine);
  for (int i = 0; i < stages; ++i, asked += step, from += step * x_stride) {
    feed.ask(i, from, feed.aligned(x), c, asked < rows, g.lane);
    copies_commit();
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if constexpr (HELD) {
      load_param(held_w[k], weight, (g.me + k * g.threads) * 8, cols, param_dtype, 1.0f);
      load_param(held_b[k], bias, (g.me + k * g.threads) * 8, cols, param_dtype, 0.0f);
    } else {
      keep_param(s_w, weight, g, k, cols, param_dtype, 1.0f);       // (read again by the same thread)
      keep_param(s_b, bias, g, k, cols, param_dtype, 0.0f);
    }
  }
  if (threadIdx.x < 32) s_sum[threadIdx.x] = s_sq[threadIdx.x] = 0.0f;
  __syncthreads();
  int stage = 0;
  // (every thread of the CTA makes as many rounds)
  for (unsigned first = blockIdx.x * g.count; first < rows; first += step, r += step, to += (long long)step * cols) {
    Eight<T> e[K];
    copies_wait(stages - 1);
    feed.take(stage, e, feed.offset(x, r, x_stride), g.lane);
    feed.ask(stage, from, feed.aligned(x), c, asked < rows, g.lane);
    copies_commit();
    asked += step;
    from += step * x_stride;
    stage = stage + 1 == stages ? 0 : stage + 1;
    Two v[K][4], t[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      pairs_of(e[k], v[k]);
      t[k] = add(add(v[k][0], v[k][1]), add(v[k][2], v[k][3]));
    }
    if (K == 2) t[0] = add(t[0], t[K - 1]);
    float sum = warp_pt(lanes(t[0]));
    if (g.warps > 1) {
      if (g.lane == 0) s_sum[g.leaf] = sum;
      __syncthreads();
      sum = over_warps<MOST / 32>(s_sum + g.first_leaf, g.lane);
    }
    const float mean = mean_of(sum, (float)cols, of);
    const Two minus_mean = twice(-mean);
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k][i] = add(v[k][i], minus_mean);
      if (!whole) keep_first(v[k], cols - (g.me + k * g.threads) * 8);
      t[k] = factor(v[k][0], v[k][0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) t[k] = fma(v[k][i], v[k][i], t[k]);
    }
    if (K == 2) t[0] = add(t[0], t[K - 1]);
    float sq = warp_pt(lanes(t[0]));
    if (g.warps > 1) {
      if (g.lane == 0) s_sq[g.leaf] = sq;
      __syncthreads();
      sq = over_warps<MOST / 32>(s_sq + g.first_leaf, g.lane);
    }
    const float rstd = inverse_root(fmaf(sq, of, eps));
    const Two rstd2 = twice(rstd);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float y[8];
      Two w[4], b[4];
      if constexpr (!HELD) {
        param(w, s_w, g, k);
        param(b, s_b, g, k);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = fma(factor(v[k][i], rstd2), HELD ? held_w[HELD ? k : 0][i] : w[i], HELD ? held_b[HELD ? k : 0][i] : b[i]);
        y[2 * i] = f.x;
        y[2 * i + 1] = f.y;
      }
      store_columns(to, y, c, k, r < rows, turn, g.lane);
    }
    if (g.me == 0 && r < rows) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
  }
}

// part: [gridDim.x][2][whole_eights(cols)] sums of the weight's and the bias' gradients, or NULL.
template <typename T, int K, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST, MOST > 256 ? 1 : K == 1 ? 3 : 2)
layer_norm_grad_kernel(const T* grad, long long grad_stride, const T* x, long long x_stride, unsigned rows, int cols,
                       const float* means, const float* rstds, const void* weight, int param_dtype, T* grad_x,
                       float* part, int threads, int stages) {
  __shared__ __align__(16) Two s_sums[2][32];
  // where the columns' sums take half of the registers, rows are read from shared memory twice
  constexpr bool LATE = K == 4;
  extern __shared__ __align__(16) char s_dynamic[];
  float* s_acc = reinterpret_cast<float*>(s_dynamic);
  dep_wait();
  dep_launch();
  const Group<MOST> g(threads);
  float4* s_w = reinterpret_cast<float4*>(s_dynamic);
  char* mine_x = reinterpret_cast<char*>(s_w + 2 * K * g.threads) +
                 g.warp * (2 * feed_bytes<T, VEC, K>(stages) + turn_bytes<T, VEC>());
  Two aw[K][4], ab[K][4];
  const bool whole = (g.me + (K - 1) * g.threads) * 8 + 8 <= cols;
  const unsigned step = gridDim.x * g.count;
  const float of = 1.0f / (float)cols;
  const Columns<T, VEC, K> c(g, cols);
  unsigned r = blockIdx.x * g.count + g.index, asked = r;
  const T* from_x = x + r * x_stride + c.read;
  const T* from_grad = grad + r * grad_stride + c.read;
  T* to = grad_x + (long long)r * cols + c.first;
  Feed<T, VEC, K> feed_x(mine_x), feed_grad(mine_x + feed_bytes<T, VEC, K>(stages));
  char* turn = mine_x + 2 * feed_bytes<T, VEC, K>(stages);
  auto ask = [&](int stage) {
    feed_x.ask(stage, from_x, feed_x.aligned(x), c, asked < rows, g.lane);
    feed_grad.ask(stage, from_grad, feed_grad.aligned(grad), c, asked < rows, g.lane);
    copies_commit();
    asked += step;
    from_x += step * x_stride;
    from_grad += step * grad_stride;
  };
  for (int i = 0; i < stages; ++i) ask(i);
  if (threadIdx.x < 64) s_sums[threadIdx.x >> 5][threadIdx.x & 31] = twice(0.0f);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (g.index == 0) keep_param(s_w, weight, g, k, cols, param_dtype, 1.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) aw[k][i] = ab[k][i] = twice(0.0f);
  }
  __syncthreads();
  float nm = r < rows ? means[r] : 0.0f, nr = r < rows ? rstds[r] : 0.0f;
  int parity = 0, stage = 0;
  for (unsigned first = blockIdx.x * g.count; first < rows;
       first += step, r += step, parity ^= 1, to += (long long)step * cols) {
    Eight<T> cx[K], cg[K];
    copies_wait(stages - 1);
    const int off_x = feed_x.offset(x, r, x_stride), off_grad = feed_grad.offset(grad, r, grad_stride);
    if (!LATE) {
      feed_x.take(stage, cx, off_x, g.lane);
      feed_grad.take(stage, cg, off_grad, g.lane);
      ask(stage);
      stage = stage + 1 == stages ? 0 : stage + 1;
    }
    const Two minus_mean = twice(-nm), rstd2 = twice(nr);
    const bool more = r + step < rows;
    nm = more ? means[r + step] : 0.0f;
    nr = more ? rstds[r + step] : 0.0f;
    Two t1[K], t2[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Two xh[4], d[4], w[4];
      param(w, s_w, g, k);
      pairs_of(LATE ? feed_x.eight(stage, k, off_x, g.lane) : cx[k], xh);
      pairs_of(LATE ? feed_grad.eight(stage, k, off_grad, g.lane) : cg[k], d);
#pragma unroll
      for (int i = 0; i < 4; ++i) xh[i] = factor(add(xh[i], minus_mean), rstd2);
      if (!whole) keep_first(xh, cols - (g.me + k * g.threads) * 8);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        aw[k][i] = fma(d[i], xh[i], aw[k][i]);
        ab[k][i] = add(ab[k][i], d[i]);
        const Two gw = factor(d[i], w[i]);
        t1[k] = i ? fma(d[i], w[i], t1[k]) : gw;
        t2[k] = i ? fma(gw, xh[i], t2[k]) : factor(gw, xh[i]);
      }
    }
#pragma unroll
    for (int d = 1; d < K; d *= 2)
#pragma unroll
      for (int k = 0; k < K; k += 2 * d) {
        t1[k] = add(t1[k], t1[k + d]);
        t2[k] = add(t2[k], t2[k + d]);
      }
    Two sums = two(lanes(t1[0]), lanes(t2[0]));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1)
      sums = add(sums, two(__shfl_xor_sync(0xffffffffu, sums.x, d), __shfl_xor_sync(0xffffffffu, sums.y, d)));
    if (g.warps > 1) {
      if (g.lane == 0) s_sums[parity][g.leaf] = sums;
      __syncthreads();
      if constexpr (MOST == 256) {     // the same tree as below, without shuffles
        const float4* q = reinterpret_cast<const float4*>(&s_sums[parity][g.first_leaf]);
        Two t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = add(two(q[i].x, q[i].y), two(q[i].z, q[i].w));
        sums = add(add(t[0], t[1]), add(t[2], t[3]));
      } else {
        // (with four eights a loop whose length is not known here: unrolled it took the registers of the columns' sums,
        // 4,096 x 16,384 in bf16 98 us against 82)
        const int leaves = K == 4 ? g.leaves : MOST / 32;
        sums = s_sums[parity][g.first_leaf + (g.lane & (leaves - 1))];
        for (int d = 1; d < leaves; d <<= 1)
          sums = add(sums, two(__shfl_xor_sync(0xffffffffu, sums.x, d), __shfl_xor_sync(0xffffffffu, sums.y, d)));
      }
    }
    if (grad_x) {
      // rstd (gw - sums.x / cols - (x - mean) rstd sums.y / cols).  (rstd^2 would pass 32 bits where rstd does not, at
      // deviations below 5e-20 without an eps; rstd sums.y / cols is as large as the result.)
      const Two minus_one = twice(-sums.x * of), minus_two = twice(-sums.y * of * rstd2.x);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Two xh[4], d[4], w[4];
        param(w, s_w, g, k);
        pairs_of(LATE ? feed_x.eight(stage, k, off_x, g.lane) : cx[k], xh);
        pairs_of(LATE ? feed_grad.eight(stage, k, off_grad, g.lane) : cg[k], d);
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Two f = factor(fma(add(xh[i], minus_mean), minus_two, fma(d[i], w[i], minus_one)), rstd2);
          y[2 * i] = f.x;
          y[2 * i + 1] = f.y;
        }
        store_columns(to, y, c, k, r < rows, turn, g.lane);
      }
    }
    if (LATE) {
      __syncwarp();
      ask(stage);
      stage = stage + 1 == stages ? 0 : stage + 1;
    }
  }
  if (!part) return;
  copies_wait(0);                      // (those past the last row write zeros)
  __syncthreads();                     // weight and rows have been read: the groups' sums take their place
  const int pitch = whole_eights(cols);
  float* mine = part + (long long)blockIdx.x * 2 * pitch;
  // several rows at a time: the groups' sums in the groups' order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (g.count > 1 && which) __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Two(&v)[4] = which ? ab[k] : aw[k];
      const int c = (g.me + k * g.threads) * 8;
      float4* to = reinterpret_cast<float4*>((g.count > 1 ? s_acc + g.index * pitch : mine + which * pitch) + c);
      if (c < cols) {
        to[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
        to[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
      }
    }
    if (g.count == 1) continue;
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      float t = s_acc[c];
      for (int j = 1; j < g.count; ++j) t += s_acc[j * pitch + c];
      mine[which * pitch + c] = t;
    }
  }
}

// grad[c] = the sum of parts rows: 32 strands of every 32nd row, then a tree.  (304 x 4,096: 10 MB, most of
// them in L2: 5 us beside the launch.)
__global__ void __launch_bounds__(1024)
layer_norm_join_kernel(const float* part, int parts, int cols, void* grad_weight, void* grad_bias, int param_dtype) {
  __shared__ float s[32][33];
  dep_wait();
  dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  void* to = blockIdx.y ? grad_bias : grad_weight;
  if (!to) return;
  const int c = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < cols) {
    const int pitch = whole_eights(cols);
    const float* p = part + (long long)blockIdx.y * pitch + c;
#pragma unroll 4
    for (int j = warp; j < parts; j += 32) t += p[(long long)j * 2 * pitch];
  }
  s[warp][lane] = t;
  __syncthreads();
  const float total = warp_pt(s[lane][warp]);
  const int of = blockIdx.x * 32 + warp;
  if (lane == 0 && of < cols) store_from_f32(to, of, total, param_dtype);
}

// Eights of columns a thread takes (two keep a row's sums over lanes and warps short), and
// the threads that take a row: as many warps as its columns need (13,107 x 5,120 in bf16, 10 warps: 53 and 92 us; with
// the next power of two, 16 of them: 86 and 113).  The gradient of wide rows takes four eights: 1,024 threads of 64
// registers each spill (4,096 x 16,384 in bf16: 182 us, 82 with 512 that take twice as much).
int eights(int64_t cols) { return cols > 256 ? 2 : 1; }
int grad_eights(int64_t cols) { return cols > 8192 ? 4 : eights(cols); }
int row_threads(int64_t cols, int eights) {
  return (int)std::max<int64_t>(1, (cols + 256 * eights - 1) / (256 * eights)) * 32;
}
// CTAs of the gradient, each of which leaves a partial sum: as many as run at once on
// the 152 SMs, by a constant, because the sums' order hangs on it.
int grad_parts(int64_t rows, int64_t cols) {
  const int threads = row_threads(cols, grad_eights(cols));
  const int64_t at_a_time = std::max(1, kThreads / threads);
  const int at_once = 152 * (threads > kThreads ? 1 : grad_eights(cols) == 1 ? 3 : 2);
  return (int)std::min<int64_t>((rows + at_a_time - 1) / at_a_time, at_once);
}

template <typename T>
bool vectors(const void* p, int64_t stride, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * sizeof(T)) | (uintptr_t)(cols * sizeof(T))) % 16 == 0;
}

// Rows that are copied ahead, and the dynamic shared memory: two, or one where 32-bit
// rows of more than 8,192 columns leave no room.
template <typename T, bool VEC, int K>
size_t room(int params, int operands, int row_threads, int threads, int* stages) {
  size_t bytes = 0;
  for (*stages = 2; *stages > 0; --*stages) {
    bytes = (size_t)params * K * 32 * row_threads +
            threads / 32 * (size_t)(operands * feed_bytes<T, VEC, K>(*stages) + turn_bytes<T, VEC>());
    if (bytes <= 226 * 1024 || *stages == 1) break;
  }
  return bytes;
}

template <typename T, int K, bool VEC, int MOST>
int forward(const void* x, int rows, int cols, int64_t x_stride, const void* weight, const void* bias, int param_dtype,
            float eps, void* out, float* mean_out, float* rstd_out, cudaStream_t s) {
  const int of_a_row = row_threads(cols, K), at_a_time = std::max(1, kThreads / of_a_row), threads = at_a_time * of_a_row;
  auto* k = layer_norm_kernel<T, K, VEC, MOST>;
  int stages = 1;
  const size_t smem = room<T, VEC, K>(MOST == 256 ? 0 : 2, 1, of_a_row, threads, &stages);
  const cudaError_t se = ensure_dyn_smem((const void*)k, smem);
  if (se != cudaSuccess) return cuda_fail(se, "det_layer_norm");
  const int per_sm = kernel_occupancy((const void*)k, threads, smem);
  if (per_sm <= 0) return cuda_fail(cudaErrorUnknown, "det_layer_norm");
  const long long grid = std::min<long long>((rows + (long long)at_a_time - 1) / at_a_time,
                                             (long long)per_sm * std::max(device_sm_count(), 1));
  launch_begin("det_layer_norm", s);
  const cudaError_t e = launch_dep(k, dim3((unsigned)grid), dim3(threads), smem, s, static_cast<const T*>(x),
                                   (unsigned)rows, cols, (long long)x_stride, weight, bias, param_dtype, eps,
                                   static_cast<T*>(out), mean_out, rstd_out, of_a_row, stages);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_layer_norm");
}

template <typename T, int K, bool VEC, int MOST>
int backward(const void* grad, int64_t grad_stride, const void* x, int64_t x_stride, int rows, int cols,
             const float* mean, const float* rstd, const void* weight, int param_dtype, void* grad_x, float* part,
             cudaStream_t s) {
  const int of_a_row = row_threads(cols, K), groups = std::max(1, kThreads / of_a_row), threads = groups * of_a_row;
  auto* k = layer_norm_grad_kernel<T, K, VEC, MOST>;
  int stages = 1;
  // weight and rows; the groups' sums take their place at the end
  const size_t sums = groups > 1 ? (size_t)groups * whole_eights(cols) * sizeof(float) : 0;
  const size_t smem = std::max(room<T, VEC, K>(1, 2, of_a_row, threads, &stages), sums);
  const cudaError_t se = ensure_dyn_smem((const void*)k, smem);
  if (se != cudaSuccess) return cuda_fail(se, "det_layer_norm_backward");
  launch_begin("det_layer_norm_backward", s);
  const cudaError_t e = launch_dep(k, dim3((unsigned)grad_parts(rows, cols)), dim3(threads), smem, s,
                                   static_cast<const T*>(grad), (long long)grad_stride, static_cast<const T*>(x),
                                   (long long)x_stride, (unsigned)rows, cols, mean, rstd, weight, param_dtype,
                                   static_cast<T*>(grad_x), part, of_a_row, stages);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_layer_norm_backward");
}

int check_rows(int dtype, int param_dtype, int64_t rows, int64_t cols) {
  if (!valid_model_dtype(dtype) || !valid_model_dtype(param_dtype)) return DET_ERR_DTYPE;
  if (rows < 0 || cols < 0 || (rows > 0 && cols == 0)) return DET_ERR_INVALID_ARG;
  if (rows >= (1LL << 31) || cols > DET_MAX_NORM_COLS) return DET_ERR_TOO_LARGE;
  return DET_OK;
}
bool misaligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % model_elem_size(dtype) != 0; }

}  // namespace
}  // namespace det

using namespace det;

// The kernels for eights() or grad_eights() and row_threads().
#define DET_NORM_PICK_T(fn, T, WIDE_K, ...)                                                                     \
  do {                                                                                                   \
    if (cols <= 256) return vec ? fn<T, 1, true, 256>(__VA_ARGS__) : fn<T, 1, false, 256>(__VA_ARGS__);  \
    if (cols <= 4096) return vec ? fn<T, 2, true, 256>(__VA_ARGS__) : fn<T, 2, false, 256>(__VA_ARGS__); \
    if (cols <= 8192) return vec ? fn<T, 2, true, 512>(__VA_ARGS__) : fn<T, 2, false, 512>(__VA_ARGS__); \
    return vec ? fn<T, WIDE_K, true, 2048 / WIDE_K>(__VA_ARGS__) : fn<T, WIDE_K, false, 2048 / WIDE_K>(__VA_ARGS__); \
  } while (0)
#define DET_NORM_PICK(fn, WIDE_K, ...)                                                 \
  do {                                                                         \
    if (dtype == DET_F32) DET_NORM_PICK_T(fn, float, WIDE_K, __VA_ARGS__);                   \
    if (dtype == DET_BF16) DET_NORM_PICK_T(fn, __nv_bfloat16, WIDE_K, __VA_ARGS__);   \
    DET_NORM_PICK_T(fn, __half, WIDE_K, __VA_ARGS__);                                 \
  } while (0)

static int norm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                        const void* bias, int param_dtype, float eps, void* out, float* mean_out, float* rstd_out,
                        bool vec, cudaStream_t s) {
  DET_NORM_PICK(forward, 2, x, (int)rows, (int)cols, x_stride, weight, bias, param_dtype, eps, out, mean_out, rstd_out, s);
}
static int norm_backward(const void* grad, int64_t grad_stride, const void* x, int64_t x_stride, int dtype, int64_t rows,
                         int64_t cols, const float* mean, const float* rstd, const void* weight, int param_dtype,
                         void* grad_x, float* part, bool vec, cudaStream_t s) {
  DET_NORM_PICK(backward, 4, grad, grad_stride, x, x_stride, (int)rows, (int)cols, mean, rstd, weight, param_dtype, grad_x,
                part, s);
}

extern "C" int det_layer_norm(const void* x, int dtype, int64_t rows, int64_t cols, int64_t x_stride,
                              const void* weight, const void* bias, int param_dtype, float eps, void* out,
                              float* mean_out, float* rstd_out, void* stream) {
  if (const int rc = check_rows(dtype, param_dtype, rows, cols)) return rc;
  if (!(eps >= 0.0f && eps < INFINITY) || x_stride < 0) return DET_ERR_INVALID_ARG;
  if (rows == 0) return DET_OK;
  if (!x || !out) return DET_ERR_INVALID_ARG;
  if (misaligned(x, dtype) || misaligned(out, dtype) || misaligned(weight, param_dtype) ||
      misaligned(bias, param_dtype) || misaligned(mean_out, DET_F32) || misaligned(rstd_out, DET_F32))
    return DET_ERR_INVALID_ARG;
  const bool vec = dtype == DET_F32 ? vectors<float>(x, x_stride, cols) && vectors<float>(out, 0, cols)
                                    : vectors<__half>(x, x_stride, cols) && vectors<__half>(out, 0, cols);
  return norm_forward(x, dtype, rows, cols, x_stride, weight, bias, param_dtype, eps, out, mean_out, rstd_out, vec,
                      as_stream(stream));
}

extern "C" size_t det_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols) {
  if (check_rows(DET_F32, DET_F32, rows, cols) != DET_OK || rows == 0) return 256;
  return 256 + align_up((size_t)grad_parts(rows, cols) * 2 * (size_t)whole_eights((int)cols) * sizeof(float), 256);
}

extern "C" int det_layer_norm_backward(const void* grad, int64_t grad_stride, const void* x, int64_t x_stride, int dtype,
                                       int64_t rows, int64_t cols, const float* mean, const float* rstd,
                                       const void* weight, int param_dtype, void* grad_x, void* grad_weight,
                                       void* grad_bias, void* workspace, size_t workspace_bytes, void* stream) {
  if (const int rc = check_rows(dtype, param_dtype, rows, cols)) return rc;
  if (grad_stride < 0 || x_stride < 0) return DET_ERR_INVALID_ARG;
  if (rows > 0 && (!grad || !x || !mean || !rstd)) return DET_ERR_INVALID_ARG;
  if (misaligned(grad, dtype) || misaligned(x, dtype) || misaligned(grad_x, dtype) || misaligned(weight, param_dtype) ||
      misaligned(grad_weight, param_dtype) || misaligned(grad_bias, param_dtype) || misaligned(mean, DET_F32) ||
      misaligned(rstd, DET_F32))
    return DET_ERR_INVALID_ARG;
  const bool params = (grad_weight || grad_bias) && cols > 0;
  if (params && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
                 workspace_bytes < det_layer_norm_backward_workspace_bytes(rows, cols)))
    return DET_ERR_WORKSPACE;
  const cudaStream_t s = as_stream(stream);
  float* part = params ? static_cast<float*>(workspace) : nullptr;
  if (rows > 0 && (params || grad_x)) {
    const bool vec = dtype == DET_F32 ? vectors<float>(x, x_stride, cols) && vectors<float>(grad, grad_stride, cols) &&
                                            vectors<float>(grad_x, 0, cols)
                                      : vectors<__half>(x, x_stride, cols) && vectors<__half>(grad, grad_stride, cols) &&
                                            vectors<__half>(grad_x, 0, cols);
    if (const int rc = norm_backward(grad, grad_stride, x, x_stride, dtype, rows, cols, mean, rstd, weight, param_dtype,
                                     grad_x, part, vec, s))
      return rc;
  }
  if (!params) return DET_OK;
  launch_begin("det_layer_norm_join", s);
  const cudaError_t e = launch_dep(layer_norm_join_kernel, dim3((unsigned)((cols + 31) / 32), 2), dim3(1024), 0, s,
                                   (const float*)part, rows > 0 ? grad_parts(rows, cols) : 0, (int)cols, grad_weight,
                                   grad_bias, param_dtype);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_layer_norm_join");
}
