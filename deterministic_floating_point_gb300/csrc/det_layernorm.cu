// det_layer_norm and its gradients.
//
// A row lies in the registers of a group of threads: 32 to 1,024 of them, eight or
// sixteen columns each (eights, the group's threads apart), so it is read once.
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
#include "det_model.cuh"

#include <algorithm>

namespace det {
namespace {

// The lanes' sums of a group, in every thread: a tree over lanes, then over
// warps through `slot` (one float a warp).  A group of one warp needs no barrier.
__device__ __forceinline__ void put_warp(float* slot, float v, int warp, int lane) {
  if (lane == 0) slot[warp] = v;
}
__device__ __forceinline__ float over_warps(const float* slot, int first_warp, int warps, int lane) {
  float v = slot[first_warp + (lane & (warps - 1))];
  for (int s = 1; s < warps; s <<= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}
template <int N>
__device__ __forceinline__ float tree(const float (&v)[N]) {
  float t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = v[i];
  return thread_pt(t);
}

// A group's place: `threads` (a power of two) of them take a row.
struct Group {
  int me, threads, warps, warp, first_warp, lane, index, count;
  __device__ __forceinline__ explicit Group(int log2_threads) {
    threads = 1 << log2_threads;
    me = threadIdx.x & (threads - 1);
    warps = threads >> 5;
    warp = threadIdx.x >> 5;
    lane = threadIdx.x & 31;
    index = threadIdx.x >> log2_threads;
    first_warp = index * warps;
    count = blockDim.x >> log2_threads;
  }
};

template <typename T, bool VEC, int K>
__device__ __forceinline__ void load_row(Eight<T> (&e)[K], const T* row, const Group& g, int cols, bool valid) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (g.me + k * g.threads) * 8;
    e[k] = load_eight<VEC>(row + c, valid ? max(0, min(8, cols - c)) : 0);
  }
}

constexpr int kThreads = 256;       // a CTA's, unless a row takes more

template <typename T, int K, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST, MOST > 256 ? 1 : K == 1 ? 4 : 3)
layer_norm_kernel(const T* x, int rows, int cols, long long x_stride, const void* weight, const void* bias,
                  int param_dtype, float eps, T* out, float* mean_out, float* rstd_out, int log2_threads) {
  __shared__ float s_sum[32], s_sq[32];
  dep_wait();
  dep_launch();
  const Group g(log2_threads);
  float w[K][8], b[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = (g.me + k * g.threads) * 8 + i;
      w[k][i] = weight && c < cols ? load_as_f32(weight, c, param_dtype) : 1.0f;
      b[k][i] = bias && c < cols ? load_as_f32(bias, c, param_dtype) : 0.0f;
    }
  const long long step = (long long)gridDim.x * g.count;
  const float of = 1.0f / (float)cols;
  long long first = (long long)blockIdx.x * g.count;       // of the CTA's rows: every thread makes as many rounds
  long long r = first + g.index;
  Eight<T> cur[K];
  load_row<T, VEC>(cur, x + r * x_stride, g, cols, r < rows);
  for (; first < rows; first += step, r += step) {
    Eight<T> next[K];
    load_row<T, VEC>(next, x + (r + step) * x_stride, g, cols, r + step < rows);
    float v[K][8], part[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      unpack_eight(cur[k], v[k]);
      part[k] = tree(v[k]);
    }
    float sum = warp_pt(tree(part));
    if (g.warps > 1) {
      put_warp(s_sum, sum, g.warp, g.lane);
      __syncthreads();
      sum = over_warps(s_sum, g.first_warp, g.warps, g.lane);
    }
    const float mean = sum * of;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int n = cols - (g.me + k * g.threads) * 8;
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[k][i] -= mean;
        q[i] = i < n ? v[k][i] * v[k][i] : 0.0f;
      }
      part[k] = tree(q);
    }
    float sq = warp_pt(tree(part));
    if (g.warps > 1) {
      put_warp(s_sq, sq, g.warp, g.lane);
      __syncthreads();
      sq = over_warps(s_sq, g.first_warp, g.warps, g.lane);
    }
    const float rstd = 1.0f / sqrtf(fmaf(sq, of, eps));
    if (r < rows) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (g.me + k * g.threads) * 8;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = fmaf(v[k][i] * rstd, w[k][i], b[k][i]);
        store_eight<VEC>(out + r * cols + c, y, max(0, min(8, cols - c)));
      }
      if (g.me == 0) {
        if (mean_out) mean_out[r] = mean;
        if (rstd_out) rstd_out[r] = rstd;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) cur[k] = next[k];
  }
}

// part: [gridDim.x][2][cols] sums of the weight's and the bias' gradients, or NULL.
template <typename T, int K, bool VEC, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 ? 2 : 1)
layer_norm_grad_kernel(const T* grad, long long grad_stride, const T* x, long long x_stride, int rows, int cols,
                       const float* means, const float* rstds, const void* weight, int param_dtype, T* grad_x,
                       float* part, int log2_threads) {
  __shared__ float s_one[2][32], s_two[2][32];
  extern __shared__ float s_acc[];
  dep_wait();
  dep_launch();
  const Group g(log2_threads);
  float w[K][8], aw[K][8], ab[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = (g.me + k * g.threads) * 8 + i;
      w[k][i] = weight && c < cols ? load_as_f32(weight, c, param_dtype) : 1.0f;
      aw[k][i] = ab[k][i] = 0.0f;
    }
  const long long step = (long long)gridDim.x * g.count;
  const float of = 1.0f / (float)cols;
  long long first = (long long)blockIdx.x * g.count;
  long long r = first + g.index;
  Eight<T> cx[K], cg[K];
  load_row<T, VEC>(cx, x + r * x_stride, g, cols, r < rows);
  load_row<T, VEC>(cg, grad + r * grad_stride, g, cols, r < rows);
  float cm = r < rows ? means[r] : 0.0f, cr = r < rows ? rstds[r] : 0.0f;
  int parity = 0;
  for (; first < rows; first += step, r += step, parity ^= 1) {
    Eight<T> nx[K], ng[K];
    const bool more = r + step < rows;
    load_row<T, VEC>(nx, x + (r + step) * x_stride, g, cols, more);
    load_row<T, VEC>(ng, grad + (r + step) * grad_stride, g, cols, more);
    const float nm = more ? means[r + step] : 0.0f, nr = more ? rstds[r + step] : 0.0f;
    float p1[K], p2[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float xh[8], d[8], q1[8], q2[8];
      unpack_eight(cx[k], xh);
      unpack_eight(cg[k], d);
      const int n = cols - (g.me + k * g.threads) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[i] = i < n ? (xh[i] - cm) * cr : 0.0f;
        aw[k][i] = fmaf(d[i], xh[i], aw[k][i]);
        ab[k][i] += d[i];
        q1[i] = d[i] * w[k][i];
        q2[i] = q1[i] * xh[i];
      }
      p1[k] = tree(q1);
      p2[k] = tree(q2);
    }
    float one = warp_pt(tree(p1)), two = warp_pt(tree(p2));
    if (g.warps > 1) {
      put_warp(s_one[parity], one, g.warp, g.lane);
      put_warp(s_two[parity], two, g.warp, g.lane);
      __syncthreads();
      one = over_warps(s_one[parity], g.first_warp, g.warps, g.lane);
      two = over_warps(s_two[parity], g.first_warp, g.warps, g.lane);
    }
    if (grad_x && r < rows) {
      one *= of;
      two *= of;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int c = (g.me + k * g.threads) * 8;
        float xh[8], d[8];
        unpack_eight(cx[k], xh);
        unpack_eight(cg[k], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = cr * (fmaf(d[i], w[k][i], -one) - (xh[i] - cm) * cr * two);
        store_eight<VEC>(grad_x + r * cols + c, d, max(0, min(8, cols - c)));
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) cx[k] = nx[k], cg[k] = ng[k];
    cm = nm;
    cr = nr;
  }
  if (!part) return;
  float* mine = part + (long long)blockIdx.x * 2 * cols;
  if (g.count == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (g.me + k * g.threads) * 8 + i;
        if (c < cols) mine[c] = aw[k][i], mine[cols + c] = ab[k][i];
      }
    return;
  }
  // several rows at a time: the groups' sums in the groups' order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = (g.me + k * g.threads) * 8 + i;
        if (c < cols) s_acc[g.index * cols + c] = which ? ab[k][i] : aw[k][i];
      }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      float t = s_acc[c];
      for (int j = 1; j < g.count; ++j) t += s_acc[j * cols + c];
      mine[which * cols + c] = t;
    }
  }
}

// grad[c] = the sum of parts rows: 32 strands of every 32nd row, then a tree.
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
    const float* p = part + (long long)blockIdx.y * cols + c;
#pragma unroll 4
    for (int j = warp; j < parts; j += 32) t += p[(long long)j * 2 * cols];
  }
  s[warp][lane] = t;
  __syncthreads();
  const float total = warp_pt(s[lane][warp]);
  const int of = blockIdx.x * 32 + warp;
  if (lane == 0 && of < cols) store_from_f32(to, of, total, param_dtype);
}

// Threads that take a row, as a logarithm: two eights each, one of up to 256 columns.
int row_threads(int64_t cols) {
  int l = 5;
  while ((16LL << l) < cols) ++l;
  return l;
}
// CTAs of the gradient, each of which leaves a partial sum: as many as run at once on
// the 152 SMs, by a constant, because the sums' order hangs on it.
int grad_parts(int64_t rows, int64_t cols) {
  const int l = row_threads(cols);
  const int64_t at_a_time = std::max<int64_t>(1, kThreads >> l);
  return (int)std::min<int64_t>((rows + at_a_time - 1) / at_a_time, l <= 8 ? 304 : 152);
}

template <typename T>
bool vectors(const void* p, int64_t stride, int64_t cols) {
  return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * sizeof(T)) | (uintptr_t)(cols * sizeof(T))) % 16 == 0;
}

template <typename T, int K, bool VEC, int MOST>
int forward(const void* x, int rows, int cols, int64_t x_stride, const void* weight, const void* bias, int param_dtype,
            float eps, void* out, float* mean_out, float* rstd_out, cudaStream_t s) {
  const int l = row_threads(cols), threads = std::max(kThreads, 1 << l), at_a_time = threads >> l;
  auto* k = layer_norm_kernel<T, K, VEC, MOST>;
  const int per_sm = kernel_occupancy((const void*)k, threads, 0);
  if (per_sm <= 0) return cuda_fail(cudaErrorUnknown, "det_layer_norm");
  const long long grid = std::min<long long>((rows + (long long)at_a_time - 1) / at_a_time,
                                             (long long)per_sm * std::max(device_sm_count(), 1));
  launch_begin("det_layer_norm", s);
  const cudaError_t e = launch_dep(k, dim3((unsigned)grid), dim3(threads), 0, s, static_cast<const T*>(x), rows, cols,
                                   (long long)x_stride, weight, bias, param_dtype, eps, static_cast<T*>(out), mean_out,
                                   rstd_out, l);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_layer_norm");
}

template <typename T, int K, bool VEC, int MOST>
int backward(const void* grad, int64_t grad_stride, const void* x, int64_t x_stride, int rows, int cols,
             const float* mean, const float* rstd, const void* weight, int param_dtype, void* grad_x, float* part,
             cudaStream_t s) {
  const int l = row_threads(cols), threads = std::max(kThreads, 1 << l), at_a_time = threads >> l;
  auto* k = layer_norm_grad_kernel<T, K, VEC, MOST>;
  const size_t smem = part && at_a_time > 1 ? (size_t)at_a_time * cols * sizeof(float) : 0;
  launch_begin("det_layer_norm_backward", s);
  const cudaError_t e = launch_dep(k, dim3((unsigned)grad_parts(rows, cols)), dim3(threads), smem, s,
                                   static_cast<const T*>(grad), (long long)grad_stride, static_cast<const T*>(x),
                                   (long long)x_stride, rows, cols, mean, rstd, weight, param_dtype,
                                   static_cast<T*>(grad_x), part, l);
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

// One eight a thread up to 256 columns, two above; CTAs of more than 256 threads where a
// row takes them.
#define DET_NORM_PICK_T(fn, T, ...)                                                                      \
  do {                                                                                                   \
    if (cols <= 256) return vec ? fn<T, 1, true, 256>(__VA_ARGS__) : fn<T, 1, false, 256>(__VA_ARGS__);  \
    if (cols <= 4096) return vec ? fn<T, 2, true, 256>(__VA_ARGS__) : fn<T, 2, false, 256>(__VA_ARGS__); \
    if (cols <= 8192) return vec ? fn<T, 2, true, 512>(__VA_ARGS__) : fn<T, 2, false, 512>(__VA_ARGS__); \
    return vec ? fn<T, 2, true, 1024>(__VA_ARGS__) : fn<T, 2, false, 1024>(__VA_ARGS__);                 \
  } while (0)
#define DET_NORM_PICK(fn, ...)                                                 \
  do {                                                                         \
    if (dtype == DET_F32) DET_NORM_PICK_T(fn, float, __VA_ARGS__);             \
    if (dtype == DET_BF16) DET_NORM_PICK_T(fn, __nv_bfloat16, __VA_ARGS__);    \
    DET_NORM_PICK_T(fn, __half, __VA_ARGS__);                                  \
  } while (0)

static int norm_forward(const void* x, int dtype, int64_t rows, int64_t cols, int64_t x_stride, const void* weight,
                        const void* bias, int param_dtype, float eps, void* out, float* mean_out, float* rstd_out,
                        bool vec, cudaStream_t s) {
  DET_NORM_PICK(forward, x, (int)rows, (int)cols, x_stride, weight, bias, param_dtype, eps, out, mean_out, rstd_out, s);
}
static int norm_backward(const void* grad, int64_t grad_stride, const void* x, int64_t x_stride, int dtype, int64_t rows,
                         int64_t cols, const float* mean, const float* rstd, const void* weight, int param_dtype,
                         void* grad_x, float* part, bool vec, cudaStream_t s) {
  DET_NORM_PICK(backward, grad, grad_stride, x, x_stride, (int)rows, (int)cols, mean, rstd, weight, param_dtype, grad_x,
                part, s);
}

extern "C" int det_layer_norm(const void* x, int dtype, int64_t rows, int64_t cols, int64_t x_stride,
                              const void* weight, const void* bias, int param_dtype, float eps, void* out,
                              float* mean_out, float* rstd_out, void* stream) {
  if (const int rc = check_rows(dtype, param_dtype, rows, cols)) return rc;
  if (!(eps >= 0.0f) || x_stride < 0) return DET_ERR_INVALID_ARG;
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
  return 256 + align_up((size_t)grad_parts(rows, cols) * 2 * (size_t)cols * sizeof(float), 256);
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
