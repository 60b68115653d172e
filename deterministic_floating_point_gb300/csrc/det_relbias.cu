// det_relative_bias and det_relative_bias_backward (include/det_model.h).
//
// The bias of a (query i, key j) pair depends on the diagonal j - i alone.
// Forward: every output is one table entry.  Backward: the sum over a bucket
// is taken diagonal by diagonal (each a sum over batch and queries in rising
// order), then over the bucket's diagonals, which are neighbours: a bucket is
// one interval of distances.  The order of the additions is fixed by indices.
#include "det_model.cuh"

#include <algorithm>

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
      if (__ldg(bounds + mid) <= n) lo = mid + 1;
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
    const int near = b > 0 ? max(__ldg(bounds + b - 1), 0) : 0;                  // least |distance|
    const int far = b < num_bounds ? __ldg(bounds + b) : 0x7fffffff;   // first |distance| beyond
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

template <typename T>
__global__ void __launch_bounds__(256)
relative_bias_kernel(const void* __restrict__ table, int table_dtype, int heads, Distances dist, int q_len, int k_len,
                     T* __restrict__ out) {
  const int h = blockIdx.z, i = blockIdx.y;
  for (int q = i; q < q_len; q += gridDim.y)
    for (int j = blockIdx.x * blockDim.x + threadIdx.x; j < k_len; j += gridDim.x * blockDim.x) {
      const int k = dist.bucket(j - q + (q_len - 1) + dist.first);
      out[((long long)h * q_len + q) * k_len + j] =
          from_f32<T>(load_as_f32(table, (long long)k * heads + h, table_dtype));
    }
}

struct GradView {
  long long stride_b, stride_h, stride_q;
  int batch, q_len, k_len;
};

// diag[h][d] = the sum of diagonal d of head h.
template <typename T>
__global__ void __launch_bounds__(256)
diagonal_sums_kernel(const T* __restrict__ grad, GradView g, float* __restrict__ diag) {
  const int d = blockIdx.x * blockDim.x + threadIdx.x, h = blockIdx.y;
  const int count = g.q_len + g.k_len - 1;
  if (d >= count) return;
  const int shift = d - (g.q_len - 1);   // key - query index
  const int i0 = max(0, -shift), i1 = min(g.q_len, g.k_len - shift);
  float sum = 0.0f;
  for (int b = 0; b < g.batch; ++b) {
    float part = 0.0f;
    const T* p = grad + b * g.stride_b + h * g.stride_h;
    for (int i = i0; i < i1; ++i) part += to_f32(p[i * g.stride_q + i + shift]);
    sum += part;
  }
  diag[(long long)h * count + d] = sum;
}

// One warp per (bucket, head): lane l adds the bucket's diagonals l, l + 32,
// ... of the interval, then the lanes are added by a tree.
__global__ void __launch_bounds__(32)
bucket_sums_kernel(const float* __restrict__ diag, Distances dist, int diagonals, int heads,
                   void* __restrict__ grad_table, int table_dtype) {
  const int k = blockIdx.x, h = blockIdx.y;
  int lo, hi;
  dist.interval(k, dist.first, dist.first + diagonals, lo, hi);
  const float* p = diag + (long long)h * diagonals - dist.first;
  float sum = 0.0f;
  for (int r = lo + (int)threadIdx.x; r < hi; r += 32) sum += p[r];
  sum = warp_pt(sum);
  if (threadIdx.x == 0) store_from_f32(grad_table, (long long)k * heads + h, sum, table_dtype);
}

int check_shape(int64_t heads, int64_t num_bounds, int64_t q_len, int64_t k_len, int64_t q_offset) {
  if (heads < 0 || num_bounds < 0 || q_len < 0 || k_len < 0) return DET_ERR_INVALID_ARG;
  const int64_t most = (1LL << 31) - 1;
  if (heads > 65535 || num_bounds > DET_MAX_BOUNDS || q_len > most || k_len > most || q_offset > most ||
      q_offset < -most || q_len + k_len + (q_offset < 0 ? -q_offset : q_offset) > most)
    return DET_ERR_TOO_LARGE;
  return DET_OK;
}

template <typename T>
int launch_bias(const void* table, int table_dtype, int heads, const Distances& dist, int q_len, int k_len, void* out,
                cudaStream_t s) {
  const dim3 grid((unsigned)std::min((k_len + 255) / 256, 1024), (unsigned)std::min(q_len, 65535), (unsigned)heads);
  launch_begin("det_relative_bias", s);
  relative_bias_kernel<T><<<grid, 256, 0, s>>>(table, table_dtype, heads, dist, q_len, k_len, static_cast<T*>(out));
  launch_end(s);
  return check_launch("det_relative_bias");
}

template <typename T>
int launch_bias_grad(const void* grad, const GradView& g, const Distances& dist, int heads, int buckets, float* diag,
                     void* grad_table, int table_dtype, cudaStream_t s) {
  const int count = g.q_len > 0 && g.k_len > 0 ? g.q_len + g.k_len - 1 : 0;
  if (count > 0) {
    launch_begin("det_relative_bias_diagonals", s);
    diagonal_sums_kernel<T><<<dim3((unsigned)((count + 255) / 256), (unsigned)heads), 256, 0, s>>>(
        static_cast<const T*>(grad), g, diag);
    launch_end(s);
    if (const int rc = check_launch("det_relative_bias_diagonals")) return rc;
  }
  launch_begin("det_relative_bias_buckets", s);
  bucket_sums_kernel<<<dim3((unsigned)buckets, (unsigned)heads), 32, 0, s>>>(diag, dist, count, heads, grad_table,
                                                                             table_dtype);
  launch_end(s);
  return check_launch("det_relative_bias_buckets");
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
  (void)bidirectional;
  if (batch < 0 || check_shape(heads, num_bounds, q_len, k_len, 0) != DET_OK) return 0;
  return align_up((size_t)heads * (size_t)(q_len + k_len) * sizeof(float) + 256, 256);
}

extern "C" int det_relative_bias_backward(const void* grad, int dtype, int64_t batch, int64_t heads, int64_t q_len,
                                          int64_t k_len, int64_t stride_b, int64_t stride_h, int64_t stride_q,
                                          const int32_t* bounds, int64_t num_bounds, int bidirectional,
                                          int64_t q_offset, void* grad_table, int table_dtype, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  if (!valid_model_dtype(dtype) || !valid_model_dtype(table_dtype)) return DET_ERR_DTYPE;
  if (batch < 0) return DET_ERR_INVALID_ARG;
  if (const int rc = check_shape(heads, num_bounds, q_len, k_len, q_offset)) return rc;
  if (batch >= (1LL << 31)) return DET_ERR_TOO_LARGE;
  if (heads == 0) return DET_OK;
  const bool none = batch == 0 || q_len == 0 || k_len == 0;
  if (!grad_table || (!none && !grad) || (num_bounds > 0 && !bounds)) return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(grad) % model_elem_size(dtype) ||
      reinterpret_cast<uintptr_t>(grad_table) % model_elem_size(table_dtype))
    return DET_ERR_INVALID_ARG;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 ||
      workspace_bytes < det_relative_bias_backward_workspace_bytes(batch, heads, q_len, k_len, num_bounds, bidirectional))
    return DET_ERR_WORKSPACE;
  const GradView g = {stride_b, stride_h, stride_q, (int)batch, none ? 0 : (int)q_len, none ? 0 : (int)k_len};
  const Distances dist = {bounds, (int)num_bounds, bidirectional ? 1 : 0, (int)(1 - q_len - q_offset)};
  const int buckets = (int)(num_bounds + 1) * (bidirectional ? 2 : 1);
  float* diag = static_cast<float*>(workspace);
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32)
    return launch_bias_grad<float>(grad, g, dist, (int)heads, buckets, diag, grad_table, table_dtype, s);
  if (dtype == DET_BF16)
    return launch_bias_grad<__nv_bfloat16>(grad, g, dist, (int)heads, buckets, diag, grad_table, table_dtype, s);
  return launch_bias_grad<__half>(grad, g, dist, (int)heads, buckets, diag, grad_table, table_dtype, s);
}
