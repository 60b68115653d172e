// det_embedding: rows of a table by token, scaled, and the table's gradient.
//
// The gradient is the row scatter-add of det_scatter_add_rows on tokens, for
// 16-bit inputs too and without its slow case, a destination that many rows
// aim at (the most frequent token of a text is met in every twentieth place):
//   1. the tokens are sorted stably (payload: the position);
//   2. every run of one token is cut into blocks of 32 by rank; a warp reduces
//      256 columns of every block that begins among its positions of the sorted
//      order, streaming through them eight rows at a time whatever runs they
//      belong to, and writes the row (or for a run of more than a block the block's
//      node);
//   3. the nodes of long runs are joined, eight warps a run and 64 columns.
// Blocks are subtrees of the canonical pairwise tree over a run's ranks, so the
// sums are those of det_scatter_add_rows bit for bit.
#include "det_sort.cuh"
#include "det_model.cuh"

#include <algorithm>

namespace det {
namespace {

constexpr int kEights = 4;      // eights a thread has in flight, a row's threads apart

// grid.x: rows, blockDim.x >> log2_threads at a time; grid.y: spans of the columns.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(256)
embedding_kernel(const T* table, int vocab, int dim, long long stride, const int32_t* tokens, int n, float scale, O* out,
                 int log2_threads) {
  dep_wait();
  dep_launch();
  const int threads = 1 << log2_threads, me = threadIdx.x & (threads - 1);
  const long long i = (long long)blockIdx.x * (blockDim.x >> log2_threads) + (threadIdx.x >> log2_threads);
  if (i >= n) return;
  const int token = tokens[i];
  const bool known = (unsigned)token < (unsigned)vocab;
  const T* row = table + (known ? token * stride : 0);
  const int c0 = (blockIdx.y * threads * kEights + me) * 8;
  Eight<T> e[kEights];
#pragma unroll
  for (int k = 0; k < kEights; ++k) {
    const int c = c0 + k * threads * 8;
    e[k] = load_eight<VEC>(row + c, known ? max(0, min(8, dim - c)) : 0);
  }
#pragma unroll
  for (int k = 0; k < kEights; ++k) {
    const int c = c0 + k * threads * 8;
    float v[8];
    unpack_eight(e[k], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = known ? __fmul_rn(v[j], scale) : 0.0f;
    store_eight<VEC>(out + i * dim + c, v, max(0, min(8, dim - c)));
  }
}

// ---------------------------------------------------------------------------
// gradient

constexpr int kBlock = 32;       // ranks of a block
constexpr int kRound = 8;        // rows in flight
constexpr int kSlice = 256;      // columns of a warp

// A run of more than one block, for the join.
struct LongRun {
  int token, start, end;
};

// The workspace after the sort's.
struct EmbedPlan {
  size_t runs, nodes, total;
};
EmbedPlan embed_plan(const SortPlan& sort, long long n, long long dim) {
  EmbedPlan p;
  p.runs = align_up(sort.total, 256);
  p.nodes = align_up(p.runs + (size_t)(n / kBlock + 1) * sizeof(LongRun), 256);
  // a window of 32 sorted positions holds at most two beginnings of a long run's blocks: of one that ends
  // in it or passes it, and of one that starts in it (two blocks of one run begin 32 positions apart,
  // and a run that starts here and is long passes the window's end)
  p.total = p.nodes + align_up((size_t)(n / kBlock + 1) * 2 * (size_t)dim * sizeof(float), 256);
  return p;
}
// The place of the node of the block that begins at sorted position q, `first` in its run.
__host__ __device__ inline long long node_slot(long long q, bool first) { return q / kBlock * 2 + (first ? 1 : 0); }

struct GradArgs {
  const int32_t* tokens;
  const int32_t* perm;           // positions in the order of their tokens
  const int32_t* seg;            // where a token's run starts in it
  const unsigned* n_valid;
  unsigned* long_runs;           // how many
  LongRun* runs;
  float* nodes;
  int n, vocab, dim;
  long long stride;
  float scale;
};

template <typename O>
__device__ __forceinline__ float finish(float sum, float scale, const O* old, bool accumulate) {
  const float v = __fmul_rn(sum, scale);
  return accumulate ? __fadd_rn(to_f32(*old), v) : v;
}

// A warp: the blocks that begin at sorted positions [w * window, (w + 1) *
// window), columns blockIdx.y * 256 and on.
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(256)
embedding_blocks_kernel(const T* grad, GradArgs a, O* out, int accumulate, int window) {
  dep_wait();
  dep_launch();
  const int lane = threadIdx.x & 31;
  const int valid = min((int)*a.n_valid, a.n);
  const long long w0 = ((long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * window;
  if (w0 >= valid) return;
  // 64 positions from w0 on, two a lane: what they hold, and where blocks begin and end
  int from[2], token[2], run0[2], run1[2];
  unsigned begins[2], ends[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long q = w0 + h * 32 + lane;
    bool in = q < valid;
    from[h] = in ? a.perm[q] : 0;
    in = in && (unsigned)from[h] < (unsigned)a.n;      // what follows an unfinished sort (its waits are bounded)
    token[h] = in ? a.tokens[from[h]] : 0;
    in = in && (unsigned)token[h] < (unsigned)a.vocab; // is left out
    run0[h] = in ? a.seg[token[h]] : 0;
    run1[h] = in ? a.seg[token[h] + 1] : 0;
    in = in && run0[h] >= 0 && run0[h] <= q && q < run1[h] && run1[h] <= valid;
    const int rank = (int)q - run0[h];
    begins[h] = __ballot_sync(0xffffffffu, in && rank % kBlock == 0);
    ends[h] = __ballot_sync(0xffffffffu, in && (rank % kBlock == kBlock - 1 || q + 1 == run1[h]));
  }
  const unsigned long long begin = begins[0] | (unsigned long long)begins[1] << 32;
  const unsigned long long end = ends[0] | (unsigned long long)ends[1] << 32;
  const unsigned long long here = begin & ((window == 32 ? 0xffffffffull : (1ull << window) - 1));
  if (here == 0) return;
  const int c = blockIdx.y * kSlice + lane * 8;
  const int nc = max(0, min(8, a.dim - c));
  const int p0 = __ffsll((long long)here) - 1;
  // the last block that begins here ends at the first end behind its beginning
  const int last = 63 - __clzll((long long)here);
  const int p1 = __ffsll((long long)(end >> last << last)) - 1;
  if (p1 < 0) return;
  float st[5][8];                // pending nodes of a block's tree: 1, 2, 4, 8, 16 rows
  int rank = 0;
  for (int p = p0; p <= p1; p += kRound) {
    Eight<T> e[kRound];
#pragma unroll
    for (int j = 0; j < kRound; ++j) {
      const int q = p + j;
      const int f = __shfl_sync(0xffffffffu, q < 32 ? from[0] : from[1], q & 31);
      e[j] = load_eight<VEC>(grad + f * a.stride + c, q <= p1 ? nc : 0);
    }
#pragma unroll
    for (int j = 0; j < kRound; ++j) {
      const int q = p + j;
      if (q > p1) break;
      if (begin >> q & 1) rank = 0;
      float v[8];
      unpack_eight(e[j], v);
      // a binary counter: the new leaf is added to the pending node of each level it completes
      int level = 0;
#pragma unroll
      for (int l = 0; l < 5; ++l) {
        if (level == l && (rank >> l & 1)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = st[l][i] + v[i];
          level = l + 1;
        }
      }
#pragma unroll
      for (int l = 0; l < 5; ++l)
        if (level == l) {
#pragma unroll
          for (int i = 0; i < 8; ++i) st[l][i] = v[i];
        }
      ++rank;
      if (!(end >> q & 1)) continue;
      // the block's node: the pending ones from the smallest up
      if (rank < kBlock) {
        bool have = false;
#pragma unroll
        for (int l = 0; l < 5; ++l)
          if (rank >> l & 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = have ? st[l][i] + v[i] : st[l][i];
            have = true;
          }
      }
      const int src = q & 31;
      const int lo = __shfl_sync(0xffffffffu, q < 32 ? run0[0] : run0[1], src);
      const int hi = __shfl_sync(0xffffffffu, q < 32 ? run1[0] : run1[1], src);
      const int tok = __shfl_sync(0xffffffffu, q < 32 ? token[0] : token[1], src);
      if (hi - lo <= kBlock) {
        O* to = out + (long long)tok * a.dim + c;
        if (accumulate) {
          float old[8];
          unpack_eight(load_eight<VEC>(to, nc), old);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fadd_rn(old[i], __fmul_rn(v[i], a.scale));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], a.scale);
        }
        store_eight<VEC>(to, v, nc);
      } else {
        const long long start = w0 + q - (rank - 1);
        float* to = a.nodes + node_slot(start, start == lo) * a.dim + c;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < nc) to[i] = v[i];
        if (start == lo && blockIdx.y == 0 && lane == 0) {
          const unsigned k = atomicAdd(a.long_runs, 1u);       // in any order: runs do not meet
          if (k <= (unsigned)(a.n / kBlock)) a.runs[k] = {tok, lo, hi};
        }
      }
    }
  }
}

// A CTA joins 64 columns of a long run: the tree over its blocks, aligned subtrees
// of them by each warp.
constexpr int kJoinWarps = 8;
template <typename O>
__global__ void __launch_bounds__(32 * kJoinWarps)
embedding_join_kernel(GradArgs a, O* out, int accumulate) {
  __shared__ float2 s_node[kJoinWarps][32];
  dep_wait();
  dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.y * 64 + lane * 2;
  const unsigned count = min(*a.long_runs, (unsigned)(a.n / kBlock) + 1u);
  for (unsigned k = blockIdx.x; k < count; k += gridDim.x) {
    const LongRun run = a.runs[k];
    const int blocks = (run.end - run.start + kBlock - 1) / kBlock;
    int span = 1;                                  // blocks of a warp
    while (span * kJoinWarps < blocks) span *= 2;
    const int b1 = min(blocks, (warp + 1) * span);
    float2 total = make_float2(absent<float>(), absent<float>());
    if (c < a.dim) {
      const bool two = c + 1 < a.dim;
      NodeCounter<float, 6> nx, ny;
      for (int b = warp * span; b < b1; b += 8) {
        float x[8], y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool in = b + j < b1;
          const float* p = a.nodes + node_slot(run.start + (long long)(b + j) * kBlock, b + j == 0) * a.dim + c;
          x[j] = in ? p[0] : absent<float>();
          y[j] = in && two ? p[1] : absent<float>();
        }
        nx.push(thread_pt(x));
        ny.push(thread_pt(y));
      }
      total = make_float2(nx.result(), ny.result());
    }
    s_node[warp][lane] = total;
    __syncthreads();
    if (warp == 0 && c < a.dim) {
      float x[kJoinWarps], y[kJoinWarps];
#pragma unroll
      for (int j = 0; j < kJoinWarps; ++j) {
        x[j] = s_node[j][lane].x;
        y[j] = s_node[j][lane].y;
      }
      O* to = out + (long long)run.token * a.dim + c;
      to[0] = from_f32<O>(finish(thread_pt(x), a.scale, to, accumulate));
      if (c + 1 < a.dim) to[1] = from_f32<O>(finish(thread_pt(y), a.scale, to + 1, accumulate));
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------

constexpr int64_t kMostDim = 1 << 21;       // 64 columns a CTA: the grid's second dimension

template <typename T>
bool vectors(const void* p, int64_t stride) {
  return (reinterpret_cast<uintptr_t>(p) | (uintptr_t)(stride * sizeof(T))) % 16 == 0;
}

template <typename T, typename O>
int forward(const void* table, int vocab, int dim, int64_t stride, const int32_t* tokens, int n, float scale, void* out,
            cudaStream_t s) {
  const bool vec = vectors<T>(table, stride) && vectors<O>(out, dim) && dim * sizeof(T) % 16 == 0;
  int l = 0;                                     // threads of a row, at most 256
  while (l < 8 && (8LL * kEights << l) < dim) ++l;
  const unsigned at_a_time = 256u >> l;
  const dim3 grid((n + at_a_time - 1) / at_a_time, (unsigned)((dim + (8LL * kEights << l) - 1) / (8LL * kEights << l)));
  launch_begin("det_embedding", s);
  const cudaError_t e =
      launch_dep(vec ? embedding_kernel<T, O, true> : embedding_kernel<T, O, false>, grid, dim3(256), 0, s,
                 static_cast<const T*>(table), vocab, dim, (long long)stride, tokens, n, scale, static_cast<O*>(out), l);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_embedding");
}

template <typename T, typename O>
int blocks(const void* grad, const GradArgs& a, int n, void* out, int accumulate, cudaStream_t s) {
  const bool vec = vectors<T>(grad, a.stride) && vectors<O>(out, a.dim) && a.dim * sizeof(T) % 16 == 0;
  const unsigned slices = (unsigned)((a.dim + kSlice - 1) / kSlice);
  // windows of 32 positions, shorter ones while they leave SMs without a warp
  int window = 32;
  while (window > 8 && (long long)slices * (n / window) < 8LL * 152) window /= 2;
  const unsigned warps = (unsigned)((n + (long long)window - 1) / window), per_cta = warps < 8 ? 1 : 8;
  launch_begin("det_embedding_blocks", s);
  const cudaError_t e = launch_dep(vec ? embedding_blocks_kernel<T, O, true> : embedding_blocks_kernel<T, O, false>,
                                   dim3((warps + per_cta - 1) / per_cta, slices), dim3(32 * per_cta), 0, s,
                                   static_cast<const T*>(grad), a, static_cast<O*>(out), accumulate, window);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_embedding_blocks");
}
template <typename O>
int join(const GradArgs& a, int n, void* out, int accumulate, cudaStream_t s) {
  // at most n / 33 long runs; the CTAs take what there are in turn
  const unsigned across = (unsigned)((a.dim + 63) / 64);
  const unsigned runs = (unsigned)std::max(1LL, std::min<long long>(n / (kBlock + 1), 8LL * 152 / across));
  launch_begin("det_embedding_join", s);
  const cudaError_t e = launch_dep(embedding_join_kernel<O>, dim3(runs, across), dim3(32 * kJoinWarps), 0, s, a,
                                   static_cast<O*>(out), accumulate);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_embedding_join");
}

int check_table(int dtype, int table_dtype, int64_t n, int64_t vocab, int64_t dim) {
  if (!valid_model_dtype(dtype) || !valid_model_dtype(table_dtype)) return DET_ERR_DTYPE;
  if (n < 0 || vocab < 0 || dim < 0) return DET_ERR_INVALID_ARG;
  if (n >= (1LL << 31) || vocab >= (1LL << 31) || dim > kMostDim) return DET_ERR_TOO_LARGE;
  return DET_OK;
}
bool misaligned(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % model_elem_size(dtype) != 0; }

}  // namespace
}  // namespace det

using namespace det;

#define DET_EMBED_PICK_T(fn, T, code, ...)                        \
  do {                                                            \
    if ((code) == DET_F32) return fn<T, float>(__VA_ARGS__);      \
    if ((code) == DET_BF16) return fn<T, __nv_bfloat16>(__VA_ARGS__); \
    return fn<T, __half>(__VA_ARGS__);                            \
  } while (0)
#define DET_EMBED_PICK(fn, first, second, ...)                                       \
  do {                                                                               \
    if ((first) == DET_F32) DET_EMBED_PICK_T(fn, float, second, __VA_ARGS__);        \
    if ((first) == DET_BF16) DET_EMBED_PICK_T(fn, __nv_bfloat16, second, __VA_ARGS__); \
    DET_EMBED_PICK_T(fn, __half, second, __VA_ARGS__);                               \
  } while (0)

static int embed_blocks(int dtype, int table_dtype, const void* grad, const GradArgs& a, int n, void* out, int accumulate,
                        cudaStream_t s) {
  DET_EMBED_PICK(blocks, dtype, table_dtype, grad, a, n, out, accumulate, s);
}

extern "C" int det_embedding(const void* table, int table_dtype, int64_t vocab, int64_t dim, int64_t table_stride,
                             const int32_t* tokens, int64_t n, float scale, void* out, int dtype, void* stream) {
  if (const int rc = check_table(dtype, table_dtype, n, vocab, dim)) return rc;
  if (table_stride < 0) return DET_ERR_INVALID_ARG;
  if (n == 0 || dim == 0) return DET_OK;
  if (!tokens || !out || (vocab > 0 && !table)) return DET_ERR_INVALID_ARG;
  if (misaligned(table, table_dtype) || misaligned(out, dtype) || misaligned(tokens, DET_F32)) return DET_ERR_INVALID_ARG;
  DET_EMBED_PICK(forward, table_dtype, dtype, table, (int)vocab, (int)dim, table_stride, tokens, (int)n, scale, out,
                 as_stream(stream));
}

extern "C" size_t det_embedding_backward_workspace_bytes(int64_t n, int64_t vocab, int64_t dim) {
  if (check_table(DET_F32, DET_F32, n, vocab, dim) != DET_OK) return 0;
  return embed_plan(make_sort_plan(n, vocab, 0, true, 0), n, dim).total;
}

extern "C" int det_embedding_backward(const void* grad, int dtype, int64_t n, int64_t dim, int64_t grad_stride,
                                      const int32_t* tokens, float scale, void* grad_table, int table_dtype,
                                      int64_t vocab, int accumulate, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (const int rc = check_table(dtype, table_dtype, n, vocab, dim)) return rc;
  if (grad_stride < 0) return DET_ERR_INVALID_ARG;
  if (vocab == 0 || dim == 0) return DET_OK;
  if (!grad_table || (n > 0 && (!grad || !tokens))) return DET_ERR_INVALID_ARG;
  if (misaligned(grad, dtype) || misaligned(grad_table, table_dtype) || misaligned(tokens, DET_F32))
    return DET_ERR_INVALID_ARG;
  const SortPlan sort = make_sort_plan(n, vocab, 0, true, 0);
  const EmbedPlan plan = embed_plan(sort, n, dim);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < plan.total) return DET_ERR_WORKSPACE;
  const cudaStream_t s = as_stream(stream);
  if (!accumulate) {
    const cudaError_t e = cudaMemsetAsync(grad_table, 0, (size_t)vocab * dim * model_elem_size(table_dtype), s);
    if (e != cudaSuccess) return cuda_fail(e, "det_embedding_backward: clear");
  }
  if (n == 0) return DET_OK;
  int buffer = 0;
  if (const int rc = enqueue_sort(sort, workspace, tokens, 0, nullptr, nullptr, s, &buffer)) return rc;
  char* w = static_cast<char*>(workspace);
  GradArgs a;
  a.tokens = tokens;
  a.perm = reinterpret_cast<const int32_t*>(w + sort.idx[buffer]);
  a.seg = reinterpret_cast<const int32_t*>(w + sort.seg);
  a.n_valid = &reinterpret_cast<SortHdr*>(w)->n_valid;
  a.long_runs = &reinterpret_cast<SortHdr*>(w)->long_segs;       // cleared by the sort, which does not use it
  a.runs = reinterpret_cast<LongRun*>(w + plan.runs);
  a.nodes = reinterpret_cast<float*>(w + plan.nodes);
  a.n = (int)n;
  a.vocab = (int)vocab;
  a.dim = (int)dim;
  a.stride = grad_stride;
  a.scale = scale;
  if (const int rc = embed_blocks(dtype, table_dtype, grad, a, (int)n, grad_table, accumulate ? 1 : 0, s)) return rc;
  if (n <= kBlock) return DET_OK;                                // no run is longer than a block
  if (table_dtype == DET_F32) return join<float>(a, (int)n, grad_table, accumulate ? 1 : 0, s);
  if (table_dtype == DET_BF16) return join<__nv_bfloat16>(a, (int)n, grad_table, accumulate ? 1 : 0, s);
  return join<__half>(a, (int)n, grad_table, accumulate ? 1 : 0, s);
}
