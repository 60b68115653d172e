// det_embedding: rows of a table by token, scaled, and the table's gradient.
//
// The gradient is the row scatter-add of det_scatter_add_rows on tokens, for
// 16-bit inputs too and without its slow case, a destination that many rows
// aim at (the most frequent token of a text is met in every twentieth place):
//   1. the positions are put in the order of their tokens, stably.  Up to 32,768 of
//      them 8 CTAs do so for an eighth of the tokens each (those with the same low
//      bits), in shared memory, in two passes of 8 bits, and without a word to each
//      other; the other SMs clear the first 96 MB of the table meanwhile.  (More: the
//      library's sort.)
//   2. every run of one token is cut into blocks of 32 by rank; a warp reduces a
//      slice of the columns of every block that begins among its positions of the
//      sorted order, streaming through them eight rows at a time whatever runs they
//      belong to, and writes the row (or for a run of more than a block the block's
//      node); CTAs among these clear the rest of the table, but for the rows that others write;
//   3. the nodes of long runs are joined, eight warps a run and 64 columns.
// Blocks are subtrees of the canonical pairwise tree over a run's ranks, so the
// sums are those of det_scatter_add_rows bit for bit.
//
// Bytes bound both.  16,384 rows of 2,048 in 32 bits to bf16: 20 us (116 MB, some rows many times: 17 at the copy's
// rate), one launch.  The gradient of 16,384 x 2,048 for 65,536 rows in bf16 (332 MB, 50 us at that rate) takes 77:
// 18 for the sort, which the clear of 96 MB fills, 49 for the sums and the rest of the clear, and about 10 for the join,
// whose launch overlaps the sums' end (11 to 17 by itself, by what the tokens are).  Added to a table in bf16, 73; at odd
// widths (2,047) 109.  (Figures below that compare two ways were taken side by side when the choice was made.)
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
  if constexpr (!VEC) {
    // element after element across the row's threads
    constexpr int N = 8;
    const int end = min(dim, (int)(blockIdx.y + 1) * threads * kEights * 8);
    for (int c = blockIdx.y * threads * kEights * 8 + me; c < end; c += N * threads) {
      float v[N];
#pragma unroll
      for (int j = 0; j < N; ++j) v[j] = known && c + j * threads < end ? to_f32(row[c + j * threads]) : 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (c + j * threads < end) out[i * dim + c + j * threads] = from_f32<O>(known ? __fmul_rn(v[j], scale) : 0.0f);
    }
  } else {
    const int c0 = (blockIdx.y * threads * kEights + me) * 8;
    Eight<T> e[kEights];
#pragma unroll
    for (int k = 0; k < kEights; ++k) {
      const int c = c0 + k * threads * 8;
      e[k] = load_eight<true>(row + c, known ? max(0, min(8, dim - c)) : 0);
    }
#pragma unroll
    for (int k = 0; k < kEights; ++k) {
      const int c = c0 + k * threads * 8;
      float v[8];
      unpack_eight(e[k], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = known ? __fmul_rn(v[j], scale) : 0.0f;
      store_eight(out + i * dim + c, v, max(0, min(8, dim - c)));
    }
  }
}

// ---------------------------------------------------------------------------
// gradient: positions by token

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32;
constexpr int kClassBits = 3, kClasses = 1 << kClassBits;          // CTAs: tokens by their low bits
constexpr int kDigitBits = 8, kDigits = 1 << kDigitBits;           // of what is left of a token
constexpr int kSortPer = 32;                                       // most positions a thread (a kernel for half of them
                                                                   // takes 6 us less where it is enough)
constexpr int kSortMost = kSortThreads * kSortPer, kPositionBits = 15;
constexpr int kSortVocab = 1 << (2 * kDigitBits + kClassBits);     // (31 bits of a record are used)
static_assert(kSortMost == 1 << kPositionBits && kPositionBits + 2 * kDigitBits <= 32, "a record is a word");

struct SortArgs {
  const int32_t* tokens;
  int n, vocab, per;             // per: positions a thread
  int32_t *perm, *run_start, *run_end;
  unsigned *n_valid, *long_runs;
  char* table;                   // to be cleared, or NULL
  long long bytes;
};

struct SortShared {
  unsigned short warp_digits[kSortWarps][kDigits];
  unsigned start[kDigits];       // of the digits' records
  unsigned scan[kSortWarps], below[kSortWarps];
  unsigned total, total_below;
  unsigned pad_[2];
  // then the records in an order (token above position)
};

// A stable pass over the records, which lie in the order of warps, steps and lanes, by
// the digit of their tokens at `shift`, to `to`, where they may have come from.
template <int PER>
__device__ __forceinline__ void sort_pass(SortShared& s, int per, const unsigned (&record)[PER], unsigned valid,
                                          int shift, unsigned* to) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned short* mine = s.warp_digits[warp];
  for (int d = lane; d < kDigits / 2; d += 32) reinterpret_cast<unsigned*>(mine)[d] = 0;
  __syncwarp();
  unsigned in_warp[PER / 2];          // two a word: as many as a warp has records
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (k >= per) break;
    const bool ok = valid >> k & 1;
    const unsigned digit = record[k] >> (kPositionBits + shift) & (kDigits - 1);
    // the lanes with the same digit, bit by bit
    unsigned same = __ballot_sync(0xffffffffu, ok);
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
      const unsigned ones = __ballot_sync(0xffffffffu, digit >> b & 1);
      same &= digit >> b & 1 ? ones : ~ones;
    }
    const unsigned ahead = __popc(same & ((1u << lane) - 1));
    const unsigned before = ok ? mine[digit] : 0;
    in_warp[k / 2] = k % 2 ? in_warp[k / 2] | (before + ahead) << 16 : before + ahead;
    __syncwarp();
    if (ok && ahead == 0) mine[digit] = (unsigned short)(before + __popc(same));
    __syncwarp();
  }
  __syncthreads();
  // a digit a thread: over the warps
  unsigned all = 0;
  if (threadIdx.x < kDigits) {
#pragma unroll 8
    for (int w = 0; w < kSortWarps; ++w) {
      const unsigned c = s.warp_digits[w][threadIdx.x];
      s.warp_digits[w][threadIdx.x] = (unsigned short)all;
      all += c;
    }
  }
  // over the digits
  unsigned scan = all;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const unsigned v = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += v;
  }
  if (lane == 31) s.scan[warp] = scan;
  __syncthreads();
  if (warp == 0) {
    unsigned v = s.scan[lane];
    const unsigned own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const unsigned u = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v += u;
    }
    s.scan[lane] = v - own;
    if (lane == 31) s.total = v;
  }
  __syncthreads();
  if (threadIdx.x < kDigits) s.start[threadIdx.x] = s.scan[warp] + scan - all;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (k >= per) break;
    if (!(valid >> k & 1)) continue;
    const unsigned digit = record[k] >> (kPositionBits + shift) & (kDigits - 1);
    to[s.start[digit] + mine[digit] + (in_warp[k / 2] >> 16 * (k % 2) & 0xffff)] = record[k];
  }
  __syncthreads();
}

// The first CTAs sort a class of tokens each; the others clear the table.
template <int PER>
__global__ void __launch_bounds__(kSortThreads, 1)
embedding_sort_kernel(SortArgs a) {
  extern __shared__ __align__(16) char s_raw[];
  dep_wait();
  dep_launch();
  if (blockIdx.x >= kClasses) {
    const float zero[8] = {};
    char* const lo = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(a.table) + 31) & ~(uintptr_t)31);
    char* const hi = reinterpret_cast<char*>(reinterpret_cast<uintptr_t>(a.table + a.bytes) & ~(uintptr_t)31);
    const long long thread = (long long)(blockIdx.x - kClasses) * kSortThreads + threadIdx.x;
    const long long threads = (long long)(gridDim.x - kClasses) * kSortThreads;
    if (hi <= lo) {
      for (long long i = thread; i < a.bytes; i += threads) a.table[i] = 0;
      return;
    }
    if (thread < 32 && a.table + thread < lo) a.table[thread] = 0;
    if (thread < 32 && hi + thread < a.table + a.bytes) hi[thread] = 0;
    for (char* p = lo + thread * 32; p < hi; p += threads * 32) st_256(reinterpret_cast<float*>(p), zero);
    return;
  }
  SortShared& s = *reinterpret_cast<SortShared*>(s_raw);
  unsigned* order = reinterpret_cast<unsigned*>(s_raw + sizeof(SortShared));
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned record[PER], valid = 0;
  {
    // the class' records in the order of their positions, and how many records lower classes have
    const int first = warp * 32 * a.per + lane;
    unsigned mine = 0, below = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = first + 32 * k;
      const int token = k < a.per && i < a.n ? a.tokens[i] : -1;
      record[k] = (unsigned)token >> kClassBits << kPositionBits | (unsigned)i;
      const bool known = (unsigned)token < (unsigned)a.vocab;
      if (known && (token & (kClasses - 1)) == (int)blockIdx.x) valid |= 1u << k;
      mine += __popc(__ballot_sync(0xffffffffu, valid >> k & 1));
      below += __popc(__ballot_sync(0xffffffffu, known && (token & (kClasses - 1)) < (int)blockIdx.x));
    }
    if (lane == 0) {
      s.scan[warp] = mine;
      s.below[warp] = below;
    }
    __syncthreads();
    if (warp == 0) {
      unsigned v = s.scan[lane], u = s.below[lane];
      const unsigned own = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const unsigned up = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += up;
        u += __shfl_xor_sync(0xffffffffu, u, d);
      }
      s.scan[lane] = v - own;
      if (lane == 31) {
        s.total = v;
        s.total_below = u;
      }
    }
    __syncthreads();
    unsigned at = s.scan[warp];
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const unsigned ok = __ballot_sync(0xffffffffu, valid >> k & 1);
      if (valid >> k & 1) order[at + __popc(ok & ((1u << lane) - 1))] = record[k];
      at += __popc(ok);
    }
    __syncthreads();
  }
  const int total = (int)s.total, base = (int)s.total_below;
  const int per = (total + kSortThreads - 1) / kSortThreads, first = warp * 32 * per + lane;
  auto load = [&](const unsigned* from) {
    valid = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int q = first + 32 * k;
      if (k < per && q < total) {
        valid |= 1u << k;
        record[k] = from[q];
      }
    }
  };
  load(order);
  sort_pass(s, per, record, valid, 0, order);
  load(order);
  sort_pass(s, per, record, valid, kDigitBits, order);
  // the order, and where runs begin and end in it
  for (int q = threadIdx.x; q < total; q += kSortThreads) {
    const unsigned t = order[q] >> kPositionBits;
    const int token = (int)(t << kClassBits | blockIdx.x);
    a.perm[base + q] = (int32_t)(order[q] & (kSortMost - 1));
    if (q == 0 || order[q - 1] >> kPositionBits != t) a.run_start[token] = base + q;
    if (q + 1 == total || order[q + 1] >> kPositionBits != t) a.run_end[token] = base + q + 1;
  }
  if (threadIdx.x == 0 && blockIdx.x == kClasses - 1) {
    *a.n_valid = (unsigned)(base + total);
    *a.long_runs = 0;
  }
}

// ---------------------------------------------------------------------------
// gradient: sums

constexpr int kBlock = 32;       // ranks of a block
constexpr int kEight = 8;        // rows that a warp asks for at a time, and of a whole subtree
constexpr int kStages = 2;       // such groups in shared memory or on their way
// columns of a lane, a 16-byte vector, and of a warp
template <typename T> constexpr int kCols = 16 / sizeof(T);

template <typename T> constexpr int kSlice = 32 * kCols<T>;

// A run of more than one block, for the join.
struct LongRun {
  int token, start, end;
};

// The workspace: that of the library's sort, or a header and the order and runs of the
// small one's; then long runs and nodes.
struct EmbedPlan {
  bool small_sort;
  SortPlan sort;
  size_t perm, run_start, run_end, runs, nodes, total;
};
EmbedPlan embed_plan(long long n, long long vocab, long long dim) {
  EmbedPlan p;
  // (gradient of 20,000 x 2,048 in bf16 for 65,536 rows: 97 us, 134 by the library's sort.  32,768 places of one token,
  // which one CTA sorts alone, 2,048 wide: 150 us for 65,536 rows and 123 for 3; by the library's sort 362 and 93.)
  p.small_sort = n <= kSortMost && vocab <= kSortVocab;
  size_t at;
  if (p.small_sort) {
    p.perm = kHeaderBytes;
    p.run_start = align_up(p.perm + (size_t)n * 4, 256);
    p.run_end = align_up(p.run_start + (size_t)vocab * 4, 256);
    at = p.run_end + (size_t)vocab * 4;
  } else {
    p.sort = make_sort_plan(n, vocab, 0, true, 0);
    p.perm = p.run_start = p.run_end = 0;
    at = p.sort.total;
  }
  p.runs = align_up(at, 256);
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
  const int32_t *run_start, *run_end;   // a token's run in it; of tokens that occur
  const unsigned* n_valid;
  unsigned* long_runs;           // how many
  LongRun* runs;
  float* nodes;
  int n, vocab, dim;
  long long stride;
  float scale;
  int sum_ctas, slices, clear_ctas;   // CTAs that sum (a number of windows each, times slices of the columns) and that clear
  int clear_from, clear_rows;         // the first row that is still to be cleared, and the rows of a warp (at most 32)
};

// (A row that is not added to counts as +0.0: a sum of -0.0 becomes +0.0, as det_scatter_add_rows has it.)
template <typename O>
__device__ __forceinline__ float finish(float sum, float scale, const O* old, bool accumulate) {
  return __fadd_rn(accumulate ? to_f32(*old) : 0.0f, __fmul_rn(sum, scale));
}

// A lane's columns of a row: 16 bytes of T.  VEC: aligned, and all or none of them.
template <typename T> struct Vec16 { uint4 q; };
__device__ __forceinline__ void pairs_of(const Vec16<float>& e, Two (&v)[2]) {
  v[0] = two(__uint_as_float(e.q.x), __uint_as_float(e.q.y));
  v[1] = two(__uint_as_float(e.q.z), __uint_as_float(e.q.w));
}
// A warp's columns of a row, from p on, `left` of them, to a place in shared memory; those
// that are not there 0.  VEC: 16-byte vectors; else in 32 bits element by element and in 16 bits the
// words that hold them (the lower half of the first may be an element before them, beside them in a
// word); `any` is aligned.
constexpr int kPlace = 33;               // 16-byte units of a place: 256 elements of 16 bits from the middle of a word on
template <bool VEC, typename T>
__device__ __forceinline__ void copy_row(uint4* to, const T* p, const void* any, int left, int lane) {
  const unsigned dst = smem_u32(to);
  auto copy4 = [&](int word, const void* from, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 4 * word), "l"(bytes > 0 ? from : any), "r"(bytes)
                 : "memory");
  };
  if constexpr (VEC) {
    const bool ok = lane * kCols<T> < left;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + 16 * lane), "l"(ok ? p + lane * kCols<T> : any),
                 "r"(ok ? 16 : 0)
                 : "memory");
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j) copy4(32 * j + lane, p + 32 * j + lane, 32 * j + lane < left ? 4 : 0);
  } else {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const int halves = left + (int)(at >> 1 & 1);         // from the first word on
    const char* words = reinterpret_cast<const char*>(at & ~(uintptr_t)3);
#pragma unroll
    for (int j = 0; j < 5; ++j) {
      const int i = 32 * j + lane;
      if (j < 4 || lane == 0) copy4(i, words + 4 * i, max(0, min(2, halves - 2 * i)) * 2);
    }
  }
}
// A lane's columns of it; odd: the row starts in the middle of a word.
template <bool VEC, typename T>
__device__ __forceinline__ Vec16<T> take_row(const uint4* from, bool odd, int lane) {
  Vec16<T> v{from[lane]};
  if constexpr (!VEC && sizeof(T) == 2) {
    if (odd) {
      const unsigned next = reinterpret_cast<const unsigned*>(from + lane)[4];
      v.q = make_uint4(__funnelshift_r(v.q.x, v.q.y, 16), __funnelshift_r(v.q.y, v.q.z, 16),
                       __funnelshift_r(v.q.z, v.q.w, 16), __funnelshift_r(v.q.w, next, 16));
    }
  }
  return v;
}
template <typename T>
__device__ __forceinline__ void pairs_of(const Vec16<T>& e, Two (&v)[4]) {
  const unsigned w[4] = {e.q.x, e.q.y, e.q.z, e.q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_two(w[i], v[i].x, v[i].y, T());
}
// to = node + v, the earlier one on the left
template <int N> __device__ __forceinline__ void join(const Two (&v)[N], const Two (&node)[N], Two (&to)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) to[i] = add(node[i], v[i]);
}
// The first n of 2 P columns.
template <bool VEC, typename O, int N>
__device__ __forceinline__ void load_cols(float (&v)[N], const O* p, int n) {
  if (VEC && n == N) {
    constexpr int W = N * (int)sizeof(O) / 4;
    unsigned w[W];
    if constexpr (W % 4 == 0) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned*>(p) + i);
        w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
      }
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x, w[1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if constexpr (sizeof(O) == 4) v[i] = __uint_as_float(w[i]);
      else unpack_two(w[i], v[2 * i], v[2 * i + 1], O());
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
template <bool VEC, typename O, int P>
__device__ __forceinline__ void store_cols(O* p, const Two (&v)[P], int n) {
  if (VEC && n == 2 * P) {
    if constexpr (sizeof(O) == 4) {
#pragma unroll
      for (int i = 0; i < P; i += 2) *reinterpret_cast<float4*>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
    } else if constexpr (P == 4) {
      *reinterpret_cast<uint4*>(p) = make_uint4(pack_two<O>(v[0].x, v[0].y), pack_two<O>(v[1].x, v[1].y),
                                                pack_two<O>(v[2].x, v[2].y), pack_two<O>(v[3].x, v[3].y));
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack_two<O>(v[0].x, v[0].y), pack_two<O>(v[1].x, v[1].y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (2 * i < n) p[2 * i] = from_f32<O>(v[i].x);
      if (2 * i + 1 < n) p[2 * i + 1] = from_f32<O>(v[i].y);
    }
  }
}

template <typename O>
__device__ __forceinline__ void clear_rows(O* out, const GradArgs& a, long long warp) {
  const int lane = threadIdx.x & 31;
  const int valid = min((int)*a.n_valid, a.n);
  const long long r0 = a.clear_from + warp * a.clear_rows, r = r0 + lane;
  // A row that a token names is written by its sum.  run_start is written for such rows only: what it holds for another
  // leads to no position of that token.
  bool skip = r >= a.vocab || lane >= a.clear_rows;
  if (!skip) {
    const int q = a.run_start[r];
    const int from = (unsigned)q < (unsigned)valid ? a.perm[q] : -1;
    skip = (unsigned)from < (unsigned)a.n && a.tokens[from] == (int)r;
  }
  const unsigned mask = __ballot_sync(0xffffffffu, !skip);
  const size_t bytes = (size_t)a.dim * sizeof(O);
  const bool vectors = (reinterpret_cast<uintptr_t>(out) | bytes) % 16 == 0;
  for (int i = 0; i < a.clear_rows; ++i) {
    if (!(mask >> i & 1)) continue;
    O* row = out + (r0 + i) * a.dim;
    if (vectors) {
      for (int c = lane; c < (int)(bytes / 16); c += 32) reinterpret_cast<uint4*>(row)[c] = make_uint4(0, 0, 0, 0);
    } else {
      for (int c = lane; c < a.dim; c += 32) row[c] = from_f32<O>(0.0f);
    }
  }
}

// A warp: the blocks that begin at sorted positions [w * window, (w + 1) *
// window), columns slice * kSlice and on.
constexpr int kEnd = 32, kLong = 64, kFirst = 128;     // of a position: it ends its block, its run is long, its block is the run's first
template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(256, 2)
embedding_blocks_kernel(const T* grad, GradArgs a, O* out, int accumulate, int window) {
  dep_wait();
  dep_launch();
  // CTAs that clear are spread among those that sum
  const long long ctas = (long long)a.sum_ctas + a.clear_ctas;
  const int cleared = (int)(blockIdx.x * (long long)a.clear_ctas / ctas);
  if ((blockIdx.x + 1LL) * a.clear_ctas / ctas > cleared) {
    clear_rows(out, a, (long long)cleared * (blockDim.x >> 5) + (threadIdx.x >> 5));
    return;
  }
  const int cta = blockIdx.x - cleared, slice = cta % a.slices;
  const int lane = threadIdx.x & 31;
  const int valid = min((int)*a.n_valid, a.n);
  const long long w0 = ((long long)(cta / a.slices) * (blockDim.x >> 5) + (threadIdx.x >> 5)) * window;
  if (w0 >= valid) return;
  // 64 positions from w0 on, two a lane: what they hold, and where blocks begin and end
  __shared__ int4 s_meta[256 / 32][64];          // position, token, rank in its block and flags
  int4* meta = s_meta[threadIdx.x >> 5];
  unsigned begins[2], ends[2], wholes[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const long long q = w0 + h * 32 + lane;
    bool in = q < valid;
    const int from = in ? a.perm[q] : 0;
    in = in && (unsigned)from < (unsigned)a.n;         // what follows an unfinished sort (its waits are bounded)
    const int token = in ? a.tokens[from] : 0;
    in = in && (unsigned)token < (unsigned)a.vocab;    // is left out
    const int lo = in ? a.run_start[token] : 0;
    const int hi = in ? a.run_end[token] : 0;
    in = in && lo >= 0 && lo <= q && q < hi && hi <= valid;
    const int rank = (int)q - lo;
    const bool begin = in && rank % kBlock == 0, end = in && (rank % kBlock == kBlock - 1 || q + 1 == hi);
    begins[h] = __ballot_sync(0xffffffffu, begin);
    ends[h] = __ballot_sync(0xffffffffu, end);
    wholes[h] = __ballot_sync(0xffffffffu, in && rank % kEight == 0 && q + kEight <= hi);   // eight rows of one block
    meta[h * 32 + lane] = make_int4(in ? from : 0, token, rank % kBlock | (end ? kEnd : 0) | (hi - lo > kBlock ? kLong : 0) |
                                                              (rank < kBlock ? kFirst : 0), 0);
  }
  __syncwarp();
  const unsigned long long begin = begins[0] | (unsigned long long)begins[1] << 32;
  const unsigned long long end = ends[0] | (unsigned long long)ends[1] << 32;
  const unsigned long long whole = wholes[0] | (unsigned long long)wholes[1] << 32;
  const unsigned long long here = begin & ((window == 32 ? 0xffffffffull : (1ull << window) - 1));
  if (here == 0) return;
  constexpr int COLS = kCols<T>, PAIRS = COLS / 2;
  const int c = slice * kSlice<T> + lane * COLS;
  const int nc = max(0, min(COLS, a.dim - c));
  const int p0 = __ffsll((long long)here) - 1;
  // the last block that begins here ends at the first end behind its beginning
  const int last = 63 - __clzll((long long)here);
  const int p1 = __ffsll((long long)(end >> last << last)) - 1;
  if (p1 < 0) return;
  // rows come through the warp's ring in groups: eight of one block that are a subtree, or up to
  // eight up to the next such
  extern __shared__ __align__(16) uint4 s_rows[];        // [warps][kStages][kEight][kPlace]
  uint4(*rows)[kEight][kPlace] = reinterpret_cast<uint4(*)[kEight][kPlace]>(s_rows) + (threadIdx.x >> 5) * kStages;
  const uintptr_t grad_odd = reinterpret_cast<uintptr_t>(grad) >> 1;
  const T* slice_grad = grad + slice * kSlice<T>;
  const int left = a.dim - slice * kSlice<T>;
  const void* any = reinterpret_cast<const void*>(reinterpret_cast<uintptr_t>(grad) & ~(uintptr_t)3);
  auto group = [&](int p) {
    if (whole >> p & 1) return kEight;
    const int to_next = (whole >> p) ? __ffsll((long long)(whole >> p)) - 1 : kEight;
    return min(kEight, min(to_next, p1 + 1 - p));
  };
  auto ask = [&](int p, int stage) {
    if (p <= p1) {
      const int n = group(p);
#pragma unroll
      for (int j = 0; j < kEight; ++j)
        if (j < n) copy_row<VEC>(rows[stage][j], slice_grad + meta[p + j].x * a.stride, VEC ? grad : any, left, lane);
      p += n;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return p;
  };
  int asked = p0;
#pragma unroll
  for (int g = 0; g < kStages; ++g) asked = ask(asked, g);
  Two st[5][PAIRS];              // pending nodes of a block's tree: 1, 2, 4, 8, 16 rows
  int stage = 0;
  for (int p = p0; p <= p1;) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    if (!VEC) __syncwarp();            // (a lane reads what others have copied)
    const uint4(*row)[kPlace] = rows[stage];
    auto take = [&](int j) {
      return take_row<VEC, T>(row[j], (grad_odd ^ (meta[p + j].x & (unsigned)a.stride)) & 1, lane);
    };
    const int n = group(p);
    const bool eight = whole >> p & 1;
    for (int q = eight ? p + kEight - 1 : p; q < p + n; ++q) {
      const int4 m = meta[q];
      const int rank = m.z & (kBlock - 1);
      // a binary counter: the new node, a row or eight, is added to the pending node of each level it
      // completes; the whole block's goes to the first place.  (A row is unpacked in each case, where its place is
      // known: values that change places cost more instructions than the sums.)
      Two v[PAIRS];
      if (eight) {
        Two x[PAIRS], y[PAIRS];
        pairs_of(take(0), x);
        pairs_of(take(1), v);
        join(v, x, x);
        pairs_of(take(2), y);
        pairs_of(take(3), v);
        join(v, y, y);
        join(y, x, x);
        pairs_of(take(4), y);
        pairs_of(take(5), v);
        join(v, y, y);
        Two z[PAIRS];
        pairs_of(take(6), z);
        pairs_of(take(7), v);
        join(v, z, z);
        join(z, y, y);
        switch (rank / kEight) {
          case 1: join(y, x, v); join(v, st[3], st[4]); break;
          case 3: join(y, x, v); join(v, st[3], v); join(v, st[4], st[0]); break;
          default: join(y, x, st[3]);
        }
      } else if (rank == 0 && (m.z & kEnd)) {
        pairs_of(take(q - p), v);              // a token that occurs once, or a run's last row by itself
      } else {
        const Vec16<T> one = take(q - p);
        switch (__ffs(~rank) - 1) {
          case 0: pairs_of(one, st[0]); break;
          case 1: pairs_of(one, v); join(v, st[0], st[1]); break;
          default: pairs_of(one, v); join(v, st[0], v); join(v, st[1], st[2]);      // 2: an eighth row comes with its eight
        }
      }
      if (!(m.z & kEnd)) continue;
      // the block's node: the pending ones from the smallest up
      if (rank > 0) {
        const int count = rank + 1 == kBlock ? 1 : rank + 1;
        bool have = false;
#pragma unroll
        for (int l = 0; l < 5; ++l)
          if (count >> l & 1) {
            if (have) {
              join(v, st[l], v);
            } else {
#pragma unroll
              for (int i = 0; i < PAIRS; ++i) v[i] = st[l][i];
            }
            have = true;
          }
      }
      const bool last_node = !(m.z & kLong);
      if (last_node) {
        O* to = out + (long long)m.y * a.dim + c;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = mul(v[i], twice(a.scale));
        float old[COLS] = {};          // (as in finish())
        if (accumulate) load_cols<VEC>(old, to, nc);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) v[i] = add(two(old[2 * i], old[2 * i + 1]), v[i]);
        store_cols<VEC>(to, v, nc);
      } else {
        const long long start = w0 + q - rank;
        store_cols<VEC>(a.nodes + node_slot(start, m.z & kFirst) * a.dim + c, v, nc);
        if ((m.z & kFirst) && slice == 0 && lane == 0) {
          const unsigned k = atomicAdd(a.long_runs, 1u);       // in any order: runs do not meet
          if (k <= (unsigned)(a.n / kBlock)) a.runs[k] = {m.y, (int)start, a.run_end[m.y]};
        }
      }
    }
    if (!VEC) __syncwarp();
    asked = ask(asked, stage);
    p += n;
    stage = stage + 1 == kStages ? 0 : stage + 1;
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

// Bytes that are cleared beside the sort, in the 18 us that it takes for 16,384 positions.  (All of a table of 268 MB
// before the sort: 42 us more.)
constexpr size_t kClearWithSort = 96 << 20;

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
int blocks(const void* grad, GradArgs a, int n, void* out, int accumulate, cudaStream_t s) {
  // vectors where every row of every operand starts on 16 bytes (rows of nodes do in the workspace then)
  const bool vec = vectors<T>(grad, a.stride) && vectors<O>(out, a.dim) && a.dim * sizeof(T) % 16 == 0;
  const unsigned slices = (unsigned)((a.dim + kSlice<T> - 1) / kSlice<T>);
  // windows of 32 positions, shorter ones while there are fewer than 8 warps an SM (500 x 1,024 in bf16: 26 us, with
  // 32 positions 32; 16,384 x 2,048: 87 us with 16 positions, 79 with 32)
  int window = 32;
  while (window > 8 && (long long)slices * (n / window) < 8LL * 152) window /= 2;
  const unsigned warps = (unsigned)((n + (long long)window - 1) / window);
  constexpr unsigned per_cta = 8;
  auto* kernel = vec ? embedding_blocks_kernel<T, O, true> : embedding_blocks_kernel<T, O, false>;
  const size_t smem = (size_t)per_cta * kStages * kEight * kPlace * 16;
  const cudaError_t se = ensure_dyn_smem((const void*)kernel, smem);
  if (se != cudaSuccess) return cuda_fail(se, "det_embedding_blocks");
  const long long sums = (long long)((warps + per_cta - 1) / per_cta) * slices;
  // rows of about 32 KB for a warp that clears (2,048 x 4,096 in bf16 for 32,000 rows: 4 rows 58 us, 16 73; 2,048 x 512
  // for 262,144: 4 rows 58, 16 48)
  a.clear_rows = (int)std::max<size_t>(2, std::min<size_t>(16, (32 << 10) / (a.dim * sizeof(O))));
  const long long clears = (a.vocab - a.clear_from + (long long)a.clear_rows * per_cta - 1) / (a.clear_rows * per_cta);
  if (sums + clears >= (1LL << 31)) return DET_ERR_TOO_LARGE;
  a.slices = (int)slices;
  a.sum_ctas = (int)sums;
  a.clear_ctas = (int)clears;
  launch_begin("det_embedding_blocks", s);
  const cudaError_t e = launch_dep(kernel, dim3((unsigned)(sums + clears)), dim3(32 * per_cta), smem, s,
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

int small_sort(const GradArgs& a, int n, int vocab, void* table, size_t bytes, cudaStream_t s) {
  SortArgs g;
  g.tokens = a.tokens;
  g.n = n;
  g.vocab = vocab;
  g.per = (n + kSortThreads - 1) / kSortThreads;
  g.perm = const_cast<int32_t*>(a.perm);
  g.run_start = const_cast<int32_t*>(a.run_start);
  g.run_end = const_cast<int32_t*>(a.run_end);
  g.n_valid = const_cast<unsigned*>(a.n_valid);
  g.long_runs = a.long_runs;
  g.table = static_cast<char*>(table);
  g.bytes = (long long)bytes;
  auto* kernel = g.per > kSortPer / 2 ? embedding_sort_kernel<kSortPer> : embedding_sort_kernel<kSortPer / 2>;
  const cudaError_t se = ensure_dyn_smem((const void*)kernel, sizeof(SortShared) + (size_t)kSortMost * 4);
  if (se != cudaSuccess) return cuda_fail(se, "det_embedding_sort");
  // CTAs that clear: one on each other SM, fewer for small tables
  const long long clear =
      table ? std::min<long long>(std::max(device_sm_count() - kClasses, 1), (long long)(bytes / (kSortThreads * 32)) + 1) : 0;
  launch_begin("det_embedding_sort", s);
  const cudaError_t e = launch_dep(kernel, dim3((unsigned)(kClasses + clear)), dim3(kSortThreads),
                                   sizeof(SortShared) + (size_t)g.per * kSortThreads * 4, s, g);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_embedding_sort");
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
  return embed_plan(n, vocab, dim).total;
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
  const EmbedPlan plan = embed_plan(n, vocab, dim);
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 || workspace_bytes < plan.total) return DET_ERR_WORKSPACE;
  const cudaStream_t s = as_stream(stream);
  const size_t table_bytes = (size_t)vocab * dim * model_elem_size(table_dtype);
  if (!accumulate && n == 0) {
    const cudaError_t e = cudaMemsetAsync(grad_table, 0, table_bytes, s);
    if (e != cudaSuccess) return cuda_fail(e, "det_embedding_backward: clear");
  }
  if (n == 0) return DET_OK;
  char* w = static_cast<char*>(workspace);
  SortHdr* header = reinterpret_cast<SortHdr*>(w);
  GradArgs a;
  a.tokens = tokens;
  a.n_valid = &header->n_valid;
  a.clear_from = (int)vocab;                                     // nothing
  a.long_runs = &header->long_segs;                              // cleared by either sort, neither of which uses it
  if (plan.small_sort) {
    a.perm = reinterpret_cast<int32_t*>(w + plan.perm);
    a.run_start = reinterpret_cast<int32_t*>(w + plan.run_start);
    a.run_end = reinterpret_cast<int32_t*>(w + plan.run_end);
    const size_t row_bytes = (size_t)dim * model_elem_size(table_dtype);
    if (!accumulate) a.clear_from = (int)std::min<int64_t>(vocab, (int64_t)(kClearWithSort / row_bytes) + 1);
    if (const int rc = small_sort(a, (int)n, (int)vocab, accumulate ? nullptr : grad_table, a.clear_from * row_bytes, s)) return rc;
  } else {
    int buffer = 0;
    if (const int rc = enqueue_sort(plan.sort, workspace, tokens, 0, nullptr, nullptr, s, &buffer)) return rc;
    a.perm = reinterpret_cast<const int32_t*>(w + plan.sort.idx[buffer]);
    a.run_start = reinterpret_cast<const int32_t*>(w + plan.sort.seg);
    a.run_end = a.run_start + 1;
    if (!accumulate) a.clear_from = 0;
  }
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
