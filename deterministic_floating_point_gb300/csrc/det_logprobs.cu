// det_token_logprobs and det_token_logprobs_backward (include/det_model.h).
//
// A row's statistics are S = sum exp(x - m) and T = sum exp(x - m) (x - m)
// with m the row's maximum: lse = m + log S, entropy = log S - T / S, the log
// probability of a token (x[token] - m) - log S.  A row is read once.  The order
// of the additions is fixed by element index: thread t of 256 takes the 4-byte
// words t, t + 256, ... of the row (two elements of the 16-bit types), 32 of
// them to a chunk; its sums over a chunk are relative to its own largest element
// so far, chunks are added in order within a part of the row, parts in order,
// and the threads by a tree.  So a row's bits depend neither on the other rows
// nor on its alignment nor on how many CTAs share it.
//
// What bounds it: the bytes in 32 bits (4,096 x 49,152: 118 us, the measured
// copy bandwidth), in 16 bits nearly as much the instructions, 7.6 an element at
// 64% of the issue slots (4,096 x 98,304 bf16: 124 us, 95%).  Rows that start at an
// odd element read each word of shared memory twice (4,096 x 100,003 bf16: 161 us,
// 75%).  With alternatives a CTA's row end takes 2 to 5 us more, half of it hidden
// by the SM's other CTA (4,096 x 98,304: one of them 143 us, 20 of them 188).
#include "det_model.cuh"

#include <algorithm>
#include <type_traits>

namespace det {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kWords = 32;      // 4-byte words of a thread's chunk
constexpr int kPartWords = 4;   // a row's last chunk goes by this many
constexpr int kBest = 6;         // most threads of a warp that the bound for the alternatives is drawn from
constexpr int kMaxJobs = 128;    // reads for a row's alternatives that the warps share

template <typename T> struct Word;   // what a 4-byte word of a row holds
template <> struct Word<float> {
  static constexpr int N = 1;
  static constexpr unsigned kMasked = 0xff800000u;   // -inf
  static __device__ __forceinline__ float get(unsigned w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
  static __device__ __forceinline__ unsigned pack(float a, float) { return __float_as_uint(a); }
};
template <> struct Word<__nv_bfloat16> {
  static constexpr int N = 2;
  static constexpr unsigned kMasked = 0xff80ff80u;
  static __device__ __forceinline__ float get(unsigned w, int j) {
    return __uint_as_float(j ? (w & 0xffff0000u) : (w << 16));
  }
  static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    unsigned r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ unsigned pack(float a, float b) {   // to nearest
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&v);
  }
};
template <> struct Word<__half> {
  static constexpr int N = 2;
  static constexpr unsigned kMasked = 0xfc00fc00u;
  static __device__ __forceinline__ float get(unsigned w, int j) {
    return __half2float(__ushort_as_half((unsigned short)(j ? (w >> 16) : w)));
  }
  static __device__ __forceinline__ unsigned larger(unsigned a, unsigned b) {
    unsigned r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ unsigned pack(float a, float b) {   // to nearest
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned*>(&v);
  }
};

// Two 32-bit lanes in a 64-bit register.
__device__ __forceinline__ unsigned long long pack_f32x2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(unsigned long long v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ unsigned long long add_f32x2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma_f32x2(unsigned long long a, unsigned long long b,
                                                        unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Word w of a row (elements N w, N w + 1), with masked logits past its end.
template <typename T>
__device__ __forceinline__ unsigned load_word(const T* row, long long w, long long vocab, bool words_aligned) {
  if constexpr (Word<T>::N == 1) {
    return w < vocab ? __float_as_uint(row[w]) : Word<T>::kMasked;
  } else {
    const long long e = 2 * w;
    const unsigned short* p = reinterpret_cast<const unsigned short*>(row);
    if (e + 1 < vocab) {
      if (words_aligned) return *reinterpret_cast<const unsigned*>(p + e);
      return (unsigned)p[e] | ((unsigned)p[e + 1] << 16);
    }
    if (e < vocab) return (unsigned)p[e] | (Word<T>::kMasked & 0xffff0000u);
    return Word<T>::kMasked;
  }
}

// A thread's (or row's) statistics in units of log 2: the largest logit m,
// and S = sum 2^y, T = sum 2^y y with y = x log2(e) - ref.  Where m is near 0
// (near_max()), ref is the product m log2(e) rounded, so y takes one fused
// operation for an element; otherwise (finite masks, infinities, NaN) ref is the
// exact product, and y = (x - m) log2(e).
//
// Near: at x = m the former y is what the rounding of ref left, up to half a unit
// of its last place.  That is at most 1 up to 2^24, and the logarithm of S takes it
// out again; at -1e10 it would be 440, and 2^y overflows.  (2,048 x 100,003 f32, three
// quarters of the logits around -1e7: 119 us, and 250 with a bound of 2^20.)
constexpr float kNearMost = 16777216.0f;
struct Stat {
  float m, s, t;
};
template <typename T> __device__ __forceinline__ bool near_max(float m) {
  // in f16 also: the bound for masked logits, m - 150 and a little, is a finite value
  return m >= (std::is_same<T, __half>::value ? -60000.0f : -kNearMost) && m <= kNearMost;
}
// The reference of a near maximum: the rounded product, the same number wherever
// it is used.  As a plain product it may be fused with the addition that takes
// it; a sum would then be scaled by 2 to the rounding's residue each time it is
// brought to its own maximum (rows of equal logits, -1e9: log p was 25 to 62 off).
__device__ __forceinline__ float near_ref(float m) { return __fmul_rn(m, kLog2e); }
// The reference of `from` less that of m, in units of log 2 (0 where they are equal).
template <typename T> __device__ __forceinline__ float ref_step(float from, float m) {
  const bool a = near_max<T>(from), b = near_max<T>(m);
  if (a && b) return __fsub_rn(near_ref(from), near_ref(m));
  if (a) return -__fmaf_rn(m, kLog2e, -near_ref(from));
  if (b) return __fmaf_rn(from, kLog2e, -near_ref(m));
  return __fmul_rn(from - m, kLog2e);
}
// S and T brought to the reference of m, which is not below st.m.
template <typename T> __device__ __forceinline__ void raise_to(Stat& st, float m) {
  if (st.m != kNegInf) {
    const float d = ref_step<T>(st.m, m), f = exp2_approx(d);
    st.t = f > 0.0f ? f * fmaf(st.s, d, st.t) : f;   // no 0 * inf; NaN stays
    st.s *= f;
  }
  st.m = m;
}

// The sorted list of a warp's best keys, the largest in lane 0; a key is the
// value's order key above the complement of its index, so no two are equal
// and the lowest index wins among equal values.
__device__ __forceinline__ void list_insert(unsigned long long& mine, unsigned long long key, int lane) {
  const int pos = __popc(__ballot_sync(0xffffffffu, mine > key));
  const unsigned long long up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane > pos) mine = up;
  else if (lane == pos) mine = key;
}

struct RowOut {
  float *logprob, *entropy, *lse, *top_logprob;
  int32_t* top_index;
};

// A row streams through shared memory in chunks of 256 threads x 32 words,
// word i of thread t of chunk c being word (32 c + i) 256 + t of the row (a
// 4-byte word: two elements of the 16-bit types).  One bulk copy fetches a
// chunk, kStages - 1 ahead of its use and across the ends of rows.  It takes the
// 16-byte blocks that lie inside the row, and puts them where the row's bytes
// have their place modulo 16, so that nothing outside a row is read; the few
// words at a row's ends that no block holds (its edges) are fetched by their threads
// a row ahead.  In a 16-bit row that starts at an odd element a thread's
// word lies in two words of shared memory.
constexpr int kChunkWords = kRowThreads * kWords;
constexpr int kChunkBytes = kChunkWords * 4;
constexpr int kStages = 3;
constexpr int kStageBytes = kChunkBytes + 32;   // a row's start modulo 16, and the block behind the chunk

struct Stream {
  alignas(16) unsigned char stage[kStages][kStageBytes];
  unsigned long long full[kStages], empty[kStages];
  int filled[kStages];   // the round of the stage's last copy, or -1
};
// The copies that are still on their way, waited for by one thread (each for at
// most kWaitNs): after a wait has given up, before the stages serve anything else
// or the CTA ends.  Round r of a stage completes phase r of its barrier.
__device__ __noinline__ void land_copies(Stream& st) {
  for (int i = 0; i < kStages; ++i)
    if (st.filled[i] >= 0) mbar_wait(&st.full[i], st.filled[i] & 1, kWaitNs);
}

// Where the parts of a row lie.
template <typename T>
struct RowMap {
  static constexpr int N = Word<T>::N;
  const T* row;
  int vocab, words;
  long long bytes;        // of the row
  int off;                // the row's start modulo 16
  long long in0, in1;     // the bytes of the row's whole 16-byte blocks, from its start
  int head, tail;         // words [0, head) and [tail, words) are edges

  __device__ __forceinline__ RowMap(const T* row_, int vocab_) : row(row_), vocab(vocab_) {
    words = (vocab + N - 1) / N;
    bytes = (long long)vocab * (int)sizeof(T);
    off = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    in0 = (16 - off) & 15;
    in1 = max(in0, ((bytes + off) & ~15LL) - off);
    tail = (int)(in1 >> 2);
    head = min((int)((in0 + 3) >> 2), tail);
    if (in1 == in0) head = tail = 0;   // no whole block: every word (at most 8) is an edge
  }
  __device__ __forceinline__ bool odd() const { return N == 2 && (off & 2); }
  // Whether chunk c has edges at the row's end, or masked words.
  __device__ __forceinline__ bool ragged(int c) const { return (long long)(c + 1) * kChunkWords > tail; }
  // The thread's word among the last edges, or -1.
  __device__ __forceinline__ int tail_word() const {
    const int w = tail + (((int)threadIdx.x - tail) & (kRowThreads - 1));
    return w < words ? w : -1;
  }
  // Fetch chunk c into a stage (one thread).
  __device__ __forceinline__ void fetch(Stream& st, int stage, int c) const {
    const long long lo = (long long)c * kChunkBytes;             // of the chunk, from the row's start
    const long long from = c == 0 ? in0 : lo - off;              // a 16-byte boundary
    const long long to = min(in1, lo - off + kStageBytes);
    const unsigned n = to > from ? (unsigned)(to - from) : 0u;
    mbar_arrive_expect_tx(&st.full[stage], n);
    if (n)
      bulk_copy_g2s(st.stage[stage] + (from - (lo - off)), reinterpret_cast<const char*>(row) + from, n, &st.full[stage]);
  }
};

// NW of the thread's words, from word i0 up, of a chunk that has arrived;
// odd_shift is 16 in a row that starts at an odd element, else 0 (SHIFT: may be 16).
template <bool SHIFT, int NW>
__device__ __forceinline__ void read_words(const unsigned char* stage, int off, int i0, unsigned odd_shift,
                                           unsigned (&x)[NW]) {
  const unsigned* p = reinterpret_cast<const unsigned*>(stage + (off & ~3)) + i0 * kRowThreads + threadIdx.x;
#pragma unroll
  for (int i = 0; i < NW; ++i) x[i] = p[i * kRowThreads];
  if (SHIFT) {
#pragma unroll
    for (int i = 0; i < NW; ++i) x[i] = __funnelshift_r(x[i], p[i * kRowThreads + 1], odd_shift);
  }
}
// Edges from where their threads hold them, and masked logits past the end;
// w0 is the thread's first of these words.
template <typename T, int NW>
__device__ __forceinline__ void set_edges(const RowMap<T>& map, int w0, unsigned head, unsigned tail, int tail_word,
                                          unsigned (&x)[NW]) {
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int w = w0 + i * kRowThreads;
    if (w < map.head) x[i] = head;
    if (w >= map.tail) x[i] = w == tail_word ? tail : Word<T>::kMasked;
  }
}

// Of a thread's elements: the chunk of the largest, and the largest of the
// other chunks.
struct Best {
  int chunk;
  float others;
};

// A row is cut into at most four parts of whole chunks, and a thread joins
// its statistics of the parts in order; so the parts may be the work of one
// CTA after the other or of a cluster's CTAs at once, with the same bits.
constexpr int kParts = 4;
__host__ __device__ inline int chunks_per_part(int chunks) { return (chunks + kParts - 1) / kParts; }

// A later part joined to the parts before it.
template <typename T>
__device__ __forceinline__ void join_part(Stat& st, Best& best, Stat part, const Best& part_best) {
  const float m = max_nan(st.m, part.m);
  if (!(part.m <= st.m)) {
    best.chunk = part_best.chunk;
    best.others = max_nan(part_best.others, st.m);
  } else {
    best.others = max_nan(best.others, part.m);
  }
  raise_to<T>(st, m);
  raise_to<T>(part, m);
  st.s += part.s;
  st.t += part.t;
}

// The largest of NW words.
template <typename T, int NW>
__device__ __forceinline__ float largest_of(const unsigned (&x)[NW]) {
  unsigned mx[NW / 2];
#pragma unroll
  for (int i = 0; i < NW / 2; ++i) mx[i] = Word<T>::larger(x[i], x[i + NW / 2]);
#pragma unroll
  for (int s = NW / 4; s > 0; s >>= 1)
#pragma unroll
    for (int i = 0; i < s; ++i) mx[i] = Word<T>::larger(mx[i], mx[i + s]);
  const float m = Word<T>::get(mx[0], 0);
  return Word<T>::N == 2 ? max_nan(m, Word<T>::get(mx[0], 1)) : m;
}

// The statistics brought to the largest of words of chunk c, before they are added.
template <typename T>
__device__ __forceinline__ void raise_words(Stat& st, Best& best, int c, float m) {
  if (!(m <= st.m)) {   // a new maximum, or NaN
    if (c != best.chunk) best.others = st.m;   // else another part of the same chunk
    best.chunk = c;
    raise_to<T>(st, max_nan(st.m, m));
  } else if (c != best.chunk) {
    best.others = max_nan(best.others, m);
  }
}

// NW words added; near_max(st.m).
template <typename T, int NW>
__device__ __forceinline__ void add_words(Stat& st, const unsigned (&x)[NW]) {
  constexpr int N = Word<T>::N;
  unsigned long long s2 = 0, t2 = 0;   // of elements 0 and 1 of the words (f32: even and odd words)
  const float ref = -near_ref(st.m);
  const unsigned long long c = pack_f32x2(kLog2e, kLog2e), minus = pack_f32x2(ref, ref);
  // 2^y is 0 from y = -127 on: a bound of -150 for x - m changes no term, and
  // without it 0 * inf for a masked logit.  16-bit logits are bounded in
  // pairs, by a value below m - 150 in every rounding.
  const float low = st.m - 150.0f - fabsf(st.m) * 0.015625f;
  const unsigned low2 = N == 2 ? Word<T>::pack(low, low) : 0u;
#pragma unroll
  for (int i = 0; i < NW; i += 3 - N) {
    unsigned long long v;
    if constexpr (N == 2) {
      const unsigned w = Word<T>::larger(x[i], low2);
      v = pack_f32x2(Word<T>::get(w, 0), Word<T>::get(w, 1));
    } else {
      v = pack_f32x2(max_nan(__uint_as_float(x[i]), low), max_nan(__uint_as_float(x[i + 1]), low));
    }
    v = fma_f32x2(v, c, minus);
    const float2 y = unpack_f32x2(v);
    const unsigned long long e = pack_f32x2(exp2_approx(y.x), exp2_approx(y.y));
    s2 = add_f32x2(s2, e);
    t2 = fma_f32x2(e, v, t2);
  }
  const float2 s = unpack_f32x2(s2), t = unpack_f32x2(t2);
  st.s += s.x + s.y;
  st.t += t.x + t.y;
}

// Whether NW words hold m alone, and it is neither +inf nor NaN.
template <typename T, int NW>
__device__ __forceinline__ bool all_equal(const unsigned (&x)[NW], float m) {
  unsigned differ = 0;
#pragma unroll
  for (int i = 1; i < NW; ++i) differ |= x[i] ^ x[0];
  return differ == 0 && Word<T>::get(x[0], 0) == m && Word<T>::get(x[0], Word<T>::N - 1) == m && m < -kNegInf;
}

// The same for a maximum far from 0 (or -inf, inf, NaN), word by word.
template <typename T>
__device__ __forceinline__ void add_far_word(Stat& st, unsigned x) {
  const float base = st.m == kNegInf ? 0.0f : st.m;
#pragma unroll
  for (int j = 0; j < Word<T>::N; ++j) {
    const float y = max_nan((Word<T>::get(x, j) - base) * kLog2e, -200.0f), e = exp2_approx(y);
    st.s += e;
    st.t = fmaf(e, y, st.t);
  }
}

// Shared memory of a row's end.
struct RowEnd {
  unsigned best[kBest * kRowWarps];        // the order keys of every warp's best threads
  float s[kRowWarps], t[kRowWarps];
  int jobs[2];                             // of a first and a second list; 0 between the rows' ends
  unsigned job[kMaxJobs];                  // chunk x 256 + thread: words to be read again
  int count[kRowWarps];                    // of a warp's list
  unsigned long long list[kRowWarps][32];  // elements that reach the bound, of a warp's jobs
};
static_assert(DET_MAX_TOP_K <= 32, "a lane per alternative");

// Threads of a warp that the bound for k alternatives is drawn from: some more
// than k in all the warps.
__device__ __forceinline__ int best_per_warp(int k) { return k == 0 ? 1 : (k + kRowWarps - 1) / kRowWarps + 1 + (k > 8); }
static_assert((DET_MAX_TOP_K + kRowWarps - 1) / kRowWarps + 2 <= kBest, "room for the largest k");

// A lower bound of the row's k-th largest element: the k-th largest of the best
// threads' order keys or a little less, by cutting the interval in which it is
// to a quarter a few times.  Every warp finds it for itself.
__device__ __forceinline__ unsigned kth_best(const RowEnd& end, int count, int k, int lane) {
  static_assert(kBest * kRowWarps <= 64, "two keys a lane");
  const bool in_a = lane < count, in_b = lane + 32 < count;
  const unsigned a = in_a ? end.best[lane] : 0u, b = in_b ? end.best[lane + 32] : 0u;
  // at least k keys reach low, and high is the largest
  unsigned low = __reduce_min_sync(0xffffffffu, in_b ? min(a, b) : in_a ? a : 0xffffffffu);
  const unsigned high = __reduce_max_sync(0xffffffffu, max(a, b));
  unsigned width = high - low;
#pragma unroll 1
  for (int i = 0; i < 3 && width >= 4; ++i) {
    width /= 4;
    unsigned up = 0;
#pragma unroll
    for (int q = 1; q < 4; ++q) {
      const unsigned mid = low + q * width;
      const int reach = __popc(__ballot_sync(0xffffffffu, in_a && a >= mid)) +
                        __popc(__ballot_sync(0xffffffffu, in_b && b >= mid));
      if (reach >= k) up = q * width;
    }
    low += up;
  }
  return low;
}

// The words that a warp reads again: of every 8th job, or, where there were too
// many, of its own threads: the 32 words of the chunk with a thread's best, or those
// of every chunk if another one has an element that reaches the bound too.
struct Jobs {
  const unsigned* list;
  int next, count;             // of the list; count < 0: of the warp's threads
  unsigned one, all;           // threads whose best chunk is to be read, or every chunk from `chunk` up
  int chunk, chunks;

  __device__ __forceinline__ bool any() const { return count < 0 ? (one | all) != 0 : next < count; }
  // Chunk x 256 + thread of the next one; best_chunk: of the lane's thread.
  __device__ __forceinline__ unsigned take(int best_chunk) {
    const unsigned first = threadIdx.x & ~31u;   // of the warp's threads
    if (count >= 0) {
      const unsigned job = list[next];
      next += kRowWarps;
      return job;
    }
    if (one) {
      const int owner = __ffs(one) - 1;
      one &= one - 1;
      // -1, in a row given up before the thread had an element: any chunk will do
      return (unsigned)max(__shfl_sync(0xffffffffu, best_chunk, owner), 0) * kRowThreads + first + owner;
    }
    const unsigned job = (unsigned)chunk * kRowThreads + first + __ffs(all) - 1;
    if (++chunk == chunks) {
      chunk = 0;
      all &= all - 1;
    }
    return job;
  }
};

// The lane's word of a job and what it holds.
template <typename T> struct Found {
  const T* row;
  int vocab, words;
  bool aligned;
  unsigned floor_key;

  __device__ __forceinline__ int at(unsigned job) const {
    return (int)((job / kRowThreads * kWords + (threadIdx.x & 31)) * kRowThreads + job % kRowThreads);
  }
  __device__ __forceinline__ unsigned load(int w) const { return w < words ? load_word(row, w, vocab, aligned) : 0u; }
  // Element j of word w: its order key above the complement of its index if it reaches the bound, else 0.
  __device__ __forceinline__ unsigned long long key(int w, unsigned word, int j) const {
    const int e = w * Word<T>::N + j;
    const unsigned ek = order_key(Word<T>::get(word, j));
    return w < words && e < vocab && ek >= floor_key ? ((unsigned long long)ek << 32) | (unsigned)~(unsigned)e : 0ull;
  }
};

// A warp whose elements do not fit its list (many equal ones): its k best, kept in order.
template <typename T>
__device__ __noinline__ int sorted_list(Jobs jobs, int best_chunk, Found<T> found, int k, unsigned long long* list) {
  static_assert(kWords == 32, "a lane per word");
  const int lane = threadIdx.x & 31;
  unsigned long long mine = 0;   // below every key
  while (jobs.any()) {
    const int w = found.at(jobs.take(best_chunk));
    const unsigned word = found.load(w);
#pragma unroll 1
    for (int j = 0; j < Word<T>::N; ++j) {
      const unsigned long long key = found.key(w, word, j);
      unsigned hits = __ballot_sync(0xffffffffu, key > __shfl_sync(0xffffffffu, mine, k - 1));
      while (hits) {
        const int src = __ffs(hits) - 1;
        hits &= hits - 1;
        list_insert(mine, __shfl_sync(0xffffffffu, key, src), lane);
      }
    }
  }
  const int count = min(k, __popc(__ballot_sync(0xffffffffu, mine != 0)));
  if (lane < count) list[lane] = mine;
  return count;
}

// The last of the top_k alternatives, where only elements equal to the bound are
// left: those of the lowest indices (one warp).
template <typename T>
__device__ __noinline__ void fill_equal(Found<T> found, unsigned equal, const RowEnd& end, int top_k, float base,
                                        float log_s, long long r, const RowOut& out) {
  const int lane = threadIdx.x & 31;
  int rank = (int)__reduce_add_sync(0xffffffffu, lane < kRowWarps ? (unsigned)end.count[lane] : 0u);
  const float log_p = (key_value(equal) - base) - log_s;
  for (int w0 = 0; w0 < found.words && rank < top_k; w0 += 32) {
    const unsigned word = found.load(w0 + lane);
    unsigned hits[Word<T>::N];
    int mine = rank;
#pragma unroll
    for (int j = 0; j < Word<T>::N; ++j) {
      const bool is = w0 + lane < found.words && (w0 + lane) * Word<T>::N + j < found.vocab &&
                      order_key(Word<T>::get(word, j)) == equal;
      hits[j] = __ballot_sync(0xffffffffu, is);
      mine += __popc(hits[j] & ((1u << lane) - 1));
      rank += __popc(hits[j]);
    }
#pragma unroll
    for (int j = 0; j < Word<T>::N; ++j) {
      if (!((hits[j] >> lane) & 1)) continue;
      if (mine < top_k) {
        if (out.top_index) out.top_index[r * top_k + mine] = (w0 + lane) * Word<T>::N + j;
        if (out.top_logprob) out.top_logprob[r * top_k + mine] = log_p;
      }
      ++mine;
    }
  }
}

// The alternatives that were not found, in a row given up (one warp): index -1.
__device__ __noinline__ void fill_missing(const RowEnd& end, int top_k, long long r, const RowOut& out) {
  const int lane = threadIdx.x & 31;
  const int found = (int)__reduce_add_sync(0xffffffffu, lane < kRowWarps ? (unsigned)end.count[lane] : 0u);
  for (int rank = found + lane; rank < top_k; rank += 32) {
    if (out.top_index) out.top_index[r * top_k + rank] = -1;
    if (out.top_logprob) out.top_logprob[r * top_k + rank] = __uint_as_float(0x7fc00000u);
  }
}

// The threads' statistics joined, the row's results and its top_k largest
// elements: only threads whose best reaches the k-th best of the warps' best
// ones are looked through again, as jobs that the warps share.
//
// It runs once a row: its instructions are mostly fetched anew, and it is one
// chain of dependent steps, about half of which the SM's other CTA hides.  What
// counts is little code, few steps, even shares, and reads of the row that
// are on their way while the sums are joined.
template <typename T>
__device__ __forceinline__ void finish_row(Stat st, const Best& best, const T* row, int vocab, long long r, int tok,
                                           int top_k, RowEnd& end, const RowOut& out) {
  constexpr int kAhead = 4;   // reads in flight
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T raw = from_f32<T>(0.0f);   // the token's logit, used at the end
  if (tok >= 0 && tok < vocab) raw = row[tok];
  const float largest = st.m;
  unsigned left = order_key(largest);
  const int each = best_per_warp(top_k);
#pragma unroll 1
  for (int j = 0; j < each; ++j) {
    const unsigned top = __reduce_max_sync(0xffffffffu, left);
    if (lane == 0) end.best[each * warp + j] = top;
    const int owner = __ffs(__ballot_sync(0xffffffffu, left == top)) - 1;
    if (lane == owner) left = 0u;
  }
  __syncthreads();
  const float m = key_value(__reduce_max_sync(0xffffffffu, end.best[each * (lane & (kRowWarps - 1))]));
  Jobs jobs = {end.job, warp, 0, 0u, 0u, 0, 0};
  Found<T> found = {row, vocab, 0, false, 0u};
  unsigned floor_key = 0;
  int at[kAhead];
  unsigned word[kAhead];
  if (top_k > 0) {
    floor_key = kth_best(end, each * kRowWarps, top_k, lane);
    found.words = (vocab + Word<T>::N - 1) / Word<T>::N;
    found.aligned = (reinterpret_cast<uintptr_t>(row) & 3) == 0;
    jobs.chunks = (found.words + kChunkWords - 1) / kChunkWords;
    // With too many elements at the bound (the mask's value, in a row with
    // fewer than k others) those above it are listed, and the lowest of the equal
    // ones fill the rest; with too many above it the warps take their own threads.
#pragma unroll 1
    for (int list = 0; list < 3; ++list) {
      found.floor_key = list == 1 ? floor_key + 1 : floor_key;
      const bool reaches = order_key(largest) >= found.floor_key;
      const bool others = reaches && order_key(best.others) >= found.floor_key;
      jobs.one = __ballot_sync(0xffffffffu, reaches && !others);
      jobs.all = __ballot_sync(0xffffffffu, others);
      jobs.count = -1;
      if (list == 2) break;
      const int single = __popc(jobs.one), many = __popc(jobs.all);
      if (single + many > 0) {
        const long long wanted = single + (long long)many * jobs.chunks;
        const int n = (int)min(wanted, (long long)kMaxJobs + 1);   // so that the sum of 8 stays small
        int base = 0;
        if (lane == 0) base = atomicAdd(&end.jobs[list], n);
        base = __shfl_sync(0xffffffffu, base, 0);
        if (base + n <= kMaxJobs) {
          const unsigned before = (1u << lane) - 1;
          if (reaches && !others)
            end.job[base + __popc(jobs.one & before)] = (unsigned)max(best.chunk, 0) * kRowThreads + threadIdx.x;
          if (others)
            for (int c = 0; c < jobs.chunks; ++c)
              end.job[base + single + __popc(jobs.all & before) * jobs.chunks + c] = (unsigned)c * kRowThreads + threadIdx.x;
        }
      }
      __syncthreads();
      jobs.count = end.jobs[list];
      if (jobs.count <= kMaxJobs) break;
      if (floor_key == 0xffffffffu) list = 1;   // nothing is above NaN
    }
  }
  const Jobs from_the_start = jobs;
  int loads = 0;
#pragma unroll
  for (int a = 0; a < kAhead; ++a) {
    if (!jobs.any()) break;
    at[a] = found.at(jobs.take(best.chunk));
    word[a] = found.load(at[a]);
    loads = a + 1;
  }
  raise_to<T>(st, m);
  float s = warp_pt(st.s), t = warp_pt(st.t);
  if (lane == 0) {
    end.s[warp] = s;
    end.t[warp] = t;
  }
  if (top_k > 0) {
    int count = 0;
    while (true) {
#pragma unroll 1
      for (int a = 0; a < loads; ++a) {   // the first of the arrays, which move up
#pragma unroll 1
        for (int j = 0; j < Word<T>::N; ++j) {
          const unsigned long long key = found.key(at[0], word[0], j);
          const unsigned hits = __ballot_sync(0xffffffffu, key != 0);
          const int slot = count + __popc(hits & ((1u << lane) - 1));
          if (key != 0 && slot < 32) end.list[warp][slot] = key;
          count += __popc(hits);
        }
#pragma unroll
        for (int i = 0; i + 1 < kAhead; ++i) {
          word[i] = word[i + 1];
          at[i] = at[i + 1];
        }
      }
      if (!jobs.any() || count > 32) break;
      at[0] = found.at(jobs.take(best.chunk));
      word[0] = found.load(at[0]);
      loads = 1;
    }
    if (count > 32) {
      __syncwarp();
      count = sorted_list(from_the_start, best.chunk, found, top_k, end.list[warp]);
    }
    if (lane == 0) end.count[warp] = count;
  }
  __syncthreads();
  if (threadIdx.x == 0) end.jobs[0] = end.jobs[1] = 0;
  s = end.s[lane & (kRowWarps - 1)];
  t = end.t[lane & (kRowWarps - 1)];
#pragma unroll
  for (int d = 1; d < kRowWarps; d <<= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, d);
    t += __shfl_xor_sync(0xffffffffu, t, d);
  }
  const bool empty = m == kNegInf;
  const float base = empty ? 0.0f : m;
  // log of the sum relative to exp(m): the reference is m log2(e) up to its rounding
  const float log_2s = empty ? 0.0f : logf(s);
  const float log_s = near_max<T>(m) ? fmaf(-kLn2, __fmaf_rn(m, kLog2e, -near_ref(m)), log_2s) : log_2s;
  if (threadIdx.x == 0) {
    if (out.lse) out.lse[r] = empty ? kNegInf : base + log_s;
    if (out.entropy) out.entropy[r] = empty ? 0.0f : log_2s - kLn2 * (t / s);
    if (out.logprob) out.logprob[r] = tok >= 0 && tok < vocab ? (to_f32(raw) - base) - log_s : 0.0f;
  }
  if (top_k > 0) {
    // the ranks of the warp's list among all lists, an element after the other
    unsigned long long v[kRowWarps];
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) v[w] = lane < end.count[w] ? end.list[w][lane] : 0ull;
    const int count = end.count[warp];
    int rank = top_k;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const unsigned long long key = end.list[warp][i];
      int above = 0;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) above += __popc(__ballot_sync(0xffffffffu, v[w] > key));
      if (lane == i) rank = above;
    }
    if (rank < top_k) {
      const unsigned long long key = end.list[warp][lane];
      if (out.top_index) out.top_index[r * top_k + rank] = (int32_t)~(unsigned)key;
      if (out.top_logprob) out.top_logprob[r * top_k + rank] = (key_value((unsigned)(key >> 32)) - base) - log_s;
    }
    if (warp == 0) {
      if (found.floor_key != floor_key) fill_equal(found, floor_key, end, top_k, base, log_s, r, out);
      else if (isnan(m)) fill_missing(end, top_k, r, out);
    }
  }
}

// What a CTA of a cluster leaves of its part for the first one.
struct PartStats {
  float m[kRowThreads], s[kRowThreads], t[kRowThreads], others[kRowThreads], chunk[kRowThreads];
};
static_assert(sizeof(PartStats) <= sizeof(Stream::stage), "it fits the stages");

// Persistent: CTA b takes the rows b, b + gridDim.x, ...; SPLIT: a cluster of a
// CTA per part takes a row (1 x 131,072 bf16: 17 us -> 12).  A wait for a copy that
// does not end within kWaitNs gives up: the row's results, and those of the CTA's
// rows after it, are NaN then.
template <typename T, bool SPLIT>
__global__ void __launch_bounds__(kRowThreads, 2)
token_logprobs_kernel(const T* logits, long long rows, int vocab, long long row_stride, const int32_t* tokens, int top_k,
                      RowOut out) {
  extern __shared__ __align__(16) unsigned char dynamic[];
  Stream& stream = *reinterpret_cast<Stream*>(dynamic);
  __shared__ RowEnd end;
  const int lane = threadIdx.x & 31;
  const int chunks = max(1, (int)(((long long)vocab + Word<T>::N * kChunkWords - 1) / (Word<T>::N * kChunkWords)));
  const int per_part = chunks_per_part(chunks), parts = (chunks + per_part - 1) / per_part;
  const int rank = SPLIT ? blockIdx.x % parts : 0;
  const int c0 = SPLIT ? rank * per_part : 0, c1 = SPLIT ? min(c0 + per_part, chunks) : chunks;
  const long long row0 = SPLIT ? blockIdx.x / parts : blockIdx.x, row_step = SPLIT ? rows : gridDim.x;
  if (threadIdx.x == 0) {
    end.jobs[0] = end.jobs[1] = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&stream.full[i], 1);
      mbar_init(&stream.empty[i], kRowWarps);
      stream.filled[i] = -1;
    }
  }
  __syncthreads();
  dep_wait();   // launched early: all loads come after, and none is a read-only one, which need not
  dep_launch();
  // the next chunk to fetch, its stage and how often the stage was filled
  long long next_row = row0;
  int next_chunk = c0, next_stage = 0, next_round = 0;
  bool gave_up = false;
  auto fetch_next = [&](bool mine) {
    if (next_row >= rows) return;
    if (mine) {
      if (next_round > 0 && !gave_up) gave_up = !mbar_wait(&stream.empty[next_stage], (next_round - 1) & 1, kWaitNs);
      if (!gave_up) {
        stream.filled[next_stage] = next_round;
        RowMap<T>(logits + next_row * row_stride, vocab).fetch(stream, next_stage, next_chunk);
      }
    }
    if (++next_chunk == c1) {
      next_chunk = c0;
      next_row += row_step;
    }
    if (++next_stage == kStages) {
      next_stage = 0;
      ++next_round;
    }
  };
  for (int i = 0; i < kStages - 1; ++i) fetch_next(threadIdx.x == 0);
  // a thread's edges of the row after the current one
  unsigned head_ahead = 0, tail_ahead = 0;
  int token_ahead = -1;   // and its token (one thread)
  auto load_edges = [&](long long r) {
    if (r >= rows) return;
    if (threadIdx.x == 0 && out.logprob) token_ahead = tokens[r];
    const RowMap<T> map(logits + r * row_stride, vocab);
    const bool aligned = (map.off & 3) == 0;
    if ((int)threadIdx.x < map.head) head_ahead = load_word(map.row, threadIdx.x, vocab, aligned);
    const int w = map.tail_word();
    if (w >= 0) tail_ahead = load_word(map.row, w, vocab, aligned);
  };
  load_edges(row0);
  int stage = 0, round = 0, turn = 0;
  for (long long r = row0; r < rows; r += row_step) {
    const RowMap<T> map(logits + r * row_stride, vocab);
    const unsigned head = head_ahead, tail = tail_ahead;
    const int token = token_ahead;
    load_edges(r + row_step);
    Stat st = {kNegInf, 0.0f, 0.0f}, all = st;   // of the part, and of the parts before it
    Best best = {-1, kNegInf}, all_best = best;
    const unsigned odd_shift = map.odd() ? 16u : 0u;
    const int tail_word = map.tail_word();
    int part_end = per_part;
    for (int c = c0; c < c1; ++c) {
      // the warps take turns at waiting for the stage that all have read and filling it
      fetch_next(threadIdx.x == turn * 32);
      turn = (turn + 1) & (kRowWarps - 1);
      if (!gave_up) gave_up = !mbar_wait(&stream.full[stage], round & 1, kWaitNs);
      const unsigned char* words = stream.stage[stage];
      // read words (all of the thread's, or kPartWords at a time in the row's
      // last chunk if it is not whole), then bring the maximum up, then add
      auto release = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(&stream.empty[stage]);
      };
      auto step = [&](auto shift, auto count, int i0, bool ragged) {
        constexpr int NW = decltype(count)::value;
        constexpr bool kAll = NW == kWords;   // the chunk's only step
        const int w0 = c * kChunkWords + i0 * kRowThreads + threadIdx.x;
        unsigned x[NW];
        read_words<decltype(shift)::value>(words, map.off, i0, odd_shift, x);
        if (ragged) set_edges(map, w0, head, tail, tail_word, x);
        else if (w0 < map.head) x[0] = head;   // the first words of a row
        raise_words<T>(st, best, c, largest_of<T>(x));
        const bool near = near_max<T>(st.m), all_near = __all_sync(0xffffffffu, near);
        if (kAll && all_near) release();
        if (near) {
          add_words<T>(st, x);
        } else if (st.m == kNegInf) {
          // masked logits alone add nothing
        } else if (all_equal<T>(x, st.m)) {
          st.s += (float)(NW * Word<T>::N);   // masked by the type's lowest value: 1 each, and nothing to T
        } else {
#pragma unroll 1
          for (int i = 0; i < NW; ++i) {
            unsigned y[1];
            read_words<true>(words, map.off, i0 + i, odd_shift, y);
            set_edges(map, w0 + i * kRowThreads, head, tail, tail_word, y);
            add_far_word<T>(st, y[0]);
          }
        }
        if (kAll && !all_near) release();
      };
      using std::integral_constant;
      if ((c + 1LL) * kChunkWords <= map.words) {
        const bool ragged = map.ragged(c);
        if (odd_shift == 0 && !ragged) {
          step(integral_constant<bool, false>(), integral_constant<int, kWords>(), 0, false);
        } else {
          step(integral_constant<bool, true>(), integral_constant<int, kWords>(), 0, ragged);
        }
      } else {
#pragma unroll 1
        for (int i0 = 0; i0 < kWords && c * kChunkWords + i0 * kRowThreads < map.words; i0 += kPartWords)
          step(integral_constant<bool, true>(), integral_constant<int, kPartWords>(), i0, true);
        release();
      }
      if (++stage == kStages) {
        stage = 0;
        ++round;
      }
      if (!SPLIT && (c + 1 == part_end || c + 1 == c1)) {
        join_part<T>(all, all_best, st, best);
        st = {kNegInf, 0.0f, 0.0f};
        best = {-1, kNegInf};
        part_end += per_part;
      }
    }
    if (SPLIT) {
      if (__syncthreads_or(gave_up)) {   // the stages have been read
        if (threadIdx.x == 0) land_copies(stream);
        __syncthreads();
      }
      PartStats& left = *reinterpret_cast<PartStats*>(stream.stage);
      left.m[threadIdx.x] = gave_up ? __uint_as_float(0x7fc00000u) : st.m;
      left.s[threadIdx.x] = st.s;
      left.t[threadIdx.x] = st.t;
      left.others[threadIdx.x] = best.others;
      left.chunk[threadIdx.x] = __int_as_float(best.chunk);
      cluster_sync_all();
      if (rank == 0)
        for (int p = 0; p < parts; ++p) {
          const Stat part = {ld_dsmem(&left.m[threadIdx.x], p), ld_dsmem(&left.s[threadIdx.x], p),
                             ld_dsmem(&left.t[threadIdx.x], p)};
          const Best part_best = {__float_as_int(ld_dsmem(&left.chunk[threadIdx.x], p)),
                                  ld_dsmem(&left.others[threadIdx.x], p)};
          join_part<T>(all, all_best, part, part_best);
        }
      cluster_sync_all();   // no CTA leaves before its part is read
      if (rank != 0) return;
    } else if (gave_up) {
      all.m = __uint_as_float(0x7fc00000u);
    }
    finish_row(all, all_best, map.row, vocab, r, token, top_k, end, out);
  }
  if (!SPLIT && __syncthreads_or(gave_up) && threadIdx.x == 0) land_copies(stream);
}

// ---------------------------------------------------------------------------
// The gradient: elementwise once lse and the entropy are known.

constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;   // 16-byte vectors of a thread
// From this magnitude on 32 bits hold lse to 2^-14 or worse (nothing of log S
// is left of it in a row at the types' lowest values): the row is summed again, by
// each of its CTAs, which read the whole row twice more.  Ten times the time where
// every row is so (1,021 x 100,003 f32 1,176 us instead of 119; a tenth of them 230).
constexpr float kLseFar = 1024.0f;

// The maximum and the log of the sum relative to it of a whole row.
template <typename T>
__device__ float2 row_max_and_log_sum(const T* row, long long vocab) {
  __shared__ float sh[2][kGradThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float m = kNegInf, s = 0.0f;
  for (long long e = threadIdx.x; e < vocab; e += kGradThreads) m = fmaxf(m, to_f32(row[e]));
  for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) sh[0][warp] = m;
  __syncthreads();
  for (int w = 0; w < kGradThreads / 32; ++w) m = fmaxf(m, sh[0][w]);
  for (long long e = threadIdx.x; e < vocab; e += kGradThreads) s += exp2_approx((to_f32(row[e]) - m) * kLog2e);
  s = warp_pt(s);
  if (lane == 0) sh[1][warp] = s;
  __syncthreads();
  s = 0.0f;
  for (int w = 0; w < kGradThreads / 32; ++w) s += sh[1][w];
  return make_float2(m, logf(s));
}

// grad[v] = [v == token] g_l - p (c + g_h log p) with c = g_l + g_h * entropy.
struct GradRow {
  float base, log_s;   // log p = (x - base) - log_s
  float gl, gh, c;
  __device__ __forceinline__ float at(float x) const {
    // p is 0 from -150 on already; without the bound 0 * inf for a masked logit
    const float lp = max_nan((x - base) - log_s, -150.0f);
    return -exp2_approx(lp * kLog2e) * fmaf(gh, lp, c);
  }
};

// Bound by the bytes: each logit is read and its gradient written once (4,096 x
// 65,536 bf16 154 us, 1,021 x 100,003 f32 119 us, both the measured copy
// bandwidth).  A CTA takes 256 x 4 vectors of 16 bytes of a row, counted from the row's
// first 16-byte boundary (the same one of both rows: SAME_PHASE), and the
// row's first CTA the elements before it and behind the last vector.  Where
// the rows' boundaries differ it goes by elements.
template <typename T, bool SAME_PHASE>
__global__ void __launch_bounds__(kGradThreads)
token_logprobs_grad_kernel(const T* __restrict__ logits, int vocab, long long row_stride,
                           const int32_t* __restrict__ tokens, const float* __restrict__ lse,
                           const float* __restrict__ entropy, const float* __restrict__ grad_logprob,
                           const float* __restrict__ grad_entropy, T* __restrict__ grad, long long grad_stride,
                           unsigned ctas_per_row) {
  constexpr int E = 16 / sizeof(T), N = Word<T>::N;
  const unsigned r = blockIdx.x / ctas_per_row, part = blockIdx.x - r * ctas_per_row;
  const T* row = logits + r * row_stride;
  T* g = grad + r * grad_stride;
  const int head = SAME_PHASE ? min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(T), vocab) : 0;
  const int vecs = SAME_PHASE ? (vocab - head) / E : 0;
  const int v0 = part * (kGradThreads * kGradVecs) + threadIdx.x;
  uint4 x[kGradVecs];
  if constexpr (SAME_PHASE) {
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i)
      if (v0 + i * kGradThreads < vecs) x[i] = __ldg(reinterpret_cast<const uint4*>(row + head) + v0 + i * kGradThreads);
  }
  const float l = lse[r];
  const int tok = grad_logprob ? tokens[r] : -1;
  GradRow q;
  q.gl = tok >= 0 && tok < vocab ? grad_logprob[r] : 0.0f;
  q.gh = grad_entropy ? grad_entropy[r] : 0.0f;
  q.c = grad_entropy ? fmaf(q.gh, entropy[r], q.gl) : q.gl;
  q.base = l;
  q.log_s = 0.0f;
  if (fabsf(l) >= kLseFar && fabsf(l) < INFINITY) {
    const float2 ms = row_max_and_log_sum(row, vocab);
    q.base = ms.x;
    q.log_s = ms.y;
  }
  if (l == kNegInf) {   // a row without a logit above -inf: 0 throughout
    q.gl = q.gh = q.c = 0.0f;
    q.base = 0.0f;
  }
  if constexpr (SAME_PHASE) {
#pragma unroll
    for (int i = 0; i < kGradVecs; ++i) {
      const int v = v0 + i * kGradThreads;
      if (v >= vecs) break;
      const unsigned w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      float d[E];
#pragma unroll
      for (int j = 0; j < E; ++j) d[j] = q.at(Word<T>::get(w[j / N], j % N));
      const int at = tok - head - v * E;   // the token's place in the vector
      if (at >= 0 && at < E) {
#pragma unroll
        for (int j = 0; j < E; ++j) d[j] += j == at ? q.gl : 0.0f;
      }
      uint4 o;
      if constexpr (N == 1) {
        o = make_uint4(__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3]));
      } else {
        unsigned y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = Word<T>::pack(d[2 * j], d[2 * j + 1]);
        o = make_uint4(y[0], y[1], y[2], y[3]);
      }
      reinterpret_cast<uint4*>(g + head)[v] = o;
    }
    if (part > 0) return;
    for (int k = threadIdx.x; k < vocab - vecs * E; k += kGradThreads) {
      const int e = k < head ? k : vecs * E + k;
      g[e] = from_f32<T>(q.at(to_f32(row[e])) + (e == tok ? q.gl : 0.0f));
    }
  } else {
    const int first = part * (kGradThreads * kGradVecs * E);
    for (int e = first + threadIdx.x; e < min(first + kGradThreads * kGradVecs * E, vocab); e += kGradThreads)
      g[e] = from_f32<T>(q.at(to_f32(row[e])) + (e == tok ? q.gl : 0.0f));
  }
}

template <typename T>
int launch_logprobs(const void* logits, long long rows, int vocab, long long stride, const int32_t* tokens, int top_k,
                    const RowOut& out, cudaStream_t s) {
  const long long per_chunk = (long long)Word<T>::N * kChunkWords;
  const int chunks = (int)std::max(1LL, (vocab + per_chunk - 1) / per_chunk);
  const int per_part = chunks_per_part(chunks), parts = (chunks + per_part - 1) / per_part;
  const long long resident = 2LL * std::max(device_sm_count(), 1);
  // A row per cluster while every CTA is resident at once: SMs would stand idle
  // otherwise.  With more rows the parts of a row gain nothing.
  const bool split = parts > 1 && rows * parts <= resident;
  auto kernel = split ? token_logprobs_kernel<T, true> : token_logprobs_kernel<T, false>;
  if (const cudaError_t e = ensure_dyn_smem(reinterpret_cast<const void*>(kernel), sizeof(Stream)))
    return cuda_fail(e, "det_token_logprobs");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(split ? rows * parts : std::min(rows, resident)));
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = sizeof(Stream);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split ? 2 : 1;
  launch_begin("det_token_logprobs", s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<const T*>(logits), rows, vocab, stride, tokens,
                                           top_k, out);
  launch_end(s);
  return e == cudaSuccess ? DET_OK : cuda_fail(e, "det_token_logprobs");
}

template <typename T>
int launch_grad(const void* logits, long long rows, long long vocab, long long stride, const int32_t* tokens,
                const float* lse, const float* entropy, const float* gl, const float* gh, void* grad,
                long long grad_stride, cudaStream_t s) {
  const long long per = (long long)kGradThreads * kGradVecs * (16 / sizeof(T)), ctas = (vocab + per - 1) / per;
  if (rows * ctas >= (1LL << 31)) return DET_ERR_TOO_LARGE;
  // every row pair starts at the same place of a 16-byte block
  const bool same = ((reinterpret_cast<uintptr_t>(logits) ^ reinterpret_cast<uintptr_t>(grad)) % 16 == 0) &&
                    (rows == 1 || (stride - grad_stride) * (long long)sizeof(T) % 16 == 0);
  launch_begin("det_token_logprobs_backward", s);
  if (same)
    token_logprobs_grad_kernel<T, true><<<(unsigned)(rows * ctas), kGradThreads, 0, s>>>(
        static_cast<const T*>(logits), (int)vocab, stride, tokens, lse, entropy, gl, gh, static_cast<T*>(grad),
        grad_stride, (unsigned)ctas);
  else
    token_logprobs_grad_kernel<T, false><<<(unsigned)(rows * ctas), kGradThreads, 0, s>>>(
        static_cast<const T*>(logits), (int)vocab, stride, tokens, lse, entropy, gl, gh, static_cast<T*>(grad),
        grad_stride, (unsigned)ctas);
  launch_end(s);
  return check_launch("det_token_logprobs_backward");
}

}  // namespace
}  // namespace det

using namespace det;

extern "C" int det_token_logprobs(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride,
                                  const int32_t* tokens, int dtype, float* logprob_out, float* entropy_out,
                                  float* lse_out, int top_k, float* top_logprob_out, int32_t* top_index_out,
                                  void* stream) {
  if (!valid_model_dtype(dtype)) return DET_ERR_DTYPE;
  if (rows < 0 || vocab < 0 || row_stride < 0 || top_k < 0 || top_k > DET_MAX_TOP_K || top_k > vocab)
    return DET_ERR_INVALID_ARG;
  if (rows >= (1LL << 31) || vocab > (1LL << 30)) return DET_ERR_TOO_LARGE;
  if (rows == 0) return DET_OK;
  if ((vocab > 0 && !logits) || (logprob_out && !tokens)) return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % model_elem_size(dtype)) return DET_ERR_INVALID_ARG;
  const RowOut out = {logprob_out, entropy_out, lse_out, top_logprob_out, top_index_out};
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32) return launch_logprobs<float>(logits, rows, (int)vocab, row_stride, tokens, top_k, out, s);
  if (dtype == DET_BF16) return launch_logprobs<__nv_bfloat16>(logits, rows, (int)vocab, row_stride, tokens, top_k, out, s);
  return launch_logprobs<__half>(logits, rows, (int)vocab, row_stride, tokens, top_k, out, s);
}

extern "C" int det_token_logprobs_backward(const void* logits, int64_t rows, int64_t vocab, int64_t row_stride,
                                           const int32_t* tokens, int dtype, const float* lse, const float* entropy,
                                           const float* grad_logprob, const float* grad_entropy, void* grad_logits,
                                           int64_t grad_row_stride, void* stream) {
  if (!valid_model_dtype(dtype)) return DET_ERR_DTYPE;
  if (rows < 0 || vocab < 0 || row_stride < 0) return DET_ERR_INVALID_ARG;
  if (rows > 1 && grad_row_stride < vocab) return DET_ERR_INVALID_ARG;   // rows of the result would overlap
  if (rows >= (1LL << 31) || vocab >= (1LL << 28)) return DET_ERR_TOO_LARGE;
  if (rows == 0 || vocab == 0) return DET_OK;
  if (!logits || !lse || !grad_logits || (grad_logprob && !tokens) || (grad_entropy && !entropy))
    return DET_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % model_elem_size(dtype) ||
      reinterpret_cast<uintptr_t>(grad_logits) % model_elem_size(dtype))
    return DET_ERR_INVALID_ARG;
  const cudaStream_t s = as_stream(stream);
  if (dtype == DET_F32)
    return launch_grad<float>(logits, rows, vocab, row_stride, tokens, lse, entropy, grad_logprob, grad_entropy,
                              grad_logits, grad_row_stride, s);
  if (dtype == DET_BF16)
    return launch_grad<__nv_bfloat16>(logits, rows, vocab, row_stride, tokens, lse, entropy, grad_logprob,
                                      grad_entropy, grad_logits, grad_row_stride, s);
  return launch_grad<__half>(logits, rows, vocab, row_stride, tokens, lse, entropy, grad_logprob, grad_entropy,
                             grad_logits, grad_row_stride, s);
}
